// prompt.cu -- rkv_prompt_attn: causal grouped-query attention over the
// packed prompts of a batch (one layer a call), on fp32 tensors; bf16 ones take
// prompt_tc.cu.
//
//   o[i] = sum_{j <= i} exp(z_ij - lse_i) v_j,  z_ij = scale <q_i, k_j>,
//   lse_i = log sum_{j <= i} exp(z_ij)
#include "internal.h"
#include "serve.cuh"

namespace rkv {
namespace {

// One CTA per (T/16*R query rows, query head): FFMA products, see serve.cuh.
template <int D, int R, int T>
__global__ void __launch_bounds__(T) prompt_ffma_kernel(const PromptArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    FTile<D, T / 16 * R> &t = *reinterpret_cast<FTile<D, T / 16 * R> *>(smem);
    int32_t *s_cu = reinterpret_cast<int32_t *>(smem + sizeof(FTile<D, T / 16 * R>));
    constexpr int ROWS = T / 16 * R;
    __shared__ SeqTile s_tile;
    if (!load_offsets(a.cu, a.B, a.n_tokens, a.n_tokens, s_cu, a.status)) return;
    const int tile = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
    if (threadIdx.x < 32) {
        SeqTile w{-1, 0};
        if (tile < tiles_from(s_cu, a.B, ROWS, 0)) w = find_tile(s_cu, a.B, a.n_tokens, ROWS, tile);
        if (threadIdx.x == 0) s_tile = w;
    }
    __syncthreads();
    const SeqTile w = s_tile;
    if (w.b < 0) return;
    const int64_t t0 = s_cu[w.b];
    const int n = s_cu[w.b + 1] - s_cu[w.b], r0 = w.blk * ROWS, h = hq / (a.Hq / a.H);
    const float *q = static_cast<const float *>(a.q) + (int64_t)hq * D;
    const float *k = static_cast<const float *>(a.k) + (int64_t)h * D;
    const float *v = static_cast<const float *>(a.v) + (int64_t)h * D;
    constexpr int V4 = D / 4;
    for (int i = threadIdx.x; i < ROWS * V4; i += T) {
        const int r = i / V4, d = i % V4 * 4;
        const float4 x = r0 + r < n ? ld4(q + (t0 + r0 + r) * a.q_stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(&t.q[r][d]) = x;
    }
    FState<D, R> st;
    st.init();
    const int last = min(r0 + ROWS, n);
    // a key tile's K and V are on their way to registers while the tile before is worked on
    constexpr int N = FT_KEYS * V4 / T;
    float4 kr[N], vr[N];
    auto load = [&](int j0) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int e = i * T + threadIdx.x, r = e / V4, d = e % V4 * 4;
            const bool in = j0 + r < n;
            kr[i] = in ? ld4(k + (t0 + j0 + r) * a.k_stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
            vr[i] = in ? ld4(v + (t0 + j0 + r) * a.v_stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    load(0);
    for (int j0 = 0; j0 < last; j0 += FT_KEYS) {
        __syncthreads();
        int odd = 0;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int e = i * T + threadIdx.x, r = e / V4, d = e % V4 * 4;
            odd |= odd4(vr[i]);
            *reinterpret_cast<float4 *>(&t.k[r][d]) = kr[i];
            *reinterpret_cast<float4 *>(&t.v[r][d]) = vr[i];
        }
        odd = __syncthreads_or(odd);
        if (j0 + FT_KEYS < last) load(j0 + FT_KEYS);
        ftile_step<D, R, ROWS>(t, st, a.qscale, j0 + FT_KEYS > r0, odd != 0,
                         [&](int row, int key) { return j0 + key > r0 + row; });
    }
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int r = r0 + ty * R + i;
        if (r >= n) continue;
        float *o = static_cast<float *>(a.out) + (t0 + r) * a.out_stride + (int64_t)hq * D;
        const float inv = 1.f / st.l[i];
#pragma unroll
        for (int j = 0; j < D / 64; j++)
            st4(o + tx * 4 + 64 * j, make_float4(st.o[i][4 * j] * inv, st.o[i][4 * j + 1] * inv,
                                                 st.o[i][4 * j + 2] * inv, st.o[i][4 * j + 3] * inv));
        if (a.lse && tx == 0) a.lse[(t0 + r) * a.Hq + hq] = (st.m[i] + log2f(st.l[i])) * LN2;
    }
}

template <int D, int R, int T>
cudaError_t launch_ffma(const PromptArgs &a, cudaStream_t s) {
    const size_t smem = sizeof(FTile<D, T / 16 * R>) + (size_t)(a.B + 1) * 4;
    cudaError_t e = cudaFuncSetAttribute(prompt_ffma_kernel<D, R, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)(a.n_tokens / (T / 16 * R) + a.B) * a.Hq;
    if (tiles >= (1ll << 31)) return cudaErrorNotSupported;
    prompt_ffma_kernel<D, R, T><<<(unsigned)tiles, T, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Tiles of 32 rows where those of 64 would not give two CTAs to each of the 148
// SMs: prompts of 512, 1,000 and 77 tokens with 4 heads of 64 take 76 us, and 100
// with 64 rows; one of 2,048 tokens with 32 heads takes 777 us, and 606 with 64.
// Of D = 128 the larger tiles have 128 rows, by 16 warps on the one CTA that an SM
// holds: 2,048 tokens, 32 heads, 1.04 ms (33 TFLOP/s), and 1.31 with 64 rows.
cudaError_t launch_prompt(const PromptArgs &a, int D, cudaStream_t s) {
    if ((int64_t)(a.n_tokens / 64 + a.B) * a.Hq < 296) return D == 64 ? launch_ffma<64, 2, 256>(a, s) : launch_ffma<128, 2, 256>(a, s);
    return D == 64 ? launch_ffma<64, 4, 256>(a, s) : launch_ffma<128, 4, 512>(a, s);
}

}  // namespace rkv
