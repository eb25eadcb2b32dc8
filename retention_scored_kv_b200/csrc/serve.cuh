// serve.cuh -- what the kernels of the serving operators share: the packed
// sequences of a batch (offsets `cu`), their query tiles in order of cost, and
// the fp32 attention tile.
#pragma once

#include "common.cuh"

namespace rkv {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// --------------------------------------------------- launches in pairs ----
// The second kernel of a pair is set up while the first still runs
// (launch_dependents in the first, launch_after on the host) and waits for its
// end, and for its writes, at wait_for_launcher.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launcher() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class Args>
cudaError_t launch_after(void (*kernel)(Args), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, const Args &a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ------------------------------------------------------ packed sequences ----
// Copies the offsets cu[0..B] to shared memory (unless NULL) and checks them: non-negative,
// non-decreasing, cu[B] <= n_tokens and no sequence longer than `longest`.
// Every thread of the block calls it; false (and RKV_DEV_BAD_INPUT) means that
// the whole call computes nothing.
__device__ __forceinline__ bool load_offsets(const int32_t *cu, int B, int n_tokens, int longest, int32_t *s_cu,
                                             int32_t *status) {
    int bad = 0;
    for (int i = threadIdx.x; i <= B; i += blockDim.x) {
        const int32_t v = __ldg(cu + i);
        if (s_cu) s_cu[i] = v;
        if (v < 0 || v > n_tokens) bad = 1;
        if (i > 0) {
            const int32_t u = __ldg(cu + i - 1);
            if (u < 0 || v < u || v - u > longest) bad = 1;
        }
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) set_status(status, RKV_DEV_BAD_INPUT);
    return bad == 0;
}

// One query tile of a packed batch: rows [blk*rows, ...) of sequence b.
struct SeqTile {
    int b, blk;
};

// Query tiles with block index >= m over all sequences.
__device__ __forceinline__ int tiles_from(const int32_t *cu, int B, int rows, int m) {
    int n = 0;
    for (int b = threadIdx.x & 31; b < B; b += 32) {
        const int nb = (cu[b + 1] - cu[b] + rows - 1) / rows;
        n += nb > m ? nb - m : 0;
    }
    return __reduce_add_sync(0xFFFFFFFFu, n);
}

// Tile number r when the batch's tiles are ordered by block index, highest
// first (under a causal mask a tile's cost grows with its index, so the long
// tiles start first and the short ones fill the tail).  A whole warp calls it;
// r must be below tiles_from(.., 0).  Bisection for the block index, then the
// i-th sequence that has such a block: no list of tiles is stored.
__device__ __forceinline__ SeqTile find_tile(const int32_t *cu, int B, int n_tokens, int rows, int r) {
    int lo = 0, hi = (n_tokens + rows - 1) / rows;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles_from(cu, B, rows, mid) > r) lo = mid;
        else hi = mid;
    }
    int i = r - tiles_from(cu, B, rows, lo + 1);
    SeqTile t{0, lo};
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + (threadIdx.x & 31);
        const bool has = b < B && (cu[b + 1] - cu[b] + rows - 1) / rows > lo;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, has);
        const int n = __popc(m);
        if (i < n) {
            t.b = b0 + (int)__fns(m, 0, i + 1);
            break;
        }
        i -= n;
    }
    return t;
}

// ------------------------------------------------------ fp32 attention tile ----
// T/16*R query rows against FT_KEYS keys at a time on the CUDA cores, one pass over
// the keys with each row's running maximum and sum.  T threads: thread (ty, tx)
// of a T/16 x 16 grid has rows ty*R..+R-1 and keys tx + 16*j of the scores, then
// the same rows and D/16 columns of the output.  Products and sums are fp32: the
// operands and results of this path are fp32 and a 16-bit product would lose
// them.  R = 4 loads each operand from shared memory for four products; R = 2
// cuts the work finer.
constexpr int FT_KEYS = 64;

template <int D, int ROWS>
struct FTile {
    float q[ROWS][D + 4];
    float k[FT_KEYS][D + 4];
    float v[FT_KEYS][D];
    float p[ROWS][FT_KEYS + 4];
};

template <int D, int R>
struct FState {
    float o[R][D / 16];  // columns tx*4 + 64*j + e
    float m[R], l[R];
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int i = 0; i < R; i++) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; j++) o[i][j] = 0.f;
        }
    }
};

// One key tile.  masked(row, key) tells whether the pair is left out; it is
// only asked when `any_mask`.  `odd`: some value of v is infinite or NaN, and
// left-out pairs must not touch it (0 * NaN is NaN), so they are marked by a
// negative weight and skipped.  The caller synchronises before and after.
template <int D, int R, int ROWS, class Mask>
__device__ __forceinline__ void ftile_step(FTile<D, ROWS> &t, FState<D, R> &st, float qscale, bool any_mask, bool odd,
                                           Mask masked) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    float s[R][4];
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[R], b[4];
#pragma unroll
        for (int i = 0; i < R; i++) a[i] = *reinterpret_cast<const float4 *>(&t.q[ty * R + i][d]);
#pragma unroll
        for (int j = 0; j < 4; j++) b[j] = *reinterpret_cast<const float4 *>(&t.k[tx + 16 * j][d]);
#pragma unroll
        for (int i = 0; i < R; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < R; i++) {
        uint32_t out = 0;
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            s[i][j] *= qscale;
            if (any_mask && masked(ty * R + i, tx + 16 * j)) {
                out |= 1u << j;
                s[i][j] = -INFINITY;
            }
            mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const float mn = fmaxf(st.m[i], mx);
        const float ms = mn == -INFINITY ? 0.f : mn;  // a row that has seen nothing yet
        const float f = exp2f(st.m[i] - ms);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const bool gone = (out >> j) & 1u;
            const float p = gone ? 0.f : exp2f(s[i][j] - ms);
            sum += p;
            t.p[ty * R + i][tx + 16 * j] = gone ? -1.f : p;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        st.m[i] = mn;
        st.l[i] = st.l[i] * f + sum;
#pragma unroll
        for (int j = 0; j < D / 16; j++) st.o[i][j] *= f;
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
    for (int n = 0; n < FT_KEYS; n += 4) {
        float4 w[R];
#pragma unroll
        for (int i = 0; i < R; i++) w[i] = *reinterpret_cast<const float4 *>(&t.p[ty * R + i][n]);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float4 v[D / 64];
#pragma unroll
            for (int j = 0; j < D / 64; j++) v[j] = *reinterpret_cast<const float4 *>(&t.v[n + e][tx * 4 + 64 * j]);
#pragma unroll
            for (int i = 0; i < R; i++) {
                float p = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
                if (p < 0.f) {
                    if (odd) continue;
                    p = 0.f;
                }
#pragma unroll
                for (int j = 0; j < D / 64; j++) {
                    st.o[i][4 * j + 0] = fmaf(p, v[j].x, st.o[i][4 * j + 0]);
                    st.o[i][4 * j + 1] = fmaf(p, v[j].y, st.o[i][4 * j + 1]);
                    st.o[i][4 * j + 2] = fmaf(p, v[j].z, st.o[i][4 * j + 2]);
                    st.o[i][4 * j + 3] = fmaf(p, v[j].w, st.o[i][4 * j + 3]);
                }
            }
        }
    }
    __syncwarp();
}

__device__ __forceinline__ bool odd4(float4 x) {
    return !(fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY && fabsf(x.z) < INFINITY && fabsf(x.w) < INFINITY);
}

__device__ __forceinline__ float4 ld4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ void st4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }

}  // namespace rkv
