// tree.cu -- rkv_tree_attn: attention of a tree of drafted tokens over the
// ragged paged cache.  Row (node i, query head g of the group) of KV head c
// attends the head's kept cache entries and the drafted tokens j of its own
// sequence with bit j of mask[i] set:
//   o = sum_{kept cache} exp(z - lse) v + sum_{j in mask[i]} exp(z_j - lse) v_j
// This file: fp32 pools; bf16 ones take tree_tc.cu.
#include "internal.h"
#include "serve.cuh"

namespace rkv {
namespace {

// Tiles of 32 rows: two CTAs or more to an SM, and little waste on small trees.
// 33 and 50 nodes over 2,000 entries a head (32/8 heads, 8 layers) take 1.36 ms
// with D = 128 and 0.79 with D = 64; in tiles of 64 rows 1.46 and 0.87; 3 and 5
// nodes of D = 64 0.17 and 0.26.
constexpr int R = 2, T = 256, TREE_ROWS = T / 16 * R;

// What key a row of a key tile is.
constexpr int32_t KEY_CACHE = -1, KEY_NONE = -2;  // >= 0: drafted token

// One CTA per (head, 32 rows, part of the keys).  The keys of a head are its
// cache pages and then its drafted tokens in groups of 16; a tile of 64 is four
// of either.  Parts of one (head, rows) meet through records in the workspace:
// the last to arrive joins them in ascending order, so the result does not
// depend on which one that is.
template <int D>
__global__ void __launch_bounds__(T) tree_ffma_kernel(const TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    FTile<D, TREE_ROWS> &t = *reinterpret_cast<FTile<D, TREE_ROWS> *>(smem);
    int32_t *s_cu = reinterpret_cast<int32_t *>(smem + sizeof(FTile<D, TREE_ROWS>));
    constexpr int ROWS = TREE_ROWS;
    __shared__ unsigned long long s_mask[64];
    // what the rows of three key tiles are: of the one that is worked on, the one
    // whose K and V are on their way, and the one that is being looked up
    __shared__ int32_t s_key[3][FT_KEYS];
    __shared__ const float *s_k[3][FT_KEYS], *s_v[3][FT_KEYS];
    __shared__ int s_some[3][2];
    __shared__ int s_last;
    if (!load_offsets(a.cu, a.B, a.n_tokens, a.max_nodes, s_cu, a.status)) return;
    const int part = blockIdx.x % a.parts, item = blockIdx.x / a.parts;
    const int c = item / a.row_tiles, r0 = item % a.row_tiles * ROWS;
    const int b = c / a.LH, lh = c % a.LH, G = a.G;
    const int t0 = s_cu[b], nodes = s_cu[b + 1] - t0, rows = nodes * G;
    if (r0 >= rows) return;
    const int m = clamp_len(__ldg(a.len + c), a.max_pages, a.status);
    const int np = (m + PAGE - 1) / PAGE, tiles = (np + (nodes + PAGE - 1) / PAGE + 3) / 4;
    if (threadIdx.x < nodes) s_mask[threadIdx.x] = __ldg(a.mask + t0 + threadIdx.x);
    constexpr int V4 = D / 4;
    const float *q = static_cast<const float *>(a.q);
    for (int i = threadIdx.x; i < ROWS * V4; i += T) {
        const int r = r0 + i / V4, d = i % V4 * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) x = ld4(q + ((int64_t)(t0 + r / G) * a.LH * G + lh * G + r % G) * D + d);
        *reinterpret_cast<float4 *>(&t.q[i / V4][d]) = x;
    }
    FState<D, R> st;
    st.init();
    const int begin = (int)((int64_t)tiles * part / a.parts), last = (int)((int64_t)tiles * (part + 1) / a.parts);
    // row threadIdx.x of tile j: its page and keep word first, its place afterwards
    int32_t page = -1;
    uint32_t word = 0xFFFFu;
    auto fetch = [&](int j) {
        const int u = j * 4 + threadIdx.x / PAGE;
        if (threadIdx.x >= FT_KEYS || u >= np) return;
        page = __ldg(a.block_table + (int64_t)c * a.max_pages + u);
        if (a.keep_mask) word = __ldg(a.keep_mask + (int64_t)c * a.max_pages + u);
    };
    auto find = [&](int j) {
        if (threadIdx.x >= FT_KEYS) return;
        const int u = j * 4 + threadIdx.x / PAGE, off = threadIdx.x % PAGE, buf = j % 3;
        int32_t kind = KEY_NONE;
        const float *kr = nullptr, *vr = nullptr;
        if (u < np) {
            if (!(word >> off & 1) || u * PAGE + off >= m) {
                // does not count: its page, if it is none, is not looked at either
            } else if (page < 0 || page >= a.n_pages) {
                set_status(a.status, RKV_DEV_BAD_INPUT);
            } else {
                kind = KEY_CACHE;
                kr = static_cast<const float *>(a.k_pool) + ((int64_t)page * PAGE + off) * D;
                vr = static_cast<const float *>(a.v_pool) + ((int64_t)page * PAGE + off) * D;
            }
        } else {
            const int i = (u - np) * PAGE + off;
            if (i < nodes) {
                kind = i;
                kr = static_cast<const float *>(a.k_draft) + ((int64_t)(t0 + i) * a.LH + lh) * D;
                vr = static_cast<const float *>(a.v_draft) + ((int64_t)(t0 + i) * a.LH + lh) * D;
            }
        }
        s_key[buf][threadIdx.x] = kind;
        s_k[buf][threadIdx.x] = kr;
        s_v[buf][threadIdx.x] = vr;
        const bool some = __any_sync(0xFFFFFFFFu, kind != KEY_CACHE);
        if ((threadIdx.x & 31) == 0) s_some[buf][threadIdx.x >> 5] = some;
    };
    constexpr int N = FT_KEYS * V4 / T;
    float4 kr[N], vr[N];
    auto load = [&](int j) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int e = i * T + threadIdx.x, r = e / V4, d = e % V4 * 4;
            const float *kp = s_k[j % 3][r], *vp = s_v[j % 3][r];
            kr[i] = kp ? ld4(kp + d) : make_float4(0.f, 0.f, 0.f, 0.f);
            vr[i] = kp ? ld4(vp + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    if (begin < last) {
        fetch(begin);
        find(begin);
        fetch(begin + 1);
        find(begin + 1);
        __syncthreads();
        load(begin);
    }
    for (int j0 = begin; j0 < last; j0++) {
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
        if (j0 + 1 < last) load(j0 + 1);
        if (j0 + 2 < last) fetch(j0 + 2);
        const int buf = j0 % 3;
        ftile_step<D, R, ROWS>(t, st, a.qscale, (s_some[buf][0] | s_some[buf][1]) != 0, odd != 0, [&](int row, int key) {
            const int32_t kind = s_key[buf][key];
            if (kind == KEY_CACHE) return false;
            const int node = (r0 + row) / G;
            return kind == KEY_NONE || node >= nodes || !(s_mask[node] >> kind & 1ull);
        });
        if (j0 + 2 < last) find(j0 + 2);
    }
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    constexpr int REC = ROWS * (D + 2);  // per part: output sums, then maxima and sums
    if (a.parts > 1) {
        float *rec = a.rec + ((int64_t)item * a.parts + part) * REC;
#pragma unroll
        for (int i = 0; i < R; i++) {
            const int r = ty * R + i;
#pragma unroll
            for (int j = 0; j < D / 64; j++)
                st4(rec + r * D + tx * 4 + 64 * j, make_float4(st.o[i][4 * j], st.o[i][4 * j + 1], st.o[i][4 * j + 2],
                                                               st.o[i][4 * j + 3]));
            if (tx == 0) {
                rec[ROWS * D + r] = st.m[i];
                rec[ROWS * D + ROWS + r] = st.l[i];
            }
        }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_last = atomicAdd(a.ticket + item, 1u) == (uint32_t)a.parts - 1u;
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        if (threadIdx.x == 0) a.ticket[item] = 0u;
        st.init();
        for (int p = 0; p < a.parts; p++) {
            const float *rp = a.rec + ((int64_t)item * a.parts + p) * REC;
#pragma unroll
            for (int i = 0; i < R; i++) {
                const int r = ty * R + i;
                const float mp = __ldcg(rp + ROWS * D + r), lp = __ldcg(rp + ROWS * D + ROWS + r);
                const float mn = fmaxf(st.m[i], mp), ms = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(st.m[i] - ms), g = exp2f(mp - ms);
                st.m[i] = mn;
                st.l[i] = st.l[i] * f + lp * g;
#pragma unroll
                for (int j = 0; j < D / 64; j++) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(rp + r * D + tx * 4 + 64 * j));
                    st.o[i][4 * j + 0] = st.o[i][4 * j + 0] * f + x.x * g;
                    st.o[i][4 * j + 1] = st.o[i][4 * j + 1] * f + x.y * g;
                    st.o[i][4 * j + 2] = st.o[i][4 * j + 2] * f + x.z * g;
                    st.o[i][4 * j + 3] = st.o[i][4 * j + 3] * f + x.w * g;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int r = r0 + ty * R + i;
        if (r >= rows) continue;
        const int64_t at = (int64_t)(t0 + r / G) * a.LH * G + lh * G + r % G;
        float *o = static_cast<float *>(a.out) + at * D;
        const bool none = st.m[i] == -INFINITY && st.l[i] == 0.f;
        const float inv = none ? 0.f : 1.f / st.l[i];
#pragma unroll
        for (int j = 0; j < D / 64; j++)
            st4(o + tx * 4 + 64 * j, make_float4(st.o[i][4 * j] * inv, st.o[i][4 * j + 1] * inv,
                                                 st.o[i][4 * j + 2] * inv, st.o[i][4 * j + 3] * inv));
        if (a.lse && tx == 0) a.lse[at] = none ? -INFINITY : (st.m[i] + log2f(st.l[i])) * LN2;
    }
}

template <int D>
cudaError_t launch_ffma(const TreeArgs &a, cudaStream_t s) {
    const size_t smem = sizeof(FTile<D, TREE_ROWS>) + (size_t)(a.B + 1) * 4;
    cudaError_t e = cudaFuncSetAttribute(tree_ffma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (int64_t)a.C * a.row_tiles * a.parts;
    if (ctas >= (1ll << 31)) return cudaErrorNotSupported;
    tree_ffma_kernel<D><<<(unsigned)ctas, T, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Parts of each (head, rows): enough for two CTAs on each of the 148 SMs when
// there are few of them, up to 16.
static int ffma_parts(int64_t items) {
    const int64_t p = (295 + items) / items;
    return (int)(p > 16 ? 16 : p);
}

TreeLayout tree_layout(int dtype, int D, int G, int64_t C, int max_nodes) {
    TreeLayout L{};
    if (dtype == RKV_BF16) {
        L.nt = 128 / G < max_nodes ? 128 / G : max_nodes;
        L.rec_tiles = max_nodes > L.nt ? 2 : 1;
        L.head_bytes = TREE_CTAS * sizeof(int4);
        // a CTA's range begins and ends inside an item at most: two records
        L.rec_floats = (size_t)TREE_CTAS * 2 * L.rec_tiles * 128 * (D + 2);
        return L;
    }
    L.row_tiles = (max_nodes * G + TREE_ROWS - 1) / TREE_ROWS;
    const int64_t items = C * L.row_tiles;
    L.parts = ffma_parts(items);
    // as many tickets for every max_nodes: calls of different sizes share a
    // workspace, and a record of one must not land on another's (zeroed) tickets
    L.head_bytes = (size_t)C * ((TREE_MAX_NODES * G + TREE_ROWS - 1) / TREE_ROWS) * 4;
    L.rec_floats = L.parts > 1 ? (size_t)items * L.parts * TREE_ROWS * (D + 2) : 0;
    return L;
}

cudaError_t launch_tree(const TreeArgs &a, int D, cudaStream_t s) {
    return D == 64 ? launch_ffma<64>(a, s) : launch_ffma<128>(a, s);
}

}  // namespace rkv
