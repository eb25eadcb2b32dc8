// attn_tc.cuh -- the part of the tensor-core attention kernels (prompt_tc.cu,
// tree_tc.cu) that is the same: a tile of 128 query rows against 128 keys, one
// tensor-memory lane a row, with the running maximum and sum of the softmax.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "serve.cuh"
#include "tc5.cuh"

namespace rkv {

constexpr int QR = 128, KR = 128;   // rows of a query tile, of a key tile
constexpr int TC_THREADS = 384;     // 8 softmax warps, 4 others
constexpr float RESCALE = 8.f;

// Tensor memory: scores of tile 0 and 1 (the weights replace them, two bf16 a
// column), then the outputs.
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;

template <int D>
struct TcCfg {
    static constexpr int TILE = 128 * D * 2;  // bytes of a tile
    static constexpr int PLANE = 128 * 128;   // 64 columns of it
};

// Position in a ring of n slots and the parity of the wait for its use.
struct Ring {
    int slot = 0;
    uint32_t turn = 0;
    __device__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            turn ^= 1;
        }
    }
};

// S = Q K^T into tensor memory.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t s, const void *q, const void *k, uint32_t idesc) {
    const uint32_t q0 = smem_u32(q), k0 = smem_u32(k);
#pragma unroll
    for (int e = 0; e < D / 16; e++) {
        const uint32_t off = (e / 4) * TcCfg<D>::PLANE + (e % 4) * 32;
        mma_ss(s, tile_desc(q0 + off, 16), tile_desc(k0 + off, 16), idesc, e > 0);
    }
}

// O (+)= P V.
template <int D>
__device__ __forceinline__ void mma_output(uint32_t o, uint32_t p, const void *v, uint32_t idesc, bool first) {
    const uint32_t v0 = smem_u32(v);
#pragma unroll
    for (int e = 0; e < KR / 16; e++)
        mma_ts(o, p + e * 8, tile_desc(v0 + e * 2048, TcCfg<D>::PLANE), idesc, !first || e > 0);
}

// One row's S of a key tile to P.  m: the row's reference maximum of the raw
// scores (-inf: nothing seen), l: the sum of its fp32 weights so far.  The
// output is rescaled only when the maximum has grown by more than RESCALE: the
// weights then stay below 2^RESCALE, far inside fp32 and bf16 range.  mask(s)
// sets scores to -inf; done() waits for the product of the previous tile (a
// bounded wait: false gives up).
template <int D, class Mask, class Done>
__device__ __forceinline__ bool softmax_tile(uint32_t ts, uint32_t to, bool first, float qscale, float &m, float &l,
                                             uint64_t *p_full, Mask mask, Done done) {
    uint32_t s[4][32];
#pragma unroll
    for (int c = 0; c < 4; c++) tmem_ld32(s[c], ts + c * 32);
#pragma unroll
    for (int c = 0; c < 4; c++) tmem_wait_ld32(s[c]);
    mask(s);
    float mx[4];
#pragma unroll
    for (int c = 0; c < 4; c++) {
        mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int e = 1; e < 32; e++) mx[c] = fmaxf(mx[c], __uint_as_float(s[c][e]));
    }
    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    if (__any_sync(0xFFFFFFFFu, first || (mt - m) * qscale > RESCALE)) {
        // the whole warp moves to its new maxima (O is read and written by warps)
        const float mn = fmaxf(m, mt);
        if (!first) {
            const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * qscale);
            l *= f;
            if (!done()) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(o, to + c);
                tmem_wait_ld32(o);
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(to + c, o);
            }
        }
        m = mn;
    }
    const float ref = m == -INFINITY ? 0.f : m * qscale;
    const float2 qs = make_float2(qscale, qscale), mm = make_float2(-ref, -ref);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int half = 0; half < 2; half++) {
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 32; e++) {
            const int c = half * 64 + 2 * e;
            float2 z = ffma2(make_float2(__uint_as_float(s[c / 32][c % 32]), __uint_as_float(s[c / 32][c % 32 + 1])), qs, mm);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            sum[e & 1] = fadd2(sum[e & 1], z);
            p[e] = pack_bf16(z.x, z.y);
        }
        tmem_st32(ts + half * 32, p);
    }
    sum[0] = fadd2(sum[0], sum[1]);
    l += sum[0].x + sum[0].y;
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(p_full);
    return true;
}

// 16 bytes of V without their infinite and NaN values; true if there were any.
__device__ __forceinline__ bool drop_odd(uint4 &v) {
    uint32_t bad = 0, *p = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t m = __vcmpeq2(p[e] & 0x7F807F80u, 0x7F807F80u);
        bad |= m;
        p[e] &= ~m;
    }
    return bad != 0;
}

// 32 columns of a row of bf16 results.
__device__ __forceinline__ void store32(__nv_bfloat16 *out, const float (&f)[32]) {
#pragma unroll
    for (int e = 0; e < 32; e += 8)
        *reinterpret_cast<uint4 *>(out + e) =
            make_uint4(pack_bf16(f[e], f[e + 1]), pack_bf16(f[e + 2], f[e + 3]), pack_bf16(f[e + 4], f[e + 5]),
                       pack_bf16(f[e + 6], f[e + 7]));
}

// Add the infinite and NaN values among 32 columns of one row of V, which the
// tensor core was not shown.
__device__ __forceinline__ void add_odd(float (&o)[32], const __nv_bfloat16 *v) {
#pragma unroll
    for (int e = 0; e < 32; e++) {
        const float f = __bfloat162float(v[e]);
        if (!(fabsf(f) < INFINITY)) o[e] += f;
    }
}

}  // namespace rkv
