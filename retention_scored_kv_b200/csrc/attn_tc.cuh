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

// Code size matters in these kernels: their roles run at the same time and share
// the SM's instruction cache.  Measured in the tree kernel: 96 KB with everything
// unrolled and inlined, 59 % of fetches hit and masked tiles took 5 times as
// long; 72 KB, 93 % hit.  Hence the rolled loops, single instances of the large
// pieces and the calls that are kept out of line.

// Bounded wait on an mbarrier phase for warps that wait beside computing ones:
// try_wait with a time hint suspends the warp until the phase ends, where polling
// would take issue slots from the softmax warps.
__device__ __forceinline__ bool try_wait_hint(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}
static __device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, int32_t *status, int site) {
    for (int i = 0; i < 2000; i++)
        if (try_wait_hint(bar, parity)) return true;
    return mbar_wait(bar, parity, status, site);
}
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, int32_t *status, int site) {
    return try_wait_hint(bar, parity) || wait_on(bar, parity, status, site);
}

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

// The largest of three; NaN if any is.  (Three operands at the rate of two.)
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// ex2 that stays where it is written among its like.
__device__ __forceinline__ float ex2_in_order(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// -inf where the bit of `in` is clear.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], uint32_t in) {
#pragma unroll
    for (int e = 0; e < 32; e++) s[e] = in & (1u << e) ? s[e] : 0xFF800000u;
}

// The largest of 32 scores and mx; NaN if any is.
__device__ __forceinline__ float max32(const uint32_t (&s)[32], float mx) {
    float a[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; e += 8)
#pragma unroll
        for (int i = 0; i < 4; i++)
            a[i] = max_nan(a[i], __uint_as_float(s[e + 2 * i]), __uint_as_float(s[e + 2 * i + 1]));
    return max_nan(max_nan(a[0], a[1], a[2]), a[3], a[3]);
}

// 32 scores to weights 2^(s * qscale - ref): bf16 over the scores' place, fp32
// into the sums.  The rounding puts each weight off by at most 2^-8 of itself,
// and the result by at most 2^-8 sum p |v|, as much as the result's own rounding
// where the v agree in sign: measured against 64 bits 1.9e-3 of the result's norm
// in all, where the result's rounding alone gives 1.4e-3.  A second product with
// the weights' low halves would take the tensor pipe half as long again.
// All exponentials go to the special function unit: a quarter or an eighth of
// them as polynomials on the FMA pipe measured no faster (8K prompts 2.99 ms
// without, 3.03 with), since the waits between roles bound the loop.
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], uint32_t tp, float qscale, float ref, float2 (&sum)[2]) {
    const float2 qs = make_float2(qscale, qscale), mm = make_float2(-ref, -ref);
    constexpr int LAG = 4;  // pairs between an exponential and its use: the unit's latency
    float2 z[16];
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16 + LAG; e++) {
        if (e < 16) {
            const float2 x = ffma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), qs, mm);
            z[e].x = ex2_in_order(x.x);
            z[e].y = ex2_in_order(x.y);
        }
        if (e >= LAG) {
            sum[e & 1] = fadd2(sum[e & 1], z[e - LAG]);
            p[e - LAG] = pack_bf16(z[e - LAG].x, z[e - LAG].y);
        }
    }
    tmem_st16(tp, p);
}

// One row's S of a key tile to P.  m: the row's reference maximum of the raw
// scores (-inf: nothing seen), l: the sum of its fp32 weights so far.  The
// output is rescaled only when the maximum has grown by more than RESCALE: the
// weights then stay below 2^RESCALE, far inside fp32 and bf16 range.  A NaN
// score, or one of +inf, makes the maximum and so the whole row NaN.
// S is read twice, 32 columns at a time, once for the maximum and once for the
// weights, instead of being held in 128 registers.  P of columns 32c..+31 lies
// over S's 16c..+15, which are read by then.  P is handed on in halves (p_full[0],
// [1]), so that the product of the first runs under the exponentials of the
// second.  masked: mask(c) gives the columns of 32c..+31 that count, and the rest
// become -inf in S.  done() waits for the product of the previous tile (a bounded
// wait: false gives up).
template <int D, class Mask, class Done>
__device__ __forceinline__ bool softmax_tile(uint32_t ts, uint32_t to, bool first, float qscale, float &m, float &l,
                                             uint64_t *p_full, bool masked, Mask mask, Done done) {
    uint32_t a[32], b[32];
    float mt = -INFINITY;
    auto look = [&](int c, uint32_t(&s)[32]) {
        if (masked) {
            const uint32_t in = mask(c);
            if (!__all_sync(0xFFFFFFFFu, in == 0xFFFFFFFFu)) {
                mask32(s, in);
                tmem_st32(ts + c * 32, s);
            }
        }
        mt = max32(s, mt);
    };
    tmem_ld32(a, ts);
#pragma unroll 1
    for (int c = 0; c < 4; c += 2) {
        tmem_wait_ld32(a);
        tmem_ld32(b, ts + (c + 1) * 32);
        look(c, a);
        tmem_wait_ld32(b);
        if (c == 0) tmem_ld32(a, ts + 64);
        look(c + 1, b);
    }
    if (masked) tmem_wait_st();
    tmem_ld32(a, ts);
    const bool grow = first || !((mt - m) * qscale <= RESCALE || mt == -INFINITY);
    if (__any_sync(0xFFFFFFFFu, grow)) {
        // O is read and written by warps; a row that need not stays as it is, so
        // that its result does not depend on the rows beside it
        float mn = grow ? max_nan(m, mt, mt) : m;
        if (mn == INFINITY) mn = NAN;
        if (!first) {
            const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * qscale);
            l *= f;
            if (!done()) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                tmem_ld32(b, to + c);
                tmem_wait_ld32(b);
#pragma unroll
                for (int e = 0; e < 32; e++) b[e] = __float_as_uint(__uint_as_float(b[e]) * f);
                tmem_st32(to + c, b);
            }
        }
        m = mn;
    }
    const float ref = m == -INFINITY ? 0.f : m * qscale;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
    for (int c = 0; c < 4; c += 2) {
        tmem_wait_ld32(a);
        tmem_ld32(b, ts + (c + 1) * 32);
        weights32(a, ts + c * 16, qscale, ref, sum);
        tmem_wait_ld32(b);
        if (c == 0) tmem_ld32(a, ts + 64);
        weights32(b, ts + c * 16 + 16, qscale, ref, sum);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(p_full + (c >> 1));
    }
    sum[0] = fadd2(sum[0], sum[1]);
    l += sum[0].x + sum[0].y;
    return true;
}

// 16 bytes of V without their infinite and NaN values (exponent field all ones);
// true if there were any.
__device__ __forceinline__ bool drop_odd(uint4 &v) {
    uint32_t bad = 0, *p = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int e = 0; e < 4; e++) {
        // adding one to an all-ones field carries into the bit above it
        const uint32_t m = ((p[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
        bad |= m;
        p[e] &= ~((m >> 15) * 0xFFFFu);
    }
    return bad != 0;
}

// 16 columns of a warp's 32 rows of bf16 results, lane i's row at out + at (where
// `here`): through shared memory, so that a store instruction writes 32 bytes of
// 16 rows instead of 16 bytes of 32.  Whole warp.
__device__ __forceinline__ void store_rows(uint4 *stage, __nv_bfloat16 *out, int64_t at, uint32_t rows, const float (&f)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 2; e++)  // a row's two pieces change places in every second group of four rows: no bank conflicts
        stage[lane * 2 + (e ^ (lane >> 2 & 1))] =
            make_uint4(pack_bf16(f[8 * e], f[8 * e + 1]), pack_bf16(f[8 * e + 2], f[8 * e + 3]),
                       pack_bf16(f[8 * e + 4], f[8 * e + 5]), pack_bf16(f[8 * e + 6], f[8 * e + 7]));
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 2; r++) {
        const int row = r * 16 + lane / 2;
        const int64_t to = __shfl_sync(0xFFFFFFFFu, at, row);
        const uint4 v = stage[row * 2 + ((lane & 1) ^ (row >> 2 & 1))];
        if (rows >> row & 1) *reinterpret_cast<uint4 *>(out + to + (lane & 1) * 8) = v;
    }
    __syncwarp();
}

// Add the infinite and NaN values of one row of V, which the tensor core was not
// shown, to columns [lo, hi) of this lane's row of O (`sees`: the row attends it).
// Whole warp; rare, and kept out of line.
template <int D>
static __device__ __noinline__ void add_odd(uint32_t to, const __nv_bfloat16 *v, bool sees, int lo = 0, int hi = D) {
#pragma unroll 1
    for (int c = lo; c < hi; c++) {
        const float f = __bfloat162float(v[c]);
        const bool odd = sees && !(fabsf(f) < INFINITY);
        if (!__any_sync(0xFFFFFFFFu, odd)) continue;
        uint32_t o;
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(o) : "r"(to + c));
        asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(o)::"memory");
        if (odd) o = __float_as_uint(__uint_as_float(o) + f);
        __syncwarp();
        asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(to + c), "r"(o) : "memory");
        tmem_wait_st();
    }
}

}  // namespace rkv
