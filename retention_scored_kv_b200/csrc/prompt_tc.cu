// prompt_tc.cu -- rkv_prompt_attn on bf16: both products on the fifth-
// generation tensor cores, accumulators in tensor memory.
//
// A CTA works on 256 query rows of one query head: two tiles of 128 rows (one
// tensor-memory lane a row) against the same key tiles of 128.  Per key tile
//   S_i = Q_i K^T        (128 x 128, tensor memory)
//   P_i = exp(S_i - m_i) (warpgroup i: one thread a row, bf16 over S's columns)
//   O_i += P_i V         (128 x D, tensor memory; P as the left operand)
// While warpgroup 0 turns S_0 into P_0 the tensor core runs S_1, O_1 and back:
// the exponentials of a tile (128 x 128 over 16 a cycle) take as long as its two
// products, so the two have to overlap.
//
// Measured (one B200, 32/8 heads of 128): one prompt of 32,768 tokens 8.06 ms,
// 1,090 TFLOP/s, 66 % of the measured burst rate of bf16 products and 80 % of the
// sustained one (the board runs at its power cap, near 1.6 GHz); 8,192 tokens
// 0.52 ms.  The tensor pipe and the special function unit are busy 55 % each.
//
// Warps 0-3 and 4-7: softmax of tile 0 and 1, and the output.  Warp 8: TMA loads
// through a ring of shared-memory slots, and the next piece of work.  Warp 9:
// issues the products.  Warps 10, 11: V of the last two key tiles of a piece of
// work, before the tensor core reads it: rows past the sequence's end become
// zero and infinite or NaN values (which would reach rows that do not attend
// them, as 0 * NaN) too; the output adds the latter for the rows that do.
#include "attn_tc.cuh"

namespace rkv {
namespace {

template <int D>
struct Cfg {
    static constexpr int TILE = TcCfg<D>::TILE, PLANE = TcCfg<D>::PLANE;
    static constexpr int SLOTS = D == 128 ? 4 : 8;         // K and V tiles in flight (five measure the same)
    static constexpr int SMEM = (2 + SLOTS) * TILE + 1024; // two query tiles; alignment of the swizzle's period
};

// A piece of work.
struct Work {
    int b, blk, hq, odd;  // odd: bit t: V of the t-th of the last two key tiles held infinities or NaN
    int t0, n;            // first token and length of the sequence
};

struct Shared {
    uint64_t full[8], empty[8];            // K / V slots
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2][2], o_done[2], o_free[2];  // p_full: by halves of the keys
    uint64_t v_last[8], v_ready[8];        // a slot's V of the last key tiles: loaded, and mended (full is not used)
    uint64_t w_full[2], w_empty[2];        // pieces of work
    Work work[2];
    uint4 stage[8][32 * 2];                // results of a warp's rows, 16 columns
    uint32_t tmem;
};

// What a piece of work consists of: key tiles of each query tile.
struct Shape {
    int nk0, nk1, nk;
    __device__ Shape(int blk, int n) {
        nk0 = 2 * blk + 1;
        nk1 = nk0 * QR < n ? nk0 + 1 : 0;
        nk = nk1 ? nk1 : nk0;
    }
};

template <int D>
struct Ctx {
    Shared *sh;
    unsigned char *q, *kv;
    int32_t *status;
    __device__ bool wait(uint64_t *bar, uint32_t parity, int site) const { return tc_wait(bar, parity, status, site); }
    __device__ unsigned char *slot(int i) const { return kv + (size_t)i * Cfg<D>::TILE; }
};

// ------------------------------------------------------------ warp 8: loads ----
template <int D>
__device__ void load_role(const Ctx<D> &x, const PromptArgs &a, const CUtensorMap *tq, const CUtensorMap *tk,
                          const CUtensorMap *tv) {
    using C = Cfg<D>;
    const int lane = threadIdx.x & 31, G = a.Hq / a.H;
    const int total = tiles_from(a.cu, a.B, 2 * QR, 0) * a.Hq;
    Ring kv, w;
    uint32_t q_turn[2] = {0, 0};
    for (;; w.next(2)) {
        int tile = 0;
        if (lane == 0) tile = (int)atomicAdd(a.next, 1u);
        tile = __shfl_sync(0xFFFFFFFFu, tile, 0);
        const bool end = tile >= total;
        SeqTile t{-1, 0};
        if (!end) t = find_tile(a.cu, a.B, a.n_tokens, 2 * QR, tile / a.Hq);
        int ok = 1;
        if (lane == 0) {
            ok = x.wait(&x.sh->w_empty[w.slot], w.turn ^ 1u, 0x400);
            Work wk{t.b, t.blk, tile % a.Hq, 0, 0, 0};
            if (!end) {
                wk.t0 = a.cu[t.b];
                wk.n = a.cu[t.b + 1] - wk.t0;
            }
            if (ok) {
                x.sh->work[w.slot] = wk;
                mbar_arrive(&x.sh->w_full[w.slot]);
            }
            if (ok && !end) {
                const Shape s(wk.blk, wk.n);
                const int h = wk.hq / G, planes = D / 64;
                auto query = [&](int i) {
                    if (!x.wait(&x.sh->q_empty[i], q_turn[i] ^ 1u, 0x401)) return false;
                    q_turn[i] ^= 1u;
                    mbar_arrive_expect_tx(&x.sh->q_full[i], C::TILE);
                    tma_tile(x.q + i * C::TILE, tq, 0, wk.t0 + (2 * wk.blk + i) * QR, wk.hq * planes, &x.sh->q_full[i]);
                    return true;
                };
                auto tile_of = [&](const CUtensorMap *m, int j) {
                    if (!x.wait(&x.sh->empty[kv.slot], kv.turn ^ 1u, 0x402)) return false;
                    uint64_t *bar = m == tv && j >= 2 * wk.blk ? &x.sh->v_last[kv.slot] : &x.sh->full[kv.slot];
                    mbar_arrive_expect_tx(bar, C::TILE);
                    tma_tile(x.slot(kv.slot), m, 0, wk.t0 + j * KR, h * planes, bar);
                    kv.next(C::SLOTS);
                    return true;
                };
                ok = query(0) && tile_of(tk, 0) && (!s.nk1 || query(1)) && tile_of(tv, 0);
                for (int j = 1; ok && j < s.nk; j++) ok = tile_of(tk, j) && tile_of(tv, j);
            }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok || end) return;
    }
}

// ---------------------------------------------------------- warp 9: products ----
// S = Q K^T into tensor memory.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t s, uint64_t q, uint64_t k, uint32_t idesc) {
#pragma unroll
    for (int e = 0; e < D / 16; e++) {
        const uint32_t off = (e / 4) * Cfg<D>::PLANE + (e % 4) * 32;
        mma_ss(s, desc_at(q, off), desc_at(k, off), idesc, e > 0);
    }
}

// O (+)= P V over half of the keys.
template <int D>
__device__ __forceinline__ void mma_output(uint32_t o, uint32_t p, uint64_t v, uint32_t idesc, int half, bool first) {
    p += half * 32;
    v = desc_at(v, half * 64 * 128);
#pragma unroll
    for (int e = 0; e < 4; e++) mma_ts(o, p + e * 8, desc_at(v, e * 2048), idesc, e > 0 || !first);
}

template <int D>
__device__ void mma_role(const Ctx<D> &x, bool neg) {
    using C = Cfg<D>;
    Shared *sh = x.sh;
    const uint32_t tmem = sh->tmem;
    const uint32_t qk = mma_desc(QR, KR, false, neg), pv = mma_desc(QR, D, true, false);
    Ring kv, w;
    uint32_t q_turn = 0, p_turn = 0, f_turn = 0;  // q_full, p_full, o_free: a bit for each tile
    uint32_t kv_turn = 0, v_turn = 0;             // full, v_ready: a bit for each slot
    const uint64_t q_desc = tile_desc(smem_u32(x.q), 16), k_desc = tile_desc(smem_u32(x.kv), 16),
                   v_desc = tile_desc(smem_u32(x.kv), C::PLANE);
    for (;; w.next(2)) {
        if (!x.wait(&sh->w_full[w.slot], w.turn, 0x410)) return;
        const int b = sh->work[w.slot].b, blk = sh->work[w.slot].blk, len = sh->work[w.slot].n;
        mbar_arrive(&sh->w_empty[w.slot]);
        if (b < 0) return;
        const Shape s(blk, len);
        // step j: O_i += P_i V of key tile j - 1, then S_i of key tile j
        for (int j = 0; j <= s.nk; j++) {
            int vslot = 0;
            if (j > 0) {
                vslot = kv.slot;
                if (j - 1 >= 2 * blk) {
                    if (!x.wait(&sh->v_ready[vslot], v_turn >> vslot & 1u, 0x413)) return;
                    v_turn ^= 1u << vslot;
                } else {
                    if (!x.wait(&sh->full[vslot], kv_turn >> vslot & 1u, 0x414)) return;
                    kv_turn ^= 1u << vslot;
                }
                kv.next(C::SLOTS);
            }
            const int kslot = kv.slot;
            bool k_here = false;
#pragma unroll 1
            for (int i = 0; i < 2; i++) {
                const int nk = i ? s.nk1 : s.nk0;
                if (j > nk) continue;
                const uint32_t o = tmem + TM_O + i * D, p = tmem + TM_S + i * 128;
                if (j > 0) {
                    if (j == 1) {
                        if (!x.wait(&sh->o_free[i], (f_turn >> i & 1u) ^ 1u, 0x415)) return;
                        f_turn ^= 1u << i;
                    }
                    const uint64_t v = desc_at(v_desc, vslot * C::TILE);
                    if (!x.wait(&sh->p_full[i][0], p_turn >> i & 1u, 0x416)) return;
                    tc_fence_after();
                    mma_output<D>(o, p, v, pv, 0, j == 1);
                    if (!x.wait(&sh->p_full[i][1], p_turn >> i & 1u, 0x418)) return;
                    p_turn ^= 1u << i;
                    tc_fence_after();
                    mma_output<D>(o, p, v, pv, 1, false);
                    mma_commit(&sh->o_done[i]);
                } else if (nk > 0) {
                    if (!x.wait(&sh->q_full[i], q_turn >> i & 1u, 0x412)) return;
                    q_turn ^= 1u << i;
                }
                if (j < nk) {
                    if (!k_here) {
                        if (!x.wait(&sh->full[kslot], kv_turn >> kslot & 1u, 0x417)) return;
                        kv_turn ^= 1u << kslot;
                        k_here = true;
                    }
                    tc_fence_after();
                    mma_scores<D>(p, desc_at(q_desc, i * C::TILE), desc_at(k_desc, kslot * C::TILE), qk);
                    mma_commit(&sh->s_full[i]);
                    if (j + 1 == nk) mma_commit(&sh->q_empty[i]);
                }
            }
            if (j > 0) mma_commit(&sh->empty[vslot]);
            if (j < s.nk) {
                mma_commit(&sh->empty[kslot]);
                kv.next(C::SLOTS);
            }
        }
    }
}

// ------------------------------------------------- warps 10, 11: V's last tiles ----
template <int D>
__device__ void mend_role(const Ctx<D> &x) {
    using C = Cfg<D>;
    Shared *sh = x.sh;
    const int t = threadIdx.x - 320;
    Ring kv, w;
    uint32_t turn = 0;  // v_last: a bit for each slot
    for (;; w.next(2)) {
        if (!x.wait(&sh->w_full[w.slot], w.turn, 0x420)) return;
        const Work wk = sh->work[w.slot];
        if (wk.b >= 0) {
            const Shape s(wk.blk, wk.n);
            for (int j = 0; j < s.nk; j++) {
                kv.next(C::SLOTS);  // K
                if (j >= 2 * wk.blk) {
                    if (!x.wait(&sh->v_last[kv.slot], turn >> kv.slot & 1u, 0x421)) return;
                    turn ^= 1u << kv.slot;
                    const int rows = wk.n - j * KR;  // rows of the sequence from here on
                    uint4 *tile = reinterpret_cast<uint4 *>(x.slot(kv.slot));
                    uint32_t odd = 0;
                    for (int i = t; i < C::TILE / 16; i += 64) {
                        const int row = (i >> 3) & 127;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (row < rows) {
                            v = tile[i];
                            if (!drop_odd(v)) continue;
                            odd = 1;
                        }
                        tile[i] = v;
                    }
                    if (odd) atomicOr(&sh->work[w.slot].odd, 1 << (j - 2 * wk.blk));
                    fence_async_shared();
                    __syncwarp();
                    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->v_ready[kv.slot]);
                }
                kv.next(C::SLOTS);  // V
            }
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->w_empty[w.slot]);
        if (wk.b < 0) return;
    }
}

// ------------------------------------------------------ warps 0-7: softmax ----
template <int D>
__device__ void softmax_role(const Ctx<D> &x, const PromptArgs &a) {
    Shared *sh = x.sh;
    const int i = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(row & 96) << 16;
    const uint32_t ts = sh->tmem + TM_S + i * 128 + lanes, to = sh->tmem + TM_O + i * D + lanes;
    const float qscale = fabsf(a.qscale);
    uint32_t s_turn = 0, d_turn = 0;  // d_turn: parity of the next product to complete
    Ring w;
    for (;; w.next(2)) {
        if (!x.wait(&sh->w_full[w.slot], w.turn, 0x431)) return;
        const Work wk = sh->work[w.slot];
        if (wk.b < 0) return;
        const Shape sp(wk.blk, wk.n);
        const int nk = i ? sp.nk1 : sp.nk0;
        if (nk) {
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < nk; j++) {
                if (!x.wait(&sh->s_full[i], s_turn, 0x432)) return;
                s_turn ^= 1u;
                tc_fence_after();
                // the product of tile j - 1 has parity d_turn ^ 1 once tile j's is awaited
                auto done = [&] { return x.wait(&sh->o_done[i], d_turn ^ 1u, 0x430); };
                auto causal = [&](int c) {
                    const int last = row - c * 32;  // column of the row's own token
                    return last < 0 ? 0u : 0xFFFFFFFFu >> (31 - min(last, 31));
                };
                const bool ok = softmax_tile<D>(ts, to, j == 0, qscale, m, l, sh->p_full[i], j + 1 == nk, causal, done);
                if (!ok) return;
                d_turn ^= 1u;
            }
            if (!x.wait(&sh->o_done[i], d_turn ^ 1u, 0x433)) return;
            tc_fence_after();
            const int r = (2 * wk.blk + i) * QR + row;  // row of the sequence
            const int odd = *(volatile int *)&sh->work[w.slot].odd;
            const bool here = r < wk.n;
            const float inv = m == -INFINITY ? NAN : __fdividef(1.f, l);  // every score -inf: 0 / 0
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (int64_t)wk.hq * D;
            if (__any_sync(0xFFFFFFFFu, odd)) {
                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + (int64_t)(wk.hq / (a.Hq / a.H)) * D;
                for (int j = 2 * wk.blk * KR; j < min(wk.n, nk * KR); j++) add_odd<D>(to, v + (wk.t0 + j) * a.v_stride, j <= r);
            }
            const uint32_t rows = __ballot_sync(0xFFFFFFFFu, here);
            const int64_t at = (wk.t0 + (int64_t)r) * a.out_stride;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_read16(o, to + c);
                float f[16];
#pragma unroll
                for (int e = 0; e < 16; e++) f[e] = __uint_as_float(o[e]) * inv;
                store_rows(sh->stage[threadIdx.x >> 5], out + c, at, rows, f);
            }
            tc_fence_before();
            if (here && a.lse) a.lse[(wk.t0 + (int64_t)r) * a.Hq + wk.hq] = (m * qscale + __log2f(l)) * LN2;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->o_free[i]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->w_empty[w.slot]);
    }
}

template <int D>
__global__ void __launch_bounds__(TC_THREADS, 1) prompt_tc_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap tq,
                                                               const __grid_constant__ CUtensorMap tk,
                                                               const __grid_constant__ CUtensorMap tv) {
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) Shared sh;
    unsigned char *tiles = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 256) {
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < 8; s++) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
            mbar_init(&sh.v_last[s], 1);
            mbar_init(&sh.v_ready[s], 2);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 4);
            mbar_init(&sh.p_full[i][1], 4);
            mbar_init(&sh.o_done[i], 1);
            mbar_init(&sh.o_free[i], 4);
            mbar_init(&sh.w_full[i], 1);
            mbar_init(&sh.w_empty[i], 11);  // products, eight softmax warps, two mending warps
        }
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&sh.tmem, TM_COLS);
    const bool ok = load_offsets(a.cu, a.B, a.n_tokens, a.n_tokens, nullptr, a.status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Ctx<D> x{&sh, tiles, tiles + 2 * Cfg<D>::TILE, a.status};
    if (ok) {
        if (warp < 8) softmax_role<D>(x, a);
        else if (warp == 8) load_role<D>(x, a, &tq, &tk, &tv);
        else if (warp > 9) mend_role<D>(x);
        else if (elect_one()) mma_role<D>(x, a.qscale < 0.f);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(sh.tmem, TM_COLS);
    }
    // the last CTA to leave puts the counters back
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(a.next + 1, 1u) == gridDim.x - 1) {
            a.next[0] = 0u;
            a.next[1] = 0u;
        }
    }
}

template <int D>
cudaError_t launch(const PromptArgs &a, int sms, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                   cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)(a.n_tokens / (2 * QR) + a.B) * a.Hq;  // upper bound
    prompt_tc_kernel<D><<<(unsigned)(tiles < sms ? tiles : sms), TC_THREADS, Cfg<D>::SMEM, s>>>(a, tq, tk, tv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_tc(const PromptArgs &a, int D, int sms, const CUtensorMap &tq, const CUtensorMap &tk,
                             const CUtensorMap &tv, cudaStream_t s) {
    return D == 64 ? launch<64>(a, sms, tq, tk, tv, s) : launch<128>(a, sms, tq, tk, tv, s);
}

}  // namespace rkv
