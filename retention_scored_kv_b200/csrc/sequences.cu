// sequences.cu -- whole sequences in the paged cache: rkv_append_tokens (many
// tokens per sequence) and rkv_fork_sequences (copying, moving and freeing).
// Both move bytes; each is a plan launch (one scan over the heads decides
// which pages are taken and given back) and a launch that moves the rows.
#include "internal.h"
#include "serve.cuh"

namespace rkv {
namespace {

constexpr int PLAN_THREADS = 1024;

__device__ __forceinline__ int pages_of(int n) { return (n + PAGE - 1) / PAGE; }

// ---------------------------------------------------------------- append ----
// Plan: head c needs pages_of(len + n) - pages_of(len) new pages; heads pop in
// ascending order.  base[c] = its length before the call (-1: the head takes
// nothing), pop[c] = index of its first page on the free stack (later ones
// below it).  A head that would leave its table takes no page; one that finds
// too few pages is skipped, and so is every later head that needs one.  Each
// thread has a run of consecutive heads, so that one scan does for all.
__global__ void __launch_bounds__(PLAN_THREADS) append_plan_kernel(const AppendTokensArgs a) {
    extern __shared__ int32_t s_cu[];
    __shared__ uint32_t scan[33];
    __shared__ int s_short;
    launch_dependents();
    if (threadIdx.x == 0) {
        s_short = INT32_MAX;
        a.plan[0] = 0;
    }
    if (!load_offsets(a.cu, a.B, a.n_new, a.n_new, s_cu, a.status)) return;
    const int top = min(max(*a.free_top, 0), a.n_pages);
    const int per = (a.C + PLAN_THREADS - 1) / PLAN_THREADS, c0 = min(a.C, (int)threadIdx.x * per), c1 = min(a.C, c0 + per);
    // pages that head c needs; -1: the head takes nothing (bits: why)
    auto look = [&](int c, int &len, int &n, int &bits) {
        const int b = c / a.LH;
        n = s_cu[b + 1] - s_cu[b];
        len = a.len[c];
        bits = 0;
        if (n == 0) return -1;
        const int32_t p0 = __ldg(a.pos0 + b);
        if (len < 0 || p0 < 0 || (int64_t)p0 + n > INT32_MAX) bits = RKV_DEV_BAD_INPUT;
        else if ((int64_t)len + n > (int64_t)a.max_pages * PAGE) bits = RKV_DEV_TABLE_OVERFLOW;
        return bits ? -1 : pages_of(len + n) - pages_of(len);
    };
    uint32_t sum = 0, total;
    for (int c = c0; c < c1; c++) {
        int len, n, bits;
        sum += (uint32_t)max(0, look(c, len, n, bits));
    }
    uint32_t before = block_exclusive_scan(sum, scan, &total);
    for (int c = c0; c < c1; c++) {
        int len, n, bits;
        const int need = look(c, len, n, bits);
        if (need > 0 && (int64_t)before + need > (int64_t)top) {
            bits = RKV_DEV_POOL_EXHAUSTED;
            atomicMin(&s_short, (int)before);  // pages taken by the heads before the first that fails
        }
        const bool ok = need >= 0 && !bits;
        a.base[c] = ok ? len : -1;
        a.pop[c] = top - 1 - (int)before;
        if (ok) a.len[c] = len + n;
        if (bits) set_status(a.status, bits);
        before += (uint32_t)max(0, need);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *a.free_top = top - (int)min((uint32_t)s_short, total);
        a.plan[0] = 1;
    }
}

// A warp takes 32 tokens of one head; the warps of a CTA and the CTAs in order
// take neighbouring heads of the same tokens, whose rows are neighbours in k_new
// and v_new (in the order of one head's tokens the reads are 256 bytes in every
// 64 KB).  Lane i finds where token i goes (its page is in the table, or the
// head's next one on the stack, which is then entered in the table); the warp
// then copies the rows in 16-byte pieces.  15,653 tokens of 256 heads of 128 bf16
// (4.15 GB read and written) take 0.76 ms, 83 % of the measured copy rate (1.01 ms
// in the order of one head's tokens and with half the warps).
constexpr int MOVE_THREADS = 256;
template <int CH>  // 16-byte pieces of a row
__global__ void __launch_bounds__(MOVE_THREADS, 4) append_rows_kernel(const AppendTokensArgs a) {
    extern __shared__ int32_t s_cu[];  // offsets, then blocks of 32 tokens before each sequence
    __shared__ uint32_t scan[33];
    wait_for_launcher();
    if (a.plan[0] == 0) return;
    int32_t *s_pre = s_cu + a.B + 1;
    const int per = (a.B + MOVE_THREADS - 1) / MOVE_THREADS;
    const int q0 = min(a.B, (int)threadIdx.x * per), q1 = min(a.B, q0 + per);
    uint32_t sum = 0, blocks;
    for (int q = q0; q < q1; q++) sum += (uint32_t)(__ldg(a.cu + q + 1) - __ldg(a.cu + q) + 31) / 32;
    uint32_t pre = block_exclusive_scan(sum, scan, &blocks);
    for (int q = q0; q < q1; q++) {
        s_cu[q] = __ldg(a.cu + q);
        s_pre[q] = (int32_t)pre;
        pre += (uint32_t)(__ldg(a.cu + q + 1) - s_cu[q] + 31) / 32;
    }
    if (threadIdx.x == 0) s_cu[a.B] = __ldg(a.cu + a.B);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (MOVE_THREADS / 32), groups = (int64_t)blocks * a.LH;
    for (int64_t g = (int64_t)blockIdx.x * (MOVE_THREADS / 32) + (threadIdx.x >> 5); g < groups; g += warps) {
        const int block = (int)(g / a.LH), lh = (int)(g % a.LH);
        int b = 0, hi = a.B;  // the last sequence with s_pre <= block that is not empty
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (s_pre[mid] <= block) b = mid;
            else hi = mid;
        }
        const int j0 = (block - s_pre[b]) * 32, n = min(32, s_cu[b + 1] - s_cu[b] - j0);
        const int c = b * a.LH + lh, base = a.base[c];
        if (base < 0) continue;
        int64_t dst = -1, src = 0;
        if (lane < n) {
            const int j = j0 + lane, slot = base + j, p = slot / PAGE, have = pages_of(base);
            int64_t row = s_cu[b] + j;
            if (a.tok) row = __ldg(a.tok + row);
            int32_t *entry = a.block_table + (int64_t)c * a.max_pages + p;
            const int32_t page = p < have ? *entry : a.free_stack[a.pop[c] - (p - have)];
            if (p >= have && slot % PAGE == 0) *entry = page;
            if (page < 0 || page >= a.n_pages || row < 0 || row >= a.n_rows) {
                set_status(a.status, RKV_DEV_BAD_INPUT);
            } else {
                src = row * a.LH + lh;
                dst = (int64_t)page * PAGE + slot % PAGE;
                a.pos_pool[dst] = __ldg(a.pos0 + b) + j;
                a.lb_pool[dst] = __ldg(a.lb_new + src);
            }
        }
        constexpr int PER = 32 / CH, UN = 4;  // rows a warp moves at once, steps in flight
#pragma unroll 1
        for (int k0 = 0; k0 < n; k0 += PER * UN) {
            uint4 xk[UN], xv[UN];
            int64_t to[UN];
#pragma unroll
            for (int u = 0; u < UN; u++) {
                const int k = k0 + u * PER + lane / CH;
                to[u] = __shfl_sync(0xFFFFFFFFu, dst, k & 31);
                const int64_t from = __shfl_sync(0xFFFFFFFFu, src, k & 31);
                if (k >= 32) to[u] = -1;
                if (to[u] >= 0) {
                    xk[u] = __ldcs(static_cast<const uint4 *>(a.k_new) + from * CH + lane % CH);
                    xv[u] = __ldcs(static_cast<const uint4 *>(a.v_new) + from * CH + lane % CH);
                }
            }
#pragma unroll
            for (int u = 0; u < UN; u++)
                if (to[u] >= 0) {
                    static_cast<uint4 *>(a.k_pool)[to[u] * CH + lane % CH] = xk[u];
                    static_cast<uint4 *>(a.v_pool)[to[u] * CH + lane % CH] = xv[u];
                }
        }
    }
}

// ------------------------------------------------------------------ fork ----
// The slot that goes on with a sequence's own pages: the sequence's slot
// itself if it continues it, else the first slot that does.
__device__ __forceinline__ int heir_of(const int32_t *parent, int B, int s) {
    if (parent[s] == s) return s;
    for (int b = 0; b < B; b++)
        if (parent[b] == s) return b;
    return -1;
}

// Plan of the fork, and the pages of ended sequences pushed onto the stack.
// Every CTA scans all heads (how many pages each gives back and takes) and
// pushes the pages of its own share of them; CTA 0 writes the plan.
__global__ void __launch_bounds__(PLAN_THREADS) fork_plan_kernel(const ForkArgs a) {
    __shared__ int32_t s_par[FORK_MAX_B], s_heir[FORK_MAX_B];
    __shared__ uint32_t scan[33];
    launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) a.plan[0] = 0;
    int bad = 0;
    if (threadIdx.x < a.B) {
        const int32_t p = __ldg(a.parent + threadIdx.x);
        s_par[threadIdx.x] = p;
        bad = p < -1 || p >= a.B;
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        if (threadIdx.x == 0) set_status(a.status, RKV_DEV_BAD_INPUT);
        return;
    }
    if (threadIdx.x < a.B) s_heir[threadIdx.x] = heir_of(s_par, a.B, threadIdx.x);
    __syncthreads();
    const int top = min(max(*a.free_top, 0), a.n_pages);
    int64_t gives = 0, takes = 0;
    for (int pass = 0; pass < 2; pass++) {
        // first the totals, then (if the stack holds enough) the pushes and the plan.  More pages than the pool has
        // mean lengths or a stack that contradict one another: the indices below would leave the stack
        if (pass == 1 && (top + gives > a.n_pages || top + gives < takes)) {
            if (threadIdx.x == 0) set_status(a.status, top + gives > a.n_pages ? RKV_DEV_BAD_INPUT : RKV_DEV_POOL_EXHAUSTED);
            return;
        }
        int64_t given = 0, taken = 0;
        for (int c0 = 0; c0 < a.C; c0 += PLAN_THREADS) {
            const int c = c0 + threadIdx.x;
            int give = 0, take = 0, n = 0;
            if (c < a.C) {
                const int b = c / a.LH, lh = c % a.LH, p = s_par[b];
                if (s_heir[b] < 0) give = pages_of(clamp_len(a.len[c], a.max_pages, a.status));
                if (p >= 0) {
                    n = clamp_len(a.len[p * a.LH + lh], a.max_pages, a.status);
                    if (s_heir[p] != b) take = pages_of(n);
                }
            }
            uint32_t tg, tt;
            const int64_t g0 = given + block_exclusive_scan((uint32_t)give, scan, &tg);
            const int64_t t0 = taken + block_exclusive_scan((uint32_t)take, scan, &tt);
            given += tg;
            taken += tt;
            if (pass == 1 && c < a.C) {
                if (blockIdx.x == 0) {
                    a.old[c] = clamp_len(a.len[c], a.max_pages, a.status);
                    a.base[c] = n;
                    a.pop[c] = top + (int)gives - 1 - (int)t0;
                }
                // CTAs take the heads in turn, so that those of one ended sequence spread
                if (c % (int)gridDim.x == (int)blockIdx.x && give > 0) {
                    const int32_t *from = a.block_table + (int64_t)c * a.max_pages;
                    int32_t *to = a.free_stack + (top + (int)g0);
                    bool odd = false;
                    for (int k = 0; k < give; k++) {
                        const int32_t page = from[k];
                        odd |= page < 0 || page >= a.n_pages;
                        to[k] = page;
                    }
                    if (odd) set_status(a.status, RKV_DEV_BAD_INPUT);
                }
            }
        }
        gives = given;
        takes = taken;
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.plan[1] = top + (int)gives - (int)takes;
        a.plan[0] = 1;
    }
}

// A block of FORK_COLS table indices of one (layer, head) over all slots at a
// time; a CTA takes every a.chunks-th block up to the longest of the slots' heads
// (a table can be long and nearly empty).  The old entries of the block are read
// first, then the new ones written, so that slots may exchange their pages
// freely.  A page that several slots copy is read once: eight samples of a 32 x 8
// heads cache with 2,048 entries a head move 2.1 GB in 0.41 ms, 79 % of the
// measured copy rate.
constexpr int FORK_COLS = 8, FORK_THREADS = 256;
template <int CH>
__global__ void __launch_bounds__(FORK_THREADS) fork_rows_kernel(const ForkArgs a) {
    __shared__ int32_t s_par[FORK_MAX_B], s_heir[FORK_MAX_B], s_n[FORK_MAX_B], s_pop[FORK_MAX_B];
    __shared__ int32_t s_old[FORK_MAX_B][FORK_COLS], s_new[FORK_MAX_B][FORK_COLS];
    __shared__ int s_pages;
    wait_for_launcher();
    if (a.plan[0] == 0) return;
    const int lh = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
    if (threadIdx.x == 0) s_pages = 0;
    __syncthreads();
    if (threadIdx.x < a.B) {
        s_par[threadIdx.x] = __ldg(a.parent + threadIdx.x);
        s_n[threadIdx.x] = a.base[threadIdx.x * a.LH + lh];
        s_pop[threadIdx.x] = a.pop[threadIdx.x * a.LH + lh];
        atomicMax(&s_pages, pages_of(max(s_n[threadIdx.x], a.old[threadIdx.x * a.LH + lh])));
        if (chunk == 0) a.len[threadIdx.x * a.LH + lh] = s_n[threadIdx.x];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.free_top = a.plan[1];
    __syncthreads();
    if (threadIdx.x < a.B) s_heir[threadIdx.x] = heir_of(s_par, a.B, threadIdx.x);
    const int pages = s_pages;
    for (int p0 = chunk * FORK_COLS; p0 < pages; p0 += a.chunks * FORK_COLS) {
        for (int i = threadIdx.x; i < a.B * FORK_COLS; i += FORK_THREADS) {
            const int b = i / FORK_COLS, p = p0 + i % FORK_COLS;
            s_old[b][i % FORK_COLS] = p < a.max_pages ? a.block_table[((int64_t)b * a.LH + lh) * a.max_pages + p] : -1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.B * FORK_COLS; i += FORK_THREADS) {
            const int b = i / FORK_COLS, k = i % FORK_COLS, p = p0 + k, s = s_par[b];
            int32_t page = -1;
            if (s >= 0 && p < pages_of(s_n[b])) page = s_heir[s] == b ? s_old[s][k] : a.free_stack[s_pop[b] - p];
            s_new[b][k] = page;
            if (p < a.max_pages && page != s_old[b][k]) a.block_table[((int64_t)b * a.LH + lh) * a.max_pages + p] = page;
        }
        __syncthreads();
        // a warp per (source sequence, column): the page's rows to every slot that copies it
        const int lane = threadIdx.x & 31;
        for (int w = threadIdx.x >> 5; w < a.B * FORK_COLS; w += FORK_THREADS / 32) {
            const int s = w / FORK_COLS, k = w % FORK_COLS, heir = s_heir[s];
            if (heir < 0 || p0 + k >= pages_of(s_n[heir])) continue;
            uint32_t lo = 0, hi = 0;  // slots that copy s
            lo = __ballot_sync(0xFFFFFFFFu, lane < a.B && s_par[lane] == s && heir != lane);
            hi = __ballot_sync(0xFFFFFFFFu, lane + 32 < a.B && s_par[lane + 32] == s && heir != lane + 32);
            uint64_t to = (uint64_t)hi << 32 | lo;
            if (!to) continue;
            const int rows = min(PAGE, s_n[heir] - (p0 + k) * PAGE);
            const int32_t from = s_old[s][k];
            if (from < 0 || from >= a.n_pages) {
                set_status(a.status, RKV_DEV_BAD_INPUT);
                continue;
            }
            constexpr int UN = CH / 2;  // 16 rows of CH pieces over 32 lanes
            uint4 xk[UN], xv[UN];
            int32_t pos = 0;
            float lb = 0.f;
            const int64_t f0 = (int64_t)from * PAGE * CH;
#pragma unroll
            for (int u = 0; u < UN; u++)
                if ((u * 32 + lane) / CH < rows) {
                    xk[u] = __ldcs(static_cast<const uint4 *>(a.k_pool) + f0 + u * 32 + lane);
                    xv[u] = __ldcs(static_cast<const uint4 *>(a.v_pool) + f0 + u * 32 + lane);
                }
            if (lane < rows) {
                pos = a.pos_pool[(int64_t)from * PAGE + lane];
                lb = a.lb_pool[(int64_t)from * PAGE + lane];
            }
            while (to) {
                const int b = __ffsll((long long)to) - 1;
                to &= to - 1;
                const int32_t page = s_new[b][k];
                if (page < 0 || page >= a.n_pages) {
                    set_status(a.status, RKV_DEV_BAD_INPUT);
                    continue;
                }
                const int64_t d0 = (int64_t)page * PAGE * CH;
#pragma unroll
                for (int u = 0; u < UN; u++)
                    if ((u * 32 + lane) / CH < rows) {
                        static_cast<uint4 *>(a.k_pool)[d0 + u * 32 + lane] = xk[u];
                        static_cast<uint4 *>(a.v_pool)[d0 + u * 32 + lane] = xv[u];
                    }
                if (lane < rows) {
                    a.pos_pool[(int64_t)page * PAGE + lane] = pos;
                    a.lb_pool[(int64_t)page * PAGE + lane] = lb;
                }
            }
        }
        __syncthreads();
    }
    // What the tables hold past those blocks, which no head reaches, becomes -1: eight loads in flight, and a store
    // only where something stood.  A table of 8,192 pages a head for heads of 500 entries costs 29 us of the 101
    // that eight slots of 32 x 8 heads take (10 of 50 us with four slots of 28 x 4).
    constexpr int UN = 8;
    int p = (pages + FORK_COLS - 1) / FORK_COLS * FORK_COLS + chunk * FORK_THREADS + (int)threadIdx.x;
    for (; p < a.max_pages; p += a.chunks * FORK_THREADS) {
        int32_t *column = a.block_table + (int64_t)lh * a.max_pages + p;
        const int64_t slot = (int64_t)a.LH * a.max_pages;
        for (int b0 = 0; b0 < a.B; b0 += UN) {
            int32_t page[UN];
#pragma unroll
            for (int u = 0; u < UN; u++) page[u] = b0 + u < a.B ? column[(b0 + u) * slot] : -1;
#pragma unroll
            for (int u = 0; u < UN; u++)
                if (page[u] != -1) column[(b0 + u) * slot] = -1;
        }
    }
}

template <int CH>
cudaError_t append_rows(const AppendTokensArgs &a, cudaStream_t s) {
    const int64_t groups = ((int64_t)a.n_new / 32 + a.B) * a.LH, per = MOVE_THREADS / 32;  // at most
    const int64_t ctas = (groups + per - 1) / per;
    return launch_after(append_rows_kernel<CH>, (unsigned)(ctas < 148 * 4 ? ctas : 148 * 4), MOVE_THREADS,
                        (size_t)(2 * a.B + 1) * 4, s, a);
}

template <int CH>
cudaError_t fork_rows(ForkArgs a, cudaStream_t s) {
    const int blocks = (a.max_pages + FORK_COLS - 1) / FORK_COLS, want = (148 * 64 + a.LH - 1) / a.LH;
    a.chunks = blocks < want ? blocks : want;
    if ((int64_t)a.LH * a.chunks >= (1ll << 31)) return cudaErrorNotSupported;
    return launch_after(fork_rows_kernel<CH>, (unsigned)(a.LH * a.chunks), FORK_THREADS, 0, s, a);
}

}  // namespace

cudaError_t launch_append_tokens(const AppendTokensArgs &a, int row_bytes, cudaStream_t s) {
    append_plan_kernel<<<1, PLAN_THREADS, (a.B + 1) * 4, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return row_bytes == 128 ? append_rows<8>(a, s) : row_bytes == 256 ? append_rows<16>(a, s) : append_rows<32>(a, s);
}

cudaError_t launch_fork(const ForkArgs &a, int row_bytes, cudaStream_t s) {
    const int64_t want = ((int64_t)a.C + 31) / 32;
    fork_plan_kernel<<<(unsigned)(want < 148 ? want : 148), PLAN_THREADS, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return row_bytes == 128 ? fork_rows<8>(a, s) : row_bytes == 256 ? fork_rows<16>(a, s) : fork_rows<32>(a, s);
}

}  // namespace rkv
