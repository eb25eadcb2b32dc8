// tree_tc.cu -- rkv_tree_attn on bf16 pools: both products on the fifth-
// generation tensor cores, K and V pages gathered by TMA.
//
// Per KV head the query rows are (drafted token, query head of the group), the
// keys its cache pages and then its drafted tokens in groups of 16 rows; a key
// tile is eight such groups.  An item is a head with at most two query tiles of
// whole tokens (nt = 128 / G tokens each).  With two tiles both meet every key
// tile, so K and V are read once for 256 rows; with one tile the two softmax
// warpgroups take the key tiles in turn, each with its own running state, and
// join at the end.
//
// All items' key tiles in order, plus COST per item for its queries and results,
// are cut into one equal range per CTA: the work is bound by the bytes of K and
// V, and heads differ in length by orders of magnitude.  An item cut by a range's
// end leaves its parts' unnormalised outputs, maxima and sums in the workspace,
// and tree_join_kernel joins them in ascending order.
//
// Warps 0-7: softmax and results.  Warp 8: items, queries, K, and a record of
// each key tile (pages, keep words) that the others follow.  Warp 9: issues the
// products.  Warp 10: V.  Warp 11: V of key tiles with rows that do not count:
// those become zero (0 * NaN would reach every row), and infinite or NaN values
// of drafted tokens too (not every row attends them; the results add them for
// those that do).
//
// Measured (one B200, calls one after the other for some tenths of a second): 24
// nodes over 256 heads of 13,107 entries on average, 1.74 GB, 0.36 ms, 73 % of the
// measured copy rate (0.31 ms, 85 %, for the first 50 ms); 16 trees of 1 to 64
// nodes over 4,608 heads of 512 entries, 1.55 GB, 0.58 ms, 41 %; one token of 8
// sequences over 896 heads of 512 entries, 0.214 GB, 90 us, 36 %.  Short items pay for
// their ends (the results of one and the first scores of the next do not overlap
// within a warpgroup) and for instructions fetched anew.
#include "attn_tc.cuh"

namespace rkv {
namespace {

constexpr int COST = 1;       // an item's queries and results, in key tiles
constexpr int MIN_RANGE = 4;  // key tiles of a CTA at least: a cut costs a record and a join
constexpr int WORDS = 8;      // ring of key tiles' keep words
constexpr int ITEMS = 4;      // ring of items

// A key tile lies as its eight groups of 16 rows, each two blocks of 8 rows, each
// D/64 planes of 8 lines of 128 bytes.  One TMA box is then a whole page (the
// boxes' number, not their size, bounds the loads), and the 8-row blocks of a
// tile are evenly spaced, as one descriptor needs them.
template <int D>
struct Cfg {
    static constexpr int TILE = TcCfg<D>::TILE;
    static constexpr int GROUP = PAGE * D * 2, BLOCK = GROUP / 2;
    static constexpr int ROOM = 227 * 1024 - 1024;  // of shared memory, less the alignment of the swizzle's period
};

// Shared memory: two query tiles of as many rows as the call's tiles have (the
// products read 128 rows from there on: what lies behind only gives rows that do
// not count), and slots for K and V tiles with the rest.  More slots are more
// bytes in flight: 2 + 2 with 128 rows of D = 128, 2 + 3 with 96, 3 + 3 up to 40.
struct Room {
    int plane, tile;  // bytes of 64 columns of a query tile, and of the tile
    int ks, vs;       // slots, at most 4 each
    __host__ __device__ Room(int rows, int D, int room) {
        plane = (rows + 7) / 8 * 1024;
        tile = plane * (D / 64);
        const int n = (room - 2 * tile) / (128 * D * 2);
        ks = n / 2 > 4 ? 4 : n / 2;
        vs = n - ks > 4 ? 4 : n - ks;
    }
};

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Item {
    int c, lh;                    // head: of all, of its sequence
    int t0, node0, nodes;         // first token of the sequence, of the item (in the sequence); the sequence's tokens
    int rows[2];                  // rows of the query tiles (rows[1] = 0: one tile)
    int lo, hi, np, len;          // key tiles of this part; cache pages and entries of the head
    int rec;                      // -1: the item is whole; else the record of this part
    int odd;                      // V of some drafted token held infinities or NaN
};

// A key tile.
struct __align__(16) Tile {
    uint16_t word[8];             // bit r: row r of group g counts
    int32_t page[8];              // page of the pool, or first row of the draft
    uint32_t live, drafts;        // groups with a row that counts (END: no more tiles), and those of drafted tokens
    uint32_t part;                // some row does not count, or is of a drafted token
    uint32_t item_lh;             // slot of the item, and lh << 8
};
constexpr uint32_t END = 0xFFFFFFFFu;

struct Shared {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t v_part[4], v_ready[4]; // a slot's V of a partial tile: loaded, and mended (v_full is not used)
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2][2], o_done[2], o_free, ml_full;  // p_full: by halves of the keys
    uint64_t w_full[ITEMS], w_empty[ITEMS]; // items
    uint64_t t_full[WORDS], t_empty[WORDS]; // tiles' records
    Item item[ITEMS];
    Tile tile[WORDS];
    uint4 stage[8][32 * 2];         // results of a warp's rows, 16 columns: from a row a lane to whole sectors
    float2 ml[2][2][QR];            // one-tile items: maximum and sum of both warpgroups (by item, warpgroup)
    uint32_t tmem;
    int c0, p0;                     // first head of this CTA's range and the work before it
    int begin, end, total;
};

template <int D>
struct Ctx {
    Shared *sh;
    unsigned char *q, *kv;
    int32_t *status;
    Room room;
    __device__ bool wait(uint64_t *bar, uint32_t parity, int site) const { return wait_on(bar, parity, status, site); }
    // in line, for the waits that every tile's path goes through
    __device__ bool wait_near(uint64_t *bar, uint32_t parity, int site) const { return tc_wait(bar, parity, status, site); }
    __device__ unsigned char *k_slot(int i) const { return kv + i * Cfg<D>::TILE; }
    __device__ unsigned char *v_slot(int i) const { return kv + (room.ks + i) * Cfg<D>::TILE; }
};

// Key tiles of head c and items it is cut into.
struct Head {
    int t0, nodes, len, np, tiles, items;
    __device__ Head(const TreeArgs &a, int32_t from, int32_t to, int32_t n, int32_t *status) {
        t0 = from;
        nodes = to - from;
        len = clamp_len(n, a.max_pages, status);
        np = ceil_div(len, PAGE);
        tiles = ceil_div(np + ceil_div(nodes, PAGE), 8);
        items = nodes == 0 ? 0 : nodes <= a.nt ? 1 : ceil_div(nodes, 2 * a.nt);
    }
    __device__ Head(const TreeArgs &a, int c, int32_t *status)
        : Head(a, __ldg(a.cu + c / a.LH), __ldg(a.cu + c / a.LH + 1), __ldg(a.len + c), status) {}
};

// Start of CTA i's range when `total` is cut into n.
__device__ __forceinline__ int cut(int total, int i, int n) { return (int)((int64_t)total * i / n); }
// CTA whose range holds position x.
static __device__ __noinline__ int cta_of(int total, int x, int n) {
    int i = (int)((int64_t)x * n / total);
    while (cut(total, i + 1, n) <= x) i++;
    while (cut(total, i, n) > x) i--;
    return i;
}

// ------------------------------------------------- warps 8 and 10: loads ----
// Every lane waits for itself, so that each may read what the phase brought, and the vote lets no lane run ahead by
// a phase (the next but one has the same parity) and all give up together.  Lane 0 waiting for all, with a shuffle
// and a __syncwarp behind it, measured 414 us on 24 nodes over 13,107 entries a head, and this 360.
static __device__ __noinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int32_t *status, int site) {
    return __all_sync(0xFFFFFFFFu, tc_wait(bar, parity, status, site));
}

// Whether the phase is over, without waiting; whole warp.
__device__ __forceinline__ bool warp_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// Pages (or rows of the draft) and keep words of a head's groups of 16 rows: 32
// of them at a time, one a lane, read a batch ahead.
struct Groups {
    const int32_t *table;
    const uint16_t *keep;
    int np, len, nodes, t0;
    int32_t page, next_page;
    uint32_t word, next_word;
    __device__ void start(const TreeArgs &a, const Item &it) {
        table = a.block_table + (int64_t)it.c * a.max_pages;
        keep = a.keep_mask ? a.keep_mask + (int64_t)it.c * a.max_pages : nullptr;
        np = it.np;
        len = it.len;
        nodes = it.nodes;
        t0 = it.t0;
        fetch(it.lo * 8 + (threadIdx.x & 31));
    }
    __device__ void fetch(int u) {
        next_page = 0;
        next_word = 0;
        if (u < np) {
            next_page = __ldg(table + u);
            next_word = keep ? __ldg(keep + u) : 0xFFFFu;
        } else if ((u - np) * PAGE < nodes) {
            next_page = t0 + (u - np) * PAGE;
            next_word = 0xFFFFu;
        }
    }
    // Tile j (`at`-th of this part): lanes 0-7 get its groups; whole warp.
    __device__ void tile(int j, int at, int n_pages, int32_t *status, int32_t &pg, uint32_t &wd, bool &draft) {
        const int lane = threadIdx.x & 31;
        if ((at & 3) == 0) {
            const int u = j * 8 + lane, in = u < np ? len - u * PAGE : nodes - (u - np) * PAGE;
            page = next_page;
            word = in < PAGE && in > 0 ? next_word & ((1u << in) - 1u) : next_word;
            if (u < np && (uint32_t)page >= (uint32_t)n_pages) {
                if (word) set_status(status, RKV_DEV_BAD_INPUT);
                word = 0;
            }
            fetch(u + 32);
        }
        pg = __shfl_sync(0xFFFFFFFFu, page, (at & 3) * 8 + (lane & 7));
        wd = __shfl_sync(0xFFFFFFFFu, word, (at & 3) * 8 + (lane & 7));
        draft = j * 8 + (lane & 7) >= np;
        if (lane >= 8) wd = 0;
    }
};

// The eight groups of a key tile: pages of the pool, or (drafts) two blocks of 8
// rows each of the drafted tokens; only those with their bit in live.  Whole
// warp; one elected thread issues, with the operands in uniform registers.
template <int D>
static __device__ __noinline__ void issue_tile(unsigned char *dst, const CUtensorMap *pool, const CUtensorMap *draft_map,
                                               const int32_t *pages, uint32_t live, uint32_t drafts, int lh, uint64_t *bar) {
    using C = Cfg<D>;
    if (elect_one()) {
        mbar_arrive_expect_tx(bar, __popc(live) * C::GROUP);
        int32_t pg[8];
        *reinterpret_cast<int4 *>(pg) = *reinterpret_cast<const int4 *>(pages);
        *reinterpret_cast<int4 *>(pg + 4) = *reinterpret_cast<const int4 *>(pages + 4);
        const uint32_t paged = live & ~drafts;
#pragma unroll
        for (int g = 0; g < 8; g++)
            if (paged >> g & 1) tma_load_4d(dst + g * C::GROUP, pool, 0, 0, 0, pg[g] * 2, bar);
#pragma unroll 1
        for (uint32_t left = live & drafts; left; left &= left - 1) {
            const int g = __ffs(left) - 1, row = pages[g];
            tma_tile(dst + g * C::GROUP, draft_map, 0, row, lh * (D / 64), bar);
            tma_tile(dst + g * C::GROUP + C::BLOCK, draft_map, 0, row + 8, lh * (D / 64), bar);
        }
    }
    __syncwarp();
}

// Warp 8.  An item's head, its first pages and (where the ring has room) the item
// itself are read and handed on while the item before it is loaded, so that
// short heads follow without a gap.
template <int D>
__device__ void load_role(const Ctx<D> &x, const TreeArgs &a, int n, const CUtensorMap *tq, const CUtensorMap *tk,
                          const CUtensorMap *dk) {
    using C = Cfg<D>;
    Shared *sh = x.sh;
    const int lane = threadIdx.x & 31, begin = sh->begin, end = sh->end;
    Ring kr, w, qr, tr;
    int c = sh->c0, lh = c % a.LH, b = c / a.LH, k = 0, pre = sh->p0;  // next head, item of it, work before that
    int32_t r0 = __ldg(a.cu + b), r1 = __ldg(a.cu + b + 1), rn = __ldg(a.len + c);  // of head c
    Head h(a, r0, r1, rn, a.status);
    Groups groups, ahead;
    Item it{}, now{};
    bool posted = false;
    auto wait = [&](uint64_t *bar, uint32_t parity, int site) { return warp_wait(bar, parity, a.status, site); };
    // Turn by turn: the tiles of the item found before and, behind the first of
    // them, the search for the next one; the first turn only searches.
#pragma unroll 1
    for (bool first = true, have = true; have; first = false) {
        if (!first) {
            if (!posted) {
                if (!wait(&sh->w_empty[w.slot], w.turn ^ 1u, 0x440)) return;
                posted = true;
                if (lane == 0) {
                    sh->item[w.slot] = it;
                    mbar_arrive(&sh->w_full[w.slot]);
                }
                w.next(ITEMS);
            }
            now = it;
            groups = ahead;
            posted = false;
        }
        // the slot of the item that was posted last
        const uint32_t item_lh = (uint32_t)((w.slot + ITEMS - 1) % ITEMS) | (uint32_t)now.lh << 8;
        // raw lengths and offsets of the head after h, used after the first tile
        const int lh2 = lh + 1 == a.LH ? 0 : lh + 1, b2 = min(lh2 ? b : b + 1, a.B - 1);
        r0 = __ldg(a.cu + b2);
        r1 = __ldg(a.cu + b2 + 1);
        rn = __ldg(a.len + min(c + 1, a.C - 1));
#pragma unroll 1
        for (int j = now.lo; j < now.hi || first; j++) {
            if (!first) {
                int32_t pg;
                uint32_t wd;
                bool draft;
                groups.tile(j, j - now.lo, a.n_pages, a.status, pg, wd, draft);
                const uint32_t live = __ballot_sync(0xFFFFFFFFu, wd != 0);
                const uint32_t part = __ballot_sync(0xFFFFFFFFu, lane < 8 && (wd != 0xFFFFu || draft));
                const uint32_t drafts = __ballot_sync(0xFFFFFFFFu, wd != 0 && draft);
                if (!wait(&sh->t_empty[tr.slot], tr.turn ^ 1u, 0x443)) return;
                Tile *t = &sh->tile[tr.slot];
                if (lane < 8) {
                    t->word[lane] = (uint16_t)wd;
                    t->page[lane] = pg;
                }
                if (lane == 0) {
                    t->live = live;
                    t->drafts = drafts;
                    t->part = part;
                    t->item_lh = item_lh;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->t_full[tr.slot]);
                tr.next(WORDS);
                if (!wait(&sh->k_empty[kr.slot], kr.turn ^ 1u, 0x442)) return;
                issue_tile<D>(x.k_slot(kr.slot), tk, dk, t->page, live, drafts, now.lh, &sh->k_full[kr.slot]);
                kr.next(x.room.ks);
                if (j > now.lo) continue;
                // the item's one or two query tiles, behind its first key tile: their
                // slots are free only when the products of the item before are done
#pragma unroll 1
                for (int i = 0; i < (now.rows[1] ? 2 : 1); i++) {
                    if (!wait(&sh->q_empty[qr.slot], qr.turn ^ 1u, 0x441)) return;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&sh->q_full[qr.slot], (uint32_t)(a.nt * a.G * D * 2));
#pragma unroll
                        for (int p = 0; p < D / 64; p++)
                            tma_tile(x.q + qr.slot * x.room.tile + p * x.room.plane, tq, p * 64, now.lh * a.G,
                                     now.t0 + now.node0 + i * a.nt, &sh->q_full[qr.slot]);
                    }
                    __syncwarp();
                    qr.next(2);
                }
                k++;
                pre += h.tiles + COST;
            }
            // the next item of the range: part of an item that has tiles in it
            for (bool raw = !first;; raw = false) {
                it.node0 = k * 2 * a.nt;
                it.lo = max(0, min(h.tiles, begin - pre - COST));
                it.hi = max(0, min(h.tiles, end - pre - COST));
                if (pre >= end) break;
                if (it.node0 < h.nodes) {
                    if (it.lo < it.hi) break;
                    k++;
                    pre += h.tiles + COST;
                    continue;
                }
                k = 0;
                if (++c >= a.C) break;
                if (++lh == a.LH) {
                    lh = 0;
                    b++;
                }
                if (!raw) {
                    r0 = __ldg(a.cu + b);
                    r1 = __ldg(a.cu + b + 1);
                    rn = __ldg(a.len + c);
                }
                h = Head(a, r0, r1, rn, a.status);
            }
            have = c < a.C && pre < end;
            if (have) {
                it.c = c;
                it.lh = lh;
                it.t0 = h.t0;
                it.nodes = h.nodes;
                it.np = h.np;
                it.len = h.len;
                const int left = h.nodes - it.node0;
                it.rows[0] = min(left, a.nt) * a.G;
                it.rows[1] = left > a.nt ? min(left - a.nt, a.nt) * a.G : 0;
                it.rec = -1;
                if (it.lo > 0 || it.hi < h.tiles) {
                    it.rec = 2 * (int)blockIdx.x + (it.lo == 0 ? 1 : 0);
                    if (it.lo == 0 && lane == 0)  // the item's first part: it describes the item to the join
                        a.join[blockIdx.x] = make_int4(c, it.node0, cta_of(sh->total, pre + COST + h.tiles - 1, n), 0);
                }
                ahead.start(a, it);
                if (!first && warp_test(&sh->w_empty[w.slot], w.turn ^ 1u)) {
                    posted = true;
                    if (lane == 0) {
                        sh->item[w.slot] = it;
                        mbar_arrive(&sh->w_full[w.slot]);
                    }
                    w.next(ITEMS);
                }
            }
            if (first) break;
        }
    }
    // the end: an item without rows, a tile that is none
    if (!wait(&sh->w_empty[w.slot], w.turn ^ 1u, 0x444) || !wait(&sh->t_empty[tr.slot], tr.turn ^ 1u, 0x445)) return;
    if (lane == 0) {
        sh->item[w.slot].rows[0] = 0;
        mbar_arrive(&sh->w_full[w.slot]);
        sh->tile[tr.slot].live = END;
        mbar_arrive(&sh->t_full[tr.slot]);
    }
}

// Warp 10: V.
template <int D>
__device__ void value_role(const Ctx<D> &x, const TreeArgs &a, const CUtensorMap *tv, const CUtensorMap *dv) {
    Shared *sh = x.sh;
#pragma unroll 1
    for (Ring vr, tr;; vr.next(x.room.vs), tr.next(WORDS)) {
        if (!warp_wait(&sh->t_full[tr.slot], tr.turn, a.status, 0x446)) return;
        const Tile *t = &sh->tile[tr.slot];
        const uint32_t live = t->live;
        if (live == END) return;
        if (!warp_wait(&sh->v_empty[vr.slot], vr.turn ^ 1u, a.status, 0x447)) return;
        issue_tile<D>(x.v_slot(vr.slot), tv, dv, t->page, live, t->drafts, t->item_lh >> 8,
                      t->part ? &sh->v_part[vr.slot] : &sh->v_full[vr.slot]);
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->t_empty[tr.slot]);
    }
}

// ---------------------------------------------------------- warp 9: products ----
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t s, uint64_t q, int q_plane, uint64_t k, uint32_t idesc) {
#pragma unroll
    for (int e = 0; e < D / 16; e++)
        mma_ss(s, desc_at(q, (e / 4) * q_plane + (e % 4) * 32), desc_at(k, (e / 4) * 1024 + (e % 4) * 32), idesc, e > 0);
}

template <int D>
__device__ __forceinline__ void mma_output(uint32_t o, uint32_t p, uint64_t v, uint32_t idesc, int half, bool first) {
    p += half * 32;
    v = desc_at(v, half * 4 * Cfg<D>::GROUP);
#pragma unroll
    for (int g = 0; g < 4; g++) mma_ts(o, p + g * 8, desc_at(v, g * Cfg<D>::GROUP), idesc, g > 0 || !first);
}

template <int D>
__device__ void mma_role(const Ctx<D> &x, bool neg) {
    using C = Cfg<D>;
    Shared *sh = x.sh;
    const uint32_t tmem = sh->tmem;
    const uint32_t qk = mma_desc(QR, KR, false, neg), pv = mma_desc(QR, D, true, false);
    Ring w, qr;
    int kslot = 0, vslot = 0, tile_no = 0;  // slots of the next K and V; key tiles so far, mod WORDS
    uint32_t k_turn = 0, v_turn = 0, r_turn = 0, q_turn = 0;  // k_full, v_full, v_ready, q_full: a bit for each slot
    uint32_t p_turn = 0, f_turn = 0;                          // p_full: a bit for each tile; o_free
    const uint64_t q_desc = tile_desc(smem_u32(x.q), 16), k_desc = tile_desc(smem_u32(x.k_slot(0)), 16, C::BLOCK),
                   v_desc = tile_desc(smem_u32(x.v_slot(0)), 1024, C::BLOCK);
    for (;; w.next(ITEMS)) {
        if (!x.wait(&sh->w_full[w.slot], w.turn, 0x450)) return;
        const Item *it = &sh->item[w.slot];
        const int rows0 = it->rows[0], two = it->rows[1] > 0, n = it->hi - it->lo;
        mbar_arrive(&sh->w_empty[w.slot]);
        if (rows0 == 0) return;
        int qs0 = qr.slot, qs1 = qr.slot;  // query tiles' slots
        for (int i = 0; i <= two; i++) {
            if (!x.wait(&sh->q_full[qr.slot], q_turn >> qr.slot & 1u, 0x451)) return;
            q_turn ^= 1u << qr.slot;
            qs1 = qr.slot;
            qr.next(2);
        }
        // Step t does O_i += P_i V of key tile t - ahead and S_i of key tile t: for
        // both i with two query tiles (ahead = 1), else for i = t mod 2 (ahead = 2).
        const int ahead = two ? 1 : 2;
#pragma unroll 1
        for (int t = 0; t < n + ahead; t++) {
            const int j = t - ahead;
            if (j >= 0) {
                const int part = *(volatile uint32_t *)&sh->tile[(tile_no + j) % WORDS].part != 0;
                if (part) {
                    if (!x.wait(&sh->v_ready[vslot], r_turn >> vslot & 1u, 0x453)) return;
                    r_turn ^= 1u << vslot;
                } else {
                    if (!x.wait(&sh->v_full[vslot], v_turn >> vslot & 1u, 0x454)) return;
                    v_turn ^= 1u << vslot;
                }
                if (j == 0) {
                    if (!x.wait(&sh->o_free, f_turn ^ 1u, 0x455)) return;
                    f_turn ^= 1u;
                }
            }
#pragma unroll 1
            for (int q = 0; q <= two; q++) {
                const int i = two ? q : t & 1;
                const uint32_t o = tmem + TM_O + i * D, p = tmem + TM_S + i * 128;
                if (j >= 0) {
                    const uint64_t v = desc_at(v_desc, vslot * C::TILE);
                    if (!x.wait_near(&sh->p_full[i][0], p_turn >> i & 1u, 0x456)) return;
                    tc_fence_after();
                    mma_output<D>(o, p, v, pv, 0, j < ahead);
                    if (!x.wait_near(&sh->p_full[i][1], p_turn >> i & 1u, 0x457)) return;
                    p_turn ^= 1u << i;
                    tc_fence_after();
                    mma_output<D>(o, p, v, pv, 1, false);
                    mma_commit(&sh->o_done[i]);
                }
                if (t < n) {
                    if (q == 0) {
                        if (!x.wait(&sh->k_full[kslot], k_turn >> kslot & 1u, 0x452)) return;
                        k_turn ^= 1u << kslot;
                    }
                    const int qs = q ? qs1 : qs0;
                    tc_fence_after();
                    mma_scores<D>(p, desc_at(q_desc, qs * x.room.tile), x.room.plane, desc_at(k_desc, kslot * C::TILE), qk);
                    mma_commit(&sh->s_full[i]);
                    if (q == two) mma_commit(&sh->k_empty[kslot]);
                    if (t == n - 1) mma_commit(&sh->q_empty[qs]);
                }
            }
            if (j >= 0) {
                mma_commit(&sh->v_empty[vslot]);
                vslot = vslot + 1 == x.room.vs ? 0 : vslot + 1;
            }
            if (t < n) kslot = kslot + 1 == x.room.ks ? 0 : kslot + 1;
        }
        tile_no = (tile_no + n) % WORDS;
    }
}

// --------------------------------------------------- warp 11: V's odd rows ----
template <int D>
__device__ void mend_role(const Ctx<D> &x) {
    using C = Cfg<D>;
    Shared *sh = x.sh;
    const int lane = threadIdx.x & 31;
    // a row is D/8 pieces of 16 bytes: line row % 8 of each plane of block row / 8
    constexpr int PIECES = D / 8, ROWS = 32 / PIECES;  // rows the warp takes at once
    const int piece = (lane / 8 % (D / 64)) * 64 + lane % 8;
    const uint32_t mine = (ROWS == 2 ? 0x5555u : 0x1111u) << (lane / PIECES);
    uint32_t turn = 0;  // v_part: a bit for each slot
#pragma unroll 1
    for (Ring vr, tr;; vr.next(x.room.vs), tr.next(WORDS)) {
        if (!x.wait(&sh->t_full[tr.slot], tr.turn, 0x460)) return;
        const Tile *t = &sh->tile[tr.slot];
        const uint32_t live = t->live, drafts = t->drafts;
        if (live == END) return;
        if (t->part) {
            if (!x.wait(&sh->v_part[vr.slot], turn >> vr.slot & 1u, 0x461)) return;
            turn ^= 1u << vr.slot;
            bool odd = false;
#pragma unroll 1
            for (int g = 0; g < 8; g++) {
                const uint32_t word = t->word[g];
                const bool draft = drafts >> g & 1;
                if (word == 0xFFFFu && !draft) continue;
                uint4 *group = reinterpret_cast<uint4 *>(x.v_slot(vr.slot) + g * C::GROUP) + piece;
                auto row = [&](int r) { return group + (r >> 3) * (C::BLOCK / 16) + (r & 7) * 8; };
                // every ROWS-th row is this part of the warp's: those that do not count
#pragma unroll 1
                for (uint32_t gone = ~word & mine; gone; gone &= gone - 1) *row(__ffs(gone) - 1) = make_uint4(0, 0, 0, 0);
                if (!draft) continue;
#pragma unroll 1
                for (uint32_t left = word & mine; left; left &= left - 1) {
                    uint4 *p = row(__ffs(left) - 1), v = *p;
                    if (drop_odd(v)) {
                        odd = true;
                        *p = v;
                    }
                }
            }
            if (odd) atomicOr(&sh->item[t->item_lh & 255u].odd, 1);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->v_ready[vr.slot]);
        }
        __syncwarp();  // all lanes have read the record, which may be written anew from here on
        if (lane == 0) mbar_arrive(&sh->t_empty[tr.slot]);
    }
}

// ------------------------------------------------------ warps 0-7: softmax ----
template <int D>
__device__ void softmax_role(const Ctx<D> &x, const TreeArgs &a) {
    Shared *sh = x.sh;
    const int i = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(row & 96) << 16;
    const uint32_t ts = sh->tmem + TM_S + i * 128 + lanes, o0 = sh->tmem + TM_O + lanes, to = o0 + i * D;
    const float qscale = fabsf(a.qscale);
    const int row_node = row / a.G, row_g = row % a.G;
    uint32_t s_turn = 0, d_turn[2] = {0, 0}, x_turn = 0;  // d_turn: parity of the next product to complete
    int tile_no = 0;
    uint32_t flip = 0;
    Ring w;
    for (;; w.next(ITEMS)) {
        if (!x.wait(&sh->w_full[w.slot], w.turn, 0x470)) return;
        const Item it = sh->item[w.slot];
        if (it.rows[0] == 0) return;
        const bool two = it.rows[1] > 0;
        const int n = it.hi - it.lo, rows = two ? it.rows[i] : it.rows[0];
        const bool warp_here = (row & 96) < rows;  // some row of this warp counts
        const int node = it.node0 + (two ? i * a.nt : 0) + row_node;
        unsigned long long mask = 0;
        if (row < rows) mask = __ldg(a.mask + it.t0 + node);
        float m = -INFINITY, l = 0.f;
        int mine = 0;
#pragma unroll 1
        for (int j = two ? 0 : i; j < n; j += two ? 1 : 2, mine++) {
            // every lane sees this phase before the warp goes on: the next can follow once lane 0 has arrived, and a lane
            // left behind would take the one after for its own (the same parity) or wait in vain
            if (!__all_sync(0xFFFFFFFFu, x.wait_near(&sh->s_full[i], s_turn, 0x471))) return;
            s_turn ^= 1u;
            if (warp_here) {
                tc_fence_after();
                const Tile *t = &sh->tile[(tile_no + j) % WORDS];
                const uint32_t part = *(volatile const uint32_t *)&t->part;
                auto done = [&] { return x.wait(&sh->o_done[i], d_turn[i] ^ 1u, 0x472); };
                uint32_t bits[4];
                if (part) {
                    const uint4 w4 = *reinterpret_cast<const uint4 *>(t->word);
                    bits[0] = w4.x;
                    bits[1] = w4.y;
                    bits[2] = w4.z;
                    bits[3] = w4.w;
                    const int first = it.np - (it.lo + j) * 8;  // group of the tile with which the draft begins
                    if (first < 8) {
                        // the draft's 64 bits from bit 16 * first of the tile's 128 on
                        const int at = 16 * first;
                        const unsigned long long lo = at < 64 ? (at < 0 ? mask >> -at : mask << at) : 0ull;
                        const unsigned long long hi = at >= 64 ? mask << (at - 64) : at > 0 ? mask >> (64 - at) : 0ull;
                        const unsigned long long c_lo = at >= 64 ? ~0ull : at > 0 ? (1ull << at) - 1ull : 0ull;
                        const unsigned long long c_hi = at > 64 ? (1ull << (at - 64)) - 1ull : 0ull;
                        bits[0] &= (uint32_t)(lo | c_lo);
                        bits[1] &= (uint32_t)((lo | c_lo) >> 32);
                        bits[2] &= (uint32_t)(hi | c_hi);
                        bits[3] &= (uint32_t)((hi | c_hi) >> 32);
                    }
                }
                auto columns = [&](int c) { return c < 2 ? (c ? bits[1] : bits[0]) : (c == 2 ? bits[2] : bits[3]); };
                const bool ok =
                    softmax_tile<D>(ts, to, mine == 0, qscale, m, l, sh->p_full[i], part != 0, columns, done);
                if (!ok) return;
            } else if (lane == 0) {
                mbar_arrive(&sh->p_full[i][0]);
                mbar_arrive(&sh->p_full[i][1]);
            }
            d_turn[i] ^= 1u;
        }
        tile_no += n;
        // products of the other warpgroup
        const int theirs = two ? n : i ? (n + 1) / 2 : n / 2;
        if (theirs & 1) d_turn[i ^ 1] ^= 1u;
        if (mine && !x.wait(&sh->o_done[i], d_turn[i] ^ 1u, 0x473)) return;
        float scale0 = 1.f, scale1 = 0.f;  // one tile: of O_0 and O_1
        int c_lo = 0, c_hi = D;
        if (!two) {
            // join the two warpgroups' states; each finishes half of the columns
            sh->ml[flip][i][row] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->ml_full);
            if (!x.wait(&sh->ml_full, x_turn, 0x474)) return;
            x_turn ^= 1u;
            if (theirs && !x.wait(&sh->o_done[i ^ 1], d_turn[i ^ 1] ^ 1u, 0x475)) return;
            const float2 s0 = sh->ml[flip][0][row], s1 = sh->ml[flip][1][row];
            flip ^= 1u;
            m = max_nan(s0.x, s1.x, s1.x);  // a NaN row (softmax_tile) stays one
            if (m != -INFINITY) {
                scale0 = s0.x == m ? 1.f : ex2((s0.x - m) * qscale);
                scale1 = s1.x == m ? 1.f : ex2((s1.x - m) * qscale);
            }
            l = s0.y * scale0 + s1.y * scale1;
            c_lo = i * (D / 2);
            c_hi = c_lo + D / 2;
        }
        tc_fence_after();
        if (warp_here) {
            const int odd = *(volatile int *)&sh->item[w.slot].odd;
            const bool here = row < rows;
            const bool none = m == -INFINITY;
            const int64_t at = (int64_t)(it.t0 + node) * a.LH * a.G + it.lh * a.G + row_g;  // row of q and out
            const float inv = it.rec >= 0 ? 1.f : none ? 0.f : __fdividef(1.f, l);
            float *rec = nullptr;
            if (it.rec >= 0) rec = a.rec + ((int64_t)it.rec * a.rec_tiles + (two ? i : 0)) * (QR * (D + 2)) + row;
            if (__any_sync(0xFFFFFFFFu, odd)) {
                scale0 = fmaxf(scale0, 0x1p-100f);  // infinite values pass, finite ones vanish as with 0
                for (int d = 0; d < it.nodes; d++)
                    add_odd<D>(two ? to : o0, static_cast<const __nv_bfloat16 *>(a.v_draft) + ((int64_t)(it.t0 + d) * a.LH + it.lh) * D,
                               here && (mask >> d & 1ull), c_lo, c_hi);
            }
            const uint32_t rows_here = __ballot_sync(0xFFFFFFFFu, here);
            const uint32_t first = two ? to : o0;
            scale0 *= inv;
            scale1 *= inv;
#pragma unroll 1
            for (int c = c_lo; c < c_hi; c += 16) {
                uint32_t o[16];
                float f[16];
                tmem_read16(o, first + c);
#pragma unroll
                for (int e = 0; e < 16; e++) f[e] = __uint_as_float(o[e]) * scale0;
                if (!two && n > 1) {
                    tmem_read16(o, o0 + D + c);
#pragma unroll
                    for (int e = 0; e < 16; e++) f[e] = fmaf(__uint_as_float(o[e]), scale1, f[e]);
                }
                if (it.rec < 0) {
                    store_rows(sh->stage[threadIdx.x >> 5], static_cast<__nv_bfloat16 *>(a.out) + c, at * D, rows_here, f);
                } else if (here) {
#pragma unroll
                    for (int e = 0; e < 16; e++) rec[(c + e) * QR] = f[e];
                }
                __syncwarp();
            }
            if (here && c_lo == 0) {
                if (rec) {
                    rec[D * QR] = m;
                    rec[(D + 1) * QR] = l;
                } else if (a.lse) {
                    a.lse[at] = none ? -INFINITY : (m * qscale + __log2f(l)) * LN2;
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&sh->o_free);
            mbar_arrive(&sh->w_empty[w.slot]);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(TC_THREADS, 1)
    tree_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap dk,
                   const __grid_constant__ CUtensorMap dv) {
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) unsigned char sh_raw[sizeof(Shared)];
    Shared &sh = *reinterpret_cast<Shared *>(sh_raw);
    __shared__ uint32_t scan[33];
    unsigned char *tiles = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5;
    launch_dependents();
    if (threadIdx.x == 256) {
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
        prefetch_tensormap(&dk);
        prefetch_tensormap(&dv);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < ITEMS; s++) {
            mbar_init(&sh.w_full[s], 1);
            mbar_init(&sh.w_empty[s], 9);  // products, eight softmax warps
        }
        for (int s = 0; s < 4; s++) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.k_empty[s], 1);
            mbar_init(&sh.v_full[s], 1);
            mbar_init(&sh.v_empty[s], 1);
            mbar_init(&sh.v_part[s], 1);
            mbar_init(&sh.v_ready[s], 1);
        }
        for (int s = 0; s < WORDS; s++) {
            mbar_init(&sh.t_full[s], 1);
            mbar_init(&sh.t_empty[s], 2);  // V, mending
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 4);
            mbar_init(&sh.p_full[i][1], 4);
            mbar_init(&sh.o_done[i], 1);
        }
        mbar_init(&sh.o_free, 8);
        mbar_init(&sh.ml_full, 8);
        fence_mbar_init();
        a.join[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    if (warp == 9) tmem_alloc(&sh.tmem, TM_COLS);
    const bool good = load_offsets(a.cu, a.B, a.n_tokens, a.max_nodes, nullptr, a.status);
    // work of all heads before each thread's share of them, and where this CTA's range begins
    int n = 1;
    if (good) {
        const int per = ceil_div(a.C, TC_THREADS), c_lo = min(a.C, (int)threadIdx.x * per), c_hi = min(a.C, c_lo + per);
        uint32_t sum = 0, total;
        for (int c = c_lo; c < c_hi; c++) {
            const Head h(a, c, nullptr);
            sum += (uint32_t)(h.items * (h.tiles + COST));
        }
        uint32_t pre = block_exclusive_scan(sum, scan, &total);
        n = max(1, min((int)gridDim.x, (int)(total / MIN_RANGE)));
        const int i = (int)blockIdx.x, begin = i < n ? cut((int)total, i, n) : 0, end = i < n ? cut((int)total, i + 1, n) : 0;
        if (threadIdx.x == 0) {
            sh.begin = begin;
            sh.end = end;
            sh.total = (int)total;
            sh.c0 = 0;
            sh.p0 = 0;
        }
        __syncthreads();
        if (begin < end && (uint32_t)begin >= pre && (uint32_t)begin < pre + sum)
            for (int c = c_lo; c < c_hi; c++) {
                const Head h(a, c, nullptr);
                const uint32_t wgt = (uint32_t)(h.items * (h.tiles + COST));
                if ((uint32_t)begin < pre + wgt) {
                    sh.c0 = c;
                    sh.p0 = (int)pre;
                    break;
                }
                pre += wgt;
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Room room(a.nt * a.G, D, Cfg<D>::ROOM - (int)sizeof(Shared) - 256);
    const Ctx<D> x{&sh, tiles, tiles + 2 * room.tile, a.status, room};
    if (good && sh.begin < sh.end) {
        if (warp < 8) softmax_role<D>(x, a);
        else if (warp == 8) load_role<D>(x, a, n, &tq, &tk, &dk);
        else if (warp == 10) value_role<D>(x, a, &tv, &dv);
        else if (warp == 11) mend_role<D>(x);
        else if (elect_one()) mma_role<D>(x, a.qscale < 0.f);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(sh.tmem, TM_COLS);
    }
}

// Joins the parts of the items that ranges' ends have cut: CTA (x, tile, 32
// columns) those of the item whose first part CTA x had; one thread a row.
template <int D>
__global__ void __launch_bounds__(QR) tree_join_kernel(const TreeArgs a) {
    wait_for_launcher();
    const int4 d = a.join[blockIdx.x];
    if (d.x < 0) return;
    const int c = d.x, node0 = d.y, last = d.z, tile = blockIdx.y, col = blockIdx.z * 32, row = threadIdx.x;
    const int b = c / a.LH, lh = c % a.LH, t0 = __ldg(a.cu + b), nodes = __ldg(a.cu + b + 1) - t0;
    const int node = node0 + tile * a.nt + row / a.G;
    if (row >= a.nt * a.G || node >= nodes) return;
    const float qscale = fabsf(a.qscale);
    const int first = (int)blockIdx.x;
    auto rec = [&](int p) { return a.rec + ((int64_t)(2 * p + (p == first)) * a.rec_tiles + tile) * (QR * (D + 2)) + row; };
    float m = -INFINITY;
    for (int p = first; p <= last; p++) {
        const float mp = __ldcg(rec(p) + D * QR);
        m = max_nan(m, mp, mp);  // a NaN row in any part is one in all
    }
    float l = 0.f, f[32];
#pragma unroll
    for (int e = 0; e < 32; e++) f[e] = 0.f;
    for (int p = first; p <= last; p++) {
        const float *r = rec(p);
        const float mp = __ldcg(r + D * QR);
        if (mp == -INFINITY) continue;  // the part's rows were all left out
        const float s = mp == m ? 1.f : ex2((mp - m) * qscale);
        l += __ldcg(r + (D + 1) * QR) * s;
#pragma unroll
        for (int e = 0; e < 32; e++) f[e] = fmaf(__ldcg(r + (col + e) * QR), s, f[e]);
    }
    // An infinite drafted value times a part's scale of 0 is NaN, where an item that is not cut gives the infinite
    // value: such columns are joined again with scales that are not 0.  (A look at every value in the first pass
    // costs a call of single tokens 5 of 93 us.)
    float nan = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e++) nan += f[e];
    if (nan != nan) {
#pragma unroll
        for (int e = 0; e < 32; e++) {
            if (f[e] == f[e]) continue;
            f[e] = 0.f;
#pragma unroll 1
            for (int p = first; p <= last; p++) {
                const float mp = __ldcg(rec(p) + D * QR);
                if (mp != -INFINITY) f[e] = fmaf(__ldcg(rec(p) + (col + e) * QR), mp == m ? 1.f : fmaxf(ex2((mp - m) * qscale), 0x1p-100f), f[e]);
            }
        }
    }
    const int64_t at = (int64_t)(t0 + node) * a.LH * a.G + (int64_t)lh * a.G + row % a.G;
    const bool none = m == -INFINITY;
    const float inv = none ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 32; e++) f[e] *= inv;
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + col);
#pragma unroll
    for (int e = 0; e < 4; e++)
        out[e] = make_uint4(pack_bf16(f[8 * e], f[8 * e + 1]), pack_bf16(f[8 * e + 2], f[8 * e + 3]),
                            pack_bf16(f[8 * e + 4], f[8 * e + 5]), pack_bf16(f[8 * e + 6], f[8 * e + 7]));
    if (a.lse && col == 0) a.lse[at] = none ? -INFINITY : (m * qscale + log2f(l)) * LN2;
}

template <int D>
cudaError_t launch(const TreeArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                   const CUtensorMap &dk, const CUtensorMap &dv, cudaStream_t s) {
    const Room room(a.nt * a.G, D, Cfg<D>::ROOM - (int)sizeof(Shared) - 256);
    // as much whatever the rows: a products' read of 128 rows stays inside
    const int smem = Cfg<D>::ROOM - (int)sizeof(Shared) - 256 + 1024;
    if (room.ks < 2 || room.vs < 2) return cudaErrorNotSupported;
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    tree_tc_kernel<D><<<TREE_CTAS, TC_THREADS, smem, s>>>(a, tq, tk, tv, dk, dv);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_after(tree_join_kernel<D>, dim3(TREE_CTAS, a.rec_tiles, D / 32), QR, 0, s, a);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs &a, int D, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                           const CUtensorMap &dk, const CUtensorMap &dv, cudaStream_t s) {
    return D == 64 ? launch<64>(a, tq, tk, tv, dk, dv, s) : launch<128>(a, tq, tk, tv, dk, dv, s);
}

}  // namespace rkv
