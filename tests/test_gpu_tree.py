"""rkv_tree_attn against the operator's definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import workloads
from tests.serve_helpers import DTYPES, assert_attention, attend64, starts

pytestmark = pytest.mark.gpu


def make(rkv, have, B, L, H, G, D, dtype, max_nodes, seed=1, max_pages=None):
    cfg = workloads.small_config(L=L, H=H, G=G, D=D, B=B, T0=40000, kv_dtype=dtype)
    dc = workloads.ragged_cache(cfg, seed, have, device="cuda", max_pages=max_pages)
    cache = rkv.Cache.from_tensors(dc, B, L, H, H * G)
    return dc, cache, rkv.Workspace(cache, max_nodes=max_nodes)


def draft(T, L, H, G, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h: torch.randn(T, L, h, D, generator=g, device="cuda").to(DTYPES[dtype])  # noqa: E731
    return r(H * G), r(H), r(H)


def tree_masks(nodes, seed=0, blank=()):
    r, out = np.random.default_rng(seed), []
    for n in nodes:
        m = []
        for i in range(n):
            m.append((m[r.integers(0, i)] if i and r.random() < 0.9 else 0) | 1 << i)
        out += [0 if i in blank else x for i, x in enumerate(m)]
    return torch.from_numpy(np.array(out, np.uint64).view(np.int64)).cuda()


def keep_words(sel, frac, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = torch.rand(*sel.keep_mask.shape, 16, generator=g, device="cuda") < frac
    sel.keep_mask.copy_((bits.int() << torch.arange(16, device="cuda")).sum(-1).to(torch.int16))
    return bits.reshape(bits.shape[0], -1)


def check(dc, q, kd, vd, mask, nodes, scale, out, lse, keep=None, first=0):
    L, H, D = kd.shape[1:]
    G, at, words = q.shape[2] // H, first, mask.cpu().numpy().view(np.uint64)
    lens = [int(x) for x in dc.len.cpu()]
    for b, n in enumerate(nodes):
        sees = torch.tensor([[bool(int(words[at + i]) >> j & 1) for j in range(n)] for i in range(n)], device="cuda").reshape(n, n)
        for l in range(L if n else 0):
            for h in range(H):
                c = (b * L + l) * H + h
                m = lens[c]
                pages = dc.block_table[c, : -(-m // 16)].long()
                here = keep[c, :m] if keep is not None else torch.ones(m, dtype=torch.bool, device="cuda")
                k = torch.cat([dc.k_pool[pages].reshape(-1, D)[:m][here], kd[at: at + n, l, h]])
                v = torch.cat([dc.v_pool[pages].reshape(-1, D)[:m][here], vd[at: at + n, l, h]])
                allowed = torch.cat([torch.ones(n, int(here.sum()), dtype=torch.bool, device="cuda"), sees], 1)
                qq = q[at: at + n, l, h * G: h * G + G].reshape(n * G, D)
                ref = attend64(qq, k, v, scale, allowed.repeat_interleave(G, 0))
                assert_attention(out[at: at + n, l, h * G: h * G + G].reshape(n * G, D),
                                 lse[at: at + n, l, h * G: h * G + G].reshape(-1), ref, out.dtype, k.shape[0])
        at += n


def outputs(q):
    return torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,H,G,D", [(1, 2, 1, 64), (2, 1, 4, 128), (1, 2, 7, 128), (1, 1, 8, 64), (1, 1, 12, 128)])
@pytest.mark.parametrize("nodes", [[1, 1, 1], [5, 0, 64], [17, 33, 16], [64, 64, 63]], ids=str)
def test_tree_matches_definition(rkv, nodes, L, H, G, D, dtype):
    rng = np.random.default_rng(sum(nodes) + G)
    have = rng.choice([0, 1, 15, 16, 17, 127, 128, 129, 250, 600], 3 * L * H)
    dc, cache, ws = make(rkv, have, 3, L, H, G, D, dtype, 64)
    q, kd, vd = draft(sum(nodes), L, H, G, D, dtype)
    mask, scale = tree_masks(nodes), 1 / math.sqrt(D)
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, scale, None, out, lse, ws, max_nodes=max(nodes))
    check(dc, q, kd, vd, mask, nodes, scale, out, lse)
    again, _ = outputs(q)
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, scale, None, again, None, ws, max_nodes=64)
    assert ws.status() == 0
    check(dc, q, kd, vd, mask, nodes, scale, again, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("frac", [0.0, 0.1, 0.9])
def test_keep_masks_and_rows_that_attend_nothing(rkv, frac, dtype):
    nodes = [9, 20]
    dc, cache, ws = make(rkv, [0, 40, 333, 16, 700, 5, 0, 128], 2, 2, 2, 4, 128, dtype, 20)
    sel = rkv.Selection.empty(cache)
    keep = keep_words(sel, frac, 3)
    q, kd, vd = draft(29, 2, 2, 4, 128, dtype)
    mask = tree_masks(nodes, blank=(2, 8))
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, 0.09, sel, out, lse, ws, max_nodes=20)
    check(dc, q, kd, vd, mask, nodes, 0.09, out, lse, keep)
    assert ws.status() == 0
    if frac == 0.0:
        assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_ragged_heads(rkv, dtype):
    """One long head among short ones: its keys are shared out and joined."""
    nodes = [24]
    dc, cache, ws = make(rkv, [30000, 3, 0, 9000, 16, 17, 2000, 100], 1, 4, 2, 4, 128, dtype, 24)
    q, kd, vd = draft(24, 4, 2, 4, 128, dtype)
    mask = tree_masks(nodes, seed=4)
    out, lse = outputs(q)
    for scale in (0.088, 0.6):
        rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, scale, None, out, lse, ws, max_nodes=24)
        check(dc, q, kd, vd, mask, nodes, scale, out, lse)
    first = out.clone()
    for _ in range(3):  # the same bits whatever order the parts end in
        rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, 0.6, None, out, lse, ws, max_nodes=24)
        assert torch.equal(first, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_odd_values_in_places_that_do_not_count(rkv, dtype, bad):
    """Free pages, rows past a head's end, evicted rows and rows behind the last sequence may hold anything;
    a drafted token's odd V reaches only the tokens that attend it."""
    nodes, D = [6, 18], 128
    have = [0, 40, 333, 16, 130, 5, 0, 129]
    dc, cache, ws = make(rkv, have, 2, 2, 2, 4, D, dtype, 18)
    sel = rkv.Selection.empty(cache)
    keep = keep_words(sel, 0.7, 5)
    live = torch.zeros(dc.n_pages, 16, dtype=torch.bool, device="cuda")
    for c, n in enumerate(have):
        for s in range(n):
            if keep[c, s]:
                live[int(dc.block_table[c, s // 16]), s % 16] = True
    dc.k_pool[~live] = bad
    dc.v_pool[~live] = bad
    q, kd, vd = draft(27, 2, 2, 4, D, dtype)
    for x in (q, kd, vd):
        x[24:] = bad
    mask = tree_masks([6, 18, 3])
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, 0.09, sel, out, lse, ws, max_nodes=18)
    check(dc, q, kd, vd, mask, nodes, 0.09, out, lse, keep)
    assert bool((out[24:] == 7).all()) and bool((lse[24:] == 7).all())
    clean = out.clone()
    vd[6 + 3, 1, 0, 77] = bad  # node 3 of the second tree
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, 0.09, sel, out, lse, ws, max_nodes=18)
    hit = torch.zeros_like(out, dtype=torch.bool)
    words = mask.cpu().numpy().view(np.uint64)
    for i in range(18):
        if int(words[6 + i]) >> 3 & 1:
            hit[6 + i, 1, 0:4, 77] = True
    assert bool(hit.any()) and torch.equal(out[~hit], clean[~hit])
    got = out[hit].float()
    assert bool(torch.isnan(got).all()) if math.isnan(bad) else bool((got == bad).all())
    assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_is_a_decode_step_after_its_append(rkv, dtype):
    """mask 1: the same attention as appending the token and decoding over the cache."""
    have = [0, 40, 333, 16, 130, 5, 15, 129]
    dc, cache, ws = make(rkv, have, 2, 2, 2, 4, 64, dtype, 1)
    q, kd, vd = draft(2, 2, 2, 4, 64, dtype)
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts([1, 1]), q, kd, vd, torch.ones(2, dtype=torch.int64, device="cuda"), 0.125, None, out, lse, ws,
                  max_nodes=1)
    t = torch.tensor([40001, 40002], dtype=torch.int32, device="cuda")
    rkv.append(cache, t, kd.reshape(8, 64), vd.reshape(8, 64), torch.zeros(8, device="cuda"), ws)
    o2, l2 = torch.empty(2, 2, 8, 64, device="cuda"), torch.empty(2, 2, 8, device="cuda")
    rkv.paged_decode_attn(cache, q.float(), 0.125, None, o2, l2, None, ws)
    # both are within their own bounds of the same value: 2e-3 of the row's norm for the decode step,
    # two bf16 half steps of sum p |v| (at most its largest |v|) for the tree
    lim = 2e-3 * o2.norm(dim=-1, keepdim=True) + (2 * 2.0 ** -8 * 6.0 if dtype == "bf16" else 1e-4)
    assert bool(((out.float() - o2).abs() <= lim).all())
    assert bool(((lse - l2).abs() <= 1e-4 + 2e-5 * l2.abs()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages_lengths_and_offsets(rkv, dtype):
    have = [40, 64, 33, 20]
    dc, cache, ws = make(rkv, have, 2, 1, 2, 2, 64, dtype, 8, max_pages=6)
    q, kd, vd = draft(9, 1, 2, 2, 64, dtype)
    mask = tree_masks([4, 5])
    out, lse = outputs(q)
    for cu in ([0, 9, 4], [-1, 3, 9], [0, 4, 10]):  # the second sequence of [0, 1, 10] would also be too long
        rkv.tree_attn(cache, torch.tensor(cu, dtype=torch.int32, device="cuda"), q, kd, vd, mask, 0.1, None, out, lse, ws, max_nodes=8)
        assert bool((out == 7).all()) and ws.status() == rkv.DEV_BAD_INPUT
        rkv.workspace_init(ws)
    rkv.tree_attn(cache, starts([0, 9]), q, kd, vd, mask, 0.1, None, out, lse, ws, max_nodes=8)
    assert bool((out == 7).all()) and ws.status() == rkv.DEV_BAD_INPUT
    rkv.workspace_init(ws)
    # a page id outside the pool: its rows count as evicted
    dc.block_table[1, 1] = dc.n_pages
    dc.block_table[2, 0] = -1
    keep = torch.ones(4, 6 * 16, dtype=torch.bool, device="cuda")
    keep[1, 16:32] = False
    keep[2, :16] = False
    rkv.tree_attn(cache, starts([4, 5]), q, kd, vd, mask, 0.1, None, out, lse, ws, max_nodes=8)
    assert ws.status() == rkv.DEV_BAD_INPUT
    dc.block_table[1, 1] = dc.block_table[2, 0] = 0  # for the definition's gather: masked there
    check(dc, q, kd, vd, mask, [4, 5], 0.1, out, lse, keep)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed_with_other_trees(rkv, dtype):
    dc, cache, ws = make(rkv, [900, 40, 333, 16, 130, 5, 15, 129], 2, 2, 2, 4, 128, dtype, 40)
    q, kd, vd = draft(50, 2, 2, 4, 128, dtype)
    mask, cu = tree_masks([10, 40]), starts([10, 40])
    out, lse = outputs(q)
    args = (cache, cu, q, kd, vd, mask, 0.09, None, out, lse, ws)
    rkv.tree_attn(*args, max_nodes=40)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rkv.tree_attn(*args, max_nodes=40)
        rkv.tree_attn(*args, max_nodes=40)
    for seed, nodes in ((2, [10, 40]), (3, [40, 1]), (4, [0, 40])):
        for x, y in zip((q, kd, vd), draft(50, 2, 2, 4, 128, dtype, seed)):
            x.copy_(y)
        mask[: sum(nodes)] = tree_masks(nodes, seed)
        cu.copy_(starts(nodes))
        dc.len[0] = 100 * seed
        graph.replay()
        check(dc, q, kd, vd, mask, nodes, 0.09, out, lse)
    assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.4])
def test_scales_of_zero_and_below(rkv, scale, dtype):
    """0: the mean of what is attended; negative: the order of the logits turns round."""
    nodes = [5, 40]
    dc, cache, ws = make(rkv, [200, 40, 0, 129], 2, 1, 2, 4, 64, dtype, 40)
    q, kd, vd = draft(45, 1, 2, 4, 64, dtype)
    mask = tree_masks(nodes, blank=(1,))
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, scale, None, out, lse, ws, max_nodes=40)
    check(dc, q, kd, vd, mask, nodes, scale, out, lse)


def test_calls_of_different_sizes_share_a_workspace(rkv):
    """Small trees after large ones and back, in turn with the decode step's calls."""
    for dtype in ("bf16", "f32"):
        dc, cache, ws = make(rkv, [900, 40, 333, 16], 1, 2, 2, 4, 128, dtype, 64)
        for n in (64, 1, 30, 64, 3, 64):
            q, kd, vd = draft(n, 2, 2, 4, 128, dtype, n)
            mask = tree_masks([n], n)
            out, lse = outputs(q)
            rkv.tree_attn(cache, starts([n]), q, kd, vd, mask, 0.09, None, out, lse, ws, max_nodes=n)
            check(dc, q, kd, vd, mask, [n], 0.09, out, lse)
            o2 = torch.empty(1, 2, 8, 128, device="cuda")
            rkv.paged_decode_attn(cache, q[:1].float().contiguous(), 0.09, None, o2, None, None, ws)
        assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_trees_at_all(rkv, dtype):
    dc, cache, ws = make(rkv, [200, 40, 0, 129], 2, 1, 2, 4, 64, dtype, 8)
    q, kd, vd = draft(3, 1, 2, 4, 64, dtype)
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts([0, 0], first=1), q, kd, vd, tree_masks([3]), 0.1, None, out, lse, ws, max_nodes=8)
    assert bool((out == 7).all()) and bool((lse == 7).all()) and ws.status() == 0


@pytest.mark.parametrize("G,nodes,D", [(7, [1, 1, 1], 128), (1, [1, 1, 1], 64), (4, [3, 1, 9], 128)])
def test_warps_without_rows_over_many_key_tiles(rkv, G, nodes, D):
    """Few rows: three of a warpgroup's four warps have none and only pass the key tiles on, many hundred of them,
    whole and partial ones in turn.  No wait gives up and every call gives the same bits."""
    have = [20000, 1, 130, 9000, 128, 0, 5000, 127, 30000, 16, 3000, 257]
    dc, cache, ws = make(rkv, have, 3, 2, 2, G, D, "bf16", max(nodes))
    sel = rkv.Selection.empty(cache)
    keep = keep_words(sel, 0.995, 6)  # about every second key tile is whole
    q, kd, vd = draft(sum(nodes), 2, 2, G, D, "bf16")
    mask, cu = tree_masks(nodes), starts(nodes)
    out, lse = outputs(q)
    rkv.tree_attn(cache, cu, q, kd, vd, mask, 0.09, sel, out, lse, ws, max_nodes=max(nodes))
    check(dc, q, kd, vd, mask, nodes, 0.09, out, lse, keep)
    again, l2 = outputs(q)
    for _ in range(200):
        rkv.tree_attn(cache, cu, q, kd, vd, mask, 0.09, sel, again, l2, ws, max_nodes=max(nodes))
    assert torch.equal(out, again) and torch.equal(lse, l2) and ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,nodes", [(4, [9]), (7, [1]), (8, [20])], ids=str)
@pytest.mark.parametrize("have", [[470, 150], [0, 40, 127, 1000, 6000]], ids=str)
def test_nan_keys_and_queries(rkv, have, G, nodes, dtype):
    """A NaN in a key or a query makes out and lse of the rows that attend it NaN, and changes no other row: on heads
    of one key tile (470 entries are four, cut after the third), of two query tiles (20 nodes of 8 heads), and on
    heads cut into parts."""
    n, H, D = nodes[0], len(have), 128
    dc, cache, ws = make(rkv, have, 1, 1, H, G, D, dtype, n)
    q, kd, vd = draft(n, 1, H, G, D, dtype)
    mask, cu = tree_masks(nodes), starts(nodes)
    words = mask.cpu().numpy().view(np.uint64)
    clean, cl = outputs(q)
    rkv.tree_attn(cache, cu, q, kd, vd, mask, 0.09, None, clean, cl, ws, max_nodes=n)
    check(dc, q, kd, vd, mask, nodes, 0.09, clean, cl)

    def run_with(place, hit, what):
        old = place.clone()
        place.fill_(math.nan)
        out, lse = outputs(q)
        rkv.tree_attn(cache, cu, q, kd, vd, mask, 0.09, None, out, lse, ws, max_nodes=n)
        place.copy_(old)
        assert bool(torch.isnan(out[hit].float()).all()), f"{what}: out"
        assert bool(torch.isnan(lse[hit]).all()), f"{what}: lse {lse[hit]}"
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], cl[~hit]), f"{what}: other rows"

    rows = lambda: torch.zeros(n, 1, H * G, dtype=torch.bool, device="cuda")  # noqa: E731
    for h, m in enumerate(have):
        for slot in sorted({0, m // 2, m - 54, m - 1}) if m else ():
            if slot < 0:
                continue
            hit = rows()
            hit[:, 0, h * G: h * G + G] = True
            page = int(dc.block_table[h, slot // 16])
            run_with(dc.k_pool[page, slot % 16, 5], hit, f"key {slot} of head {h}")
        for j in (0, n - 1):
            hit = rows()
            for i in range(n):
                hit[i, 0, h * G: h * G + G] = bool(int(words[i]) >> j & 1)
            run_with(kd[j, 0, h, 5], hit, f"drafted key {j} of head {h}")
        hit = rows()
        hit[n // 2, 0, h * G + G - 1] = True
        run_with(q[n // 2, 0, h * G + G - 1, 5], hit, f"query of head {h}")
    assert ws.status() == 0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("nodes", [[9], [40]], ids=str)
def test_odd_drafted_values_far_below_the_maximum(rkv, nodes, bad):
    """Cached logits near +200, drafted ones near -200: the drafted weights are 0 in fp32, but not in the definition,
    so an infinite drafted value is the result of the rows that attend it, whether or not a range's end cuts their
    head (384 entries are three key tiles and the draft a fourth, alone behind the cut; 150 and the draft are two)."""
    have, G, D, n = [384, 150], 4, 128, nodes[0]
    dc, cache, ws = make(rkv, have, 1, 1, 2, G, D, "bf16", n)
    q, kd, vd = draft(n, 1, 2, G, D, "bf16")
    q.fill_(1.0)
    kd.fill_(-200.0 / D)
    dc.k_pool.fill_(200.0 / D)
    mask, cu = tree_masks(nodes), starts(nodes)
    words = mask.cpu().numpy().view(np.uint64)
    clean, cl = outputs(q)
    rkv.tree_attn(cache, cu, q, kd, vd, mask, 1.0, None, clean, cl, ws, max_nodes=n)
    check(dc, q, kd, vd, mask, nodes, 1.0, clean, cl)
    for h in range(2):
        keep = vd[3, 0, h, 77].clone()
        vd[3, 0, h, 77] = bad
        out, lse = outputs(q)
        rkv.tree_attn(cache, cu, q, kd, vd, mask, 1.0, None, out, lse, ws, max_nodes=n)
        vd[3, 0, h, 77] = keep
        hit = torch.zeros_like(out, dtype=torch.bool)
        for i in range(n):
            if int(words[i]) >> 3 & 1:
                hit[i, 0, h * G: h * G + G, 77] = True
        got = out[hit].float()
        assert bool(torch.isnan(got).all()) if math.isnan(bad) else bool((got == bad).all()), f"head {h}: {got}"
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, cl)
    assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_page_that_no_kept_entry_lies_on_is_not_looked_at(rkv, dtype):
    """A page id outside the pool is bad input only where an entry that counts lies on it."""
    dc, cache, ws = make(rkv, [40, 64, 33, 20], 2, 1, 2, 2, 64, dtype, 8, max_pages=6)
    q, kd, vd = draft(9, 1, 2, 2, 64, dtype)
    mask, cu = tree_masks([4, 5]), starts([4, 5])
    sel = rkv.Selection.empty(cache)
    keep = torch.ones(4, 6 * 16, dtype=torch.bool, device="cuda")
    keep[1, 16:32] = False
    keep[2, 32] = False
    sel.keep_mask.copy_((keep.view(4, 6, 16).int() << torch.arange(16, device="cuda")).sum(-1).to(torch.int16))
    out, lse = outputs(q)
    dc.block_table[1, 1] = dc.n_pages
    dc.block_table[2, 2] = -1   # its kept bits lie past the head's 33 entries
    rkv.tree_attn(cache, cu, q, kd, vd, mask, 0.1, sel, out, lse, ws, max_nodes=8)
    assert ws.status() == 0
    dc.block_table[1, 1] = dc.block_table[2, 2] = 0  # for the definition's gather: masked there
    check(dc, q, kd, vd, mask, [4, 5], 0.1, out, lse, keep)
    dc.block_table[2, 1] = -1
    rkv.tree_attn(cache, cu, q, kd, vd, mask, 0.1, sel, out, lse, ws, max_nodes=8)
    assert ws.status() == rkv.DEV_BAD_INPUT


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,D", [(13, 64), (16, 128), (33, 64), (33, 128), (64, 64), (64, 128)])
def test_many_query_heads_on_one_kv_head(rkv, G, D, dtype):
    """Up to 64 query heads a KV head: query tiles of two whole tokens, up to sixteen items of a head."""
    nodes, scale = [1, 64, 7, 0], 1 / math.sqrt(D)
    dc, cache, ws = make(rkv, [130, 0, 17, 600, 16, 250, 40, 5], 4, 1, 2, G, D, dtype, 64)
    q, kd, vd = draft(sum(nodes), 1, 2, G, D, dtype)
    mask = tree_masks(nodes, blank=(3,))
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, scale, None, out, lse, ws, max_nodes=64)
    check(dc, q, kd, vd, mask, nodes, scale, out, lse)
    assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_against_the_decode_step_in_its_own_rounding(rkv, dtype):
    """As test_one_token_is_a_decode_step_after_its_append, in bounds that scale with the row.  The tree is off by half
    a step of the pool type from each rounded weight, relative to sum p |v|, and from the result; the decode
    step by 2e-3 of the row's norm."""
    have = [0, 40, 333, 16, 130, 5, 15, 129]
    dc, cache, ws = make(rkv, have, 2, 2, 2, 4, 64, dtype, 1)
    q, kd, vd = draft(2, 2, 2, 4, 64, dtype)
    out, lse = outputs(q)
    rkv.tree_attn(cache, starts([1, 1]), q, kd, vd, torch.ones(2, dtype=torch.int64, device="cuda"), 0.125, None, out, lse, ws,
                  max_nodes=1)
    t = torch.tensor([40001, 40002], dtype=torch.int32, device="cuda")
    rkv.append(cache, t, kd.reshape(8, 64), vd.reshape(8, 64), torch.zeros(8, device="cuda"), ws)
    o2 = torch.empty(2, 2, 8, 64, device="cuda")
    rkv.paged_decode_attn(cache, q.float(), 0.125, None, o2, None, None, ws)
    half = torch.finfo(out.dtype).eps / 2
    for c, m in enumerate(have):
        b, (l, h) = c // 4, divmod(c % 4, 2)
        pages = dc.block_table[c, : -(-(m + 1) // 16)].long()
        k, v = (x[pages].reshape(-1, 64)[: m + 1] for x in (dc.k_pool, dc.v_pool))
        ref = attend64(q[b, l, h * 4: h * 4 + 4], k, v, 0.125, torch.ones(4, m + 1, dtype=torch.bool, device="cuda"))
        got, want = out[b, l, h * 4: h * 4 + 4].double(), o2[b, l, h * 4: h * 4 + 4].double()
        lim = (half if dtype == "bf16" else 2.0 ** -16) * (1 + 2 ** -6) * (ref[2] + want.abs()) + 2e-3 * ref[0].norm(dim=-1, keepdim=True)
        assert bool(((got - want).abs() <= lim).all())
    assert ws.status() == 0
