"""rkv_append_tokens and rkv_fork_sequences against a cache kept as lists:
tables, lengths, stack and pools bit for bit."""
import math

import numpy as np
import pytest
import torch

import workloads
from tests.serve_helpers import DTYPES, ListCache, starts

pytestmark = pytest.mark.gpu


def make(rkv, lengths, B, L=2, H=2, D=64, dtype="bf16", seed=1, max_pages=None, spare=40, max_nodes=0):
    cfg = workloads.small_config(L=L, H=H, G=2, D=D, B=B, T0=4000, kv_dtype=dtype)
    need = sum(-(-int(n) // 16) for n in lengths)
    dc = workloads.ragged_cache(cfg, seed, lengths, device="cuda", n_pages=need + spare, max_pages=max_pages)
    cache = rkv.Cache.from_tensors(dc, B, L, H, 2 * H)
    return dc, cache, rkv.Workspace(cache, max_nodes=max_nodes)


def rows(n, L, H, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(n, L, H, D, generator=g, device="cuda").to(DTYPES[dtype]) for _ in range(2))
    return k, v, -torch.rand(n, L, H, generator=g, device="cuda")


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("lens", [[1, 1, 1], [0, 17, 3], [200, 0, 33], [16, 15, 1]], ids=str)
@pytest.mark.parametrize("gather", [False, True])
def test_append_tokens(rkv, lens, dtype, D, gather):
    have = [0, 15, 16, 17, 31, 1, 0, 48, 100, 5, 32, 2]
    dc, cache, ws = make(rkv, have, 3, D=D, dtype=dtype, max_pages=24, spare=120)
    n = sum(lens)
    k, v, lb = rows(2 * n + 1 if gather else n, 2, 2, D, dtype)
    k[0, 0, 0, 1] = math.nan  # values are moved, not computed with
    tok = torch.randperm(2 * n + 1, device="cuda")[:n].to(torch.int32) if gather else None
    if gather:
        tok[-1] = tok[0]  # the same row twice
    pos0 = torch.tensor([5, 4000, 2**31 - 300], dtype=torch.int32, device="cuda")
    want = ListCache(dc)
    for _ in range(2):  # twice: the second starts in the middle of pages the first began
        want.append(4, starts(lens), pos0, k, v, lb, tok)
        rkv.append_tokens(cache, starts(lens), pos0, k, v, lb, ws, tok=tok)
        want.assert_same(dc)
    # 200 tokens twice do not fit a table of 24 pages beside the 17 to 48 entries that some heads hold
    full = any(n + 2 * lens[c // 4] > 24 * 16 for c, n in enumerate(have))
    assert ws.status() == (rkv.DEV_TABLE_OVERFLOW if full else 0)


def test_append_tokens_is_append_for_one(rkv):
    have = [0, 15, 16, 17, 31, 1, 0, 48]
    a, ca, wa = make(rkv, have, 2)
    b, cb, wb = make(rkv, have, 2)
    k, v, lb = rows(2, 2, 2, 64, "bf16")
    t = torch.tensor([7, 9], dtype=torch.int32, device="cuda")
    for _ in range(3):
        rkv.append(ca, t, k, v, lb, wa)
        rkv.append_tokens(cb, starts([1, 1]), t, k, v, lb, wb)
    ListCache(a).assert_same(b)


def test_append_many_rows_to_many_heads(rkv):
    """More rows than one sweep of the grid moves, odd heads, rows behind the last sequence unread."""
    rng = np.random.default_rng(3)
    have = rng.integers(0, 60, 5 * 3 * 7)
    dc, cache, ws = make(rkv, have, 5, L=3, H=7, D=64, max_pages=300, spare=9000)
    lens = [1500, 0, 2777, 1, 801]
    k, v, lb = rows(sum(lens) + 5, 3, 7, 64, "bf16")
    pos0 = torch.arange(5, dtype=torch.int32, device="cuda")
    want = ListCache(dc)
    table, at = want.tables, starts(lens)
    rkv.append_tokens(cache, at, pos0, k, v, lb, ws)
    assert ws.status() == 0
    got = ListCache(dc)
    free = list(want.free)
    for c, n in enumerate(have):
        b, (l, h) = c // 21, divmod(c % 21, 7)
        m, s = lens[b], int(at[b])
        need = -(-(n + m) // 16) - -(-n // 16)
        assert got.tables[c] == table[c] + [free.pop() for _ in range(need)] and got.lens[c] == n + m
        t = torch.tensor(got.tables[c], dtype=torch.long)
        assert torch.equal(got.k[t].reshape(-1, 64)[n: n + m], k[s: s + m, l, h].cpu())
        assert torch.equal(got.v[t].reshape(-1, 64)[n: n + m], v[s: s + m, l, h].cpu())
        assert torch.equal(got.lb[t].reshape(-1)[n: n + m], lb[s: s + m, l, h].cpu())
        assert torch.equal(got.pos[t].reshape(-1)[n: n + m], torch.arange(b, b + m, dtype=torch.int32))
        assert torch.equal(got.k[t].reshape(-1, 64)[:n], want.k[t].reshape(-1, 64)[:n])
    assert got.free == free


def test_append_tokens_errors_on_the_device(rkv):
    # a head without room in its table takes nothing; the others go on
    have = [0, 62, 3, 64]
    dc, cache, ws = make(rkv, have, 1, max_pages=4)
    k, v, lb = rows(3, 2, 2, 64, "bf16")
    pos0 = torch.tensor([70], dtype=torch.int32, device="cuda")
    want = ListCache(dc)
    want.append(4, starts([3]), pos0, k, v, lb)
    rkv.append_tokens(cache, starts([3]), pos0, k, v, lb, ws)
    want.assert_same(dc)
    assert ws.status() == rkv.DEV_TABLE_OVERFLOW
    # too few pages: the first head that finds too few and later ones that need some take nothing
    have = [1, 16, 3, 16, 15, 16, 2, 14]
    dc, cache, ws = make(rkv, have, 2, max_pages=8, spare=3)
    k, v, lb = rows(40, 2, 2, 64, "bf16")
    pos0 = torch.tensor([70, 80], dtype=torch.int32, device="cuda")
    want = ListCache(dc)
    want.append(4, starts([38, 2]), pos0, k, v, lb)
    rkv.append_tokens(cache, starts([38, 2]), pos0, k, v, lb, ws)
    want.assert_same(dc)
    assert ws.status() == rkv.DEV_POOL_EXHAUSTED
    # offsets that decrease: nothing happens; rows of tok outside the input are left out
    dc, cache, ws = make(rkv, have, 2, max_pages=8)
    want = ListCache(dc)
    cu = torch.tensor([0, 9, 5], dtype=torch.int32, device="cuda")
    rkv.append_tokens(cache, cu, pos0, k, v, lb, ws)
    want.assert_same(dc)
    assert ws.status() == rkv.DEV_BAD_INPUT
    rkv.workspace_init(ws)
    tok = torch.tensor([1, -1, 40, 2], dtype=torch.int32, device="cuda")
    rkv.append_tokens(cache, starts([2, 2]), pos0, k, v, lb, ws, tok=tok)
    assert ws.status() == rkv.DEV_BAD_INPUT and int(dc.len[0]) == 3
    rkv.workspace_init(ws)
    before = dc.len.clone()
    rkv.append_tokens(cache, starts([2, 2]), torch.tensor([-3, 2**31 - 2], dtype=torch.int32, device="cuda"), k, v, lb, ws)
    assert ws.status() == rkv.DEV_BAD_INPUT and torch.equal(dc.len, before)


PARENTS = [[0, 1, 2, 3], [0, 0, 0, 0], [3, 2, 1, 0], [1, 2, 3, 0], [-1, -1, -1, -1], [0, 3, 0, -1], [2, 2, 3, 3],
           [1, 0, 0, 1], [-1, 0, 1, 2]]


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 128)])
@pytest.mark.parametrize("parent", PARENTS, ids=str)
def test_fork(rkv, parent, dtype, D):
    have = [0, 15, 16, 17, 31, 1, 0, 48, 100, 5, 32, 200, 0, 0, 7, 64]
    dc, cache, ws = make(rkv, have, 4, D=D, dtype=dtype, spare=80)
    dc.v_pool.view(-1)[::97] = math.nan
    want = ListCache(dc)
    par = torch.tensor(parent, dtype=torch.int32, device="cuda")
    for _ in range(2):
        want.fork(4, parent)
        rkv.fork_sequences(cache, par, ws)
        want.assert_same(dc)
    assert ws.status() == 0


def test_fork_of_64_sequences_and_one(rkv):
    rng = np.random.default_rng(8)
    have = rng.integers(0, 150, 64 * 4)
    dc, cache, ws = make(rkv, have, 64, spare=2500)
    parent = [int(x) for x in rng.integers(-1, 64, 64)]
    want = ListCache(dc)
    want.fork(4, parent)
    rkv.fork_sequences(cache, torch.tensor(parent, dtype=torch.int32, device="cuda"), ws)
    want.assert_same(dc)
    dc, cache, ws = make(rkv, [3, 40, 0, 16], 1)
    want = ListCache(dc)
    for p in (0, -1):
        want.fork(4, [p])
        rkv.fork_sequences(cache, torch.tensor([p], dtype=torch.int32, device="cuda"), ws)
        want.assert_same(dc)


def test_fork_in_a_long_and_nearly_empty_table(rkv):
    have = [0, 900, 16, 1, 9, 33, 2000, 5]
    dc, cache, ws = make(rkv, have, 2, max_pages=5000, spare=300)
    want = ListCache(dc)
    for parent in ([0, 0], [1, 0], [-1, 1], [1, 1]):
        want.fork(4, parent)
        rkv.fork_sequences(cache, torch.tensor(parent, dtype=torch.int32, device="cuda"), ws)
        want.assert_same(dc)
    assert ws.status() == 0


def test_fork_without_room_or_with_bad_parents_changes_nothing(rkv):
    have = [40, 0, 16, 1, 9, 9, 9, 9]
    dc, cache, ws = make(rkv, have, 2, spare=0)
    want = ListCache(dc)
    # slot 1's four pages come back, five are needed
    rkv.fork_sequences(cache, torch.tensor([0, 0], dtype=torch.int32, device="cuda"), ws)
    want.assert_same(dc)
    assert ws.status() == rkv.DEV_POOL_EXHAUSTED
    rkv.workspace_init(ws)
    for bad in ([0, 2], [-2, 1]):
        rkv.fork_sequences(cache, torch.tensor(bad, dtype=torch.int32, device="cuda"), ws)
        want.assert_same(dc)
        assert ws.status() == rkv.DEV_BAD_INPUT
        rkv.workspace_init(ws)
    rkv.fork_sequences(cache, torch.tensor([1, 1], dtype=torch.int32, device="cuda"), ws)
    want.fork(4, [1, 1])
    want.assert_same(dc)
    assert ws.status() == 0


def test_captured_and_replayed(rkv):
    """One graph that appends and forks, replayed from the same bookkeeping with other values."""
    have = [0, 15, 16, 17, 31, 1, 0, 48]
    dc, cache, ws = make(rkv, have, 2, spare=60)
    k, v, lb = rows(9, 2, 2, 64, "bf16")
    cu, pos0 = starts([4, 5]), torch.tensor([100, 200], dtype=torch.int32, device="cuda")
    par = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    keep = dc.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rkv.append_tokens(cache, cu, pos0, k, v, lb, ws)
        rkv.fork_sequences(cache, par, ws)
    for seed, parent, lens in ((1, [1, 1], [4, 5]), (2, [1, 0], [9, 0]), (3, [-1, 0], [0, 7])):
        for f in ("k_pool", "v_pool", "pos_pool", "lb_pool", "block_table", "len", "free_stack", "free_top"):
            getattr(dc, f).copy_(getattr(keep, f))
        for x, y in zip((k, v, lb), rows(9, 2, 2, 64, "bf16", seed)):
            x.copy_(y)
        par.copy_(torch.tensor(parent))
        cu.copy_(starts(lens))
        want = ListCache(dc)
        want.append(4, cu, pos0, k, v, lb)
        want.fork(4, parent)
        graph.replay()
        want.assert_same(dc)
    assert ws.status() == 0


@pytest.mark.parametrize("parent", [[0, 1], [0, 0], [1, 0], [-1, 1], [-1, -1]], ids=str)
@pytest.mark.parametrize("max_pages", [9, 300])
def test_fork_over_a_table_with_stale_entries(rkv, parent, max_pages):
    """What a table holds past its heads' pages (a caller cut len back, or never cleared it) is -1 afterwards."""
    have = [0, 15, 16, 17, 100, 1, 0, 48]
    dc, cache, ws = make(rkv, have, 2, max_pages=max_pages, spare=80)
    for c, n in enumerate(have):
        dc.block_table[c, -(-n // 16):] = torch.randint(0, dc.n_pages, (max_pages - -(-n // 16),), device="cuda", dtype=torch.int32)
    want = ListCache(dc)
    want.fork(4, parent)
    rkv.fork_sequences(cache, torch.tensor(parent, dtype=torch.int32, device="cuda"), ws)
    want.assert_same(dc)
    assert ws.status() == 0


@pytest.mark.parametrize("parent", [[0, -1], [1, 1], [-1, -1]], ids=str)
def test_fork_with_a_stack_that_contradicts_the_tables(rkv, parent):
    """*free_top says that all pages are free while the heads hold some: pages given back would be pushed past the
    stack's end, so nothing is changed.  A page id outside the pool that is given back is recorded."""
    have = [40, 0, 16, 1, 9, 9, 30, 9]
    dc, cache, ws = make(rkv, have, 2, spare=20)
    par = torch.tensor(parent, dtype=torch.int32, device="cuda")
    real = dc.free_top.clone()
    dc.free_top.fill_(dc.n_pages)
    want = ListCache(dc)
    rkv.fork_sequences(cache, par, ws)
    want.assert_same(dc)
    assert ws.status() == rkv.DEV_BAD_INPUT
    rkv.workspace_init(ws)
    dc.free_top.copy_(real)
    want = ListCache(dc)
    want.fork(4, parent)
    rkv.fork_sequences(cache, par, ws)
    want.assert_same(dc)
    assert ws.status() == 0
    dc, cache, ws = make(rkv, have, 2, spare=20)
    for c in (0, 4):
        dc.block_table[c, 0] = dc.n_pages + 7
    rkv.fork_sequences(cache, torch.tensor([-1, -1], dtype=torch.int32, device="cuda"), ws)
    assert ws.status() == rkv.DEV_BAD_INPUT and not bool(dc.len.any())


@pytest.mark.parametrize("parent", [[0, 0, 0, 0], [0, 3, 0, -1], [1, 0, 0, 1]], ids=str)
def test_fork_of_fp32_rows_of_64(rkv, parent):
    have = [0, 15, 16, 17, 31, 1, 0, 48, 100, 5, 32, 200, 0, 0, 7, 64]
    dc, cache, ws = make(rkv, have, 4, D=64, dtype="f32", spare=80)
    want = ListCache(dc)
    for _ in range(2):
        want.fork(4, parent)
        rkv.fork_sequences(cache, torch.tensor(parent, dtype=torch.int32, device="cuda"), ws)
        want.assert_same(dc)
    assert ws.status() == 0
