"""The serving operators together, as a server runs them: prompts attend and enter the cache, a step evicts, a
sequence forks, a drafted tree attends, its accepted path is appended, and decoding goes on."""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests.gpu_helpers import compare_state, keep_flags, masked_keep, rkv_cache
from tests.oracle_helpers import host_cache
from tests.serve_helpers import DTYPES, ListCache, assert_attention, attend64, starts
from tests.test_gpu_prompt import check as check_prompt
from tests.test_gpu_tree import check as check_tree, tree_masks

pytestmark = pytest.mark.gpu


def held(lists, c):
    """K and V rows of head c in slot order, on the GPU."""
    t, n = torch.tensor(lists.tables[c], dtype=torch.long), lists.lens[c]
    D = lists.k.shape[-1]
    return lists.k[t].reshape(-1, D)[:n].cuda(), lists.v[t].reshape(-1, D)[:n].cuda()


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype,G,D", [("bf16", 4, 128), ("bf16", 7, 128), ("f32", 1, 64)])
def test_prompt_to_speculative_decoding(rkv, dtype, G, D, fused):
    B, L, H = 3, 2, 2
    Hq, LH, scale, dt = H * G, L * H, 1 / math.sqrt(D), DTYPES[dtype]
    cfg = workloads.small_config(L=L, H=H, G=G, D=D, B=B, T0=16, kv_dtype=dtype)
    dc = workloads.ragged_cache(cfg, 2, [0] * cfg.C, device="cuda", n_pages=400, max_pages=40)
    cache = rkv.Cache.from_tensors(dc, B, L, H, Hq)
    ws = rkv.Workspace(cache, max_nodes=8)
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731

    # prompts, layer by layer over slices of the rows that enter the cache
    lens = [300, 45, 130]
    T, cu = sum(lens), starts(lens)
    q, k, v = rand(T, L, Hq, D), rand(T, L, H, D), rand(T, L, H, D)
    lb = -torch.rand(T, L, H, generator=g, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(T, Hq, device="cuda")
    for l in range(L):
        rkv.prompt_attn(cache, cu, q[:, l], k[:, l], v[:, l], scale, out[:, l], lse, ws)
        check_prompt(q[:, l], k[:, l], v[:, l], out[:, l], lse, lens, scale)
    lists = ListCache(dc)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    rkv.append_tokens(cache, cu, zero, k, v, lb, ws)
    lists.append(LH, cu, zero, k, v, lb)
    lists.assert_same(dc)

    # the prefill eviction and a first token
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    budget = [400, 100, 2000]
    sel, outs = rkv.Selection.empty(cache), rkv.StepOutputs.empty(cache)
    rkv.step(cache, sel, ws, outs, q=torch.randn(B, L, Hq, D, generator=g, device="cuda"), t=t,
             m_global=torch.tensor(budget, dtype=torch.int64, device="cuda"), k_new=rand(cfg.C, D), v_new=rand(cfg.C, D),
             lb_new=-torch.rand(cfg.C, generator=g, device="cuda"), evict=True, fused=fused)
    kept = [min(m, n * LH) for m, n in zip(budget, lens)]
    assert [int(x) for x in dc.len.view(B, LH).sum(1).cpu()] == [m + LH for m in kept]

    # sequence 0 goes on twice, sequence 2 as it is, sequence 1 ends
    lists = ListCache(dc)
    rkv.fork_sequences(cache, torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda"), ws)
    lists.fork(LH, [0, 0, 2])
    lists.assert_same(dc)

    # a drafted tree for each, and its accepted path
    nodes = [8, 5, 1]
    n = sum(nodes)
    q, kd, vd, mask = rand(n, L, Hq, D), rand(n, L, H, D), rand(n, L, H, D), tree_masks(nodes, 3)
    out, lse = torch.empty_like(q), torch.empty(n, L, Hq, device="cuda")
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, scale, None, out, lse, ws, max_nodes=8)
    check_tree(dc, q, kd, vd, mask, nodes, scale, out, lse)
    words, first, path = mask.cpu().numpy().view(np.uint64), [0, 8, 13], []
    for f, m in zip(first, nodes):  # from the last drafted token up to its root
        path.append([f + j for j in range(m) if int(words[f + m - 1]) >> j & 1])
    acc, tok = starts([len(p) for p in path]), torch.tensor(sum(path, []), dtype=torch.int32, device="cuda")
    t = torch.tensor([301, 301, 131], dtype=torch.int32, device="cuda")
    lb = -torch.rand(n, L, H, generator=g, device="cuda")
    rkv.append_tokens(cache, acc, t, kd, vd, lb, ws, tok=tok)
    lists.append(LH, acc, t, kd, vd, lb, tok)
    lists.assert_same(dc)

    # decoding goes on over what is there
    qf = torch.randn(B, L, Hq, D, generator=g, device="cuda")
    t = t + torch.tensor([len(p) for p in path], dtype=torch.int32, device="cuda")
    k1, v1, lb1 = rand(cfg.C, D), rand(cfg.C, D), -torch.rand(cfg.C, generator=g, device="cuda")
    rkv.step(cache, sel, ws, outs, q=qf, t=t, m_global=None, k_new=k1, v_new=v1, lb_new=lb1, evict=False, fused=fused)
    for c in range(cfg.C):
        kc, vc = held(lists, c)
        rows = qf.view(cfg.C, G, D)[c]
        o = attend64(rows, kc, vc, scale, torch.ones(G, kc.shape[0], dtype=torch.bool, device="cuda"))[0]
        err = (outs.out.view(cfg.C, G, D)[c].double() - o).abs().amax(-1)
        assert bool((err <= 2e-3 * o.norm(dim=-1)).all())  # the decode attention's own tolerance
    lists.append(LH, starts([1] * B), t, k1.view(B, L, H, D), v1.view(B, L, H, D), lb1.view(B, L, H))
    lists.assert_same(dc)
    assert ws.status() == 0


def test_two_caches_on_two_streams(rkv):
    """Calls on workspaces of their own overlap freely: the same bits as one after the other."""
    calls, want = [], []
    for i, (nodes, have) in enumerate((([64], [3000, 17, 900, 40]), ([9], [50, 2500, 700, 0]))):
        cfg = workloads.small_config(L=2, H=2, G=4, D=128, B=1, T0=40000)
        dc = workloads.ragged_cache(cfg, i, have, device="cuda")
        cache = rkv.Cache.from_tensors(dc, 1, 2, 2, 8)
        ws = rkv.Workspace(cache, max_nodes=64)
        g = torch.Generator(device="cuda").manual_seed(i)
        q = torch.randn(nodes[0], 2, 8, 128, generator=g, device="cuda").bfloat16()
        kd, vd = (torch.randn(nodes[0], 2, 2, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        calls.append((cache, starts(nodes), q, kd, vd, tree_masks(nodes), 0.1, None, torch.empty_like(q), None, ws))
        rkv.tree_attn(*calls[-1], max_nodes=64)
        want.append(calls[-1][8].clone())
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c[8].record_stream(s)
            rkv.tree_attn(*c, max_nodes=64, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c[8], w) and c[-1].status() == 0


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_evictions_after_forks_and_accepted_rows(rkv, dtype, fused):
    """The workspace keeps a threshold window per sequence from the last eviction.  After a fork, or rows appended by
    the dozen, it belongs to other entries: what is kept must not depend on it."""
    cfg = workloads.small_config(L=2, H=2, G=4, D=64, B=3, T0=900, M=1100, kv_dtype=dtype, steps=8)
    dc = workloads.prefill_cache(cfg, 5, n_steps=100).to("cuda")
    cache, LH = rkv_cache(rkv, dc), cfg.L * cfg.H
    sel, ws, outs = rkv.Selection.empty(cache), rkv.Workspace(cache), rkv.StepOutputs.empty(cache)
    t = torch.full((3,), cfg.T0, dtype=torch.int32, device="cuda")

    def evicting_step(s, budget):
        nonlocal t
        inp = workloads.step_inputs(cfg, 5, s, "cuda")
        mg = torch.tensor(budget, dtype=torch.int64, device="cuda")
        hc, before = host_cache(dc), dc.len.cpu().numpy()
        rkv.step(cache, sel, ws, outs, q=inp["q"], t=t, m_global=mg, k_new=inp["k_new"], v_new=inp["v_new"], lb_new=inp["lb_new"],
                 evict=True, fused=fused)
        ref = oracle.step(hc, t.cpu().numpy(), mg.cpu().numpy(), inp["q"].cpu().numpy().reshape(cfg.C, cfg.G, cfg.D),
                          workloads.rows_to_host(inp["k_new"]), workloads.rows_to_host(inp["v_new"]), inp["lb_new"].cpu().numpy(),
                          evict=True, scale=cfg.scale)
        assert ws.status() == 0
        assert np.array_equal(sel.kept.cpu().numpy(), ref["kept"])
        assert np.array_equal(masked_keep(keep_flags(sel, dc.max_pages), before), ref["keep"])
        compare_state(dc, hc)
        t = t + 1

    def fork(parent):
        nonlocal t
        lists = ListCache(dc)
        lists.fork(LH, parent)
        rkv.fork_sequences(cache, torch.tensor(parent, dtype=torch.int32, device="cuda"), ws)
        lists.assert_same(dc)
        t = t[torch.tensor([max(0, p) for p in parent], device="cuda")].contiguous()

    def accept(counts, seed):
        nonlocal t
        n, dt = sum(counts), dc.k_pool.dtype
        g = torch.Generator(device="cuda").manual_seed(seed)
        k, v = (torch.randn(n, cfg.L, cfg.H, cfg.D, generator=g, device="cuda").to(dt) for _ in range(2))
        lb = -torch.rand(n, cfg.L, cfg.H, generator=g, device="cuda") * 1e-3
        lists = ListCache(dc)
        lists.append(LH, starts(counts), t, k, v, lb)
        rkv.append_tokens(cache, starts(counts), t, k, v, lb, ws)
        lists.assert_same(dc)
        t = t + torch.tensor(counts, dtype=torch.int32, device="cuda")

    # windows of three sequences far apart
    evicting_step(0, [3000, 1500, 200])
    evicting_step(1, [2990, 1490, 190])
    fork([2, 0, 1])                       # each window now belongs to another sequence
    evicting_step(2, [150, 2980, 1480])
    fork([1, 1, 1])                       # samples of one
    evicting_step(3, [2900, 2000, 100])
    accept([7, 0, 31], 1)
    evicting_step(4, [2900, 2000, 150])
    fork([-1, 2, 0])                      # one ends: nothing to keep there
    accept([0, 3, 12], 2)
    evicting_step(5, [50, 100, 2500])
    accept([40, 1, 1], 3)                 # a new sequence in its place
    evicting_step(6, [100, 60, 2000])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pools_past_32_bits(rkv, dtype):
    """Pages whose first element lies at 2^31 and beyond: append, fork and tree reach them."""
    B, L, H, G, D, n_pages, max_pages = 2, 1, 2, 4, 128, (1 << 20) + 4096, 40
    dt, C = DTYPES[dtype], B * L * H
    g = torch.Generator(device="cuda").manual_seed(1)
    zeros = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)  # noqa: E731
    k_pool, v_pool = (torch.empty(n_pages, 16, D, dtype=dt, device="cuda") for _ in range(2))
    pos, lb = zeros(n_pages, 16, dtype=torch.int32), zeros(n_pages, 16)
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")  # the top of the stack is the highest page
    cache = rkv.Cache(k_pool, v_pool, pos, lb, torch.full((C, max_pages), -1, dtype=torch.int32, device="cuda"),
                      zeros(C, dtype=torch.int32), free, torch.tensor([n_pages], dtype=torch.int32, device="cuda"), B, L, H, H * G)
    ws = rkv.Workspace(cache, max_nodes=8)
    lens = [500, 77]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    k, v, lbn = rand(577, L, H, D), rand(577, L, H, D), -torch.rand(577, L, H, generator=g, device="cuda")
    zero = zeros(B, dtype=torch.int32)
    rkv.append_tokens(cache, starts(lens), zero, k, v, lbn, ws)
    rkv.fork_sequences(cache, torch.tensor([1, 1], dtype=torch.int32, device="cuda"), ws)  # 0 ends, 1 goes on twice
    nodes = [8, 3]
    q, kd, vd, mask = rand(11, L, H * G, D), rand(11, L, H, D), rand(11, L, H, D), tree_masks(nodes, 3)
    out, lse = torch.empty_like(q), torch.empty(11, L, H * G, device="cuda")
    rkv.tree_attn(cache, starts(nodes), q, kd, vd, mask, 0.09, None, out, lse, ws, max_nodes=8)
    assert ws.status() == 0 and cache.len.tolist() == [77] * 4
    assert int(cache.block_table.max()) < n_pages and int(cache.block_table[:, :5].min()) >= 1 << 20
    for c in range(C):
        pages = cache.block_table[c, :5].long()
        for pool, rows in ((k_pool, k), (v_pool, v)):
            assert torch.equal(pool[pages].reshape(-1, D)[:77], rows[500:, 0, c % 2])
        assert torch.equal(lb[pages].reshape(-1)[:77], lbn[500:, 0, c % 2])
        assert pos[pages].reshape(-1)[:77].tolist() == list(range(77))
    check_tree(cache, q, kd, vd, mask, nodes, 0.09, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_past_32_bits(rkv, dtype):
    """1,024 prompts of 342 tokens in one projection's output of 48 heads of 128: 2.15e9 elements."""
    B, n, H, Hq, D = 1024, 342, 8, 32, 128
    cfg = workloads.small_config(L=1, H=H, G=Hq // H, D=D, B=B, T0=16, kv_dtype=dtype)
    dc = workloads.ragged_cache(cfg, 5, [0] * cfg.C, device="cuda", n_pages=4)
    cache = rkv.Cache.from_tensors(dc, B, 1, H, Hq)
    ws = rkv.Workspace(cache)
    T = B * n
    assert T * (Hq + 2 * H) * D > 2 ** 31
    qkv = torch.empty(T, (Hq + 2 * H) * D, dtype=DTYPES[dtype], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for b in (0, 511, 1022, 1023):  # the others may hold anything
        qkv[b * n: b * n + n] = torch.randn(n, qkv.shape[1], generator=g, device="cuda").to(qkv.dtype)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], dim=1))
    out, lse = torch.empty(T, Hq, D, dtype=qkv.dtype, device="cuda"), torch.empty(T, Hq, device="cuda")
    rkv.prompt_attn(cache, starts([n] * B), q, k, v, 0.09, out, lse, ws)
    for b in (0, 511, 1022, 1023):
        check_prompt(q, k, v, out, lse, [n], 0.09, first=b * n)
    assert ws.status() == 0
