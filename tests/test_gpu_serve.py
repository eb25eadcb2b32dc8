"""The serving operators together, as a server runs them: prompts attend and enter the cache, a step evicts, a
sequence forks, a drafted tree attends, its accepted path is appended, and decoding goes on."""
import math

import numpy as np
import pytest
import torch

import workloads
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
