"""rkv_prompt_attn against the operator's definition in 64 bits."""
import math

import pytest
import torch

import workloads
from tests.serve_helpers import DTYPES, assert_attention, attend64, starts

pytestmark = pytest.mark.gpu


def shape_cache(rkv, B, H, Hq, D, dtype):
    cfg = workloads.small_config(L=1, H=H, G=Hq // H, D=D, B=B, T0=16, kv_dtype=dtype)
    dc = workloads.ragged_cache(cfg, 5, [0] * cfg.C, device="cuda")
    cache = rkv.Cache.from_tensors(dc, B, 1, H, Hq)
    return cache, rkv.Workspace(cache)


def inputs(T, H, Hq, D, dtype, seed=0, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * H) * D, generator=g, device="cuda") * amp
    qkv = qkv.to(DTYPES[dtype])
    return [x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], dim=1)]


def check(q, k, v, out, lse, lens, scale, first=0):
    Hq, H, at = q.shape[1], k.shape[1], first
    for n in lens:
        below = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for h in range(Hq if n else 0):
            kv = h // (Hq // H)
            ref = attend64(q[at: at + n, h], k[at: at + n, kv], v[at: at + n, kv], scale, below)
            assert_attention(out[at: at + n, h], lse[at: at + n, h], ref, out.dtype, n)
        at += n


LENS = [[1], [2, 1, 3], [127], [128], [129, 1], [255, 256, 257], [0, 5, 0, 300, 0], [1000, 33], [1] * 40]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hq,D", [(4, 4, 64), (1, 8, 128), (4, 28, 128), (2, 4, 64)])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:6])))
def test_prompt_matches_definition(rkv, lens, H, Hq, D, dtype):
    cache, ws = shape_cache(rkv, len(lens), H, Hq, D, dtype)
    T, scale = sum(lens), 1 / math.sqrt(D)
    q, k, v = inputs(T, H, Hq, D, dtype, seed=T + D)
    out, lse = torch.empty(T, Hq, D, dtype=q.dtype, device="cuda"), torch.empty(T, Hq, device="cuda")
    rkv.prompt_attn(cache, starts(lens), q, k, v, scale, out, lse, ws)
    check(q, k, v, out, lse, lens, scale)
    assert ws.status() == 0
    again = torch.empty_like(out)
    rkv.prompt_attn(cache, starts(lens), q, k, v, scale, again, None, ws)
    assert torch.equal(out, again)  # the same bits, with and without lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_prompt_and_growing_logits(rkv, dtype):
    """Keys that grow along the sequence: the running maximum moves in every tile."""
    cache, ws = shape_cache(rkv, 1, 1, 2, 128, dtype)
    T = 2500
    q, k, v = inputs(T, 1, 2, 128, dtype, seed=9)
    ramp = torch.linspace(0.1, 6.0, T, device="cuda")[:, None, None]
    for kk in (k * ramp, k * ramp.flip(0)):
        kk = kk.to(k.dtype)
        out, lse = torch.empty(T, 2, 128, dtype=q.dtype, device="cuda"), torch.empty(T, 2, device="cuda")
        rkv.prompt_attn(cache, starts([T]), q, kk, v, 0.3, out, lse, ws)
        check(q, kk, v, out, lse, [T], 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_outside_the_sequences_stay(rkv, dtype):
    lens, first, behind = [70, 0, 131], 3, 9
    T = first + sum(lens) + behind
    cache, ws = shape_cache(rkv, 3, 2, 4, 64, dtype)
    q, k, v = inputs(T, 2, 4, 64, dtype)
    for x in (q, k, v):  # what no sequence holds may be anything
        x[:first] = math.nan
        x[T - behind:] = math.inf
    out = torch.full((T, 6, 64), 7.0, dtype=q.dtype, device="cuda")
    view, lse = out[:, 1:5], torch.full((T, 4), 7.0, device="cuda")  # a token stride wider than the heads
    rkv.prompt_attn(cache, starts(lens, first=first), q, k, v, 0.125, view, lse, ws)
    check(q, k, v, view, lse, lens, 0.125, first)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 5] == 7).all())
    assert bool((out[:first] == 7).all()) and bool((out[T - behind:] == 7).all())
    assert bool((lse[:first] == 7).all()) and bool((lse[T - behind:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 40, 130, 299])
def test_odd_values_reach_only_rows_that_attend_them(rkv, dtype, bad, at):
    """V of token `at` of the first of two sequences is odd: earlier rows and the other sequence are not touched."""
    lens = [300, 50]
    cache, ws = shape_cache(rkv, 2, 1, 2, 128, dtype)
    q, k, v = inputs(350, 1, 2, 128, dtype, seed=3)
    clean = v.clone()
    v[at, 0, 5] = bad
    out, lse = torch.empty(350, 2, 128, dtype=q.dtype, device="cuda"), torch.empty(350, 2, device="cuda")
    rkv.prompt_attn(cache, starts(lens), q, k, v, 0.1, out, lse, ws)
    want, wl = torch.empty_like(out), torch.empty_like(lse)
    rkv.prompt_attn(cache, starts(lens), q, k, clean, 0.1, want, wl, ws)
    check(q, k, clean, want, wl, lens, 0.1)
    hit = torch.zeros(350, dtype=torch.bool, device="cuda")
    hit[at:300] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse, wl)
    col = torch.arange(128, device="cuda") == 5
    assert torch.equal(out[hit][:, :, ~col], want[hit][:, :, ~col])
    got = out[hit][:, :, 5].float()
    assert bool(torch.isnan(got).all()) if math.isnan(bad) else bool((got == bad).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu", [[0, 5, 3], [-1, 5, 9], [0, 5, 21], [2, 2**31 - 1, 20]])
def test_bad_offsets_do_nothing(rkv, dtype, cu):
    cache, ws = shape_cache(rkv, 2, 2, 2, 64, dtype)
    q, k, v = inputs(20, 2, 2, 64, dtype)
    out = torch.full((20, 2, 64), 7.0, dtype=q.dtype, device="cuda")
    rkv.prompt_attn(cache, torch.tensor(cu, dtype=torch.int32, device="cuda"), q, k, v, 0.125, out, None, ws)
    assert bool((out == 7).all()) and ws.status() == rkv.DEV_BAD_INPUT


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_on_another_stream_and_replayed_on_new_values(rkv, dtype):
    lens = [200, 1, 77]
    cache, ws = shape_cache(rkv, 3, 2, 8, 128, dtype)
    T = sum(lens)
    q, k, v = inputs(T, 2, 8, 128, dtype, seed=1)
    cu = starts(lens)
    out, lse = torch.zeros(T, 8, 128, dtype=q.dtype, device="cuda"), torch.zeros(T, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rkv.prompt_attn(cache, cu, q, k, v, 0.1, out, lse, ws)  # warm-up
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rkv.prompt_attn(cache, cu, q, k, v, 0.1, out, lse, ws)
    for seed, ls in ((2, lens), (3, [3, 250, 25])):
        for x, y in zip((q, k, v), inputs(T, 2, 8, 128, dtype, seed=seed)):
            x.copy_(y)
        cu.copy_(starts(ls))
        graph.replay()
        check(q, k, v, out, lse, ls, 0.1)
    assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.4])
def test_scales_of_zero_and_below(rkv, scale, dtype):
    cache, ws = shape_cache(rkv, 2, 2, 4, 128, dtype)
    q, k, v = inputs(340, 2, 4, 128, dtype)
    out, lse = torch.empty(340, 4, 128, dtype=q.dtype, device="cuda"), torch.empty(340, 4, device="cuda")
    rkv.prompt_attn(cache, starts([300, 40]), q, k, v, scale, out, lse, ws)
    check(q, k, v, out, lse, [300, 40], scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_and_more_work_than_one_round(rkv, dtype):
    """1024 sequences, most of them empty or short, and several pieces of work for each SM."""
    lens = [(i * 37) % 11 if i % 5 else 0 for i in range(1021)] + [700, 1, 513]
    cache, ws = shape_cache(rkv, 1024, 1, 2, 64, dtype)
    T = sum(lens)
    q, k, v = inputs(T, 1, 2, 64, dtype)
    out, lse = torch.empty(T, 2, 64, dtype=q.dtype, device="cuda"), torch.empty(T, 2, device="cuda")
    rkv.prompt_attn(cache, starts(lens), q, k, v, 0.125, out, lse, ws)
    check(q, k, v, out, lse, lens, 0.125)
    assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_to_attend_and_nan_keys(rkv, dtype):
    """Only empty sequences: nothing is written.  A NaN key makes the rows that attend it NaN, and no others."""
    cache, ws = shape_cache(rkv, 2, 1, 2, 128, dtype)
    q, k, v = inputs(350, 1, 2, 128, dtype, seed=3)
    out, lse = torch.full((350, 2, 128), 7.0, dtype=q.dtype, device="cuda"), torch.full((350, 2), 7.0, device="cuda")
    rkv.prompt_attn(cache, starts([0, 0], first=5), q, k, v, 0.1, out, lse, ws)
    assert bool((out == 7).all()) and bool((lse == 7).all()) and ws.status() == 0
    k = k.clone()
    k[140, 0, 77] = math.nan
    rkv.prompt_attn(cache, starts([300, 50]), q, k, v, 0.1, out, lse, ws)
    hit = torch.zeros(350, dtype=torch.bool, device="cuda")
    hit[140:300] = True
    assert bool(torch.isnan(out[hit].float()).all()) and bool(torch.isnan(lse[hit]).all())
    k[140, 0, 77] = 0
    keep_out, keep_lse = out.clone(), lse.clone()
    rkv.prompt_attn(cache, starts([300, 50]), q, k, v, 0.1, out, lse, ws)
    check(q, k, v, out, lse, [300, 50], 0.1)
    assert torch.equal(out[~hit], keep_out[~hit]) and torch.equal(lse[~hit], keep_lse[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_of_any_stride(rkv, dtype):
    """The stride between tokens says nothing where there is only one."""
    cache, ws = shape_cache(rkv, 1, 2, 4, 64, dtype)
    q, k, v = (x.contiguous() for x in inputs(1, 2, 4, 64, dtype))
    views = [x[0].unsqueeze(1).transpose(0, 1) for x in (q, k, v)]  # [1, heads, D], 64 elements between tokens
    assert all(x.stride(0) == 64 for x in views)
    odd = [torch.as_strided(x, x.shape, (7, 64, 1)) for x in (q, k, v)]
    for qq, kk, vv in (views, odd):
        out, lse = torch.empty(4, 1, 64, dtype=q.dtype, device="cuda").transpose(0, 1), torch.empty(1, 4, device="cuda")
        rkv.prompt_attn(cache, starts([1]), qq, kk, vv, 0.125, out, lse, ws)
        check(q, k, v, out, lse, [1], 0.125)
    assert ws.status() == 0
