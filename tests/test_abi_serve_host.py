"""Host-side refusals of the serving operators: each is refused before the
first CUDA call (the pointers are placeholders that nothing may touch)."""
import ctypes

import pytest
import torch

from tests.test_abi_host import _cache, lib  # noqa: F401  (fixture)


def _prompt(rkv, so, cs, **kw):
    a = dict(cu=16, n=8, q=16, qs=1024, k=16, ks=512, v=16, vs=512, out=16, os=1024, ws=16, nbytes=None)
    a.update(kw)
    n = so.rkv_workspace_size(ctypes.byref(cs)) if a["nbytes"] is None else a["nbytes"]
    return so.rkv_prompt_attn(ctypes.byref(cs), a["cu"], a["n"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], 0.1, a["out"],
                              a["os"], None, a["ws"], n, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(cu=None), -1, "cu"), (dict(n=0), -1, "positive"), (dict(q=None), -1, "non-NULL"), (dict(out=None), -1, "non-NULL"),
    (dict(q=8), -1, "aligned"), (dict(ks=513), -1, "aligned"), (dict(qs=512), -1, "below"), (dict(vs=0), -1, "below"),
    (dict(ws=None), -1, "workspace"), (dict(nbytes=64), -3, "needed"),
])
def test_prompt_refusals(lib, kw, code, needle):  # noqa: F811
    rkv, so = lib
    assert _prompt(rkv, so, _cache(rkv), **kw) == code
    assert needle in so.rkv_last_error().decode()


@pytest.mark.parametrize("kw,needle", [(dict(D=96), "not built"), (dict(B=1025), "at most 1024"), (dict(D=256), "not built")])
def test_prompt_unsupported(lib, kw, needle):  # noqa: F811
    rkv, so = lib
    assert _prompt(rkv, so, _cache(rkv, **kw), qs=4096, ks=4096, vs=4096, os=4096) == rkv.ERR_UNSUPPORTED
    assert needle in so.rkv_last_error().decode()


def _tree(rkv, so, cs, **kw):
    a = dict(cu=16, n=8, nodes=8, q=16, k=16, v=16, mask=16, sel=None, out=16, nbytes=None)
    a.update(kw)
    n = so.rkv_tree_workspace_size(ctypes.byref(cs), max(1, min(64, a["nodes"]))) if a["nbytes"] is None else a["nbytes"]
    sel = ctypes.byref(a["sel"]) if a["sel"] is not None else None
    return so.rkv_tree_attn(ctypes.byref(cs), a["cu"], a["n"], a["nodes"], a["q"], a["k"], a["v"], a["mask"], 0.1, sel, a["out"], None,
                            16, n, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(cu=None), -1, "cu"), (dict(n=-1), -1, "positive"), (dict(nodes=0), -1, "max_nodes"), (dict(nodes=65), -1, "max_nodes"),
    (dict(mask=None), -1, "non-NULL"), (dict(k=24), -1, "aligned"), (dict(nbytes=64), -3, "needed"),
])
def test_tree_refusals(lib, kw, code, needle):  # noqa: F811
    rkv, so = lib
    assert _tree(rkv, so, _cache(rkv), **kw) == code
    assert needle in so.rkv_last_error().decode()


def test_tree_selection_workspace_and_shapes(lib):  # noqa: F811
    rkv, so = lib
    cs = _cache(rkv)
    assert _tree(rkv, so, cs, sel=rkv.SelectStruct(16, 16, 16, None, 16)) == -1
    assert "keep_mask" in so.rkv_last_error().decode()
    # the shared workspace alone is too small for trees
    base = so.rkv_workspace_size(ctypes.byref(cs))
    assert so.rkv_tree_workspace_size(ctypes.byref(cs), 8) > base
    assert _tree(rkv, so, cs, nbytes=base) == rkv.ERR_WORKSPACE_TOO_SMALL
    for n in (0, 65, -1):
        assert so.rkv_tree_workspace_size(ctypes.byref(cs), n) == 0
    assert so.rkv_tree_workspace_size(ctypes.byref(_cache(rkv, P=8)), 8) == 0
    assert _tree(rkv, so, _cache(rkv, D=32)) == rkv.ERR_UNSUPPORTED
    assert _tree(rkv, so, _cache(rkv, H=1, Hq=65)) == rkv.ERR_UNSUPPORTED
    assert "65" not in so.rkv_last_error().decode() and "64 query heads" in so.rkv_last_error().decode()


def _append(rkv, so, cs, **kw):
    a = dict(cu=16, tok=None, n_new=8, pos0=16, k=16, v=16, lb=16, n_rows=8, nbytes=None)
    a.update(kw)
    n = so.rkv_workspace_size(ctypes.byref(cs)) if a["nbytes"] is None else a["nbytes"]
    return so.rkv_append_tokens(ctypes.byref(cs), a["cu"], a["tok"], a["n_new"], a["pos0"], a["k"], a["v"], a["lb"], a["n_rows"], 16, n,
                                None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(cu=None), -1, "cu"), (dict(n_new=0), -1, "positive"), (dict(pos0=None), -1, "NULL"), (dict(lb=None), -1, "NULL"),
    (dict(k=24), -1, "aligned"), (dict(n_rows=7), -1, "n_rows"), (dict(tok=16, n_rows=0), -1, "n_rows"), (dict(nbytes=64), -3, "needed"),
])
def test_append_tokens_refusals(lib, kw, code, needle):  # noqa: F811
    rkv, so = lib
    assert _append(rkv, so, _cache(rkv), **kw) == code
    assert needle in so.rkv_last_error().decode()


def test_append_tokens_and_fork_unsupported(lib):  # noqa: F811
    rkv, so = lib
    assert _append(rkv, so, _cache(rkv, D=96)) == rkv.ERR_UNSUPPORTED
    assert _append(rkv, so, _cache(rkv, B=1025)) == rkv.ERR_UNSUPPORTED
    fork = lambda cs, parent, n=None: so.rkv_fork_sequences(  # noqa: E731
        ctypes.byref(cs), parent, 16, so.rkv_workspace_size(ctypes.byref(cs)) if n is None else n, None)
    assert fork(_cache(rkv), None) == rkv.ERR_INVALID_ARG and "parent" in so.rkv_last_error().decode()
    assert fork(_cache(rkv, B=65), 16) == rkv.ERR_UNSUPPORTED and "64" in so.rkv_last_error().decode()
    assert fork(_cache(rkv, D=32), 16) == rkv.ERR_UNSUPPORTED
    assert fork(_cache(rkv), 16, 10) == rkv.ERR_WORKSPACE_TOO_SMALL
    assert fork(_cache(rkv, k_pool=None), 16) == rkv.ERR_INVALID_ARG


def test_binding_refuses_wrong_tensors(lib):  # noqa: F811
    """The binding checks shapes, types and strides (CPU tensors stand in; nothing is launched)."""
    rkv, _ = lib
    import workloads
    cfg = workloads.small_config(L=1, H=2, G=2, D=64, B=2, T0=16)
    dc = workloads.ragged_cache(cfg, 1, [3] * cfg.C)
    cache = rkv.Cache.from_tensors(dc, 2, 1, 2, 4)
    cu = torch.zeros(3, dtype=torch.int32)
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    call = lambda **kw: rkv.prompt_attn(cache, **{**dict(cu=cu, q=q, k=k, v=k, scale=1.0, out=q, lse=None, ws=None), **kw})  # noqa: E731
    for kw in (dict(q=q.float()), dict(k=k[:4]), dict(v=k[:, :1]), dict(cu=cu.long()), dict(cu=cu[:2]), dict(lse=torch.zeros(5, 4).T),
               dict(q=torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), dict(out=q.expand(5, 4, 64)[:, :, ::2])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        rkv.fork_sequences(cache, torch.zeros(2, dtype=torch.int64), None)
    with pytest.raises(ValueError):
        rkv.tree_attn(cache, cu, q[:, None], k[:, None], k[:, None], torch.zeros(5, dtype=torch.int32), 1.0, None, q[:, None], None, None,
                      max_nodes=4)
    with pytest.raises(ValueError):
        rkv.append_tokens(cache, cu, cu[:2], k, k, torch.zeros(5, 1, 2), None)


def test_fork_refuses_tables_past_its_scan(lib):  # noqa: F811
    """1,024 heads of 2^22 pages are 2^32: the scan's sums would wrap."""
    rkv, so = lib
    fork = lambda cs: so.rkv_fork_sequences(ctypes.byref(cs), 16, 16, 64, None)  # noqa: E731
    assert fork(_cache(rkv, max_pages=1 << 22)) == rkv.ERR_UNSUPPORTED and "2^22" in so.rkv_last_error().decode()
    assert fork(_cache(rkv, max_pages=(1 << 22) - 1)) == rkv.ERR_WORKSPACE_TOO_SMALL


def test_append_refuses_more_pages_than_its_sums_hold(lib):  # noqa: F811
    """2^18 heads that each take 2^21 / 16 pages are 2^35: the plan's 32-bit sums would wrap to 0, and heads would
    take pages that are not free."""
    rkv, so = lib
    cs = _cache(rkv, L=1 << 16, H=4, Hq=4, max_pages=1 << 17)
    args = dict(tok=16, n_rows=8, nbytes=64)
    assert _append(rkv, so, cs, n_new=1 << 21, **args) == rkv.ERR_UNSUPPORTED and "2^31" in so.rkv_last_error().decode()
    # (8190 + 1) * 2^18 is below 2^31, (8191 + 1) * 2^18 is 2^31
    assert _append(rkv, so, cs, n_new=8190 * 16 + 15, **args) == rkv.ERR_WORKSPACE_TOO_SMALL
    assert _append(rkv, so, cs, n_new=8191 * 16, **args) == rkv.ERR_UNSUPPORTED


def test_tree_refuses_more_work_than_its_positions_number(lib):  # noqa: F811
    """64 query heads a KV head: two tokens a query tile, sixteen items of 64 nodes.  2^14 heads of 2^16 pages are then
    2^31 key tiles: the kernel's 32-bit ranges would wrap."""
    rkv, so = lib
    cs = _cache(rkv, L=1 << 14, H=1, Hq=64, n_pages=1 << 20, max_pages=1 << 16)
    big = 1 << 62  # the workspace is large enough; nothing is read before the refusal
    assert _tree(rkv, so, cs, nodes=64, nbytes=big) == rkv.ERR_UNSUPPORTED and "key tiles" in so.rkv_last_error().decode()


def test_binding_refuses_what_would_be_read_out_of_range(lib):  # noqa: F811
    """A keep mask of another cache's shape, and a workspace on another device (nothing is launched)."""
    rkv, _ = lib
    import types

    import workloads
    cfg = workloads.small_config(L=1, H=2, G=2, D=64, B=2, T0=16)
    cache = rkv.Cache.from_tensors(workloads.ragged_cache(cfg, 1, [3] * cfg.C), 2, 1, 2, 4)
    cu, bf = torch.zeros(3, dtype=torch.int32), torch.bfloat16
    q, k = torch.zeros(5, 1, 4, 64, dtype=bf), torch.zeros(5, 1, 2, 64, dtype=bf)
    here = types.SimpleNamespace(buf=torch.zeros(16), ptr=0, nbytes=0)
    away = types.SimpleNamespace(buf=torch.zeros(16, device="meta"), ptr=0, nbytes=0)
    sel = rkv.Selection.empty(cache)
    tree = lambda sel, ws: rkv.tree_attn(cache, cu, q, k, k, torch.zeros(5, dtype=torch.int64), 1.0, sel, q, None, ws, max_nodes=4)  # noqa: E731
    with pytest.raises(ValueError, match="ws"):
        tree(sel, away)
    with pytest.raises(ValueError, match="ws"):
        rkv.prompt_attn(cache, cu, q[:, 0], k[:, 0], k[:, 0], 1.0, q[:, 0], None, away)
    with pytest.raises(ValueError, match="ws"):
        rkv.append_tokens(cache, cu, cu[:2], k, k, torch.zeros(5, 1, 2), away)
    with pytest.raises(ValueError, match="ws"):
        rkv.fork_sequences(cache, cu[:2], away)
    sel.keep_mask = sel.keep_mask[:, 1:].contiguous()
    with pytest.raises(ValueError, match="keep_mask"):
        tree(sel, here)
    sel.keep_mask = torch.zeros(cache.C, cache.max_pages, dtype=torch.int32)
    with pytest.raises(ValueError, match="keep_mask"):
        tree(sel, here)
