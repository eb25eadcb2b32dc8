"""The serving operators around the retention-scored cache, as cases to measure.

Four operators of `retention_scored_kv_b200`: `prompt_attn` (causal attention over packed prompts),
`append_tokens` (many tokens per sequence into the paged cache), `tree_attn` (a tree of drafted tokens over
the ragged cache) and `fork_sequences` (copying, moving and freeing whole sequences' pages).

`run` computes them in plain torch where `own` is false and through the library where it is true; `exact`
restates each operator in 64 bits.
"""
import math
from types import SimpleNamespace

import numpy as np
import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _text(values):
    return ",".join(str(int(v)) for v in values)


def listed():
    # heads of an 8B-class model (32 query heads on 8 KV heads of 128), of a vision-language model (28 on 4)
    # and of a small fp32 one (4 heads of 64)
    h8, vl, tiny = dict(Hq=32, H=8, D=128), dict(Hq=28, H=4, D=128), dict(Hq=4, H=4, D=64)
    return [
        # one whole long prompt, one layer: the step before its cache is cut to 2,048 entries a head
        dict(name="prompt_32k", op="prompt", dtype="bf16", lens="32768", **h8),
        # a batch of sixteen prompts of different lengths up to 8K, packed
        dict(name="prompt_batch_8k", op="prompt", dtype="bf16",
             lens="8192,517,4099,1,7168,2048,333,6011,8191,95,1500,3777,5120,16,2600,7001", **h8),
        # short chat turns, where latency counts
        dict(name="prompt_short", op="prompt", dtype="bf16", lens="129,1,64,200", **vl),
        # the fp32 model
        dict(name="prompt_f32", op="prompt", dtype="f32", lens="512,1000,77", **tiny),
        # the prompts of four sequences enter the cache of all layers
        dict(name="append_prompts", op="append", dtype="bf16", L=32, lens="6000,4097,1,5555", have=0, gather=False, **h8),
        # the accepted paths of sixteen drafted trees enter it: one to seven tokens a sequence
        dict(name="append_accepted", op="append", dtype="bf16", L=36, lens="1,3,2,7,1,4,5,2,1,6,3,2,1,1,4,0", have=512, gather=True,
             **h8),
        # a drafted tree of 24 nodes over what is left of a 128K context (10 % of its entries)
        dict(name="tree_long", op="tree", dtype="bf16", L=32, nodes="24", have=13107, keep=1.0, blank=0, **h8),
        # sixteen trees of different sizes over 512 entries a head on average
        dict(name="tree_batch", op="tree", dtype="bf16", L=36, nodes="64,31,48,7,16,64,1,25,60,12,33,5,64,20,40,9", have=512, keep=1.0,
             blank=0, **h8),
        # single tokens of a batch of eight, over an evicting step's keep masks
        dict(name="tree_single", op="tree", dtype="bf16", L=28, nodes="1,1,1,1,1,1,1,1", have=512, keep=0.9, blank=0, **vl),
        # the fp32 model, with nodes that attend nothing drafted and heads that hold nothing
        dict(name="tree_f32", op="tree", dtype="f32", L=2, nodes="17,3", have=700, keep=0.5, blank=2, **tiny),
        # one prompt's survivors become eight parallel samples
        dict(name="fork_samples", op="fork", dtype="bf16", L=32, parent="0,0,0,0,0,0,0,0", have=2048, **h8),
        # four beams reorder: one goes on, one moves, one is copied, one ends
        dict(name="fork_beams", op="fork", dtype="bf16", L=28, parent="0,3,0,-1", have=130, **vl),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "append", "tree", "tree", "fork"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    H = rng.choice((1, 2, 4, 8))
    c = dict(op=op, dtype=dtype, H=H, Hq=H * rng.choice((1, 2, 4, 7, 8)), D=rng.choice((64, 128)))
    if op == "prompt":
        left, lens = (16384 if dtype == "bf16" else 2048), []
        for _ in range(_spread(rng, 1, 24)):
            n = _spread(rng, 1, max(1, left))
            lens.append(n)
            left = max(1, left - n)
        return dict(c, lens=_text(lens))
    B, L = _spread(rng, 1, 12), _spread(rng, 1, 32)
    rows = 6000000 // (B * L * H)  # entries of a head, so that a pool holds about 6M rows at most
    if op == "append":
        gather = rng.random() < 0.5
        return dict(c, L=L, have=_spread(rng, 1, max(1, min(2000, rows // 2))), gather=gather,
                    lens=_text([1] + [rng.choice((0, 1)) if rng.random() < 0.2 else _spread(rng, 1, 16 if gather else max(1, min(6000, rows // 4)))
                                      for _ in range(B)]))
    if op == "tree":
        return dict(c, L=L, have=_spread(rng, 1, max(1, min(20000, rows // (2 if dtype == "bf16" else 8)))), keep=rng.choice((1.0, 1.0, 0.5, 0.1)),
                    blank=rng.choice((0, 0, 3)), nodes=_text([_spread(rng, 1, 64) for _ in range(B)]))
    parent = [rng.randrange(-1, B) for _ in range(B)] + [0, 0]  # one sequence at least is copied
    return dict(c, L=L, have=_spread(rng, 1, max(1, min(8000, rows // 6))), parent=_text(parent))


def _head_lens(case, B):
    """Entries of each head: ragged, as a budget over all heads leaves them; the same for every seed."""
    LH = case["L"] * case["H"]
    if case["have"] == 0:
        return np.zeros(B * LH, np.int64)
    r = np.random.RandomState(1000 + case["have"] + 7 * B + 13 * LH)
    n = r.randint(0, 2 * case["have"] + 1, B * LH)
    n[r.random_sample(B * LH) < 0.02] = 0
    return n.astype(np.int64)


def work(case):
    eb, D, H, Hq = (2 if case["dtype"] == "bf16" else 4), case["D"], case["H"], case["Hq"]
    r = D * eb
    if case["op"] == "prompt":
        lens = _ints(case["lens"])
        T = sum(lens)
        return {"bytes": T * ((2 * Hq + 2 * H) * r + 4 * Hq), "flops": 4.0 * D * Hq * sum(n * (n + 1) / 2 for n in lens)}
    LH = case["L"] * H
    if case["op"] == "append":
        n = sum(_ints(case["lens"])) * LH
        return {"bytes": n * (2 * (2 * r + 4) + 4), "flops": 0}
    if case["op"] == "tree":
        nodes = _ints(case["nodes"])
        have = _head_lens(case, len(nodes))
        # without the keep masks every row of a head is read; of the dropped ones nothing is needed
        kept = have * case["keep"]
        per = np.repeat(np.array(nodes, np.float64), LH)
        T = sum(nodes)
        return {"bytes": kept.sum() * 2 * r + T * LH * 2 * r + T * case["L"] * Hq * (2 * r + 4),
                "flops": 4.0 * D * (Hq // H) * float((per * (kept + (per + 1) / 2)).sum())}
    parent = _ints(case["parent"])
    have = _head_lens(case, len(parent)).reshape(len(parent), LH).sum(1)
    copied = [p for p, c in zip(parent, _copies(parent)) if c]
    rows = sum(have[p] for p in copied) + sum(have[p] for p in set(copied))  # written, and read once for all copies
    return {"bytes": float(rows) * (2 * r + 8) + 8 * len(parent) * LH, "flops": 0}


def _copies(parent):
    """Whether slot b's pages are copies: it continues another slot whose pages go elsewhere."""
    heir = {}
    for b, p in enumerate(parent):
        if p >= 0 and (p not in heir or p == b):
            heir[p] = b
    return [p >= 0 and heir[p] != b for b, p in enumerate(parent)]


# ------------------------------------------------------------------ the inputs
def _cache(case, B, head_lens, room, spare, g):
    """A cache in the middle of decoding: head c holds head_lens[c] entries on pages from all over the pool.
    The bookkeeping (tables, lengths, free pages) lies in one buffer, `book`, with a snapshot beside it."""
    L, H, D, dt = case["L"], case["H"], case["D"], DTYPES[case["dtype"]]
    C = B * L * H
    need = -(-head_lens // PAGE)
    max_pages = int(max(1, (-(-(head_lens + room) // PAGE)).max()))
    n_pages = int(need.sum() + spare + 8)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    s = SimpleNamespace(B=B, L=L, H=H, Hq=case["Hq"], D=D, C=C, n_pages=n_pages, max_pages=max_pages, dtype=dt)
    sizes = [C * max_pages, C, n_pages, 1]
    s.book = torch.empty(sum(sizes), dtype=torch.int32, device="cuda")
    table, s.len, s.free_stack, s.free_top = s.book.split(sizes)
    s.block_table = table.view(C, max_pages)
    need_d = torch.from_numpy(need).cuda()
    p = torch.arange(max_pages, device="cuda")
    first = need_d.cumsum(0) - need_d
    at = (first[:, None] + p[None, :]).clamp_max(n_pages - 1)
    s.block_table.copy_(torch.where(p[None, :] < need_d[:, None], order[at], -1))
    s.len.copy_(torch.from_numpy(head_lens).cuda())
    used = int(need.sum())
    s.free_stack.fill_(-1)
    s.free_stack[: n_pages - used] = order[used:]
    s.free_top.fill_(n_pages - used)
    s.book0 = s.book.clone()
    s.k_pool = torch.randn(n_pages, PAGE, D, generator=g, device="cuda", dtype=dt)
    s.v_pool = torch.randn(n_pages, PAGE, D, generator=g, device="cuda", dtype=dt)
    s.pos_pool = torch.randint(0, 1 << 20, (n_pages, PAGE), generator=g, device="cuda", dtype=torch.int32)
    s.lb_pool = -torch.rand(n_pages, PAGE, generator=g, device="cuda")
    return s


def _handle(s, max_nodes=0):
    """What a program that calls the library keeps beside its tensors: the cache's handle and its workspace."""
    import retention_scored_kv_b200 as rkv
    s.rkv = rkv
    s.cache = rkv.Cache(s.k_pool, s.v_pool, s.pos_pool, s.lb_pool, s.block_table, s.len, s.free_stack, s.free_top, s.B, s.L, s.H, s.Hq)
    s.ws = rkv.Workspace(s.cache, max_nodes=max_nodes)


def _starts(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt, D, H, Hq = case["op"], DTYPES[case["dtype"]], case["D"], case["H"], case["Hq"]
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=dt)  # noqa: E731
    if op == "prompt":
        lens = _ints(case["lens"])
        T = sum(lens)
        s = _cache(dict(case, L=1, have=0), len(lens), np.zeros(len(lens) * H, np.int64), 16, 0, g)
        # one projection's output, as a model has it: the query, key and value heads of a token side by side
        qkv = randn(T, (Hq + 2 * H) * D)
        s.q, s.k, s.v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], dim=1))
        s.out = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
        s.lse = torch.zeros(T, Hq, device="cuda")
        s.lens, s.cu = lens, _starts(lens)
        if own:
            _handle(s)
    elif op == "append":
        lens = _ints(case["lens"])
        B, n = len(lens), sum(lens)
        have = _head_lens(case, B)
        LH = case["L"] * H
        most = np.repeat(np.array(lens), LH)
        s = _cache(case, B, have, most, int((-(-(have + most) // PAGE) + (-have // PAGE)).sum()), g)
        rows = 4 * n + 3 if case["gather"] else n
        s.k_new, s.v_new = randn(rows, case["L"], H, D), randn(rows, case["L"], H, D)
        s.lb_new = -torch.rand(rows, case["L"], H, generator=g, device="cuda")
        s.tok = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32) if case["gather"] else None
        s.pos0 = torch.randint(0, 1 << 20, (B,), generator=g, device="cuda", dtype=torch.int32)
        s.lens, s.cu = lens, _starts(lens)
        if own:
            _handle(s)
    elif op == "tree":
        nodes = _ints(case["nodes"])
        B, T = len(nodes), sum(nodes)
        s = _cache(case, B, _head_lens(case, B), 16, 0, g)
        s.q = randn(T, case["L"], Hq, D)
        s.k_draft, s.v_draft = randn(T, case["L"], H, D), randn(T, case["L"], H, D)
        r, mask = np.random.RandomState(seed % (1 << 31)), []
        for n in nodes:
            seen = []
            for i in range(n):
                up = seen[r.randint(max(0, i - 6), i)] if i else 0  # a node's parent is a recent one
                seen.append(up | 1 << i)
            for i in r.permutation(n)[: case["blank"]]:
                seen[i] = 0  # a place in the batch that no drafted token fills
            mask += seen
        s.mask = torch.from_numpy(np.array(mask, np.uint64).view(np.int64)).cuda()
        s.scale = 1.0 / math.sqrt(D)
        s.out = torch.zeros(T, case["L"], Hq, D, dtype=dt, device="cuda")
        s.lse = torch.zeros(T, case["L"], Hq, device="cuda")
        s.nodes, s.cu, s.longest = nodes, _starts(nodes), int(_head_lens(case, B).max())
        s.keep_mask = None
        if case["keep"] < 1.0:
            bits = torch.rand(s.C, s.max_pages, PAGE, generator=g, device="cuda") < case["keep"]
            s.keep_mask = (bits.to(torch.int32) << torch.arange(PAGE, device="cuda", dtype=torch.int32)).sum(-1).to(torch.int16)
        if own:
            _handle(s, max(nodes))
            s.sel = None
            if s.keep_mask is not None:
                s.sel = s.rkv.Selection.empty(s.cache)
                s.sel.keep_mask.copy_(s.keep_mask)
                s.sel.n_pre.copy_(s.len)
    else:
        parent = _ints(case["parent"])
        B = len(parent)
        have = _head_lens(case, B)
        LH = case["L"] * H
        per = (-(-have // PAGE)).reshape(B, LH).sum(1)
        s = _cache(case, B, have, 16, int(sum(per[p] for p in parent if p >= 0)), g)
        # the slots' tables take any sequence: as long as the longest
        s.parents, s.parent = parent, torch.tensor(parent, dtype=torch.int32, device="cuda")
        if own:
            _handle(s)
    s.op = op
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if s.op == "prompt":
        if own:
            s.rkv.prompt_attn(s.cache, s.cu, s.q, s.k, s.v, 1.0 / math.sqrt(s.D), s.out, s.lse, s.ws)
        else:
            _plain_prompt(s)
        return s.out, s.lse
    if s.op == "tree":
        if own:
            s.rkv.tree_attn(s.cache, s.cu, s.q, s.k_draft, s.v_draft, s.mask, s.scale, s.sel, s.out, s.lse, s.ws, max_nodes=max(s.nodes))
        else:
            _plain_tree(s)
        return s.out, s.lse
    # a server that tries a step again goes back to the bookkeeping it kept: rows past the lengths do not count
    s.book.copy_(s.book0)
    if s.op == "append":
        if own:
            s.rkv.append_tokens(s.cache, s.cu, s.pos0, s.k_new, s.v_new, s.lb_new, s.ws, tok=s.tok)
        else:
            _plain_append(s)
    elif own:
        s.rkv.fork_sequences(s.cache, s.parent, s.ws)
    else:
        _plain_fork(s)
    return s.k_pool, s.v_pool, s.pos_pool, s.lb_pool, s.block_table, s.len, s.free_top, s.free_stack


def _attend(q, k, v, scale, allowed):
    """Softmax attention in 32 bits: q [.., R, D], k and v [.., N, D], allowed broadcasts to [.., R, N]; a row
    that may see nothing gives 0 and -inf."""
    z = (q @ k.transpose(-1, -2)).mul_(scale)
    z.masked_fill_(~allowed, -math.inf)
    m = z.amax(-1, keepdim=True)
    m.masked_fill_(m == -math.inf, 0.0)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = p @ v
    return o / torch.where(l > 0, l, 1.0), (m + l.log()).squeeze(-1)


def _plain_prompt(s):
    G, at = s.Hq // s.H, 0
    for n in s.lens:
        k = s.k[at: at + n].transpose(0, 1).float()  # [H, n, D]
        v = s.v[at: at + n].transpose(0, 1).float()
        rows = max(1, min(n, (1 << 29) // (s.Hq * n)))  # query rows at a time: scores of about 2 GB
        for i in range(0, n, rows):
            e = min(n, i + rows)
            q = s.q[at + i: at + e].float().view(e - i, s.H, G, s.D).permute(1, 2, 0, 3).reshape(s.H, G * (e - i), s.D)
            sees = torch.arange(e, device="cuda")[None, :] <= torch.arange(i, e, device="cuda")[:, None]
            o, lse = _attend(q, k[:, :e], v[:, :e], 1.0 / math.sqrt(s.D), sees.repeat(G, 1))
            s.out[at + i: at + e] = o.view(s.H, G, e - i, s.D).permute(2, 0, 1, 3).reshape(e - i, s.Hq, s.D).to(s.dtype)
            s.lse[at + i: at + e] = lse.view(s.Hq, e - i).transpose(0, 1)
        at += n


def _plain_tree(s):
    G, LH, T = s.Hq // s.H, s.L * s.H, s.q.shape[0]
    n_max, pages = max(s.nodes), -(-s.longest // PAGE)
    node = torch.arange(n_max, device="cuda")
    count = s.cu[1:] - s.cu[:-1]
    there = node[None, :] < count[:, None]                               # [B, n_max]
    row = (s.cu[:-1, None] + node[None, :]).clamp_max(T - 1).long()      # rows of the packed draft
    slot = torch.arange(pages * PAGE, device="cuda")
    held = slot[None, :] < s.len[:, None]                                # [C, N]
    if s.keep_mask is not None:
        held &= (s.keep_mask[:, slot // PAGE].int() >> (slot % PAGE)[None, :]) & 1 == 1
    tree = (s.mask[row][:, :, None] >> node[None, None, :]) & 1 == 1      # [B, i, j]
    tree &= there[:, None, :]
    step = max(1, (1 << 29) // max(1, LH * n_max * G * (pages * PAGE + n_max)))  # sequences at a time
    for b in range(0, s.B, step):
        e = min(s.B, b + step)
        nb, r = e - b, row[b:e]
        table = s.block_table[b * LH: e * LH, :pages].clamp_min(0).long()
        k = torch.cat([s.k_pool[table].view(nb, LH, -1, s.D), s.k_draft[r].view(nb, n_max, LH, s.D).transpose(1, 2)], 2).float()
        v = torch.cat([s.v_pool[table].view(nb, LH, -1, s.D), s.v_draft[r].view(nb, n_max, LH, s.D).transpose(1, 2)], 2).float()
        q = s.q[r].float().view(nb, n_max, LH, G, s.D).permute(0, 2, 1, 3, 4).reshape(nb, LH, n_max * G, s.D)
        sees = torch.cat([held[b * LH: e * LH].view(nb, LH, 1, -1).expand(-1, -1, n_max * G, -1),
                          tree[b:e].repeat_interleave(G, 1)[:, None].expand(-1, LH, -1, -1)], 3)
        o, lse = _attend(q, k, v, s.scale, sees)
        o = o.view(nb, LH, n_max, G, s.D).transpose(1, 2).reshape(nb, n_max, s.L, s.Hq, s.D)
        at = r[there[b:e]]
        s.out[at] = o[there[b:e]].to(s.dtype)
        s.lse[at] = lse.view(nb, LH, n_max, G).transpose(1, 2).reshape(nb, n_max, s.L, s.Hq)[there[b:e]]


def _plain_append(s):
    LH, n = s.L * s.H, sum(s.lens)
    counts = s.cu[1:] - s.cu[:-1]
    seq = torch.repeat_interleave(torch.arange(s.B, device="cuda"), counts.long(), output_size=n)
    j = torch.arange(n, device="cuda") - s.cu[:-1][seq]
    add = counts.repeat_interleave(LH)
    have = (s.len + PAGE - 1) // PAGE
    need = (s.len + add + PAGE - 1) // PAGE - have
    first = need.cumsum(0) - need
    p = torch.arange(s.max_pages, device="cuda")
    fresh = (p[None, :] >= have[:, None]) & (p[None, :] < (have + need)[:, None])
    at = s.free_top - 1 - (first[:, None] + p[None, :] - have[:, None])
    s.block_table.copy_(torch.where(fresh, s.free_stack[at.clamp(0, s.n_pages - 1)], s.block_table))
    s.free_top.sub_(need.sum().to(torch.int32))
    head = seq[:, None] * LH + torch.arange(LH, device="cuda")[None, :]   # [n, LH]
    slot = s.len[head] + j[:, None]
    row = s.block_table[head, slot // PAGE].long() * PAGE + slot % PAGE
    src = slice(None) if s.tok is None else s.tok.long()
    s.k_pool.view(-1, s.D)[row.view(-1)] = s.k_new[src].view(-1, s.D)
    s.v_pool.view(-1, s.D)[row.view(-1)] = s.v_new[src].view(-1, s.D)
    s.lb_pool.view(-1)[row.view(-1)] = s.lb_new[src].view(-1)
    s.pos_pool.view(-1)[row.view(-1)] = (s.pos0[seq] + j).to(torch.int32).repeat_interleave(LH)
    s.len.add_(add)


def _plain_fork(s):
    LH = s.L * s.H
    copies = torch.tensor(_copies(s.parents), device="cuda")
    used = torch.zeros(s.B, dtype=torch.bool, device="cuda")
    used[s.parent[s.parent >= 0].long()] = True
    old_len, old_table = s.len.view(s.B, LH).clone(), s.block_table.view(s.B, LH, s.max_pages).clone()
    p = torch.arange(s.max_pages, device="cuda")
    full = p < (old_len[..., None] + PAGE - 1) // PAGE
    gone = old_table[full & ~used[:, None, None]]                         # heads in order, pages in order
    top = s.free_top.long()
    s.free_stack[top + torch.arange(gone.numel(), device="cuda")] = gone
    top = top + gone.numel()
    src = s.parent.clamp_min(0).long()
    new_len = torch.where((s.parent >= 0)[:, None], old_len[src], 0)
    have = p < (new_len[..., None] + PAGE - 1) // PAGE
    table = torch.where(have, old_table[src], -1)
    fresh = have & copies[:, None, None]
    from_page = table[fresh].long()
    to_page = s.free_stack[top - 1 - torch.arange(from_page.numel(), device="cuda")]
    table[fresh] = to_page
    rows = (new_len[..., None] - p * PAGE).clamp(0, PAGE)[fresh]           # rows of each page that hold entries
    live = torch.arange(PAGE, device="cuda")[None, :] < rows[:, None]
    a = (from_page[:, None] * PAGE + torch.arange(PAGE, device="cuda"))[live]
    b = (to_page.long()[:, None] * PAGE + torch.arange(PAGE, device="cuda"))[live]
    for pool in (s.k_pool.view(-1, s.D), s.v_pool.view(-1, s.D), s.pos_pool.view(-1), s.lb_pool.view(-1)):
        pool[b] = pool[a]
    s.block_table.copy_(table.view(s.C, s.max_pages))
    s.len.copy_(new_len.view(-1))
    s.free_top.copy_(top - from_page.numel())


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(s)
    if case["op"] == "tree":
        return _exact_tree(s)
    if s.n_pages * PAGE * s.D > 1 << 26:
        return None
    return _exact_append(s) if case["op"] == "append" else _exact_fork(s)


def _softmax_rows(z, v):
    lse = torch.logsumexp(z, -1)
    w = torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    return w @ v, lse


def _exact_prompt(s):
    G = s.Hq // s.H
    out, lse = torch.zeros(s.out.shape, dtype=torch.float64, device="cuda"), torch.zeros(s.lse.shape, dtype=torch.float64, device="cuda")
    at = 0
    for n in s.lens:
        for h in range(s.H):
            k, v = s.k[at: at + n, h].double(), s.v[at: at + n, h].double()
            for i in range(0, n, 4096):
                e = min(n, i + 4096)
                above = torch.ones(e - i, e, dtype=torch.bool, device="cuda").triu(i + 1)
                for g in range(h * G, h * G + G):
                    z = (s.q[at + i: at + e, g].double() @ k[:e].T) / math.sqrt(s.D)
                    z[above] = -math.inf
                    out[at + i: at + e, g], lse[at + i: at + e, g] = _softmax_rows(z, v[:e])
        at += n
    return out, lse


def _exact_tree(s):
    G, LH = s.Hq // s.H, s.L * s.H
    T = s.q.shape[0]
    out = torch.zeros(T, s.L * s.H, G, s.D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, s.L * s.H, G, dtype=torch.float64, device="cuda")
    q = s.q.view(T, LH, G, s.D)
    lens, at = s.len.tolist(), 0
    words = s.mask.cpu().numpy().view(np.uint64)
    for b, n in enumerate(s.nodes):
        sees = torch.tensor([[(int(words[at + i]) >> j) & 1 for j in range(n)] for i in range(n)], dtype=torch.bool, device="cuda")
        for h in range(LH):
            c = b * LH + h
            m = lens[c]
            pages = s.block_table[c, : -(-m // PAGE)].long()
            k = torch.cat([s.k_pool[pages].reshape(-1, s.D)[:m], s.k_draft.view(T, LH, s.D)[at: at + n, h]]).double()
            v = torch.cat([s.v_pool[pages].reshape(-1, s.D)[:m], s.v_draft.view(T, LH, s.D)[at: at + n, h]]).double()
            z = (q[at: at + n, h].double().reshape(n * G, s.D) @ k.T * s.scale).view(n, G, m + n)
            if s.keep_mask is not None:
                bits = (s.keep_mask[c].int()[:, None] >> torch.arange(PAGE, device="cuda")) & 1
                z[:, :, :m].masked_fill_(bits.reshape(-1)[:m] == 0, -math.inf)
            z[:, :, m:].masked_fill_(~sees[:, None, :], -math.inf)
            out[at: at + n, h], lse[at: at + n, h] = _softmax_rows(z, v)
        at += n
    return out.view(T, s.L, s.Hq, s.D), lse.view(T, s.L, s.Hq)


def _host(s):
    pools = [x.double().cpu().numpy() for x in (s.k_pool, s.v_pool)] + [s.pos_pool.cpu().numpy(), s.lb_pool.double().cpu().numpy()]
    free = s.free_stack[: int(s.free_top)].tolist()
    return pools, free, [[p for p in row if p >= 0] for row in s.block_table.tolist()], s.len.tolist()


def _bookkeeping(s, pools, free, tables, lens):
    table = np.full((s.C, s.max_pages), -1, np.int32)
    for c, t in enumerate(tables):
        table[c, : len(t)] = t
    return (*pools, table, np.array(lens, np.int32), np.array([len(free)], np.int32), None)


def _exact_append(s):
    pools, free, tables, lens = _host(s)
    k, v, lb = s.k_new.double().cpu().numpy(), s.v_new.double().cpu().numpy(), s.lb_new.double().cpu().numpy()
    tok, pos0, LH, cu = (s.tok.tolist() if s.tok is not None else None), s.pos0.tolist(), s.L * s.H, s.cu.tolist()
    for c in range(s.C):
        b, (l, h) = c // LH, divmod(c % LH, s.H)
        for j in range(cu[b + 1] - cu[b]):
            r = tok[cu[b] + j] if tok is not None else cu[b] + j
            if lens[c] % PAGE == 0:
                tables[c].append(free.pop())
            at = tables[c][lens[c] // PAGE], lens[c] % PAGE
            pools[0][at], pools[1][at], pools[2][at], pools[3][at] = k[r, l, h], v[r, l, h], pos0[b] + j, lb[r, l, h]
            lens[c] += 1
    return _bookkeeping(s, pools, free, tables, lens)


def _exact_fork(s):
    pools, free, tables, lens = _host(s)
    LH, copied = s.L * s.H, _copies(s.parents)
    for b in range(s.B):
        if b not in s.parents:
            for c in range(b * LH, b * LH + LH):
                free += tables[c]
    new, new_len = [[] for _ in range(s.C)], [0] * s.C
    for b, p in enumerate(s.parents):
        for h in range(LH if p >= 0 else 0):
            c, o = b * LH + h, p * LH + h
            new_len[c] = lens[o]
            new[c] = [free.pop() for _ in tables[o]] if copied[b] else tables[o]
            if copied[b]:
                for i, (x, y) in enumerate(zip(tables[o], new[c])):
                    n = min(PAGE, lens[o] - i * PAGE)
                    for pool in pools:
                        pool[y, :n] = pool[x, :n]
    return _bookkeeping(s, pools, free, new, new_len)
