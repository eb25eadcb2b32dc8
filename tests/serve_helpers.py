"""64-bit statements of the serving operators and the tolerances that follow
from their arithmetic (test code only)."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def starts(lens, device="cuda", first=0):
    return torch.tensor([first] + [first + int(x) for x in np.cumsum(lens)], dtype=torch.int32, device=device)


def attend64(q, k, v, scale, allowed):
    """Masked softmax attention in 64 bits: q [R, D], k and v [N, D], allowed [R, N].

    Returns (out, lse, weight, dz): weight = sum_j p_j |v_j| per output value,
    dz = a bound on the error of a fp32 logit's exponential (below)."""
    q, k, v = q.double(), k.double(), v.double()
    R, D = q.shape
    if k.shape[0] == 0:
        z = q.new_zeros(R)
        return q.new_zeros(R, D), z - math.inf, q.new_zeros(R, D), z[:, None]
    z = (q @ k.T) * scale
    z = torch.where(allowed, z, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    # the logit: D fp32 products and sums, half a step (2^-24) each, of terms
    # whose magnitudes add up to `size`; then one multiply by the scale, the
    # subtraction of the maximum and an exponential good to 2^-21
    size = (q.abs() @ k.abs().T) * abs(scale)
    size = torch.where(allowed, size, 0.0).amax(-1)
    dz = (D + 4) * 2.0 ** -24 * size + 2.0 ** -21
    return p @ v, lse, p @ v.abs(), dz[:, None]


def assert_attention(out, lse, ref, dtype, n_keys):
    """Kernel results against attend64's.  A weight is off by dz and, for bf16
    results, by half a bf16 step (2^-8) from rounding it for the product with V;
    so is the sum of the weights (dz) that divides; the fp32 sums over n keys
    add n half steps each; the result is rounded once."""
    o, l, weight, dz = ref
    half = torch.finfo(dtype).eps / 2
    sums = 2 * (n_keys + 8) * 2.0 ** -24
    bound = (2 * dz + sums + (half if dtype != torch.float32 else 0.0)) * weight * (1 + 2 ** -6) + half * o.abs() * (1 + 2 ** -6)
    bound = bound + 1e-37
    err = (out.double() - o).abs()
    assert bool(torch.isfinite(out.float()).all())
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"output off by {worst:.3g} times the bound"
    if lse is not None:
        empty = torch.isinf(l)
        assert bool(torch.isneginf(lse[empty]).all()) and bool(torch.isfinite(lse[~empty]).all())
        assert bool((out[empty] == 0).all())
        d = (lse.double() - l)[~empty].abs()
        lim = (dz[:, 0] + sums + 2.0 ** -22 * l.abs() + 2.0 ** -21)[~empty]
        assert bool((d <= lim).all()), f"lse off by {float((d / lim).max()):.3g} times the bound"


class ListCache:
    """The paged cache as Python lists, for whole-sequence operators: entry =
    (K row, V row, position, log-retention) as the raw tensors' slices."""

    def __init__(self, dc):
        self.k, self.v = dc.k_pool.cpu().clone(), dc.v_pool.cpu().clone()
        self.pos, self.lb = dc.pos_pool.cpu().clone(), dc.lb_pool.cpu().clone()
        self.lens = [int(x) for x in dc.len.cpu()]
        self.tables = [[int(p) for p in row[: -(-n // PAGE)]] for row, n in zip(dc.block_table.cpu(), self.lens)]
        self.free = [int(x) for x in dc.free_stack.cpu()[: int(dc.free_top.cpu()[0])]]
        self.max_pages = dc.block_table.shape[1]

    def append(self, LH, cu, pos0, k_new, v_new, lb_new, tok=None):
        k_new, v_new, lb_new = (x.cpu().reshape(x.shape[0], LH, -1) for x in (k_new, v_new, lb_new))
        cu, pos0 = [int(x) for x in cu.cpu()], [int(x) for x in pos0.cpu()]
        short = False
        for c in range(len(self.lens)):
            b, lh = divmod(c, LH)
            n = cu[b + 1] - cu[b]
            need = -(-(self.lens[c] + n) // PAGE) - -(-self.lens[c] // PAGE)
            if self.lens[c] + n > self.max_pages * PAGE or pos0[b] < 0:
                continue
            if need and (short or need > len(self.free)):
                short = True
                continue
            for j in range(n):
                r = int(tok[cu[b] + j]) if tok is not None else cu[b] + j
                slot = self.lens[c]
                if slot % PAGE == 0:
                    self.tables[c].append(self.free.pop())
                at = self.tables[c][slot // PAGE], slot % PAGE
                self.k[at], self.v[at], self.pos[at], self.lb[at] = k_new[r, lh], v_new[r, lh], pos0[b] + j, lb_new[r, lh, 0]
                self.lens[c] += 1

    def fork(self, LH, parent):
        B = len(parent)
        heir = {s: (s if parent[s] == s else parent.index(s)) for s in set(parent) if s >= 0}
        for s in range(B):
            if s not in heir:
                for c in range(s * LH, s * LH + LH):
                    self.free += self.tables[c]
        tables, lens = [[] for _ in self.tables], [0] * len(self.lens)
        for b, s in enumerate(parent):
            for lh in range(LH if s >= 0 else 0):
                c, o = b * LH + lh, s * LH + lh
                lens[c] = self.lens[o]
                if heir[s] == b:
                    tables[c] = list(self.tables[o])
                    continue
                tables[c] = [self.free.pop() for _ in self.tables[o]]
                for i, (x, y) in enumerate(zip(self.tables[o], tables[c])):
                    n = min(PAGE, lens[c] - i * PAGE)
                    for pool in (self.k, self.v, self.pos, self.lb):
                        pool[y, :n] = pool[x, :n].clone()
        self.tables, self.lens = tables, lens

    def assert_same(self, dc):
        assert [int(x) for x in dc.len.cpu()] == self.lens
        table = torch.full((len(self.tables), self.max_pages), -1, dtype=torch.int32)
        for c, t in enumerate(self.tables):
            table[c, : len(t)] = torch.tensor(t, dtype=torch.int32)
        assert torch.equal(dc.block_table.cpu(), table)
        top = int(dc.free_top.cpu()[0])
        assert top == len(self.free) and [int(x) for x in dc.free_stack.cpu()[:top]] == self.free
        for got, want in ((dc.k_pool, self.k), (dc.v_pool, self.v), (dc.pos_pool, self.pos), (dc.lb_pool, self.lb)):
            raw = torch.int16 if got.element_size() == 2 else torch.int32
            assert torch.equal(got.cpu().view(raw), want.view(raw))  # bits: a NaN is moved too
