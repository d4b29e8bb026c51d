"""Plain float64 attention over a paged cache, problems for its tests, and the
error bounds of the kernels' roundings.

Bounds.  Let A = sum_j p_j |v_j| / sum_j p_j (what the outputs' terms add up to
in magnitude).  Against the exact result,
  - a score is a 128-term fp32 sum in the tensor cores' order: at most
    128 * 2^-22 * scale * sum|q k| off (2^-22: two bits below fp32's half step
    for an accumulator that truncates), which changes p by that relatively;
  - exp2 and its argument: 2^-20 relative; fp32 sums over n keys: n * 2^-23;
  - P enters the second product as hi + lo (2^-16 relative) or as one bf16
    (2^-8 relative);
  - the output's rounding to bf16: 2^-8 of it (half a step).
So |out - exact| <= 2^-8 |exact| + (2 d + p_rel) A, |lse - exact| <= d + 2^-22 |exact|.
"""
from __future__ import annotations

import math

import torch

D = 128
P_SPLIT, P_BF16 = 2.0 ** -16, 2.0 ** -8


def keys_of(cache, pages, n, head):
    """Rows 0 .. n - 1 of one sequence and kv head, float64."""
    bs = cache.shape[1]
    pos = torch.arange(n)
    return cache[torch.tensor(pages, dtype=torch.long)[pos // bs], pos % bs, head].double()


def attention(q, k_cache, v_cache, table, cu, lens, scale, p_rel):
    """(out, lse, out bound, lse bound) in float64; all tensors on the CPU,
    sequence b's rows cu[b] .. cu[b + 1] - 1 being its last ones."""
    T, nq = q.shape[0], q.shape[1] // D
    nkv = k_cache.shape[2]
    G = nq // nkv
    out, tol = torch.zeros(T, nq, D, dtype=torch.float64), torch.zeros(T, nq, D, dtype=torch.float64)
    lse, ltol = torch.full((T, nq), -math.inf, dtype=torch.float64), torch.zeros(T, nq, dtype=torch.float64)
    x = q.view(T, nq, D).double()
    bs = k_cache.shape[1]
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo or n == 0:
            continue
        pages = table[b][:-(-n // bs)]
        for h in range(nkv):
            k, v = keys_of(k_cache, pages, n, h), keys_of(v_cache, pages, n, h)
            xh = x[lo:hi, h * G:(h + 1) * G]
            s = torch.einsum("tgd,kd->tgk", xh, k) * scale
            mag = torch.einsum("tgd,kd->tgk", xh.abs(), k.abs()) * scale
            seen = torch.arange(n)[None] <= (n - (hi - lo) + torch.arange(hi - lo))[:, None]
            s = s.masked_fill(~seen[:, None], -math.inf)
            any_seen = seen.any(-1)[:, None]
            w = torch.where(any_seen, torch.logsumexp(s, -1), torch.zeros(()).double())
            p = torch.exp(s - w[..., None])
            vz = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
            d = 128 * 2.0 ** -22 * mag.masked_fill(~seen[:, None], 0.0).amax(-1) + 2.0 ** -20 + n * 2.0 ** -23
            o = torch.einsum("tgk,kd->tgd", p, vz)
            out[lo:hi, h * G:(h + 1) * G] = o
            tol[lo:hi, h * G:(h + 1) * G] = 2.0 ** -8 * o.abs() + (2 * d + p_rel)[..., None] * \
                torch.einsum("tgk,kd->tgd", p, vz.abs())
            lse[lo:hi, h * G:(h + 1) * G] = torch.where(any_seen, w, torch.full((), -math.inf).double())
            ltol[lo:hi, h * G:(h + 1) * G] = d + 2.0 ** -22 * w.abs()
    return out.view(T, nq * D), lse, tol.view(T, nq * D), ltol


LAYOUTS = ("slots", "heads", "pairs", "padded")


def cache_pair(blocks, page, nkv, layout, fill):
    """k and v views [blocks, page, nkv, 128] of one layout: slots first, heads
    first, keys and values of a page side by side, or rows with gaps."""
    shape = (blocks, page, nkv, D)
    if layout == "slots":
        return tuple(torch.full(shape, fill, dtype=torch.bfloat16) for _ in range(2))
    if layout == "heads":
        return tuple(torch.full((blocks, nkv, page, D), fill, dtype=torch.bfloat16).transpose(1, 2) for _ in range(2))
    if layout == "pairs":
        both = torch.full((blocks, 2, page, nkv, D), fill, dtype=torch.bfloat16)
        return both[:, 0], both[:, 1]
    return tuple(torch.full((blocks, page, nkv, D + 24), fill, dtype=torch.bfloat16)[..., :D] for _ in range(2))


def on_gpu(view, blocks, page, nkv, layout):
    """The same view of the same layout on the GPU."""
    base = view._base if view._base is not None else view
    moved = base.cuda()
    return moved.as_strided(view.shape, view.stride(), view.storage_offset())


class Problem:
    """A paged cache holding `lens` keys per sequence on scattered pages, the
    queries, and everything no query may see filled with NaN: the slots past
    a sequence's keys, the pool's other pages, and (in the table) page ids."""

    def __init__(self, lens, qlens, nq, nkv, page, layout="slots", seed=0, std=1.5, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.nq, self.nkv, self.page, self.layout = list(lens), nq, nkv, page, layout
        self.cu = [0]
        for n in qlens:
            self.cu.append(self.cu[-1] + n)
        need = [-(-n // page) for n in lens]
        self.blocks = sum(need) + spare
        self.k, self.v = cache_pair(self.blocks, page, nkv, layout, math.nan)
        order = torch.randperm(self.blocks, generator=g).tolist()
        width = max(need, default=0) + 2
        self.table = []
        at = 0
        for n, keys in zip(need, lens):
            pages = order[at:at + n]
            at += n
            self.table.append(pages + [(-7, 2 ** 31 - 1)[i % 2] for i in range(width - n)])
            for i, p in enumerate(pages):
                m = min(page, keys - i * page)
                self.k[p, :m] = (torch.randn(m, nkv, D, generator=g) * std).bfloat16()
                self.v[p, :m] = torch.randn(m, nkv, D, generator=g).bfloat16()
        self.q = (torch.randn(self.cu[-1], nq * D, generator=g) * std).bfloat16()

    def gpu(self):
        t = dict(q=self.q.cuda(), block_table=torch.tensor(self.table, dtype=torch.int32).cuda().view(len(self.lens), -1),
                 seq_lens=torch.tensor(self.lens, dtype=torch.int32).cuda(),
                 cu_q=torch.tensor(self.cu, dtype=torch.int32).cuda())
        if self.layout == "pairs":
            both = self.k._base.cuda()
            t["k_cache"], t["v_cache"] = both[:, 0], both[:, 1]
        else:
            for name, c in (("k_cache", self.k), ("v_cache", self.v)):
                t[name] = on_gpu(c, self.blocks, self.page, self.nkv, self.layout)
        return t

    def expect(self, scale, p_rel):
        return attention(self.q, self.k, self.v, self.table, self.cu, self.lens, scale, p_rel)


def check(out, lse, want, where=""):
    """Every element of out (bf16) and lse (fp32) within its bound."""
    ref, rl, tol, ltol = want
    got = out.cpu().double()
    assert torch.isfinite(got).all(), where + ": out is not finite"
    worst = ((got - ref).abs() - tol).max().item() if got.numel() else 0.0
    assert worst <= 0.0, f"{where}: out past its bound by {worst:.3g}"
    if lse is not None:
        gl = lse.cpu().double()
        empty = torch.isinf(rl)
        assert torch.equal(gl[empty], rl[empty]), where + ": lse of empty rows"
        worst = ((gl - rl).abs() - ltol)[~empty].max().item() if (~empty).any() else 0.0
        assert worst <= 0.0, f"{where}: lse past its bound by {worst:.3g}"
