"""One decoder layer serving a few conversations: prompts, a fork, decode steps
and a compaction over one paged KV cache.

    python examples/decoder_layer.py

Per call of the layer: flint_qkv_fused (input norm, qkv, q/k norm, RoPE, the
cache write), flint_attn_prompt or flint_attn_decode over the cache, the
output projection (torch), and flint_moe_forward_add_norm.  Weights and inputs
are random.  The run checks itself: a token decoded after its prompt gives
what the prompt with that token gives, a fork answers as its origin does, and
a compaction changes no bit.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_w4a16_mixture_gb300 as fm  # noqa: E402
from nvfp4_w4a16_mixture_gb300 import synth  # noqa: E402

D = 128


class Pool:
    """Pages of one KV cache, the host's side: each sequence's page list and
    length, and how many sequences hold a page."""

    def __init__(self, blocks: int, page: int, kv_heads: int):
        self.page, self.blocks = page, blocks
        self.k = torch.zeros(blocks, page, kv_heads, D, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.workspace = torch.zeros(fm.flint_kv_workspace_bytes(blocks), dtype=torch.uint8, device="cuda")
        self.holders = [0] * blocks
        self.pages: dict[int, list[int]] = {}
        self.length: dict[int, int] = {}

    def take(self) -> int:
        p = self.holders.index(0)
        self.holders[p] = 1
        return p

    def grow(self, seq: int, tokens: int) -> list[int]:
        """Room for `tokens` more; the slots they go to."""
        pages, start = self.pages.setdefault(seq, []), self.length.get(seq, 0)
        while len(pages) * self.page < start + tokens:
            pages.append(self.take())
        self.length[seq] = start + tokens
        return [pages[t // self.page] * self.page + t % self.page for t in range(start, start + tokens)]

    def fork(self, seq: int, new: int) -> None:
        """`new` goes on from seq: whole pages are shared, a part-filled last
        page is copied."""
        n, pages = self.length[seq], self.pages[seq]
        whole = n // self.page
        self.pages[new], self.length[new] = pages[:whole], n
        for p in pages[:whole]:
            self.holders[p] += 1
        if n % self.page:
            self.pages[new].append(self.take())
            moves = torch.tensor([[pages[whole], self.pages[new][-1]]], dtype=torch.int32, device="cuda")
            tokens = torch.tensor([n % self.page], dtype=torch.int32, device="cuda")
            fm.flint_kv_copy_pages(self.k, self.v, moves, tokens=tokens, workspace=self.workspace)

    def free(self, seq: int) -> None:
        for p in self.pages.pop(seq):
            self.holders[p] -= 1
        del self.length[seq]

    def tables(self, seqs) -> tuple[torch.Tensor, torch.Tensor]:
        width = max(len(self.pages[s]) for s in seqs)
        rows = [self.pages[s] + [-1] * (width - len(self.pages[s])) for s in seqs]
        return (torch.tensor(rows, dtype=torch.int32, device="cuda"),
                torch.tensor([self.length[s] for s in seqs], dtype=torch.int32, device="cuda"))

    def compact(self) -> int:
        """Moves the used pages to the pool's start; how many they are."""
        seqs = list(self.pages)
        table, lens = self.tables(seqs)
        new, moves, counts = fm.flint_kv_compact_plan(table, lens, self.page, self.blocks, workspace=self.workspace)
        fm.flint_kv_copy_pages(self.k, self.v, moves, count=counts[1:], workspace=self.workspace)
        assert fm.flint_moe_status(self.workspace) == fm.FLINT_OK
        self.holders = [0] * self.blocks
        for s, row in zip(seqs, new.tolist()):
            self.pages[s] = row[:len(self.pages[s])]
            for p in self.pages[s]:
                self.holders[p] += 1
        return int(counts[0])


class Layer:
    def __init__(self, H=512, heads=16, kv_heads=2, E=16, top_k=4, I=256, SI=256, max_pos=4096, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.top_k = heads, kv_heads, top_k
        _, self.moe = synth.make_problem(1, H, E, top_k, I, SI, seed=seed, device="cuda")
        codes, scales, gs = synth.quantize_nvfp4(torch.randn((heads + 2 * kv_heads) * D, H, generator=g) * 0.03)
        self.qkv = (codes.cuda(), scales.cuda(), gs.reshape(1).float().cuda())
        self.out = (torch.randn(H, heads * D, generator=g) * 0.02).bfloat16().cuda()
        one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.norm_in, self.norm_moe, self.norm_q = one, one, one[:D].clone()
        angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * (1e6 ** (-torch.arange(64) / 64.0))[None, :]
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()

    def __call__(self, x, residual, pool: Pool, seqs, tokens):
        """The rows of x are the next tokens[i] tokens of seqs[i], packed.
        Returns the layer's output and residual, packed the same."""
        start = [pool.length.get(s, 0) for s in seqs]
        slots = [t for s, n in zip(seqs, tokens) for t in pool.grow(s, n)]
        pos = [p for a, n in zip(start, tokens) for p in range(a, a + n)]
        table, lens = pool.tables(seqs)
        q, residual = fm.flint_qkv_fused(x, residual, self.norm_in, 1e-6, *self.qkv, self.norm_q, self.norm_q, 1e-6,
                                         self.rope, torch.tensor(pos, device="cuda"), pool.k, pool.v,
                                         torch.tensor(slots, device="cuda"), self.heads, self.kv_heads)
        if all(n == 1 for n in tokens):
            attn = fm.flint_attn_decode(q, pool.k, pool.v, table, lens)
        else:
            cu = torch.tensor([0, *torch.tensor(tokens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
            attn = fm.flint_attn_prompt(q, pool.k, pool.v, table, cu, lens)
        return fm.forward_add_norm_layer(attn @ self.out.t(), residual, self.norm_moe, 1e-6, self.moe, self.top_k)


def close(a, b) -> bool:
    """Alike up to the roundings of two paths to the same rows."""
    return float((a.float() - b.float()).norm() / b.float().norm()) < 0.02


def main() -> None:
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = lambda n: torch.randn(n, 512, generator=g, device="cuda").bfloat16()  # noqa: E731
    layer, pool = Layer(), Pool(blocks=64, page=16, kv_heads=2)

    # three prompts in one packed call
    n = [100, 7, 300]
    x, r = rows(sum(n)), rows(sum(n))
    out, _ = layer(x, r, pool, [0, 1, 2], n)
    # the first one again, its last token decoded on its own
    whole = out[:100]
    layer(x[:99], r[:99], pool, [3], [99])
    last, _ = layer(x[99:100], r[99:100], pool, [3], [1])
    assert close(last, whole[99:]), "decode after a prompt differs from the longer prompt"
    # a fork, then one token for every conversation: the fork answers as its origin
    pool.fork(2, 4)
    x1, r1 = rows(1).expand(4, -1).contiguous(), rows(1).expand(4, -1).contiguous()
    out, _ = layer(x1, r1, pool, [0, 1, 2, 4], [1] * 4)
    assert torch.equal(out[2], out[3]), "a fork differs from its origin"
    # conversations end; the pool is closed up, and the answers stay the same bits
    pool.free(3)
    pool.free(1)
    table, lens = pool.tables([0, 2, 4])
    q = rows(3).repeat(1, 4)
    before = fm.flint_attn_decode(q, pool.k, pool.v, table, lens)
    used = pool.compact()
    table, lens = pool.tables([0, 2, 4])
    assert int(table.max()) < used
    assert torch.equal(before, fm.flint_attn_decode(q, pool.k, pool.v, table, lens)), "a compaction changed the answers"
    # the forks go different ways
    out, _ = layer(rows(2), rows(2), pool, [2, 4], [1, 1])
    assert not torch.equal(out[0], out[1])
    print(f"decoder layer ok: {len(pool.pages)} conversations on {used} pages")


if __name__ == "__main__":
    main()
