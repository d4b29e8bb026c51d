"""Real work of the operators around the paged key-value cache that the fused
qkv writes: attention of one new token per sequence (decode), attention of
whole prompts and prompt chunks (packed, causal), and the copying and
compacting of the cache's pages.

Each case runs in a plain form (elementary torch operations in fp32, rounded
once) or, with `own` set, through the framework's entry points, on the same
state.  Heads are 128 wide, activations and caches bf16, as in the fused qkv.
"""
import math
import random

import torch

own = False

D = 128
SCALE = D ** -0.5


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the first answer tokens of one short chat turn: latency
        {"name": "decode_short", "op": "decode", "batch": 1, "low": 611, "high": 611, "nq": 32, "nkv": 4, "page": 16, "mix": 1},
        # one user in a long document, a single sequence that has to fill the card
        {"name": "decode_long", "op": "decode", "batch": 1, "low": 32781, "high": 32781, "nq": 32, "nkv": 4, "page": 16, "mix": 2},
        # an ordinary serving batch, lengths spread over two decades
        {"name": "decode_batch", "op": "decode", "batch": 64, "low": 64, "high": 4096, "nq": 32, "nkv": 4, "page": 16, "mix": 3},
        # seven query heads to a key head, odd pages, an idle slot (length 0) and a first token (length 1)
        {"name": "decode_odd", "op": "decode", "batch": 17, "low": 0, "high": 3001, "nq": 28, "nkv": 4, "page": 24, "mix": 4},
        # a full batch of long contexts: the cache's bandwidth
        {"name": "decode_full", "op": "decode", "batch": 64, "low": 8000, "high": 32000, "nq": 32, "nkv": 8, "page": 64, "mix": 5},
        # one short question
        {"name": "prompt_short", "op": "prompt", "batch": 1, "low": 130, "high": 130, "prefix": 0, "nq": 32, "nkv": 4, "page": 16, "mix": 6},
        # one prompt of the grouped MoE path's size
        {"name": "prompt_4096", "op": "prompt", "batch": 1, "low": 4096, "high": 4096, "prefix": 0, "nq": 32, "nkv": 4, "page": 16, "mix": 7},
        # a prefill batch of different lengths packed together, one of them a single token
        {"name": "prompt_packed", "op": "prompt", "batch": 16, "low": 1, "high": 2000, "prefix": 0, "nq": 32, "nkv": 8, "page": 32, "mix": 8},
        # one chunk of a long prompt whose earlier chunks are in the cache: few rows, a long axis
        {"name": "prompt_chunk", "op": "prompt", "batch": 1, "low": 500, "high": 500, "prefix": 30011, "nq": 32, "nkv": 4, "page": 16, "mix": 9},
        # the largest prompt of the framework's own configurations
        {"name": "prompt_16384", "op": "prompt", "batch": 1, "low": 16384, "high": 16384, "prefix": 0, "nq": 32, "nkv": 4, "page": 16, "mix": 10},
        # beams or samples that part from their prompts: each takes its own copy of a part-filled last page
        {"name": "pages_fork", "op": "fork", "batch": 96, "copies": 4, "blocks": 2048, "nkv": 4, "page": 16, "mix": 11},
        # a pool in which sequences have come and gone, closed up so that its upper part is free
        {"name": "pages_compact", "op": "compact", "batch": 48, "low": 100, "high": 8000, "blocks": 24000, "nkv": 4, "page": 16, "mix": 12},
    ]


HEADS = ((32, 4), (32, 8), (28, 4), (16, 2), (8, 1), (40, 8), (12, 12), (24, 8), (16, 1))
PAGES = (4, 8, 16, 16, 24, 32, 64, 128)


def _log_int(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "prompt", "prompt", "fork", "compact"))
    nq, nkv = rng.choice(HEADS)
    page, mix = rng.choice(PAGES), rng.randrange(1 << 30)
    if op == "decode":
        batch, high = _log_int(rng, 1, 64), _log_int(rng, 16, 32000)
        high = min(high, 8_000_000 // (batch * nkv))
        return {"op": op, "batch": batch, "low": rng.choice((0, 1, high // 2)), "high": high, "nq": nq, "nkv": nkv, "page": page, "mix": mix}
    if op == "prompt":
        batch, prefix = _log_int(rng, 1, 24), rng.choice((0, 0, 0, _log_int(rng, 1, 16000)))
        high = min(_log_int(rng, 32, 8192), int(math.sqrt(2.5e9 / (batch * nq))), 50_000_000 // (batch * nq * max(1, prefix)) + 200)
        return {"op": op, "batch": batch, "low": rng.choice((1, high // 2)), "high": high, "prefix": prefix, "nq": nq, "nkv": nkv, "page": page, "mix": mix}
    blocks = _log_int(rng, 64, 400_000 // (nkv * page))
    if op == "fork":
        copies = rng.randint(1, 6)
        return {"op": op, "batch": rng.randint(1, blocks // (2 * (copies + 1))), "copies": copies, "blocks": blocks, "nkv": nkv, "page": page, "mix": mix}
    batch = _log_int(rng, 1, 48)
    high = max(page, blocks * page // (2 * batch))
    return {"op": op, "batch": batch, "low": rng.choice((0, high // 3)), "high": high, "blocks": max(blocks, batch * 2), "nkv": nkv, "page": page, "mix": mix}


def _lengths(case):
    """The sequences' lengths (prompt: of the new parts), from the case alone.
    A batch of several has the ends of its range in it."""
    rng = random.Random(case["mix"])
    low, high = case["low"], case["high"]
    n = [low if rng.random() < 0.03 else _log_int(rng, max(1, low, high // 16), high) for _ in range(case["batch"])]
    if case["batch"] > 1:
        n[0], n[-1] = high, low
    if low == 0 and case["batch"] > 2:
        n[1] = 1
    return n


def _need(lengths, page):
    return [-(-n // page) for n in lengths]


def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed((seed * 1_000_003 + case["mix"] * 7919) % (1 << 62))


def _normal(gen, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def _tables(lengths, page, blocks, gen):
    """block_table int32 [batch, widest]: every sequence's pages, scattered
    over the pool; -1 past them."""
    need = _need(lengths, page)
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def prepare(case, seed):
    """What a serving program has in hand: the caches (normalised keys, values;
    unused slots hold what earlier sequences left), the pages' tables and the
    lengths, and the new queries."""
    gen = _gen(case, seed)
    op, nkv, page = case["op"], case["nkv"], case["page"]
    st = dict(case)
    if op == "fork":
        blocks = case["blocks"]
        n = case["batch"] * case["copies"]
        order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        src = order[:case["batch"]].repeat_interleave(case["copies"])
        st["moves"] = torch.stack((src, order[case["batch"]:case["batch"] + n]), 1).contiguous()
        st["tokens"] = torch.randint(1, page + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    else:
        lengths = _lengths(case)
        total = [n + case.get("prefix", 0) for n in lengths]
        blocks = case.get("blocks") or max(1, sum(_need(total, page)) + 7)
        st["seq_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        st["block_table"] = _tables(total, page, blocks, gen)
        st["longest"] = max(total)
        if op == "decode":
            st["q"] = _normal(gen, case["batch"], case["nq"] * D, std=1.5)
        if op == "prompt":
            cu = [0]
            for n in lengths:
                cu.append(cu[-1] + n)
            st["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            st["longest_q"] = max(lengths)
            st["q"] = _normal(gen, cu[-1], case["nq"] * D, std=1.5)
    st["blocks"] = blocks
    st["k_cache"] = _normal(gen, blocks, page, nkv, D, std=1.5)
    st["v_cache"] = _normal(gen, blocks, page, nkv, D)
    return st


# -------------------------------------------------------------- plain forms
def _rows(cache, table, page, longest):
    """The first `longest` cache rows of every sequence, fp32
    [batch, nkv, longest, 128] (whatever row where a sequence is shorter)."""
    pos = torch.arange(longest, device="cuda")
    blk = table[:, pos // page].clamp(min=0).long()
    return cache[blk, pos % page].transpose(1, 2).float()


def _attend(q, k, v, visible):
    """softmax(scale q k^T) v and the log of its sum, over the visible keys; a
    row that sees none gives zeros and -inf."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(SCALE)
    s.masked_fill_(~visible, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return o, (m + total.log()).squeeze(-1)


def _plain_decode(st):
    b, nq, nkv, page, longest = st["batch"], st["nq"], st["nkv"], st["page"], max(1, st["longest"])
    k = _rows(st["k_cache"], st["block_table"], page, longest)
    v = _rows(st["v_cache"], st["block_table"], page, longest)
    seen = torch.arange(longest, device="cuda") < st["seq_lens"][:, None]
    o, lse = _attend(st["q"].float().view(b, nkv, nq // nkv, D), k, v, seen[:, None, None])
    return {"out": o.reshape(b, nq * D).to(torch.bfloat16), "lse": lse.reshape(b, nq)}


def _plain_prompt(st):
    b, nq, nkv, page, longest, lq = st["batch"], st["nq"], st["nkv"], st["page"], st["longest"], st["longest_q"]
    g, cu = nq // nkv, st["cu_q"].long()
    k = _rows(st["k_cache"], st["block_table"], page, longest)
    v = _rows(st["v_cache"], st["block_table"], page, longest)
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + torch.arange(lq, device="cuda")).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().view(b, lq, nkv, g, D).permute(0, 2, 3, 1, 4).reshape(b, nkv, g * lq, D)
    last = st["seq_lens"].long()[:, None] - n[:, None] + torch.arange(lq, device="cuda")
    seen = (torch.arange(longest, device="cuda") <= last[:, :, None])[:, None].repeat(1, 1, g, 1)
    o, lse = _attend(q, k, v, seen)
    token = torch.arange(st["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu, token, right=True) - 1
    o = o.view(b, nkv, g, lq, D)[seq, :, :, token - cu[seq]]
    lse = lse.view(b, nkv, g, lq)[seq, :, :, token - cu[seq]]
    return {"out": o.reshape(-1, nq * D).to(torch.bfloat16), "lse": lse.reshape(-1, nq)}


def _plain_copy(st, moves, tokens):
    src, dst = moves.long().unbind(1)
    first = torch.arange(st["page"], device="cuda") < tokens[:, None]
    pair, slot = first.nonzero(as_tuple=True)
    st["k_cache"][dst[pair], slot] = st["k_cache"][src[pair], slot]
    st["v_cache"][dst[pair], slot] = st["v_cache"][src[pair], slot]


def _plain_compact(st):
    table, page, blocks = st["block_table"].long(), st["page"], st["blocks"]
    used = torch.arange(table.shape[1], device="cuda") < (st["seq_lens"][:, None] + page - 1) // page
    live = torch.zeros(blocks + 1, dtype=torch.bool, device="cuda")
    live[torch.where(used, table, blocks)] = True
    live = live[:blocks]
    n_live = live.sum()
    ids = torch.arange(blocks, device="cuda")
    src = (live & (ids >= n_live)).nonzero().squeeze(1)
    dst = (~live & (ids < n_live)).nonzero().squeeze(1)
    to = ids.clone()
    to[src] = dst
    new_table = torch.where(used, to[table.clamp(min=0)], -1).to(torch.int32)
    moves = torch.full((blocks // 2, 2), -1, dtype=torch.int32, device="cuda")
    moves[:src.shape[0]] = torch.stack((src, dst), 1).to(torch.int32)
    whole = torch.full_like(src, page)
    _plain_copy(st, moves[:src.shape[0]], whole)
    return {"table": new_table, "moves": moves, "counts": torch.stack((n_live, torch.full_like(n_live, src.shape[0]))).to(torch.int32),
            "k": st["k_cache"], "v": st["v_cache"]}


# ------------------------------------------------------- the framework's own
def _workspace(fm, st, n):
    """The zeroed workspace that a program allocates once and keeps."""
    if "workspace" not in st:
        st["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _own_run(st):
    import nvfp4_w4a16_mixture_gb300 as fm
    if st["op"] == "decode":
        ws = _workspace(fm, st, fm.flint_attn_decode_workspace_bytes(st["batch"], st["nq"], st["nkv"]))
        lse = torch.empty(st["batch"], st["nq"], dtype=torch.float32, device="cuda")
        out = fm.flint_attn_decode(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"], scale=SCALE, lse=lse, workspace=ws)
        return {"out": out, "lse": lse}
    if st["op"] == "prompt":
        t = st["q"].shape[0]
        ws = _workspace(fm, st, fm.flint_attn_prompt_workspace_bytes(t, st["batch"], st["nq"], st["nkv"]))
        lse = torch.empty(t, st["nq"], dtype=torch.float32, device="cuda")
        out = fm.flint_attn_prompt(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["cu_q"], st["seq_lens"], scale=SCALE, lse=lse, workspace=ws)
        return {"out": out, "lse": lse}
    ws = _workspace(fm, st, fm.flint_kv_workspace_bytes(st["blocks"]))
    if st["op"] == "fork":
        fm.flint_kv_copy_pages(st["k_cache"], st["v_cache"], st["moves"], tokens=st["tokens"], workspace=ws)
        return {"k": st["k_cache"], "v": st["v_cache"]}
    table, moves, counts = fm.flint_kv_compact_plan(st["block_table"], st["seq_lens"], st["page"], st["blocks"], workspace=ws)
    fm.flint_kv_copy_pages(st["k_cache"], st["v_cache"], moves, count=counts[1:], workspace=ws)
    return {"table": table, "moves": moves, "counts": counts, "k": st["k_cache"], "v": st["v_cache"]}


def run(st):
    if own:
        return _own_run(st)
    if st["op"] == "decode":
        return _plain_decode(st)
    if st["op"] == "prompt":
        return _plain_prompt(st)
    if st["op"] == "fork":
        _plain_copy(st, st["moves"], st["tokens"])
        return {"k": st["k_cache"], "v": st["v_cache"]}
    return _plain_compact(st)


# --------------------------------------------------------------------- work
def work(case):
    op, nkv, page = case["op"], case["nkv"], case["page"]
    row = nkv * D * 2 * 2  # one token's keys and values
    if op == "fork":
        n = case["batch"] * case["copies"]
        return {"bytes": int(n * (page + 1) / 2 * row * 2), "flops": 0}
    lengths = _lengths(case)
    prefix = case.get("prefix", 0)
    if op == "compact":
        need = _need(lengths, page)
        live = sum(need)
        moved = live * (case["blocks"] - live) // case["blocks"]  # of scattered pages, as many lie above the live count
        return {"bytes": moved * page * row * 2 + 8 * sum(need), "flops": 0}
    heads = case["nq"] * D
    keys = sum(n + prefix for n in lengths if n)
    if op == "decode":
        return {"bytes": keys * row + case["batch"] * (heads * 4 + case["nq"] * 4), "flops": 4 * heads * keys}
    pairs = sum(n * prefix + n * (n + 1) // 2 for n in lengths)
    return {"bytes": keys * row + sum(lengths) * (heads * 4 + case["nq"] * 4), "flops": 4 * heads * pairs}


# -------------------------------------------------------------------- exact
def _exact_rows(cache, pages, n, head):
    """Rows 0 .. n - 1 of one sequence and head, fp64."""
    return cache.index_select(0, pages.long())[:, :, head].reshape(-1, D)[:n].double()


def _exact_attention(st, first):
    """out and lse of packed queries: sequence b's are first[b] .. first[b+1]-1
    and its last one sees every key."""
    q, nq, nkv, page = st["q"], st["nq"], st["nkv"], st["page"]
    g = nq // nkv
    out = torch.zeros(q.shape[0], nq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((q.shape[0], nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["seq_lens"].tolist()):
        lo, hi = first[b], first[b + 1]
        if n == 0 or hi == lo:
            continue
        pages = st["block_table"][b, :-(-n // page)]
        for h in range(nkv):
            k = _exact_rows(st["k_cache"], pages, n, h)
            v = _exact_rows(st["v_cache"], pages, n, h)
            for a in range(lo, hi, 2048):
                z = min(hi, a + 2048)
                end = n - hi + z  # keys that the block's last query sees
                x = q[a:z].view(z - a, nq, D)[:, h * g:(h + 1) * g].double()
                s = torch.einsum("tgd,kd->gtk", x, k[:end]) / math.sqrt(D)
                late = torch.ones(z - a, end, dtype=torch.bool, device="cuda").triu(end - (z - a) + 1)
                s = s.masked_fill(late, -math.inf)
                w = torch.logsumexp(s, -1)
                out[a:z, h * g:(h + 1) * g] = torch.einsum("gtk,kd->tgd", torch.exp(s - w[..., None]), v[:end])
                lse[a:z, h * g:(h + 1) * g] = w.transpose(0, 1)
    return {"out": out.reshape(q.shape[0], nq * D), "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op in ("decode", "prompt"):
        if work(case)["flops"] > 8e12:
            return None
        return _exact_attention(st, st["cu_q"].tolist() if op == "prompt" else list(range(case["batch"] + 1)))
    if op == "fork":
        before_k, before_v = st["k_cache"].clone(), st["v_cache"].clone()
        for (s, d), n in zip(st["moves"].tolist(), st["tokens"].tolist()):
            st["k_cache"][d, :n], st["v_cache"][d, :n] = before_k[s, :n], before_v[s, :n]
        return {"k": st["k_cache"], "v": st["v_cache"]}
    old, need = st["block_table"].tolist(), _need(st["seq_lens"].tolist(), page)
    live = sorted({p for row, n in zip(old, need) for p in row[:n]})
    count = len(live)
    taken = set(live)
    pairs = list(zip([p for p in live if p >= count], [p for p in range(count) if p not in taken]))
    to = dict(pairs)
    table = [[to.get(p, p) if i < n else -1 for i, p in enumerate(row)] for row, n in zip(old, need)]
    moves = pairs + [(-1, -1)] * (case["blocks"] // 2 - len(pairs))
    if pairs:
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*pairs))
        st["k_cache"][dst], st["v_cache"][dst] = st["k_cache"][src], st["v_cache"][src]
    return {"table": torch.tensor(table, dtype=torch.int32, device="cuda"), "moves": torch.tensor(moves, dtype=torch.int32, device="cuda").view(-1, 2),
            "counts": torch.tensor([count, len(pairs)], dtype=torch.int32, device="cuda"), "k": st["k_cache"], "v": st["v_cache"]}
