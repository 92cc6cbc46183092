"""The paged-cache operators of the decode library, as cases to be timed and compared.

The framework's cache rows live in pools of fixed-size pages that a page table per sequence
strings together.  Four kinds of pass go over such a cache:

  attn    the attention of each sequence's newest tokens (one token, a few, or a chunk of a
          prompt) over its pages, causal, with an optional sliding window and a few first
          tokens ("sinks") that stay visible;
  append  writing the newest key and value rows into their pages;
  branch  forking sequences (prefix pages shared), growing them (pages taken for the next
          tokens, a shared partial page copied before it is written) and that copy;
  evict   releasing finished sequences and the pages behind the others' windows, compacting
          the pages that are left and moving their rows.

``own`` False computes them with elementary torch operations in 32 bits, True through the
framework's entry points.
"""
import math
import random

import torch

own = False


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest call: one token of one short sequence (the `tiny` workload's heads and length)
        dict(name="attn_tiny_decode", op="attn", B=1, Hq=8, Hkv=2, d=128, page=16, q_lo=1, q_hi=1, ctx_lo=2047,
             ctx_hi=2047, window=0, sinks=0, fused=False, nhd=False, lens=1),
        # one token per sequence over long caches (the `h128k` workload): every K and V row is read once
        dict(name="attn_h128k_decode", op="attn", B=4, Hq=32, Hkv=8, d=128, page=64, q_lo=1, q_hi=1, ctx_lo=99999,
             ctx_hi=131071, window=0, sinks=0, fused=False, nhd=False, lens=2),
        # a local layer of the `hybrid` workload: 1024-token window, four sinks, pages behind it released
        dict(name="attn_hybrid_local_decode", op="attn", B=8, Hq=16, Hkv=8, d=256, page=64, q_lo=1, q_hi=1,
             ctx_lo=1500, ctx_hi=65535, window=1024, sinks=4, fused=True, nhd=False, lens=3),
        # a mixed batch: ragged chunks next to few-token sequences, small heads, window and sinks, odd lengths
        dict(name="attn_mixed_ragged", op="attn", B=7, Hq=16, Hkv=2, d=64, page=32, q_lo=1, q_hi=700, ctx_lo=0,
             ctx_hi=6001, window=600, sinks=5, fused=True, nhd=True, lens=4),
        # a step of chunked prefill in a running batch (the `llama8b` heads at 32K tokens): the largest case
        dict(name="attn_chunk_32k", op="attn", B=4, Hq=32, Hkv=8, d=128, page=16, q_lo=512, q_hi=512, ctx_lo=31999,
             ctx_hi=32767, window=0, sinks=0, fused=True, nhd=False, lens=5),
        # a whole prompt at once, from an empty cache
        dict(name="attn_prefill_8k", op="attn", B=1, Hq=32, Hkv=8, d=128, page=128, q_lo=8192, q_hi=8192, ctx_lo=0,
             ctx_hi=0, window=0, sinks=0, fused=True, nhd=False, lens=6),
        # the append of a decode step: one row per sequence and head
        dict(name="append_decode", op="append", B=64, Hkv=8, d=128, page=16, q_lo=1, q_hi=1, ctx_lo=100, ctx_hi=8000,
             fused=True, nhd=False, lens=7),
        # the append of a prompt chunk, ragged
        dict(name="append_chunk", op="append", B=6, Hkv=8, d=128, page=64, q_lo=300, q_hi=8192, ctx_lo=0, ctx_hi=9000,
             fused=True, nhd=True, lens=8),
        # parallel sampling from a few prompts: a handful of forks, then one token for everyone
        dict(name="branch_small", op="branch", B=16, parents=4, kids=2, Hkv=2, d=128, page=16, ctx_lo=50, ctx_hi=900,
             pages=512, grow=1, nhd=False, lens=9),
        # the same on a serving-size table
        dict(name="branch_large", op="branch", B=256, parents=60, kids=3, Hkv=8, d=128, page=64, ctx_lo=500,
             ctx_hi=5000, pages=8192, grow=3, nhd=False, lens=10),
        # a few finished sequences and short windows
        dict(name="evict_small", op="evict", B=12, Hkv=2, d=64, page=16, ctx_lo=30, ctx_hi=500, pages=512, drop=3,
             window=128, sinks=4, nhd=False, lens=11),
        # a serving-size cache in which a third of the sequences end: about 2,000 pages move
        dict(name="evict_large", op="evict", B=128, Hkv=8, d=128, page=64, ctx_lo=500, ctx_hi=6000, pages=8192,
             drop=43, window=4096, sinks=4, nhd=False, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("attn", "attn", "attn", "attn", "append", "branch", "evict"))
        c = dict(op=op, Hkv=rng.choice((1, 2, 3, 4, 8)), d=rng.choice((64, 128, 128, 256)),
                 page=rng.choice((16, 32, 64, 128, 256)), nhd=rng.random() < 0.3, lens=rng.randrange(1 << 30))
        if op in ("attn", "append"):
            kind = rng.choice(("one", "few", "chunk", "mixed"))
            c["B"] = _log_int(rng, 1, 64)
            c["q_hi"] = {"one": 1, "few": rng.randint(2, 16)}.get(kind) or _log_int(rng, 20, 8192)
            c["q_lo"] = {"one": 1, "few": 1, "chunk": max(1, c["q_hi"] * 3 // 4), "mixed": 0}[kind]
            c["ctx_hi"] = _log_int(rng, 1, 131071 if kind in ("one", "few") else 40000)
            c["ctx_lo"] = rng.choice((0, c["ctx_hi"] // 2, c["ctx_hi"]))
            c["fused"] = rng.random() < 0.5
        if op == "attn":
            c["Hq"] = c["Hkv"] * rng.choice((1, 2, 4, 4, 8, 16))
            c["window"] = 0 if rng.random() < 0.5 else _log_int(rng, 1, 8192)
            c["sinks"] = rng.choice((0, 1, 4, rng.randint(2, 100))) if c["window"] else 0
            cells = c["B"] * c["Hq"] * c["q_hi"] * (_slots(c)[1] * c["page"] + 1)
            rows = c["B"] * c["Hkv"] * c["d"] * (c["ctx_hi"] + c["q_hi"])
            if cells > 2.2e9 or rows > 6e8 or work(c)["flops"] > 1.0e12:
                continue
        elif op == "append":
            if c["B"] * c["q_hi"] > 50000 or c["B"] * (c["ctx_hi"] + c["q_hi"]) * c["Hkv"] * c["d"] > 4e8:
                continue
        elif op == "branch":
            c.update(parents=_log_int(rng, 1, 60), kids=rng.randint(1, 4), grow=rng.choice((1, 1, 3, 40)),
                     ctx_hi=_log_int(rng, 20, 5000))
            c.update(B=c["parents"] * (1 + c["kids"]) + rng.randint(0, 9), ctx_lo=rng.choice((1, c["ctx_hi"] // 2)))
            per = -(-(c["ctx_hi"] + c["grow"]) // c["page"])
            c["pages"] = c["parents"] * per + c["B"] * (2 + c["grow"] // c["page"]) + rng.randint(0, 400)
        else:
            c.update(B=_log_int(rng, 1, 128), ctx_hi=_log_int(rng, 20, 6000), window=_log_int(rng, 1, 4096),
                     sinks=rng.choice((0, 4, 33)))
            c.update(ctx_lo=rng.choice((1, c["ctx_hi"] // 2)), drop=rng.randint(0, c["B"]))
            c["pages"] = c["B"] * -(-c["ctx_hi"] // c["page"]) + rng.randint(1, 1000)
        if op in ("branch", "evict") and c["pages"] * c["page"] * c["Hkv"] * c["d"] > 5e8:
            continue
        return c


def _lengths(c):
    """Per-sequence (new tokens, tokens after them), a function of the case alone."""
    r = random.Random(c["lens"])
    q = [r.randint(c.get("q_lo", 0), c.get("q_hi", 0)) for _ in range(c["B"])]
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["B"])]
    if "q_hi" in c:
        q[r.randrange(c["B"])] = c["q_hi"]
    return q, [a + b for a, b in zip(q, ctx)]


def _visible(n, q, window, sinks):
    """(rows that some query reads, sum over the queries of the rows each reads) of one sequence."""
    if q == 0:
        return 0, 0
    if not window:
        return n, q * (n - q) + q * (q + 1) // 2
    lo = max(0, n - q - window + 1)
    pairs = 0
    for p in (range(n - q, n) if q < 9000 else ()):
        w = max(0, p - window + 1)
        pairs += p + 1 - w + min(sinks, w)
    return n - lo + min(sinks, lo), pairs


def work(c):
    rows2 = 2 * c["Hkv"] * c["d"] * 2  # bytes of one token's K and V rows
    if c["op"] == "attn":
        q, n = _lengths(c)
        seen = [_visible(b, a, c["window"], c["sinks"]) for a, b in zip(q, n)]
        return {"bytes": sum(s[0] for s in seen) * rows2 + 2 * sum(q) * c["Hq"] * c["d"] * 2,
                "flops": 4.0 * c["d"] * c["Hq"] * sum(s[1] for s in seen)}
    if c["op"] == "append":
        q, _ = _lengths(c)
        return {"bytes": 2 * sum(q) * rows2, "flops": 0}
    page_bytes = c["page"] * rows2
    _, n = _lengths(c)
    if c["op"] == "branch":
        # every fork of a partial last page is one page copied; the table rows and counts are read and written
        part = sum(1 for b in n[:c["parents"]] if b % c["page"])
        return {"bytes": 2 * part * c["kids"] * page_bytes + 2 * 4 * (c["pages"] + c["B"] * _max_pages(c)), "flops": 0}
    live = sum(_kept_pages(c, b) for b in n[c["drop"]:])
    moves = live * (1.0 - live / c["pages"])  # live pages above the first `live`, for pages in random order
    return {"bytes": 2 * moves * page_bytes + 2 * 4 * (c["pages"] + c["B"] * _max_pages(c)), "flops": 0}


def _kept_pages(c, n):
    ps = c["page"]
    return sum(1 for s in range(-(-n // ps)) if s * ps < c["sinks"] or (s + 1) * ps > n - c["window"])


def _max_pages(c):
    return -(-(c["ctx_hi"] + c.get("q_hi", 0) + c.get("grow", 0)) // c["page"])


def _slots(c):
    """(sink pages, pages from the first one a sequence's first query reads) that the plain form gathers."""
    ps = c["page"]
    if not c["window"]:
        return 0, _max_pages(c)
    return -(-c["sinks"] // ps), min(_max_pages(c), (c["window"] + c["q_hi"] - 2) // ps + 2)


# --------------------------------------------------------------------------- inputs
def _pools(c, n_pages, gen):
    """K and V pools [n_pages, Hkv, page, d], heads outside or inside the page's rows; a few rows heavy."""
    out = []
    for _ in range(2):
        if c["nhd"]:
            x = torch.randn(n_pages, c["page"], c["Hkv"], c["d"], generator=gen, device="cuda", dtype=torch.bfloat16)
            x = x.transpose(1, 2)
        else:
            x = torch.randn(n_pages, c["Hkv"], c["page"], c["d"], generator=gen, device="cuda", dtype=torch.bfloat16)
        out.append(x)
    heavy = torch.rand(n_pages, 1, c["page"], 1, generator=gen, device="cuda") < 0.01
    out[0] *= torch.where(heavy, 2.0, 1.0).to(torch.bfloat16)
    return out


def prepare(case, seed):
    c, op = case, case["op"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ps, B, mp = c["page"], c["B"], _max_pages(c)
    q, n = _lengths(c)
    s = dict(case=c)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if op in ("attn", "append"):
        window, sinks = c.get("window", 0), c.get("sinks", 0)
        # each sequence's pages that are still held (behind a window only the sinks' pages are)
        held = [(b, t) for b in range(B) for t in range(-(-n[b] // ps))
                if not window or t * ps < sinks or (t + 1) * ps > n[b] - q[b] - window]
        n_pages = len(held) + 7
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)[:len(held)]
        table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
        at = torch.tensor(held, device="cuda").reshape(-1, 2)
        table[at[:, 0], at[:, 1]] = order
        s["K"], s["V"] = _pools(c, n_pages, gen)
        begin = [0]
        for x in q:
            begin.append(begin[-1] + x)
        s.update(table=table, q_begin=i32(begin), seq_lens=i32(n), max_q=max(q))
        Hq = c.get("Hq", c["Hkv"])
        heads = (Hq, c["Hkv"], c["Hkv"])
        if c["fused"]:  # slices of one projection's output
            x = torch.randn(begin[-1], sum(heads), c["d"], generator=gen, device="cuda").to(torch.bfloat16)
            parts = x.split(heads, 1)
        else:
            parts = [torch.randn(begin[-1], h, c["d"], generator=gen, device="cuda").to(torch.bfloat16) for h in heads]
        s["Q"], s["K_new"], s["V_new"] = parts
        s["O"] = torch.empty(begin[-1], Hq, c["d"], dtype=torch.bfloat16, device="cuda")
        s["scale"] = 1.0 / math.sqrt(c["d"])
    else:
        r = random.Random(c["lens"] + 1)
        n_pages = c["pages"]
        first = c["parents"] if op == "branch" else B
        n = n[:first] + [0] * (B - first)
        need = [-(-x // ps) for x in n]
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
        b_of = torch.tensor([b for b in range(B) for _ in range(need[b])], device="cuda")
        t_of = torch.tensor([t for b in range(B) for t in range(need[b])], device="cuda")
        table[b_of, t_of] = order[:sum(need)]
        ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        ref[order[:sum(need)].long()] = 1
        # the bookkeeping in one buffer, so that one copy brings a pass back to its start
        s["book0"] = torch.cat([table.reshape(-1), ref, i32(n)])
        s["book"] = s["book0"].clone()
        s["table"] = s["book"][:B * mp].view(B, mp)
        s["ref"] = s["book"][B * mp:B * mp + n_pages]
        s["seq_lens"] = s["book"][B * mp + n_pages:]
        s["K"], s["V"] = _pools(c, n_pages, gen)
        if op == "branch":
            rows = list(range(first, first * (1 + c["kids"])))
            r.shuffle(rows)
            s["fork_src"] = i32([b for b in range(first) for _ in range(c["kids"])])
            s["fork_dst"] = i32(rows)
            s["n_new"] = i32([c["grow"] if b < first * (1 + c["kids"]) else 0 for b in range(B)])
            cap = B
        else:
            ended = [1] * c["drop"] + [0] * (B - c["drop"])
            s["ended"] = i32(ended)
            cap = max(1, n_pages // 2)
            s["n_moves"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["src"] = torch.empty(cap, dtype=torch.int32, device="cuda")
        s["dst"] = torch.empty(cap, dtype=torch.int32, device="cuda")
    if own:
        import token_level_sparse_jssa_b200 as jssa
        s["L"] = jssa.make_paged_layout(s["K"], s["V"], s["table"], c.get("Hq", c["Hkv"]), jssa.OUT_BF16)
        s["ws"] = jssa.alloc_paged_workspace(s["L"], s.get("max_q", 1))
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if op in ("branch", "evict"):
        s["book"].copy_(s["book0"])
    return (_own if own else _plain)[op](s)


def _own_attn(s):
    import token_level_sparse_jssa_b200 as jssa
    c = s["case"]
    jssa.paged_attn(s["L"], s["Q"], s["K"], s["V"], s["table"], s["q_begin"], s["max_q"], s["seq_lens"], c["window"],
                    c["sinks"], s["scale"], s["O"], None, s["ws"])
    return s["O"]


def _own_append(s):
    import token_level_sparse_jssa_b200 as jssa
    jssa.paged_append_kv(s["L"], s["K_new"], s["V_new"], s["K"], s["V"], s["table"], s["q_begin"], s["seq_lens"],
                         s["ws"])
    return s["K"], s["V"]


def _own_branch(s):
    import token_level_sparse_jssa_b200 as jssa
    jssa.pages_fork(s["L"], s["fork_src"], s["fork_dst"], s["table"], s["ref"], s["seq_lens"], s["ws"])
    jssa.pages_reserve(s["L"], s["n_new"], s["table"], s["ref"], s["seq_lens"], s["src"], s["dst"], s["ws"])
    jssa.pages_copy(s["L"], s["K"], s["V"], s["src"], s["dst"], None, s["ws"])
    return {k: s[k] for k in ("table", "ref", "seq_lens", "src", "dst", "K", "V")}


def _own_evict(s):
    import token_level_sparse_jssa_b200 as jssa
    c = s["case"]
    jssa.pages_release(s["L"], s["ended"], c["window"], c["sinks"], s["table"], s["ref"], s["seq_lens"], s["ws"])
    jssa.pages_compact(s["L"], s["table"], s["ref"], s["src"], s["dst"], s["n_moves"], s["ws"])
    jssa.pages_copy(s["L"], s["K"], s["V"], s["src"], s["dst"], s["n_moves"], s["ws"])
    return {k: s[k] for k in ("table", "ref", "seq_lens", "src", "dst", "n_moves", "K", "V")}


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hkv, d, ps, W, S = (c[k] for k in ("B", "Hq", "Hkv", "d", "page", "window", "sinks"))
    dev, qmax, mp = s["Q"].device, s["max_q"], s["table"].shape[1]
    lens, qb = s["seq_lens"].long(), s["q_begin"].long()
    nq = qb[1:] - qb[:-1]
    total = s["Q"].shape[0]
    i = torch.arange(qmax, device=dev)
    at = (qb[:-1, None] + i).clamp(max=total - 1)
    q = s["Q"][at].float().view(B, qmax, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    pos = (lens - nq)[:, None] + i
    # the pages that some query of a sequence reads, and their tokens' positions
    sink_slots, n_slots = _slots(c)
    first = (lens - nq - W + 1).clamp(min=0) // ps if W else torch.zeros_like(lens)
    slot = first[:, None] + torch.arange(n_slots, device=dev)
    if sink_slots:
        slot = torch.where(slot < sink_slots, mp, slot)  # already among the sinks' pages
        slot = torch.cat([torch.arange(sink_slots, device=dev).expand(B, -1), slot], 1)
    page = s["table"].gather(1, slot.clamp(max=mp - 1)).clamp(min=0)
    t = (slot[:, :, None] * ps + torch.arange(ps, device=dev)).reshape(B, -1)
    k = s["K"][page].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    v = s["V"][page].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    seen = (t[:, None, :] <= pos[:, :, None]) & (t < lens[:, None])[:, None, :]
    if W:
        seen &= (t[:, None, :] > pos[:, :, None] - W) | (t < S)[:, None, :]
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, -1, qmax, t.shape[1])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.exp_().view(B, Hkv, -1, t.shape[1])
    total_p = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total_p > 0, total_p, 1.0)
    o = o.view(B, Hq, qmax, d).transpose(1, 2)
    tok = torch.arange(total, device=dev)
    b_of = torch.searchsorted(qb[1:].contiguous(), tok, right=True)
    return o[b_of, tok - qb[b_of]].to(torch.bfloat16)


def _plain_append(s):
    ps, qb, lens = s["case"]["page"], s["q_begin"].long(), s["seq_lens"].long()
    tok = torch.arange(s["K_new"].shape[0], device=qb.device)
    b = torch.searchsorted(qb[1:].contiguous(), tok, right=True)
    t = lens[b] - qb[b + 1] + tok
    page, row = s["table"][b, t // ps].long(), t % ps
    s["K"][page, :, row] = s["K_new"]
    s["V"][page, :, row] = s["V_new"]
    return s["K"], s["V"]


def _plain_copy(s):
    # unused entries copy a source page onto itself
    idle = s["src"].max().clamp(min=0)
    src = torch.where(s["src"] < 0, idle, s["src"]).long()
    dst = torch.where(s["dst"] < 0, idle, s["dst"]).long()
    s["K"][dst] = s["K"][src]
    s["V"][dst] = s["V"][src]


def _free_pages(ref):
    """The free pages in ascending order, padded with n_pages."""
    n = ref.shape[0]
    free = ref <= 0
    rank = torch.where(free, free.cumsum(0) - 1, n)
    out = torch.full((n + 1,), n, dtype=torch.long, device=ref.device)
    out[rank] = torch.arange(n, device=ref.device)
    return out


def _plain_branch(s):
    ps, table, ref, lens = s["case"]["page"], s["table"], s["ref"], s["seq_lens"]
    B, mp = table.shape
    n_pages = ref.shape[0]
    dev = table.device
    # fork: the children's rows are their parents', every shared page counted once more
    a, b = s["fork_src"].long(), s["fork_dst"].long()
    table[b] = table[a]
    lens[b] = lens[a]
    shared = table[b].reshape(-1).long()
    ref.index_add_(0, shared.clamp(min=0), (shared >= 0).to(torch.int32))
    # grow: pages for the next tokens in sequence order, the lowest free ones first
    n_new, old = s["n_new"].long(), lens.long()
    slot0 = old // ps
    last = table.gather(1, slot0.clamp(max=mp - 1)[:, None])[:, 0].long()
    part = (old % ps != 0) & (n_new > 0)
    same = (last[:, None] == last[None, :]) & part[:, None] & part[None, :]
    before = same.tril(-1).sum(1)
    split = part & (ref[last.clamp(min=0)] - before > 1)
    lo = torch.where(split, slot0, -(-old // ps))
    hi = torch.where(n_new > 0, -(-(old + n_new) // ps), lo)
    slots = torch.arange(mp, device=dev)
    takes = (slots >= lo[:, None]) & (slots < hi[:, None])
    rank = takes.reshape(-1).cumsum(0).view(B, mp) - 1
    fresh = _free_pages(ref)[rank.clamp(min=0)].to(torch.int32)
    drops = torch.where(split, last, 0)
    ref.index_add_(0, drops, -split.to(torch.int32))
    ref.index_add_(0, torch.where(takes, fresh, 0).reshape(-1).long(), takes.reshape(-1).to(torch.int32))
    table.copy_(torch.where(takes, fresh, table))
    lens += s["n_new"]
    s["src"].copy_(torch.where(split, last, -1))
    s["dst"].copy_(torch.where(split, table.gather(1, slot0.clamp(max=mp - 1)[:, None])[:, 0], -1))
    _plain_copy(s)
    return {k: s[k] for k in ("table", "ref", "seq_lens", "src", "dst", "K", "V")}


def _plain_evict(s):
    c, table, ref, lens = s["case"], s["table"], s["ref"], s["seq_lens"]
    ps, mp, n_pages = c["page"], table.shape[1], ref.shape[0]
    dev = table.device
    start = torch.arange(mp, device=dev) * ps
    ended = s["ended"] != 0
    n = lens[:, None]
    behind = (start >= c["sinks"]) & (start + ps <= n - c["window"]) & (start < n)
    gone = (ended[:, None] | behind) & (table >= 0)
    ref.index_add_(0, torch.where(gone, table, 0).reshape(-1).long(), -gone.reshape(-1).to(torch.int32))
    table.masked_fill_(gone, -1)
    lens.masked_fill_(ended, 0)
    # compact: the live pages above the first n_live go to the holes below, both in ascending order
    live = ref > 0
    n_live = live.sum()
    page = torch.arange(n_pages, device=dev)
    hole, mover = ~live & (page < n_live), live & (page >= n_live)
    cap = s["src"].shape[0]
    for flag, out in ((hole, s["dst"]), (mover, s["src"])):
        got = torch.full((cap + 1,), -1, dtype=torch.int32, device=dev)
        got[torch.where(flag, flag.cumsum(0) - 1, cap)] = page.to(torch.int32)
        got[cap] = -1
        out.copy_(got[:cap])
    s["n_moves"].copy_(mover.sum()[None])
    # table entries and counts follow the pages; unused moves go through a place past the end
    a, b = (torch.where(x >= 0, x, n_pages).long() for x in (s["src"], s["dst"]))
    to = torch.arange(n_pages + 1, dtype=torch.int32, device=dev)
    to[a] = s["dst"]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    counts = torch.cat([ref, ref.new_zeros(1)])
    moved = counts[a]
    counts[a] = 0
    counts[b] = moved
    ref.copy_(counts[:n_pages])
    _plain_copy(s)
    return {k: s[k] for k in ("table", "ref", "seq_lens", "src", "dst", "n_moves", "K", "V")}


_plain = dict(attn=_plain_attn, append=_plain_append, branch=_plain_branch, evict=_plain_evict)
_own = dict(attn=_own_attn, append=_own_append, branch=_own_branch, evict=_own_evict)


# --------------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    if case["op"] == "append":
        return None  # rows as they are: nothing is computed
    s = prepare(case, seed)
    return {"attn": _exact_attn, "branch": _exact_branch, "evict": _exact_evict}[case["op"]](s)


def _exact_attn(s):
    c = s["case"]
    G, ps = c["Hq"] // c["Hkv"], c["page"]
    lens, begin, table = s["seq_lens"].tolist(), s["q_begin"].tolist(), s["table"].long()
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        lo, hi = begin[b], begin[b + 1]
        for i0 in range(lo, hi, 1024):
            i1 = min(hi, i0 + 1024)
            p0, p1 = n - hi + i0, n - hi + i1  # the block's query positions
            t = torch.arange(p1, device="cuda")
            if c["window"]:
                t = t[(t < c["sinks"]) | (t > p0 - c["window"])]
            p = torch.arange(p0, p1, device="cuda")[:, None]
            hidden = t > p
            if c["window"]:
                hidden |= (t <= p - c["window"]) & (t >= c["sinks"])
            for h in range(c["Hkv"]):
                k = s["K"][table[b, t // ps], h, t % ps].double()
                v = s["V"][table[b, t // ps], h, t % ps].double()
                for g in range(h * G, h * G + G):
                    z = (s["Q"][i0:i1, g].double() @ k.T) * s["scale"]
                    z[hidden] = -math.inf
                    out[i0:i1, g] = torch.softmax(z, 1) @ v
    return out


def _exact_branch(s):
    """Sequence by sequence, on lists."""
    ps = s["case"]["page"]
    table, ref, lens = s["table"].tolist(), s["ref"].tolist(), s["seq_lens"].tolist()
    src, dst = [-1] * len(lens), [-1] * len(lens)
    for a, b in zip(s["fork_src"].tolist(), s["fork_dst"].tolist()):
        table[b] = list(table[a])
        lens[b] = lens[a]
        for p in table[b]:
            if p >= 0:
                ref[p] += 1
    unused = iter([p for p, r in enumerate(ref) if r == 0])
    for b, add in enumerate(s["n_new"].tolist()):
        n = lens[b]
        if add > 0:
            if n % ps and ref[table[b][n // ps]] > 1:
                src[b], dst[b] = table[b][n // ps], next(unused)
                ref[src[b]] -= 1
                ref[dst[b]] = 1
                table[b][n // ps] = dst[b]
            for t in range(-(-n // ps), -(-(n + add) // ps)):
                table[b][t] = next(unused)
                ref[table[b][t]] = 1
        lens[b] = n + add
    return dict(_ints(table=table, ref=ref, seq_lens=lens, src=src, dst=dst), K=None, V=None)


def _exact_evict(s):
    c = s["case"]
    ps = c["page"]
    table, ref, lens = s["table"].tolist(), s["ref"].tolist(), s["seq_lens"].tolist()
    for b, ended in enumerate(s["ended"].tolist()):
        for t, p in enumerate(table[b]):
            keep = t * ps < c["sinks"] or (t + 1) * ps > lens[b] - c["window"]
            if p >= 0 and (ended or not keep):
                ref[p] -= 1
                table[b][t] = -1
        lens[b] = 0 if ended else lens[b]
    live = [p for p, r in enumerate(ref) if r > 0]
    moves = [p for p in live if p >= len(live)]
    holes = [p for p in range(len(live)) if ref[p] == 0]
    to = dict(zip(moves, holes))
    for p, h in to.items():
        ref[h], ref[p] = ref[p], 0
    table = [[to.get(p, p) for p in row] for row in table]
    pad = [-1] * (s["src"].shape[0] - len(moves))
    return dict(_ints(table=table, ref=ref, seq_lens=lens, src=moves + pad, dst=holes + pad, n_moves=[len(moves)]),
                K=None, V=None)


def _ints(**lists):
    return {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in lists.items()}
