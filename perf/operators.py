"""Cases for the serving operators over a paged KV cache: the page plan of a
step, the attention of packed prompts, and the attention of new tokens over
the cache.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, with ``own`` set, through libmq's
entry points as a serving loop calls them.  ``exact`` is the definition in 64
bits.  All inputs are synthetic.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128                      # head dimension of every attention of this library


# -- cases ----------------------------------------------------------------------

def listed():
    return [
        # a decode step of a few requests: 8 slots, at most 8 new pages; launch latency is all of it
        _plan("plan_decode_8", B=8, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=8192, page=16, pick=1),
        # a step that mixes prompts, chunks and single tokens, some requests idle, in pages of 64
        _plan("plan_mixed_257", B=257, new_lo=0, new_hi=512, ctx_lo=0, ctx_hi=8192, page=64, pick=2),
        # a whole 131072-token budget over thousands of requests
        _plan("plan_full_4096", B=4096, new_lo=1, new_hi=120, ctx_lo=0, ctx_hi=4096, page=16, pick=3),
        # a handful of short prompts (tests' head layout), no cache yet
        _packed("packed_short_3", B=3, lo=1, hi=300, H=8, Hkv=2, page=0, pad=5, amax=False, pick=27),
        # one prompt of the 8B layer's 8192 tokens, written to the cache, with the amax of o for the O projection
        _packed("packed_8b_8192", B=1, lo=8192, hi=8192, H=32, Hkv=8, page=64, pad=0, amax=True, pick=5),
        # a ragged prefill batch with the 70B layer's heads
        _packed("packed_ragged_16", B=16, lo=64, hi=4096, H=64, Hkv=8, page=16, pad=77, amax=False, pick=6),
        # the fourth 16384-token chunk of the chunked 131072-token prefill
        _paged("chunk_16384_at_49152", B=1, chunks=1, new_lo=16384, new_hi=16384, ctx_lo=49152, ctx_hi=49152,
               H=32, Hkv=8, page=128, pick=7),
        # a step of a serving loop: a few chunks beside many single tokens
        _paged("mixed_4_of_64", B=64, chunks=4, new_lo=300, new_hi=2048, ctx_lo=128, ctx_hi=16384, H=32, Hkv=8,
               page=16, pick=8),
        # eight draft tokens checked at once for each request
        _paged("draft_8x16", B=16, chunks=16, new_lo=8, new_hi=8, ctx_lo=1000, ctx_hi=8192, H=32, Hkv=8, page=32,
               pick=9),
        # the bench's decode step: one token over 8192 cached positions
        _paged("decode_1_at_8192", B=1, chunks=0, new_lo=1, new_hi=1, ctx_lo=8192, ctx_hi=8192, H=32, Hkv=8, page=64,
               pick=10),
        # one token over a long context
        _paged("decode_1_at_32768", B=1, chunks=0, new_lo=1, new_hi=1, ctx_lo=32768, ctx_hi=32768, H=32, Hkv=8,
               page=16, pick=11),
        # a decode batch of ragged contexts
        _paged("decode_64", B=64, chunks=0, new_lo=1, new_hi=1, ctx_lo=512, ctx_hi=8192, H=32, Hkv=8, page=16,
               pick=12),
    ]


def _plan(name, **kw):
    return {"name": name, "op": "plan", **kw}


def _packed(name, **kw):
    return {"name": name, "op": "packed", **kw}


def _paged(name, **kw):
    return {"name": name, "op": "paged", **kw}


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo + 0.5), math.log(hi + 0.5)))))))


HEADS = [(32, 8), (64, 8), (8, 2), (4, 4), (8, 1), (12, 4), (16, 16), (6, 2), (28, 4), (40, 8)]


def draw(rng):
    kind = rng.choice(["plan", "packed", "packed", "chunk", "mixed", "decode", "decode"])
    pick = rng.randrange(1 << 30)
    page = rng.choice([8, 16, 32, 64, 128, 256])
    H, Hkv = rng.choice(HEADS)
    if kind == "plan":
        new_hi = _log_int(rng, 1, 500)
        return {"op": "plan", "B": _log_int(rng, 1, min(4096, max(1, 200000 // new_hi))), "new_lo": rng.choice([0, 1]),
                "new_hi": new_hi, "ctx_lo": 0, "ctx_hi": _log_int(rng, 1, 8192), "page": page, "pick": pick}
    if kind == "packed":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(16, min(8192, 40000 // B)))
        return {"op": "packed", "B": B, "lo": _log_int(rng, 1, hi), "hi": hi, "H": H, "Hkv": Hkv,
                "page": rng.choice([0, page]), "pad": rng.choice([0, 1, 130]), "amax": rng.random() < 0.3, "pick": pick}
    if kind == "chunk":
        new_hi = _log_int(rng, 2, 4096)
        ctx_hi = _log_int(rng, 1, 40000)
        B = _log_int(rng, 1, 6)
        return {"op": "paged", "B": B, "chunks": B, "new_lo": max(1, new_hi // 3), "new_hi": new_hi,
                "ctx_lo": rng.choice([0, ctx_hi // 2, ctx_hi]), "ctx_hi": ctx_hi, "H": H, "Hkv": Hkv, "page": page,
                "pick": pick}
    if kind == "mixed":
        B = _log_int(rng, 2, 100)
        new_hi = _log_int(rng, 2, 1500)
        return {"op": "paged", "B": B, "chunks": rng.randint(1, min(B, 4)), "new_lo": max(1, new_hi // 4),
                "new_hi": new_hi, "ctx_lo": 0, "ctx_hi": _log_int(rng, 1, 8192), "H": H, "Hkv": Hkv, "page": page,
                "pick": pick}
    B = _log_int(rng, 1, 128)
    ctx_hi = _log_int(rng, 1, min(60000, 400000 // B))
    new = rng.choice([1, 1, 1, 2, 5])
    return {"op": "paged", "B": B, "chunks": B, "new_lo": new, "new_hi": new, "ctx_lo": rng.choice([0, ctx_hi // 3]),
            "ctx_hi": ctx_hi, "H": H, "Hkv": Hkv, "page": page, "pick": pick}


# -- lengths of a case ------------------------------------------------------------

def _spread(rng, lo, hi):
    return lo if lo == hi else (0 if lo == 0 and rng.random() < 0.1 else _log_int(rng, max(lo, 1), hi))


def _lengths(case):
    """(context lengths, new lengths) of the case's requests; a packed prompt has no context."""
    rng = random.Random(case["pick"])
    B = case["B"]
    if case["op"] == "packed":
        return [0] * B, [_log_int(rng, case["lo"], case["hi"]) for _ in range(B)]
    ctx = [_spread(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    if case["op"] == "plan":
        return ctx, [_spread(rng, case["new_lo"], case["new_hi"]) for _ in range(B)]
    chunked = set(rng.sample(range(B), case["chunks"]))
    return ctx, [_log_int(rng, case["new_lo"], case["new_hi"]) if b in chunked else 1 for b in range(B)]


def _pages(n, page):
    return -(-n // page)


def work(case):
    ctx, new = _lengths(case)
    T = sum(new)
    if case["op"] == "plan":
        ps = case["page"]
        fresh = sum(_pages(c + n, ps) - _pages(c, ps) for c, n in zip(ctx, new))
        partly = sum(1 for c, n in zip(ctx, new) if n and c % ps)   # a page already in the table takes tokens
        return {"bytes": 8 * case["B"] + 4 * (case["B"] + 1) + 8 * T + 8 * fresh + 4 * partly + 16, "flops": 2 * T}
    H, Hkv = case["H"], case["Hkv"]
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    b = T * (H + 2 * Hkv) * D * 2 + T * H * D * 2 + sum(ctx) * 2 * Hkv * D * 2
    if case["page"]:
        b += T * 2 * Hkv * D * 2
    return {"bytes": b, "flops": 4 * D * H * pairs}


# -- inputs -----------------------------------------------------------------------

def _table(case, ctx, new, gen_rng):
    """A block table with every page of ctx + new assigned in a shuffled pool, the pool's size, and how many pages
    each request holds before the step."""
    ps = case["page"]
    held = [_pages(c, ps) for c in ctx]
    total = [_pages(c + n, ps) for c, n in zip(ctx, new)]
    width = max(max(total), 1) + 1
    n_pages = sum(total) + 3
    ids = list(range(n_pages))
    gen_rng.shuffle(ids)
    rows, at = [], 0
    for b in range(case["B"]):
        rows.append(ids[at:at + total[b]] + [-1] * (width - total[b]))
        at += total[b]
    return rows, n_pages, held, ids[at:]


def prepare(case, seed):
    ctx, new = _lengths(case)
    rng = random.Random(seed * 7919 + 13)
    dev = "cuda"
    i32 = dict(dtype=torch.int32, device=dev)
    B, T = case["B"], sum(new)
    st = {"case": case, "ctx": ctx, "new": new}
    if case["op"] == "plan":
        # the table as the step before left it, and the pool's free pages
        ps = case["page"]
        rows, n_pages, held, spare = _table(case, ctx, new, rng)
        free, table = [], []
        for b in range(B):
            free += [p for p in rows[b][held[b]:] if p >= 0]
            table.append(rows[b][:held[b]] + [-1] * (len(rows[b]) - held[b]))
        free += spare
        rng.shuffle(free)
        st.update(ctx_lens=torch.tensor(ctx, **i32), new_lens=torch.tensor(new, **i32), free=torch.tensor(free, **i32),
                  table=torch.tensor(table, **i32), T=T + 3,      # a fixed token budget a little above the step's
                  cu=torch.zeros(B + 1, **i32), slots=torch.zeros(T + 3, dtype=torch.int64, device=dev),
                  info=torch.zeros(4, **i32))
        return st
    H, Hkv = case["H"], case["Hkv"]
    g = torch.Generator(device=dev).manual_seed(seed * 1_000_003 + case["pick"])
    pad = case.get("pad", 0)
    qkv = torch.randn(T + pad, (H + 2 * Hkv) * D, generator=g, device=dev, dtype=torch.float32)
    qkv[:, :H * D] *= 2.0           # queries a little long, so that some weights stand out
    qkv = qkv.to(torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st.update(qkv=qkv, cu=torch.tensor(cu, **i32), cu_host=cu,
              o=torch.zeros(T + pad, H * D, dtype=torch.bfloat16, device=dev), T=T + pad,
              amax=torch.zeros(1, dtype=torch.float32, device=dev))
    if case["page"]:
        ps = case["page"]
        rows, n_pages, held, _ = _table(case, ctx, new, rng)
        shape = (n_pages, Hkv, ps, D)
        k = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        v = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        table = torch.tensor(rows, **i32)
        for b in range(B):
            if held[b]:
                ids = table[b, :held[b]].long()
                for pool in (k, v):
                    pool[ids] = torch.randn(held[b], Hkv, ps, D, generator=g, device=dev).to(torch.bfloat16)
        slots = []
        for b in range(B):
            slots += [rows[b][(ctx[b] + i) // ps] * ps + (ctx[b] + i) % ps for i in range(new[b])]
        slots += [-1] * pad
        st.update(k=k, v=v, table=table, n_pages=n_pages, ctx_lens=torch.tensor(ctx, **i32),
                  slots=torch.tensor(slots, dtype=torch.int64, device=dev))
    if own:
        from nvfp4_quantized_prefill_b200 import binding as mq
        nb = (mq.mq_attention_packed_workspace_bytes(st["T"], B, H, Hkv, D) if case["op"] == "packed" else
              mq.mq_attention_paged_workspace_bytes(st["T"], B, max(new), H, Hkv, D))
        st.update(ws=torch.empty(nb, dtype=torch.uint8, device=dev), ws_bytes=nb)
    return st


# -- one pass ------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    from nvfp4_quantized_prefill_b200 import binding as mq
    c = st["case"]
    if c["op"] == "plan":
        mq.mq_paged_plan(st["ctx_lens"], st["new_lens"], c["B"], c["page"], st["free"], st["free"].numel(), st["table"],
                         st["table"].shape[1], st["T"], st["cu"], st["slots"], st["info"])
        return [st["cu"], st["slots"], st["table"], st["info"]]
    H, Hkv = c["H"], c["Hkv"]
    cols = (H + 2 * Hkv) * D
    if c["op"] == "packed":
        pool = (st["slots"], st["k"], st["v"], st["n_pages"], c["page"]) if c["page"] else (None, None, None, 0, 0)
        mq.mq_attention_packed_bf16(st["qkv"], cols, st["T"], st["cu"], c["B"], H, Hkv, D, *pool, st["o"], H * D,
                                    st["amax"] if c["amax"] else None, st["ws"], st["ws_bytes"])
        out = [st["o"]]
        if c["page"]:
            out += [st["k"], st["v"]]
        if c["amax"]:
            out.append(st["amax"].to(torch.bfloat16))      # the value is a BF16 output's
        return out
    mq.mq_attention_paged_bf16(st["qkv"], cols, st["T"], st["cu"], st["ctx_lens"], c["B"], max(st["new"]), H, Hkv, D,
                               st["slots"], st["table"], st["table"].shape[1], st["k"], st["v"], st["n_pages"],
                               c["page"], st["o"], H * D, None, st["ws"], st["ws_bytes"])
    return [st["o"], st["k"], st["v"]]


def _run_plain(st):
    c = st["case"]
    if c["op"] == "plan":
        return _plan_plain(st)
    H, Hkv = c["H"], c["Hkv"]
    G = H // Hkv
    T = sum(st["new"])
    qkv = st["qkv"][:T]
    q = qkv[:, :H * D].view(T, Hkv, G, D)
    kn = qkv[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
    vn = qkv[:, (H + Hkv) * D:].view(T, Hkv, D)
    o = st["o"]
    if c["page"]:
        page, off = st["slots"][:T] // c["page"], st["slots"][:T] % c["page"]
        st["k"][page, :, off] = kn
        st["v"][page, :, off] = vn
    for b in range(c["B"]):
        t0, t1, ctx = st["cu_host"][b], st["cu_host"][b + 1], st["ctx"][b]
        n = ctx + t1 - t0
        if c["op"] == "paged":
            ids = st["table"][b, :_pages(n, c["page"])].long()
            kb = st["k"][ids].transpose(1, 2).reshape(-1, Hkv, D)[:n].float()
            vb = st["v"][ids].transpose(1, 2).reshape(-1, Hkv, D)[:n].float()
        else:
            kb, vb = kn[t0:t1].float(), vn[t0:t1].float()
        kb, vb = kb.transpose(0, 1), vb.transpose(0, 1)                      # [Hkv, n, D]
        step = max(1, min(t1 - t0, (1 << 29) // (n * H)))                    # rows at a time: 2 GB of scores
        for r in range(t0, t1, step):
            e = min(r + step, t1)
            m = ctx + e - t0                                                # keys the last of these rows sees
            qb = q[r:e].float().permute(1, 2, 0, 3).reshape(Hkv, G * (e - r), D)
            s = torch.bmm(qb, kb[:, :m].transpose(1, 2)).view(Hkv, G, e - r, m) * (1.0 / math.sqrt(D))
            pos = torch.arange(ctx + r - t0, ctx + e - t0, device=s.device)
            s.masked_fill_(torch.arange(m, device=s.device) > pos[:, None], float("-inf"))
            s -= s.amax(-1, keepdim=True)
            s.exp_()
            l = s.sum(-1, keepdim=True)
            ob = torch.bmm(s.view(Hkv, G * (e - r), m), vb[:, :m]).view(Hkv, G, e - r, D) / l
            o[r:e] = ob.permute(2, 0, 1, 3).reshape(e - r, H * D).to(torch.bfloat16)
    out = [o]
    if c["page"]:
        out += [st["k"], st["v"]]
    if c.get("amax"):
        out.append(o[:T].float().abs().amax().view(1).to(torch.bfloat16))
    return out


def _plan_plain(st):
    """Prefix sums, a search of each token's request, and gathers."""
    c = st["case"]
    ps, T, table, free = c["page"], st["T"], st["table"], st["free"]
    ctx, new = st["ctx_lens"].long(), st["new_lens"].long()
    cu = torch.zeros(c["B"] + 1, dtype=torch.int64, device=ctx.device)
    cu[1:] = torch.cumsum(new, 0)
    held = (ctx + ps - 1) // ps
    need = (ctx + new + ps - 1) // ps - held
    base = torch.cumsum(need, 0) - need
    t = torch.arange(T, device=ctx.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp_(max=c["B"] - 1)
    live = t < cu[-1]
    pos = ctx[b] + t - cu[b]
    page = (pos // ps).clamp_(max=table.shape[1] - 1)
    fresh = live & (page >= held[b])
    taken = free[(base[b] + page - held[b]).clamp_(0, free.numel() - 1)]
    first = fresh & (pos % ps == 0)
    row, col, val = b[first], page[first], taken[first]
    table[row, col] = val
    ids = torch.where(fresh, taken, table[b, page]).long()
    st["cu"].copy_(cu)
    st["slots"].copy_(torch.where(live, ids * ps + pos % ps, torch.full_like(ids, -1)))
    st["info"].copy_(torch.stack([cu[-1], need.sum(), torch.zeros_like(cu[-1]), (ctx + new).max()]))
    return [st["cu"], st["slots"], table, st["info"]]


# -- the definition in 64 bits ------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return _plan_exact(st)
    H, Hkv = case["H"], case["Hkv"]
    G = H // Hkv
    o = torch.zeros(st["T"], H * D, dtype=torch.float64, device="cuda")
    total = 0
    for b in range(case["B"]):
        ctx, n = st["ctx"][b], st["new"][b]
        rows = st["qkv"][st["cu_host"][b]:st["cu_host"][b] + n]
        keys = rows[:, H * D:(H + Hkv) * D].reshape(n, Hkv, D)
        vals = rows[:, (H + Hkv) * D:].reshape(n, Hkv, D)
        if case["page"]:
            for i0 in range(0, n, 1 << 16):                    # the new tokens' rows of the cache
                s = st["slots"][st["cu_host"][b] + i0:st["cu_host"][b] + min(n, i0 + (1 << 16))]
                m = s.numel()
                st["k"].view(-1, Hkv, case["page"], D)[s // case["page"], :, s % case["page"]] = keys[i0:i0 + m]
                st["v"].view(-1, Hkv, case["page"], D)[s // case["page"], :, s % case["page"]] = vals[i0:i0 + m]
        for g in range(Hkv):
            kg, vg = keys[:, g].double(), vals[:, g].double()
            if ctx:
                ids = st["table"][b, :_pages(ctx, case["page"])].long()
                kg = torch.cat([st["k"][ids, g].reshape(-1, D)[:ctx].double(), kg])
                vg = torch.cat([st["v"][ids, g].reshape(-1, D)[:ctx].double(), vg])
            for h in range(g * G, (g + 1) * G):
                qh = rows[:, h * D:(h + 1) * D].double()
                for r in range(0, n, 2048):
                    e = min(n, r + 2048)
                    z = qh[r:e] @ kg[:ctx + e].T / D ** 0.5
                    z = torch.where(torch.ones(e - r, ctx + e, dtype=torch.bool, device="cuda").tril(ctx + r), z,
                                    torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                    w = torch.softmax(z, dim=1)
                    o[total + r:total + e, h * D:(h + 1) * D] = w @ vg[:ctx + e]
        total += n
    out = [o]
    if case["page"]:
        out += [st["k"], st["v"]]
    if case.get("amax"):
        out.append(o[:total].abs().amax().view(1))
    return out


def _plan_exact(st):
    """Request by request and token by token on the host."""
    c, ps = st["case"], st["case"]["page"]
    table, free = st["table"].cpu().tolist(), st["free"].cpu().tolist()
    cu, slots, taken, longest = [0], [], 0, 0
    for b in range(c["B"]):
        held = _pages(st["ctx"][b], ps)
        for i in range(st["new"][b]):
            p, off = divmod(st["ctx"][b] + i, ps)
            if off == 0 and p >= held:
                table[b][p] = free[taken]
                taken += 1
            slots.append(table[b][p] * ps + off)
        cu.append(len(slots))
        longest = max(longest, st["ctx"][b] + st["new"][b])
    slots += [-1] * (st["T"] - len(slots))
    return [torch.tensor(cu, dtype=torch.int32), torch.tensor(slots, dtype=torch.int64),
            torch.tensor(table, dtype=torch.int32), torch.tensor([cu[-1], taken, 0, longest], dtype=torch.int32)]
