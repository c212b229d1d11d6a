"""The paged serving calls on the GPU: the page plan, attention of packed
prompts and attention of new tokens over the paged cache, each against its
definition, and a serving loop of them together.

Attention tolerance, per output element, as for the single-sequence attention:
    |gpu - ref| <= 2^-8 (a + |ref|),  a = sum_j w_j |v_j| / sum_j w_j
Each weight is rounded to BF16 before the P.V product (half a step, 2^-9
relative with 8 significant bits: at most 2^-9 a) and the sum that divides is
taken over the rounded weights (its deviation, at most 2^-9 relative, is
another 2^-9 |ref| <= 2^-9 a); o is rounded to BF16 (2^-9 |ref|).  Together
2^-8 a + 2^-9 |ref|; FP32 accumulation and 2^x (2^-22 relative) fit in the
remaining 2^-9 |ref|, and where |ref| is far below a, below the 2^-9 a that a
worst-case sign pattern of the weights' roundings would need.  Pages, tables,
slots and max |o| are compared exactly."""
import random

import numpy as np
import pytest
import torch

import oracle
from mqtest import ensure_built
from nvfp4_quantized_prefill_b200 import binding as mq

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# -- the page plan -------------------------------------------------------------------

def plan_ref(ctx, new, ps, free, table, max_pages, T):
    """Request by request, token by token."""
    table = [list(r) for r in table]
    ctx, new = [max(c, 0) for c in ctx], [max(n, 0) for n in new]
    cu, slots, needed, longest, lost = [0], [], 0, 0, 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        kept = min(n, T - cu[-1])
        held = min(-(-c // ps), max_pages)
        need = min(-(-(c + kept) // ps), max_pages) - held
        for i in range(kept):
            p, off = divmod(c + i, ps)
            page = -1
            if p < max_pages:
                if p >= -(-c // ps):
                    k = needed + p - held
                    page = free[k] if k < len(free) else -1
                    table[b][p] = page
                else:
                    page = table[b][p]
            lost += page < 0
            slots.append(page * ps + off if page >= 0 else -1)
        needed += need
        longest = max(longest, c + kept)
        cu.append(cu[-1] + kept)
    slots += [-1] * (T - len(slots))
    return cu, slots, table, [sum(new), needed, sum(new) - cu[-1] + lost, longest]


def _plan(ctx, new, ps, free, table, max_pages, T, stream=None):
    B = len(ctx)
    cu = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    info = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    td, fd = _i32(table), _i32(free)
    mq.mq_paged_plan(_i32(ctx), _i32(new), B, ps, fd if len(free) else None, len(free), td, max_pages, T, cu, slots,
                     info, stream)
    return cu, slots, td, info


def _pool(ctx, new, ps, max_pages, n_free, seed):
    """A table with the pages of ctx in place and a shuffled free list."""
    rng = random.Random(seed)
    held = [min(-(-max(c, 0) // ps), max_pages) for c in ctx]
    ids = list(range(sum(held) + n_free))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-5] * (max_pages - h))
        at += h
    return table, ids[at:]


PLANS = [
    # ctx, new, page size, max_pages, free pages, T
    ([0], [1], 8, 1, 1, 1),
    ([7, 8, 9, 0], [1, 1, 1, 1], 8, 3, 4, 4),
    ([0, 5, 0, 100, 16], [0, 0, 0, 0, 0], 16, 8, 3, 5),                 # a step without new tokens
    ([3, 0, 40, 16, 15], [20, 0, 1, 16, 2], 16, 5, 9, 64),              # padding rows
    ([3, 0, 40, 16, 15], [20, 0, 1, 16, 2], 16, 5, 9, 30),              # cut at T
    ([30, 0, 10], [40, 50, 60], 16, 4, 20, 200),                        # table rows too short
    ([0, 10, 0], [100, 30, 100], 16, 20, 9, 240),                       # the free list runs out
    ([0, 10, 0], [100, 30, 100], 16, 20, 0, 240),                       # no free page at all
    ([-3, 5], [4, -2], 32, 2, 4, 8),                                    # negative lengths count as none
    ([1000] * 3, [300, 1, 257], 256, 6, 6, 600),
    ([70000, 2 ** 31 - 600], [5, 590], 128, 600, 9, 600),               # positions next to 2^31
]


@pytest.mark.parametrize("ctx,new,ps,max_pages,n_free,T", PLANS)
def test_plan_against_its_definition(ctx, new, ps, max_pages, n_free, T):
    table, free = _pool(ctx, new, ps, max_pages, n_free, 3)
    got = _plan(ctx, new, ps, free, table, max_pages, T)
    for g, r in zip(got, plan_ref(ctx, new, ps, free, table, max_pages, T)):
        assert g.tolist() == r
    assert mq.mq_check() == 0


@pytest.mark.parametrize("B,hi,ps", [(513, 40, 16), (4096, 33, 8), (16384, 9, 64)])
def test_plan_many_requests(B, hi, ps):
    rng = random.Random(B)
    ctx = [rng.randrange(0, 300) for _ in range(B)]
    new = [rng.choice([0, 1, 1, rng.randrange(0, hi)]) for _ in range(B)]
    max_pages = 300 // ps + hi // ps + 2
    table, free = _pool(ctx, new, ps, max_pages, sum(new) // ps + B, B)
    T = sum(new) + 11
    got = _plan(ctx, new, ps, free, table, max_pages, T)
    for g, r in zip(got, plan_ref(ctx, new, ps, free, table, max_pages, T)):
        assert g.tolist() == r


# -- attention -----------------------------------------------------------------------

def _qkv(n, H, Hkv, seed, q_gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, (H + 2 * Hkv) * D, generator=g)
    x[:, : H * D] *= q_gain
    return x.to(torch.bfloat16)


def _split(x, H, Hkv):
    return x[:, : H * D], x[:, H * D:(H + Hkv) * D], x[:, (H + Hkv) * D:]


def assert_close(o, ref, a, what):
    og = o.float().double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(og).all(), f"{what}: not finite"
    over = np.abs(og - ref) - 2.0 ** -8 * (a + np.abs(ref))
    if (over > 0).any():
        i = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError(f"{what}: {int((over > 0).sum())}/{over.size} outside the bound; worst at {i}: gpu "
                             f"{og[i]!r} ref {ref[i]!r} a {a[i]!r}")


class Step:
    """A batch of sequences with ctx cached and new tokens each, in a pool of
    shuffled pages whose rows nobody wrote hold NaN, and padding rows of NaN."""

    def __init__(self, ctx, new, H, Hkv, ps, seed=0, pad=0, q_gain=1.0, ld_extra=0, paged=True):
        self.ctx, self.new, self.H, self.Hkv, self.ps, self.pad = ctx, new, H, Hkv, ps, pad
        B, self.n = len(ctx), sum(new)
        self.T = self.n + pad
        cols = (H + 2 * Hkv) * D
        self.seqs = [_qkv(c + n, H, Hkv, seed * 1000 + b, q_gain) for b, (c, n) in enumerate(zip(ctx, new))]
        rows = torch.cat([s[c:] for s, c in zip(self.seqs, ctx)] +
                         [torch.full((pad, cols), float("nan"), dtype=torch.bfloat16)])
        wide = torch.full((max(self.T, 1), cols + ld_extra), float("nan"), dtype=torch.bfloat16)
        wide[: self.T, :cols] = rows
        self.qkv, self.ldqkv = wide.cuda(), cols + ld_extra
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32).tolist()
        self.o = torch.full((max(self.T, 1), H * D + ld_extra), 3.0, dtype=torch.bfloat16, device="cuda")
        self.amax = torch.full((1,), 99.0, dtype=torch.float32, device="cuda")
        self.max_pages = max(-(-(c + n) // ps) for c, n in zip(ctx, new)) + 1 if ps else 1
        if ps:
            total = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
            self.n_pages = sum(total) + 2
            ids = list(range(self.n_pages))
            random.Random(seed).shuffle(ids)
            self.table, at = [], 0
            for t in total:
                self.table.append(ids[at:at + t] + [-1] * (self.max_pages - t))
                at += t
            self.k = torch.full((self.n_pages, Hkv, ps, D), float("nan"), dtype=torch.bfloat16)
            self.v = self.k.clone()
            for b, c in enumerate(ctx):
                self._put(self.k, self.v, b, 0, c)
            self.k, self.v = self.k.cuda(), self.v.cuda()
            self.k0, self.v0 = self.k.clone(), self.v.clone()
            self.slots = [self.table[b][p // ps] * ps + p % ps for b in range(B)
                          for p in range(ctx[b], ctx[b] + new[b])] + [-1] * pad
            self.slots_d = torch.tensor(self.slots or [0], dtype=torch.int64, device="cuda")

    def _put(self, kp, vp, b, lo, hi):
        _, k, v = _split(self.seqs[b], self.H, self.Hkv)
        for p in range(lo, hi):
            page, off = self.table[b][p // self.ps], p % self.ps
            kp[page, :, off] = k[p].view(self.Hkv, D)
            vp[page, :, off] = v[p].view(self.Hkv, D)

    def packed(self, stream=None, amax=True):
        H, Hkv, B = self.H, self.Hkv, len(self.ctx)
        nb = mq.mq_attention_packed_workspace_bytes(self.T, B, H, Hkv, D)
        self.ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
        self.cu_d = _i32(self.cu)
        pool = (self.slots_d, self.k, self.v, self.n_pages, self.ps) if self.ps else (None, None, None, 0, 0)
        mq.mq_attention_packed_bf16(self.qkv, self.ldqkv, self.T, self.cu_d, B, H, Hkv, D, *pool, self.o,
                                    self.o.stride(0), self.amax if amax else None, self.ws, nb, stream)

    def paged(self, max_new=None, stream=None, amax=True):
        H, Hkv, B = self.H, self.Hkv, len(self.ctx)
        max_new = max_new or max(max(self.new), 1)
        nb = mq.mq_attention_paged_workspace_bytes(self.T, B, max_new, H, Hkv, D)
        self.ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
        self.cu_d, self.ctx_d, self.table_d = _i32(self.cu), _i32(self.ctx), _i32(self.table)
        mq.mq_attention_paged_bf16(self.qkv, self.ldqkv, self.T, self.cu_d, self.ctx_d, B, max_new, H, Hkv, D,
                                   self.slots_d, self.table_d, self.max_pages, self.k, self.v, self.n_pages, self.ps,
                                   self.o, self.o.stride(0), self.amax if amax else None, self.ws, nb, stream)

    def check(self, what, rows=None):
        torch.cuda.synchronize()
        H, Hkv = self.H, self.Hkv
        o = self.o[:, : H * D]
        for b, s in enumerate(self.seqs):
            if not self.new[b]:
                continue
            q, k, v = _split(s, H, Hkv)
            r = None if rows is None else np.array(sorted({x % self.new[b] for x in rows}), dtype=np.int64)
            ref, a = oracle.attention(q[self.ctx[b]:], k, v, H, Hkv, D, pos0=self.ctx[b], rows=r)
            og = o[self.cu[b]:self.cu[b + 1]]
            assert_close(og if r is None else og[torch.from_numpy(r).cuda()], ref, a, f"{what}, sequence {b}")
        # padding rows and the columns between rows are left as they were
        assert (self.o[self.n:] == 3.0).all() and (self.o[:, H * D:] == 3.0).all()
        if self.ps:
            kr, vr = self.k0.cpu(), self.v0.cpu()
            for b in range(len(self.ctx)):
                self._put(kr, vr, b, self.ctx[b], self.ctx[b] + self.new[b])
            assert torch.equal(self.k.cpu().view(torch.int16), kr.view(torch.int16))
            assert torch.equal(self.v.cpu().view(torch.int16), vr.view(torch.int16))
        assert mq.mq_check() == 0

    def check_amax(self):
        want = float(self.o[: self.n, : self.H * D].float().abs().max()) if self.n else 0.0
        assert float(self.amax) == want


PROMPTS = [
    # lengths, H, Hkv, page size (0: no cache), padding rows, q gain
    ([1], 1, 1, 0, 0, 1.0),
    ([77], 4, 2, 16, 3, 1.0),
    ([1, 1, 1], 8, 2, 8, 0, 1.0),
    ([127, 128, 129], 4, 4, 64, 0, 4.0),
    ([300, 0, 5, 64, 0, 65], 8, 2, 16, 131, 1.0),
    ([31, 33, 32, 500], 8, 1, 32, 0, 8.0),
    ([640, 257], 6, 2, 128, 1, 4.0),              # group of 3: 42 tokens a tile
    ([190], 7, 1, 256, 0, 1.0),                   # group of 7: 18 tokens a tile
    ([200, 3], 64, 1, 16, 0, 1.0),                # group of 64: two tokens a tile
    ([9, 40], 128, 1, 16, 0, 1.0),                # one token a tile
    ([40], 99, 1, 0, 0, 1.0),                     # 99 of 128 rows of a tile
    ([0, 0, 0], 4, 2, 16, 4, 1.0),                # nothing to do but padding
    ([1500, 700, 1, 90], 16, 4, 16, 60, 2.0),
]


@pytest.mark.parametrize("lens,H,Hkv,ps,pad,gain", PROMPTS)
def test_packed_prompts(lens, H, Hkv, ps, pad, gain):
    st = Step([0] * len(lens), lens, H, Hkv, ps, seed=len(lens) + H, pad=pad, q_gain=gain)
    st.packed()
    st.check("packed")
    st.check_amax()


CHUNKS = [
    # ctx, new, H, Hkv, page size, padding rows, q gain
    ([0], [1], 1, 1, 8, 0, 1.0),
    ([300], [1], 8, 2, 16, 0, 1.0),
    ([127, 128, 129, 0, 1], [1, 1, 1, 1, 1], 32, 8, 64, 0, 1.0),
    ([1000, 0, 17], [1, 0, 1], 4, 4, 32, 5, 4.0),                 # an idle request
    ([200, 64, 5], [8, 3, 8], 8, 2, 16, 0, 1.0),                  # draft tokens
    ([255, 256, 257], [2, 2, 2], 6, 2, 256, 0, 1.0),
    ([500], [300], 8, 2, 16, 0, 4.0),                             # a chunk
    ([0, 1000, 130], [129, 64, 65], 4, 2, 8, 7, 1.0),             # chunks, one without context
    ([900, 40, 700, 3], [1, 200, 1, 1], 8, 2, 128, 0, 1.0),       # a chunk beside single tokens
    ([100, 2000], [33, 34], 16, 4, 64, 0, 8.0),
    ([300, 7], [20, 1], 64, 1, 16, 0, 1.0),                       # two tokens a tile
    ([90], [3], 99, 1, 16, 0, 1.0),
    ([6000], [5], 16, 4, 16, 0, 2.0),
    ([0, 0], [0, 0], 4, 2, 16, 3, 1.0),
    ([33] * 40, [1] * 40, 4, 1, 16, 2, 1.0),
]


@pytest.mark.parametrize("ctx,new,H,Hkv,ps,pad,gain", CHUNKS)
def test_chunks_over_the_paged_cache(ctx, new, H, Hkv, ps, pad, gain):
    st = Step(ctx, new, H, Hkv, ps, seed=len(ctx) + H + ps, pad=pad, q_gain=gain)
    st.paged()
    st.check("paged")
    st.check_amax()


@pytest.mark.parametrize("seed", range(6))
def test_random_steps(seed):
    """Sizes, heads and pages drawn together; every row is checked."""
    rng = random.Random(seed)
    H, Hkv = rng.choice([(32, 8), (8, 2), (4, 4), (8, 1), (12, 4), (28, 4), (40, 8)])
    B = rng.choice([1, 3, 9])
    new = [rng.choice([1, 1, 7, rng.randrange(1, 200)]) for _ in range(B)]
    ctx = [rng.choice([0, 1, rng.randrange(0, 700)]) for _ in range(B)]
    ps = rng.choice([8, 16, 32, 64, 128, 256])
    st = Step(ctx, new, H, Hkv, ps, seed=100 + seed, pad=rng.choice([0, 9]), q_gain=2.0)
    st.paged(amax=False)
    st.check(f"random paged step {seed}")
    st = Step([0] * B, new, H, Hkv, ps, seed=200 + seed, pad=rng.choice([0, 9]), q_gain=2.0)
    st.packed(amax=False)
    st.check(f"random packed step {seed}")


def test_leading_dimensions():
    st = Step([0, 0], [150, 20], 8, 2, 16, seed=5, pad=3, ld_extra=24)
    st.packed()
    st.check("packed with strides")
    st = Step([40, 300], [150, 1], 8, 2, 16, seed=6, pad=3, ld_extra=8)
    st.paged()
    st.check("paged with strides")


def test_long_rows_sampled():
    """Long enough for many key tiles, several work ranges per head and split rows."""
    st = Step([0, 0], [3000, 1100], 32, 8, 64, seed=7, q_gain=2.0)
    st.packed()
    st.check("long prompts", rows=[0, 1, 63, 64, 127, 128, 1000, 1099, 2047, 2999])
    st.check_amax()
    st = Step([5000, 9000, 64], [700, 1, 1], 32, 8, 16, seed=8, q_gain=2.0)
    st.paged()
    st.check("long contexts", rows=[0, 1, 31, 32, 33, 63, 64, 500, 699])
    st.check_amax()


@pytest.mark.parametrize("max_new", [1, 4, 40, 70])
def test_max_new_may_exceed_the_rows_there_are(max_new):
    """max_new only bounds; the launch it chooses does not change the answer."""
    st = Step([70, 600, 129], [1, 1, 1], 8, 2, 16, seed=9, pad=max(0, max_new - 3))
    st.paged(max_new=max_new)
    st.check(f"max_new {max_new}")


# -- values in masked places -------------------------------------------------------------

@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("paged", [False, True])
def test_nonfinite_rows_reach_only_rows_that_attend_to_them(value, paged):
    """A bad token changes its own and later rows of its sequence, nothing
    before it and no neighbour (whose rows share its tiles)."""
    H, Hkv, bad = 8, 2, 75
    ctx, new = ([37, 0, 20], [30, 150, 40]) if paged else ([0, 0, 0], [30, 150, 40])
    st = Step(ctx, new, H, Hkv, 16, seed=11)
    for part in ("v", "k"):
        st2 = Step(ctx, new, H, Hkv, 16, seed=11)
        c0 = (H + (Hkv if part == "v" else 0)) * D
        st2.qkv[st2.cu[1] + bad, c0:c0 + Hkv * D] = value
        run = (lambda s: s.paged(amax=False)) if paged else (lambda s: s.packed(amax=False))
        run(st)
        run(st2)
        torch.cuda.synchronize()
        lo, hi = st.cu[1] + bad, st.cu[2]
        assert torch.equal(st.o[:lo], st2.o[:lo]) and torch.equal(st.o[hi:], st2.o[hi:])
        assert torch.isfinite(st2.o[:lo].float()).all() and torch.isfinite(st2.o[hi:].float()).all()
        if part == "v" or np.isnan(value):
            assert not torch.isfinite(st2.o[lo:hi].float()).any()
        assert mq.mq_check() == 0


@pytest.mark.parametrize("ctx,new,paged", [(0, 150, False), (0, 1, False), (37, 30, True), (900, 1, True), (300, 200, True)])
def test_rows_whose_every_score_is_minus_infinity_are_nan(ctx, new, paged):
    """Their softmax is 0 / 0, as in the formula; the sequence beside them is
    not touched."""
    H, Hkv = 8, 2
    st = Step([ctx, 20 if paged else 0], [new, 40], H, Hkv, 16, seed=31)
    heads = torch.arange(H) * D
    for s in st.seqs[:1]:
        s[:, heads] = 1.0
        s[:, H * D + torch.arange(Hkv) * D] = float("-inf")
    st.qkv[:new, : st.ldqkv] = st.seqs[0][ctx:].cuda()
    st._put(st.k, st.v, 0, 0, ctx)
    (st.paged if paged else st.packed)()
    torch.cuda.synchronize()
    assert torch.isnan(st.o[:new]).all()
    q, k, v = _split(st.seqs[1], H, Hkv)
    c = st.ctx[1]
    ref, a = oracle.attention(q[c:], k, v, H, Hkv, D, pos0=c)
    assert_close(st.o[new:st.n], ref, a, "the other sequence")
    assert mq.mq_check() == 0


@pytest.mark.parametrize("gone,ctx,new", [(200, 700, 1), (200, 300, 60), (129, 0, 300), (640, 3000, 5)])
def test_keys_with_a_score_of_minus_infinity_have_no_weight(gone, ctx, new):
    """The first keys of a sequence are -inf: rows behind them attend to the
    others as if those were not there."""
    H, Hkv = 8, 2
    st = Step([ctx], [new], H, Hkv, 16, seed=32)
    s = st.seqs[0]
    s[:, torch.arange(H) * D] = 1.0
    s[:gone, H * D + torch.arange(Hkv) * D] = float("-inf")
    st.qkv[:new, : st.ldqkv] = s[ctx:].cuda()
    st._put(st.k, st.v, 0, 0, ctx)
    st.paged()
    torch.cuda.synchronize()
    q, k, v = _split(s, H, Hkv)
    first = max(ctx, gone)
    ref, a = oracle.attention(q[first:], k[gone:], v[gone:], H, Hkv, D, pos0=first - gone)
    assert_close(st.o[first - ctx:new], ref, a, "rows behind the keys")
    assert torch.isnan(st.o[: first - ctx]).all()
    assert mq.mq_check() == 0


def test_bad_pages_and_slots_stay_inside_the_cache():
    """Slots outside the cache are skipped; a table entry outside it reads as
    zeros; nothing else of the pool changes and no other sequence's rows do."""
    ctx, new = [40, 40, 40], [3, 3, 3]
    good = Step(ctx, new, 8, 2, 16, seed=12)
    good.paged()
    bad = Step(ctx, new, 8, 2, 16, seed=12)
    bad.table[1][0] = -1
    bad.table[1][1] = bad.n_pages + 5
    bad.slots_d[3], bad.slots_d[4], bad.slots_d[5] = -9, bad.n_pages * 16, 1 << 40
    bad.paged()
    torch.cuda.synchronize()
    assert torch.equal(good.o[:3], bad.o[:3]) and torch.equal(good.o[6:], bad.o[6:])
    for pool, pool0 in ((bad.k, bad.k0), (bad.v, bad.v0)):
        changed = (pool.view(torch.int16) != pool0.view(torch.int16)).any(-1).any(1)       # [page, row]
        rows = {int(p) * 16 + int(r) for p, r in changed.nonzero().tolist()}
        assert rows == set(bad.slots[:3] + bad.slots[6:])
    assert mq.mq_check() == 0


def test_a_table_row_that_is_too_short_drops_the_keys_past_it():
    """Positions from max_pages * page_size on have no page: rows there attend
    to what the table holds."""
    H, Hkv, ps = 4, 2, 16
    st = Step([60], [30], H, Hkv, ps, seed=13)
    st.max_pages = 5                                     # 80 of 90 positions
    st.table = [r[:5] for r in st.table]
    st.slots_d[20:] = -1
    st.paged()
    torch.cuda.synchronize()
    q, k, v = _split(st.seqs[0], H, Hkv)
    ref, a = oracle.attention(q[60:80], k[:80], v[:80], H, Hkv, D, pos0=60)
    assert_close(st.o[:20], ref, a, "rows inside")
    for i in range(80, 90):
        ref, a = oracle.attention(q[i:i + 1], k[:80], v[:80], H, Hkv, D, pos0=79)
        assert_close(st.o[i - 60:i - 59], ref, a, f"row at {i}")
    assert mq.mq_check() == 0


def test_rows_past_max_new_are_left_as_they_were():
    """A sequence with more rows than max_new: the first max_new are computed,
    the cache gets them all."""
    H, Hkv, ps = 8, 2, 16
    st = Step([50, 0, 300], [9, 60, 1], H, Hkv, ps, seed=14)
    st.paged(max_new=5)
    torch.cuda.synchronize()
    amax = 0.0
    for b, s in enumerate(st.seqs):
        q, k, v = _split(s, H, Hkv)
        c, n = st.ctx[b], min(st.new[b], 5)
        ref, a = oracle.attention(q[c:c + n], k[:c + n], v[:c + n], H, Hkv, D, pos0=c)
        got = st.o[st.cu[b]:st.cu[b + 1]]
        assert_close(got[:n], ref, a, f"sequence {b}")
        assert (got[n:] == 3.0).all()
        amax = max(amax, float(got[:n].float().abs().max()))
    assert float(st.amax) == amax
    kr, vr = st.k0.cpu(), st.v0.cpu()
    for b in range(3):
        st._put(kr, vr, b, st.ctx[b], st.ctx[b] + st.new[b])
    assert torch.equal(st.k.cpu().view(torch.int16), kr.view(torch.int16))
    assert torch.equal(st.v.cpu().view(torch.int16), vr.view(torch.int16))
    assert mq.mq_check() == 0


@pytest.mark.parametrize("paged", [False, True])
def test_as_many_requests_as_there_may_be(paged):
    """One token each without context attends to itself alone (weight 1), so o
    is its value, bit for bit, in every head of the group."""
    B, H, Hkv, ps = mq.MQ_PAGED_MAX_REQUESTS, 4, 2, 8
    qkv = _qkv(B, H, Hkv, 41).cuda()
    cols = qkv.shape[1]
    slots = torch.randperm(B, generator=torch.Generator().manual_seed(1)).cuda() * ps
    k = torch.full((B, Hkv, ps, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    o = torch.full((B, H * D), 3.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    if paged:
        table, ctx = (slots // ps).to(torch.int32).view(B, 1).contiguous(), torch.zeros(B, dtype=torch.int32, device="cuda")
        nb = mq.mq_attention_paged_workspace_bytes(B, B, 1, H, Hkv, D)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        mq.mq_attention_paged_bf16(qkv, cols, B, cu, ctx, B, 1, H, Hkv, D, slots, table, 1, k, v, B, ps, o, H * D, None,
                                   ws, nb)
    else:
        nb = mq.mq_attention_packed_workspace_bytes(B, B, H, Hkv, D)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        mq.mq_attention_packed_bf16(qkv, cols, B, cu, B, H, Hkv, D, slots, k, v, B, ps, o, H * D, None, ws, nb)
    torch.cuda.synchronize()
    _, kn, vn = _split(qkv, H, Hkv)
    want = vn.view(B, Hkv, 1, D).expand(B, Hkv, H // Hkv, D).reshape(B, H * D)
    assert torch.equal(o, want)
    pages = slots // ps
    assert torch.equal(k[pages, :, 0].reshape(B, -1), kn) and torch.equal(v[pages, :, 0].reshape(B, -1), vn)
    assert torch.isnan(k[:, :, 1:]).all() and torch.isnan(v[:, :, 1:]).all()
    assert mq.mq_check() == 0


def test_a_cache_whose_offsets_pass_32_bits():
    """Pages beyond 2^32 bytes (and 2^31 elements) into each array."""
    H, Hkv, ps = 8, 2, 64
    n_pages = (1 << 33) // (Hkv * ps * D * 2) + 16                 # 8 GiB and a little
    st = Step([0, 200, 1000], [70, 1, 5], H, Hkv, ps, seed=15)
    high = torch.zeros(n_pages, Hkv, ps, D, dtype=torch.bfloat16, device="cuda")
    highv = torch.zeros_like(high)
    n0 = st.n_pages
    move = lambda p: n_pages - 1 - p if p % 2 else n_pages // 2 + p      # noqa: E731 (half of them past 4 GiB only)
    ids = torch.tensor([move(p) for p in range(n0)], device="cuda")
    high[ids], highv[ids] = st.k, st.v
    small = st.k, st.v
    st.table = [[move(p) if p >= 0 else p for p in r] for r in st.table]
    st.slots_d = ids[(st.slots_d // ps)] * ps + st.slots_d % ps
    st.k, st.v, st.n_pages = high, highv, n_pages
    st.paged()
    torch.cuda.synchronize()
    st.k, st.v = high[ids], highv[ids]
    inv = {move(p): p for p in range(n0)}
    st.table = [[inv.get(p, p) for p in r] for r in st.table]
    st.check("high pages")
    del small


# -- streams, graphs, and the loop -----------------------------------------------------------

def test_another_stream_and_repeated_calls_give_the_same_bits():
    s = torch.cuda.Stream()
    outs = []
    for stream in (None, s, s):
        a = Step([0, 0], [300, 77], 8, 2, 16, seed=21)
        b = Step([700, 90, 2000], [40, 1, 1], 8, 2, 16, seed=22)
        torch.cuda.synchronize()
        a.packed(stream)
        b.paged(stream=stream)
        torch.cuda.synchronize()
        outs.append((a.o, b.o))
    for x, y in outs[1:]:
        assert torch.equal(x, outs[0][0]) and torch.equal(y, outs[0][1])
    assert mq.mq_check() == 0


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own, over and over: the
    same bits as one after the other."""
    mk = lambda: (Step([0] * 5, [900, 77, 300, 1, 500], 16, 4, 16, seed=23),       # noqa: E731
                  Step([3000, 90, 2000, 64], [40, 1, 1, 300], 16, 4, 16, seed=24))
    a0, b0 = mk()
    a0.packed()
    b0.paged()
    a1, b1 = mk()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    # (arguments first, so that the calls follow one another closely)
    a1.packed(sa)
    b1.paged(stream=sb)
    torch.cuda.synchronize()
    B, H, Hkv = 5, 16, 4
    for _ in range(20):
        a1.o.fill_(3.0)
        b1.o.fill_(3.0)
        torch.cuda.synchronize()
        for _ in range(4):
            mq.mq_attention_packed_bf16(a1.qkv, a1.ldqkv, a1.T, a1.cu_d, B, H, Hkv, D, a1.slots_d, a1.k, a1.v, a1.n_pages,
                                        a1.ps, a1.o, a1.o.stride(0), a1.amax, a1.ws, a1.ws.numel(), sa)
            mq.mq_attention_paged_bf16(b1.qkv, b1.ldqkv, b1.T, b1.cu_d, b1.ctx_d, 4, 300, H, Hkv, D, b1.slots_d, b1.table_d,
                                       b1.max_pages, b1.k, b1.v, b1.n_pages, b1.ps, b1.o, b1.o.stride(0), b1.amax, b1.ws,
                                       b1.ws.numel(), sb)
        torch.cuda.synchronize()
        assert torch.equal(a1.o, a0.o) and torch.equal(b1.o, b0.o)
        assert float(a1.amax) == float(a0.amax) and float(b1.amax) == float(b0.amax)
    assert mq.mq_check() == 0


def test_captured_prompts_are_replayed_with_other_lengths():
    """A packed call by itself in a graph, max |o| included: prompts short
    enough to need no work list of their own, then others."""
    H, Hkv, T, B = 8, 2, 200, 3
    lens = [[40, 100, 60], [200, 0, 0], [1, 1, 1], [0, 0, 150], [0, 0, 0]]
    st = Step([0, 0, 0], lens[0], H, Hkv, 0, seed=25)
    nb = mq.mq_attention_packed_workspace_bytes(T, B, H, Hkv, D)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    cu = _i32([0, 0, 0, 0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.mq_attention_packed_bf16(st.qkv, st.ldqkv, T, cu, B, H, Hkv, D, None, None, None, 0, 0, st.o, H * D, st.amax,
                                    ws, nb)
    rows = st.qkv.cpu()
    for ls in lens:
        cu.copy_(_i32([0] + np.cumsum(ls).tolist()))
        st.o.fill_(3.0)
        st.amax.fill_(99.0)
        g.replay()
        torch.cuda.synchronize()
        at = 0
        for n in ls:
            if n:
                ref, a = oracle.attention(*_split(rows[at:at + n], H, Hkv), H, Hkv, D)
                assert_close(st.o[at:at + n], ref, a, f"prompt of {n} in {ls}")
            at += n
        assert (st.o[at:] == 3.0).all()
        assert float(st.amax) == (float(st.o[:at].float().abs().max()) if at else 0.0)
    assert mq.mq_check() == 0


def test_a_captured_step_is_replayed_with_other_lengths():
    """Lengths, tables and slots are device data: one captured plan + append +
    attention decodes token after token of sequences that grow."""
    H, Hkv, ps, B, steps = 8, 2, 16, 3, 40
    ctx0 = [5, 30, 0]
    seqs = [_qkv(c + steps, H, Hkv, 300 + b) for b, c in enumerate(ctx0)]
    cols, max_pages = (H + 2 * Hkv) * D, 8
    n_pages = B * max_pages
    order = list(range(n_pages))
    random.Random(4).shuffle(order)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    k = torch.full((n_pages, Hkv, ps, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    free = _i32(order)
    ctx, new = _i32(ctx0), torch.ones(B, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    info = torch.zeros(4, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(B, cols, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(B, H * D, dtype=torch.bfloat16, device="cuda")
    nb = mq.mq_attention_paged_workspace_bytes(B, B, 1, H, Hkv, D)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    # the prompts: plan, then packed attention writing the pages
    rows = torch.cat([s[:c] for s, c in zip(seqs, ctx0)]).cuda()
    T = rows.shape[0]
    zero, cu0 = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots0 = torch.zeros(T, dtype=torch.int64, device="cuda")
    mq.mq_paged_plan(zero, ctx, B, ps, free, n_pages, table, max_pages, T, cu0, slots0, info)
    o0 = torch.zeros(T, H * D, dtype=torch.bfloat16, device="cuda")
    nb0 = mq.mq_attention_packed_workspace_bytes(T, B, H, Hkv, D)
    ws0 = torch.empty(nb0, dtype=torch.uint8, device="cuda")
    mq.mq_attention_packed_bf16(rows, cols, T, cu0, B, H, Hkv, D, slots0, k, v, n_pages, ps, o0, H * D, None, ws0, nb0)
    torch.cuda.synchronize()
    assert info.tolist() == [35, 3, 0, 30]
    free.copy_(_i32(order[3:] + order[:3]))

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.mq_paged_plan(ctx, new, B, ps, free, n_pages, table, max_pages, B, cu, slots, info)
        mq.mq_attention_paged_bf16(qkv, cols, B, cu, ctx, B, 1, H, Hkv, D, slots, table, max_pages, k, v, n_pages, ps,
                                   o, H * D, None, ws, nb)
    outs = []
    for i in range(steps):
        qkv.copy_(torch.stack([s[c + i] for s, c in zip(seqs, ctx0)]))
        g.replay()
        torch.cuda.synchronize()
        outs.append(o.clone())
        assert info[2] == 0
        taken = int(info[1])
        free.copy_(torch.roll(free, -taken))
        ctx += 1
    got = torch.stack(outs, 1)                                        # [B, steps, H * D]
    for b, (s, c) in enumerate(zip(seqs, ctx0)):
        q, kk, vv = _split(s, H, Hkv)
        ref, a = oracle.attention(q, kk, vv, H, Hkv, D)
        assert_close(got[b], ref[c:], a[c:], f"decoded rows of sequence {b}")
        if c:
            at = sum(ctx0[:b])
            assert_close(o0[at:at + c], ref[:c], a[:c], f"prompt rows of sequence {b}")
    assert mq.mq_check() == 0


def test_chunked_prefill_equals_the_whole_prompt():
    """A prompt taken in chunks over the cache agrees with the one-sequence
    prefill attention, and its o feeds the quantizer by its amax."""
    H, Hkv, ps, S = 16, 4, 64, 900
    x = _qkv(S, H, Hkv, 77, 2.0)
    xd = x.cuda()
    part = torch.zeros(mq.MQ_AMAX_PARTIALS_MAX, dtype=torch.float32, device="cuda")
    whole = torch.empty(S, H * D, dtype=torch.bfloat16, device="cuda")
    mq.mq_attention_prefill_bf16(xd, S, H, Hkv, D, None, None, 0, whole, part)
    max_pages = -(-S // ps)
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    k = torch.full((max_pages, Hkv, ps, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    free = list(range(max_pages))[::-1]
    o = torch.empty_like(whole)
    at = 0
    for n in (300, 1, 450, 149):
        rows = xd[at:at + n].contiguous()
        cu, info = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
        slots = torch.zeros(n, dtype=torch.int64, device="cuda")
        amax = torch.zeros(1, dtype=torch.float32, device="cuda")
        mq.mq_paged_plan(_i32([at]), _i32([n]), 1, ps, _i32(free) if free else None, len(free), table, max_pages, n, cu,
                         slots, info)
        nb = mq.mq_attention_paged_workspace_bytes(n, 1, n, H, Hkv, D)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        mq.mq_attention_paged_bf16(rows, rows.shape[1], n, cu, _i32([at]), 1, n, H, Hkv, D, slots, table, max_pages, k,
                                   v, max_pages, ps, o[at:at + n], H * D, amax, ws, nb)
        torch.cuda.synchronize()
        assert float(amax) == float(o[at:at + n].float().abs().max())
        codes = torch.empty(n, H * D // 2, dtype=torch.uint8, device="cuda")
        sf = torch.empty(mq.mq_sf_bytes(n, H * D), dtype=torch.uint8, device="cuda")
        s_enc = torch.zeros(1, dtype=torch.float32, device="cuda")
        mq.mq_quantize_nvfp4(o[at:at + n], n, H * D, H * D, codes, sf, s_enc, amax, 1)
        torch.cuda.synchronize()
        assert abs(float(s_enc) * float(amax) - 2688.0) <= 2688.0 * 2.0 ** -22
        free = free[int(info[1]):]
        at += n
    q, kk, vv = _split(x, H, Hkv)
    ref, a = oracle.attention(q, kk, vv, H, Hkv, D)
    assert_close(whole, ref, a, "whole prompt")
    assert_close(o, ref, a, "in chunks")
    assert mq.mq_check() == 0
