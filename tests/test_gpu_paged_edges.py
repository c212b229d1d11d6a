"""Edges of the paged serving calls: plans over tables and free lists with
negative pages, host threads planning at once, steps whose rows are in the
cache already, weights whose running base lags behind, non-finite values in
items that are split, and work cut over more entries than fit shared memory.

Attention tolerance, per output element:
    |gpu - ref| <= (2^-8 + 2^-12) (a + |ref|),  a = sum_j w_j |v_j|
with the weights w of sum 1.  A weight is rounded to BF16 (8 significant bits:
at most half a step, 2^-8 of it) before its product, and the sum that divides is of
the unrounded weights, so o is off by at most 2^-8 a; o is then rounded to BF16
(2^-8 |o|).  In 2^-12: second-order terms (2^-16 a), 2^x (2^-22), and FP32 sums
of n keys, 16 at a time in the products and 64 at a time in the row sums,
at most (n / 16 + n / 64 + 64) 2^-23 < 2^-13 for n < 10000."""
import random
import threading

import numpy as np
import pytest
import torch

import oracle
from mqtest import ensure_built
from nvfp4_quantized_prefill_b200 import binding as mq
from test_gpu_paged import D, Step, _i32, _plan, _split, plan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# -- the page plan ----------------------------------------------------------------------

NEGATIVE = [
    # ctx, new, page size, table, free pages, T
    ([20], [4], 16, [[3, -1, -1]], [], 4),                          # the partly filled page got none in its step
    ([20], [4], 16, [[3, -1, -1]], [8, 9], 4),                      # new tokens before its end need no other
    ([20], [30], 16, [[3, -1, -1, 7]], [8, 9], 30),                 # .. and then do
    ([16, 20, 7], [3, 2, 1], 16, [[-1, 5], [4, -9], [6, 1]], [2], 8),   # a full page without id holds no new token
    ([20, 20], [0, 4], 16, [[3, -1], [4, -1]], [], 4),              # a request without new tokens loses none
    ([20, 20], [-3, 40], 16, [[3, -1], [4, -1]], [], 9),            # cut at T inside the page
    ([0, 5], [50, 40], 16, [[-1] * 4, [7, -1, -1, -1]], [1, -2, 3, -1, -6, 9], 90),    # free ids that are negative
    ([0, 5], [50, 40], 16, [[-1] * 4, [7, -1, -1, -1]], [1, -2, 3, -1, -6, 9], 60),
    ([40, 3], [9, 80], 16, [[1, 2], [3, 4]], [-1, -1, -1, -1, -1, -1], 89),             # rows too short as well
]


@pytest.mark.parametrize("ctx,new,ps,table,free,T", NEGATIVE)
def test_tokens_of_negative_pages_are_counted(ctx, new, ps, table, free, T):
    got = _plan(ctx, new, ps, free, table, len(table[0]), T)
    for g, r in zip(got, plan_ref(ctx, new, ps, free, table, len(table[0]), T)):
        assert g.tolist() == r
    assert int(got[3][2]) == sum(max(n, 0) for n in new) - int((got[1] >= 0).sum())
    assert mq.mq_check() == 0


@pytest.mark.parametrize("B,T_of", [(200, 1.0), (900, 0.7), (4000, 1.0), (5000, 0.9), (16384, 1.0)])
def test_negative_pages_among_many_requests(B, T_of):
    rng = random.Random(B)
    ps, max_pages = 16, 8
    ctx = [rng.randrange(0, 90) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 20, rng.randrange(0, 70)]) for _ in range(B)]
    table = [[rng.randrange(0, 99) if rng.random() < 0.8 else -1 - rng.randrange(3) for _ in range(max_pages)]
             for _ in range(B)]
    free = [rng.randrange(0, 1 << 20) if rng.random() < 0.9 else -rng.randrange(1, 9) for _ in range(sum(new) // ps)]
    T = int(sum(new) * T_of) + 3
    got = _plan(ctx, new, ps, free, table, max_pages, T)
    for g, r in zip(got, plan_ref(ctx, new, ps, free, table, max_pages, T)):
        assert g.tolist() == r
    assert mq.mq_check() == 0


def test_a_step_after_the_free_list_ran_out():
    """The first step leaves a negative page in the table; the next one's
    tokens fall into it and are reported."""
    ps, table = 16, [[3, -1, -1]]
    _, slots, table, info = _plan([16], [4], ps, [], table, 3, 4)
    assert slots.tolist() == [-1] * 4 and info.tolist() == [4, 1, 4, 20]
    _, slots, table, info = _plan([20], [4], ps, [], table.tolist(), 3, 4)
    assert slots.tolist() == [-1] * 4 and info.tolist() == [4, 0, 4, 24]


def test_host_threads_plan_at_once():
    """Calls of two sizes of shared memory from four threads, over and over."""
    def case(B):
        return dict(ctx=_i32([7] * B), new=_i32([1] * B), B=B, ps=8,
                    free=torch.arange(B, dtype=torch.int32, device="cuda"), n_free=B,
                    table=torch.full((B, 2), 5, dtype=torch.int32, device="cuda"), max_pages=2, T=B,
                    cu=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                    slots=torch.zeros(B, dtype=torch.int64, device="cuda"), info=_i32([0] * 4), s=torch.cuda.Stream())
    cases, codes = [case(B) for B in (5000, 16384, 5001, 16383)], {}
    torch.cuda.synchronize()
    go = threading.Barrier(len(cases))
    plan = mq.lib().mq_paged_plan

    def work(i, args):
        go.wait(30)
        codes[i] = {plan(*args) for _ in range(6000)}
    threads = [threading.Thread(target=work, args=(i, [x.data_ptr() if torch.is_tensor(x) else
                                                       x if isinstance(x, int) else x.cuda_stream for x in c.values()]))
               for i, c in enumerate(cases)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == {i: {0} for i in range(len(cases))}, {i: [mq.STATUS[c] for c in v] for i, v in codes.items()}
    for c in cases:
        assert c["info"].tolist() == [c["B"], 0, 0, 8] and (c["slots"] == 47).all()
    assert mq.mq_check() == 0


# -- attention ------------------------------------------------------------------------

def _close(o, ref, a, what):
    og = o.float().double().cpu().numpy().reshape(ref.shape)
    over = np.abs(og - ref) - (2.0 ** -8 + 2.0 ** -12) * (a + np.abs(ref))
    assert (over <= 0).all(), f"{what}: {int((~(over <= 0)).sum())} of {over.size} outside the bound"


@pytest.mark.parametrize("ctx,new,H,Hkv", [
    ([300], [1], 8, 2), ([127, 0, 64], [1, 1, 1], 32, 8), ([200, 5], [8, 3], 8, 2), ([500, 0], [300, 40], 4, 4),
    ([900, 40, 3000], [1, 200, 1], 8, 1)])
def test_rows_that_are_in_the_cache_already(ctx, new, H, Hkv):
    """slots NULL: the same answer as a call that writes them, the cache as it was."""
    mk = lambda: Step(ctx, new, H, Hkv, 16, seed=51, pad=2)      # noqa: E731
    st = mk()
    st.paged()
    st.check("slots given")
    st2 = mk()
    k, v = st2.k.cpu(), st2.v.cpu()
    for b in range(len(ctx)):
        st2._put(k, v, b, ctx[b], ctx[b] + new[b])
    st2.k, st2.v, st2.slots_d = k.cuda(), v.cuda(), None
    # (nothing of the batch but its queries is read)
    st2.qkv[:, H * D:] = float("nan")
    st2.paged()
    torch.cuda.synchronize()
    assert torch.equal(st2.o, st.o) and torch.equal(st2.amax, st.amax)
    for got, want in ((st2.k, k), (st2.v, v)):
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    assert mq.mq_check() == 0


def _lagging(n, H, Hkv, seed):
    """Rows whose scores, in the exponent of 2, are 0 for the first key, up to
    7.9 for key 100 and as far below 0 for all others; values that are the same at every
    position."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(n, (H + 2 * Hkv) * D)
    top = 7.9 * D ** 0.5 / 1.4426950408889634
    x[:, torch.arange(H) * D] = torch.rand(n, H, generator=g) * top
    kcol = H * D + torch.arange(Hkv) * D
    x[:, kcol] = -1.0
    x[0, kcol] = 0.0
    if n > 100:
        x[100, kcol] = 1.0
    x[:, (H + Hkv) * D:] = torch.randn(Hkv * D, generator=g).to(torch.bfloat16).float()
    x[:, (H + Hkv) * D] = 1.0
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("ctx,new,paged", [(0, 500, False), (0, 150, True), (300, 200, True), (800, 1, True),
                                           (9000, 8, True), (5000, 70, True)])
def test_a_value_that_every_key_has_comes_out(ctx, new, paged):
    """The weights lie anywhere below 2^8, the largest of a row dominates it and
    its rounding is not made up for by others: the bound with a = |ref| = |v|."""
    H, Hkv = 8, 2
    st = Step([ctx], [new], H, Hkv, 16, seed=52)
    s = st.seqs[0] = _lagging(ctx + new, H, Hkv, 53)
    st.qkv[:new] = s[ctx:].cuda()
    k, v = st.k.cpu(), st.v.cpu()
    st._put(k, v, 0, 0, ctx)
    st.k, st.v = k.cuda(), v.cuda()
    (st.paged if paged else st.packed)()
    torch.cuda.synchronize()
    _, _, v = _split(s, H, Hkv)
    want = v[ctx:].view(new, Hkv, 1, D).expand(new, Hkv, H // Hkv, D).reshape(new, H * D).double().numpy()
    _close(st.o[:new], want, np.abs(want), "one value")
    assert mq.mq_check() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("ctx,new,bad", [(3000, 8, 3), (3000, 60, 40), (700, 8, 7), (9000, 33, 0), (200, 31, 10),
                                         (20000, 4, 2)])
def test_nonfinite_rows_of_items_that_are_split(ctx, new, bad, value):
    """A bad new token over a context of many tiles: an item whose two slots
    take turns at the tiles, and items cut between CTAs."""
    H, Hkv = 8, 2
    lens = dict(ctx=[40, ctx, 2500], new=[3, new, 1])
    st = Step(lens["ctx"], lens["new"], H, Hkv, 16, seed=54)
    st.paged(amax=False)
    for part in ("v", "k"):
        st2 = Step(lens["ctx"], lens["new"], H, Hkv, 16, seed=54)
        c0 = (H + (Hkv if part == "v" else 0)) * D
        st2.qkv[st2.cu[1] + bad, c0:c0 + Hkv * D] = value
        st2.paged(amax=False)
        torch.cuda.synchronize()
        lo, hi = st.cu[1] + bad, st.cu[2]
        assert torch.equal(st.o[:lo], st2.o[:lo]) and torch.equal(st.o[hi:], st2.o[hi:])
        assert torch.isfinite(st2.o[:lo].float()).all() and torch.isfinite(st2.o[hi:].float()).all()
        rows = st2.o[lo:hi].float()
        if part == "v":
            assert torch.equal(rows, torch.full_like(rows, value)) or (np.isnan(value) and torch.isnan(rows).all())
        elif np.isnan(value):
            assert torch.isnan(rows).all()
        assert mq.mq_check() == 0


def test_long_sequences_among_more_entries_than_shared_memory_holds():
    """Over 1024 entries, and borders of the CTAs' ranges inside the long ones."""
    rng = random.Random(6)
    H, Hkv, B = 8, 2, 1300
    ctx = [rng.randrange(0, 30) for _ in range(B)]
    new = [1] * B
    for b, c, n in ((0, 4000, 1), (511, 9000, 40), (512, 2500, 1), (1299, 6000, 3)):
        ctx[b], new[b] = c, n
    st = Step(ctx, new, H, Hkv, 16, seed=55)
    st.paged(amax=False)
    torch.cuda.synchronize()
    for b in [0, 1, 2, 510, 511, 512, 513, 1298, 1299] + rng.sample(range(B), 60):
        q, k, v = _split(st.seqs[b], H, Hkv)
        ref, a = oracle.attention(q[ctx[b]:], k, v, H, Hkv, D, pos0=ctx[b])
        _close(st.o[st.cu[b]:st.cu[b + 1]], ref, a, f"sequence {b}")
    assert mq.mq_check() == 0
