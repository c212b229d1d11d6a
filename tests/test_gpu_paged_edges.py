"""Edges of the paged serving calls: plans over tables and free lists with
negative pages, and host threads planning at once."""
import random
import threading

import pytest
import torch

from mqtest import ensure_built
from nvfp4_quantized_prefill_b200 import binding as mq
from test_gpu_paged import _i32, _plan, plan_ref

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
