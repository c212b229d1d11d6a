"""Host-side checks of the paged serving calls: every refusal comes before any
device work, and the workspace queries answer 0 for what the calls refuse.
No kernel runs here."""
import pytest

from nvfp4_quantized_prefill_b200 import binding, build

BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


PLAN = dict(ctx=16, new=16, B=4, ps=16, free=16, n_free=8, table=16, max_pages=8, T=64, cu=16, slots=16, info=16,
            stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(ctx=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(slots=None), 1),
    (dict(info=None), 1), (dict(free=None), 1), (dict(n_free=-1), 1),
    (dict(B=0), 2), (dict(B=16385), 2), (dict(T=0), 2), (dict(T=(1 << 22) + 1), 2), (dict(ps=0), 2), (dict(ps=4), 2),
    (dict(ps=24), 2), (dict(ps=512), 2), (dict(max_pages=0), 2), (dict(max_pages=(1 << 24) + 1), 2),
    (dict(n_free=1 << 31), 2),
    (dict(ctx=18), 3), (dict(new=17), 3), (dict(free=18), 3), (dict(table=18), 3), (dict(cu=18), 3),
    (dict(slots=20), 3), (dict(info=18), 3)])
def test_plan_refusals(lib, change, code):
    assert lib.mq_paged_plan(*{**PLAN, **change}.values()) == code


PACKED = dict(qkv=16, ldqkv=1024, T=64, cu=16, B=4, H=4, Hkv=2, D=128, slots=16, k=16, v=16, n_pages=8, ps=16, o=16,
              ldo=512, amax=16, ws=16, nb=BIG, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(qkv=None), 1), (dict(cu=None), 1), (dict(o=None), 1), (dict(ws=None), 1),
    (dict(slots=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None, k=None), 1), (dict(nb=0), 1),
    (dict(T=0), 2), (dict(T=(1 << 22) + 1), 2), (dict(B=0), 2), (dict(B=16385), 2), (dict(D=64), 2), (dict(Hkv=3), 2),
    (dict(H=0), 2), (dict(H=1028, ldqkv=1 << 20, ldo=1 << 20), 2), (dict(Hkv=0), 2),
    (dict(H=258, Hkv=2, ldqkv=1 << 20, ldo=1 << 20), 2),
    (dict(ldqkv=1016), 2), (dict(ldo=504), 2), (dict(ps=48), 2), (dict(ps=4), 2), (dict(n_pages=0), 2),
    (dict(n_pages=1 << 31), 2),
    (dict(ldqkv=1028), 3), (dict(ldo=516), 3), (dict(qkv=24), 3), (dict(o=24), 3), (dict(ws=24), 3), (dict(k=24), 3),
    (dict(v=24), 3), (dict(cu=18), 3), (dict(slots=20), 3), (dict(amax=18), 3)])
def test_packed_attention_refusals(lib, change, code):
    assert lib.mq_attention_packed_bf16(*{**PACKED, **change}.values()) == code


PAGED = dict(qkv=16, ldqkv=1024, T=64, cu=16, ctx=16, B=4, max_new=16, H=4, Hkv=2, D=128, slots=16, table=16,
             max_pages=8, k=16, v=16, n_pages=8, ps=16, o=16, ldo=512, amax=16, ws=16, nb=BIG, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(qkv=None), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(table=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(nb=0), 1),
    (dict(T=0), 2), (dict(B=0), 2), (dict(B=16385), 2), (dict(max_new=0), 2), (dict(max_new=65), 2), (dict(D=64), 2),
    (dict(Hkv=3), 2), (dict(H=258, Hkv=2, ldqkv=1 << 20, ldo=1 << 20), 2), (dict(ldqkv=1016), 2), (dict(ldo=504), 2),
    (dict(ps=12), 2), (dict(ps=512), 2), (dict(n_pages=0), 2), (dict(max_pages=0), 2),
    (dict(max_pages=(1 << 24) + 1), 2),
    (dict(ldqkv=1028), 3), (dict(ldo=516), 3), (dict(qkv=24), 3), (dict(k=24), 3), (dict(ctx=18), 3),
    (dict(table=18), 3), (dict(slots=20), 3), (dict(ws=24), 3)])
def test_paged_attention_refusals(lib, change, code):
    assert lib.mq_attention_paged_bf16(*{**PAGED, **change}.values()) == code


def test_workspace_queries(lib):
    packed, paged = binding.mq_attention_packed_workspace_bytes, binding.mq_attention_paged_workspace_bytes
    assert packed(1, 1, 1, 1, 128) > 0 and paged(1, 1, 1, 1, 1, 128) > 0
    for bad in [(0, 1, 4, 2, 128), (8, 0, 4, 2, 128), (8, 1, 4, 3, 128), (8, 1, 4, 2, 64), (8, 1, 258, 2, 128)]:
        assert packed(*bad) == 0
        assert paged(bad[0], bad[1], 1, *bad[2:]) == 0
    assert paged(8, 1, 0, 4, 2, 128) == 0 and paged(8, 1, 9, 4, 2, 128) == 0
