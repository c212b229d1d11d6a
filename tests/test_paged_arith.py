"""CPU check of the exponential that the paged attention evaluates on the FMA
pipes (no GPU): its steps in binary32, with the constants of the source, against
2^x in 64 bits."""
import os
import re

import numpy as np

from nvfp4_quantized_prefill_b200 import build

F = np.float32


def _source():
    text = open(os.path.join(build.CSRC, "mq_attention_paged.cu")).read()
    at = text.index("void exp2_pair_fma(")
    return text[at:text.index("\n}\n", at)]


def _fma(a, b, c):
    # the product of two binary32 is exact in binary64
    return (a.astype(np.float64) * b.astype(np.float64) + c.astype(np.float64)).astype(F)


def _exp2(x):
    """The function's steps; every constant is read from the source."""
    body = _source()
    num = r"(-?\d+\.\d+(?:e-?\d+)?)f"
    low = re.search(r"fmaxf\(x0, " + num + r"\)", body)
    shift = re.search(r"fadd2\(x, pack2\(" + num, body)
    first = re.search(r"ffma2\(f, twice\(" + num + r"\), twice\(" + num + r"\)\)", body)
    coeff = [F(c) for c in first.groups() + tuple(re.findall(r"ffma2\(p, f, twice\(" + num + r"\)\)", body))]
    assert len(coeff) == 6 and coeff[-1] == 1
    x = np.maximum(x.astype(F), F(low.group(1)))
    magic = F(shift.group(1))
    t = (x + magic).astype(F)
    n = (t - magic).astype(F)
    f = _fma(n, np.full_like(n, -1), x)
    p = _fma(f, np.full_like(f, coeff[0]), np.full_like(f, coeff[1]))
    for c in coeff[2:]:
        p = _fma(p, f, np.full_like(f, c))
    bits = (t.view(np.uint32) << np.uint32(23)) + p.view(np.uint32)
    return bits.view(F)


def test_exp2_on_the_fma_pipes_is_as_exact_as_the_transcendental_unit():
    """Least error 9.1e-8 of the quintic, a rounding of 2^-24 in its last step
    (relative to p >= 0.7: 8.5e-8) and those before it scaled by |f| <= 1/2 (half
    a step of 0.7, 3e-8, times 1/2, and less): below 2^-22 = 2.4e-7 together."""
    rng = np.random.default_rng(1)
    x = np.concatenate([np.linspace(-126, 8, 2_000_001), rng.uniform(-2, 2, 1_000_000), np.arange(-126, 128),
                        np.arange(-125, 127) + 0.5, np.nextafter(np.arange(-125, 127) + F(0.5), F(200)),
                        rng.uniform(8, 127.4, 200_000)]).astype(F)
    want = np.exp2(x.astype(np.float64))
    got = _exp2(x).astype(np.float64)
    assert (np.abs(got - want) <= 2.0 ** -22 * want).all()
    whole = np.arange(-126, 128)
    assert (_exp2(whole) == np.ldexp(np.ones(whole.size), whole)).all()      # (numpy's binary32 exp2 is not exact there)


def test_exp2_of_masked_scores_is_zero():
    gone = np.array([-np.inf, -3e38, -1e6, -200, -128, -127.5, -127], dtype=F)
    assert (_exp2(gone) == 0).all()
    tail = np.linspace(-127, -126, 100_001).astype(F)
    assert (np.abs(_exp2(tail)) <= 2.0 ** -126).all()
