"""The bounds that the whole-cache operators are held to, tried on faults on the host:
a lost page, a coarser query, a sum or an output that is off are outside them."""
import numpy as np
import pytest

from tests.dense_bounds import TightCase, flat_lse

CASES = {"one_sequence": dict(lens=[3000]), "long": dict(lens=[6000], sink=True), "e4m3": dict(lens=[4000], fmt=1),
         "no_window": dict(lens=[2500], window=False, rope_base=10000.0)}


def answer(case, q=None, drop=()):
    """o and lse of query 0 in 64 bits, without the entries `drop`, for another query."""
    keep = case.q
    if q is not None:
        case.q = q
    e = np.setdiff1d(case.entries(0, 0), drop)
    o, lse, _, _ = super(TightCase, case).attention(0, 0, e)
    case.q = keep
    return o, lse


def outside(case, o, lse):
    eo, el, to, tl = case.attention(0, 0)
    return bool((np.abs(lse - el) > tl).any() or (np.abs(o - eo) > to).any())


@pytest.mark.parametrize("name", list(CASES))
def test_faults_are_outside_the_bounds(name):
    case = TightCase(900 + list(CASES).index(name), **CASES[name])
    n = case.lens[0]
    o, lse = answer(case)
    assert not outside(case, o, lse)
    # what the arithmetic does: bf16 outputs
    bits = o.astype(np.float32).view(np.uint32)
    assert not outside(case, ((bits + 0x8000) & 0xFFFF0000).view(np.float32).astype(np.float64), lse)
    rng = np.random.default_rng(1)
    # any page; a single entry shows where all weigh the same (flat_lse) or each has a head of its own
    for p in rng.choice(n // 64, 8, replace=False):
        assert outside(case, *answer(case, drop=np.arange(64 * p, 64 * p + 64)))
    top = np.abs(case.q).max(2, keepdims=True)
    cut = np.trunc(case.q / (top * 2.0 ** -16)) * (top * 2.0 ** -16)
    assert outside(case, *answer(case, q=cut.astype(np.float32)))
    assert outside(case, o, lse + 2.0 ** -9)
    assert outside(case, o * (1 + 2.0 ** -6), lse)


@pytest.mark.parametrize("n", [1, 64, 1000, 70129])
def test_one_key_more_or_less_is_outside_the_flat_bound(n):
    lse, tol = flat_lse(n)
    assert abs(lse - np.log(n)) <= tol and abs(np.log(n + 1) - lse) > 2 * tol and (n == 1 or abs(np.log(n - 1) - lse) > 2 * tol)
