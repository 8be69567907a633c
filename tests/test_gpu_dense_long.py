"""csa2_dense_attn over sequences of up to 1,048,576 entries, so many of them that a run
holds a whole one: what sums, weights and references keep over that length."""
import numpy as np
import pytest
import torch

from tests.dense_long import HEADS, LongCase, bf16_values, codes_of, repeated_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_sparse_attention_layer_gb300 import build, csa2
    build.build()
    csa2.load()


def queries(rng, B, size):
    return bf16_values(rng.standard_normal((B, HEADS, 512)) * size / np.sqrt(512))


@pytest.mark.parametrize("fmt,B,n", [(0, 152, 1 << 20), (1, 152, 1 << 20), (0, 230, 500003), (1, 3, 1 << 20),
                                     (0, 152, 128 * 128), (0, 152, 128 * 128 + 1), (1, 152, 256 * 128 + 70)])
def test_positive_values_of_a_long_sequence(fmt, B, n):
    """Values of one sign under flat attention: the output's sum only grows, and every
    step's truncation has the same sign.  A logit's error is at most 1e-5 of its terms,
    |q| |k| < 0.3 x 6 x 512 / sqrt(512), in sum 4e-4 at most."""
    rng = np.random.default_rng(n + fmt)
    nib = rng.integers(4, 8, (64 * 64, 512))
    scales = np.full((64 * 64, 32 if fmt else 16), 0x38 if fmt else 127, np.uint8)     # 1.0
    case = LongCase(codes_of(nib), scales, repeated_pages(B, (n + 63) // 64, 64), [n - b % 2 for b in range(B)],
                    queries(rng, B, 0.3), fmt)
    d = case.cuda()
    case.check(d, sorted({0, 1 % B, B // 2, B - 1}), 4e-4)
    assert int(d.status) == 0 and bool(torch.isfinite(d.o).all())
