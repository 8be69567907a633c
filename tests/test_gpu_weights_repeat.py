"""csa2_attn_weights over many runs of a few tiles, again and again: the same
bits, and those of the definition."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_layer_gb300 import csa2
from tests.dense_case import DenseCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,k", [(0, None), (1, None), (0, 200), (1, 200)])
def test_weights_of_short_runs_repeat(fmt, k):
    case = DenseCase(71 + fmt, [130 + 40 * (i % 7) for i in range(260)], fmt=fmt)
    d = case.cuda()
    rng = np.random.default_rng(3)
    idx = it = None
    if k:
        idx = np.full((case.B, k), -1, np.int32)
        for b, n in enumerate(case.lens):
            e = np.sort(rng.choice(n, min(n, k), replace=False))
            idx[b, :e.size] = e
        it = torch.from_numpy(idx).cuda()
    csa2.csa2_dense_attn(d.cache, d.batch, d.q, case.sm_scale, d.o, d.lse, swa=d.swa)
    first = None
    for _ in range(60):
        acc = torch.zeros((case.B, case.E), device="cuda")
        csa2.csa2_attn_weights(d.cache, d.batch, d.q, case.sm_scale, d.lse, acc, idx=it, swa=d.swa)
        first = acc if first is None else first
        assert torch.equal(acc, first)
    want, tol = case.weights(d.lse.cpu().numpy(), idx)
    assert (np.abs(first.cpu().numpy() - want) <= tol).all() and int(d.status) == 0
