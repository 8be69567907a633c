"""Queries that hold a NaN or an infinity: what they touch is NaN, nothing else is."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_layer_gb300 import csa2
from tests.dense_case import DenseCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_sparse_attention_layer_gb300 import build
    build.build()
    csa2.load()


@pytest.mark.parametrize("nq,selected", [(1, False), (1, True), (3, False), (3, True)])
def test_weights_of_a_poisoned_query_are_nan(nq, selected):
    """The entries that it sees get NaN, not a large weight; the others keep theirs."""
    case = DenseCase(81, [300, 200], nq=nq)
    d = case.cuda()
    csa2.csa2_dense_attn(d.cache, d.batch, d.q, case.sm_scale, d.o, d.lse, swa=d.swa)
    idx = it = None
    if selected:
        idx = np.full((case.B * nq, 40), -1, np.int32)
        for r in range(idx.shape[0]):
            idx[r, :30] = np.sort(case.rng.choice(150, 30, replace=False))
        it = torch.from_numpy(idx).cuda()
    bad = nq - 1                                   # the last query of sequence 0
    d.q[bad, 5, 77] = float("nan")
    acc = torch.zeros((2, 300), device="cuda")
    csa2.csa2_attn_weights(d.cache, d.batch, d.q, case.sm_scale, d.lse, acc, idx=it, swa=d.swa)
    got = acc.cpu().numpy()
    want, tol = case.weights(d.lse.cpu().numpy(), idx)
    sees = np.zeros((2, 300), bool)
    sees[0, idx[bad][idx[bad] >= 0] if selected else case.entries(0, nq - 1)] = True
    assert np.array_equal(np.isnan(got), sees)
    assert (np.abs(got - want)[~sees] <= tol[~sees]).all() and int(d.status) == 0
