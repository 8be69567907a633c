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


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,nq", [([300], 1), ([9000, 130], 1), ([700], 3)])
def test_a_poisoned_head_is_nan_and_the_others_are_right(lens, nq, bad):
    """Whole rows, rows cut into parts, several queries.  Logits that fall by hundreds from the first entries
    on, so that a reference that followed them down would leave the range."""
    case = DenseCase(83, lens, nq=nq, q_scale=40.0, window=len(lens) == 2)
    d = case.cuda()
    heads = [0, 9, 33]
    d.q[0, heads, 200] = bad
    csa2.csa2_dense_attn(d.cache, d.batch, d.q, case.sm_scale, d.o, d.lse, swa=d.swa)
    o, lse = d.o.float().cpu().numpy(), d.lse.cpu().numpy()
    assert np.isnan(lse[0, heads]).all() and np.isnan(o[0, heads]).all()
    rest = [h for h in range(64) if h not in heads]
    eo, el, to, tl = case.attention(0, 0)
    assert (np.abs(lse[0, rest] - el[rest]) <= tl[rest]).all() and (np.abs(o[0, rest] - eo[rest]) <= to[rest]).all()
    case.check_attention(d.o, d.lse, rows=range(1, case.B * nq))


def test_falling_logits_beside_a_poisoned_head():
    """Head 0 of a query is NaN; head 1's logits fall from 0 to -400 over the sequence."""
    import oracle
    case = DenseCase(84, [128 * 6], window=False)
    x = np.zeros((768, 512))
    x[:, :256] = -np.repeat(np.arange(6) / 4.0, 128)[:, None]                  # 0, -0.25, ... as FP4 holds them
    x[:, 256:] = case.rng.integers(1, 4, (768, 256))
    codes, scales = oracle.KV_FORMATS[0][0](x.astype(np.float32))
    at = case.slots(0, np.arange(768))
    case.kv_codes[at], case.kv_scales[at] = codes, scales
    q = np.zeros((200, 64, 512), np.float32)
    q[:, :, :256] = 320 / 256
    case.q, case.nq, case.B = q, 200, 1
    case.q_pos = np.full((1, 200), 767)
    case.q_bits = (q.view(np.uint32) >> 16).astype(np.uint16)
    d = case.cuda()
    d.q[:, 0, 3] = float("nan")
    csa2.csa2_dense_attn(d.cache, d.batch, d.q, 1.0, d.o, d.lse)
    o, lse = d.o.float().cpu().numpy(), d.lse.cpu().numpy()
    eo, el, to, tl = case.attention(0, 0)
    assert np.isnan(lse[:, 0]).all() and np.isnan(o[:, 0]).all()
    assert (np.abs(lse[:, 1:] - el[1:]) <= tl[1:]).all() and (np.abs(o[:, 1:] - eo[1:]) <= to[1:]).all()


def test_eviction_by_weights_that_are_not_numbers():
    """A NaN is above +inf, one with its sign set below -inf; ties go to the lower index."""
    case = DenseCase(85, [400], window=False)
    d = case.cuda()
    acc = case.rng.standard_normal((1, 400)).astype(np.float32)
    acc[0, [10, 399, 77]] = np.nan
    acc[0, [11, 200]] = np.inf
    acc[0, [12, 300]] = -np.inf
    bits = acc.view(np.uint32)
    bits[0, [13, 14]] = 0xFFC00000
    key = np.where(bits[0] >> 31, ~bits[0], bits[0] | 0x80000000)
    for keep in (1, 3, 4, 5, 100, 395, 396, 397, 398, 399):
        kept = torch.empty((1, keep), dtype=torch.int32, device="cuda")
        n_out = torch.empty(1, dtype=torch.int64, device="cuda")
        dst = [torch.zeros((448, 256), dtype=torch.uint8, device="cuda"), torch.zeros((448, 16), dtype=torch.uint8, device="cuda")]
        table = torch.arange(7, dtype=torch.int32, device="cuda")[None].contiguous()
        csa2.csa2_evict(d.cache, csa2.cache_struct(dst[0], dst[1], table), d.n, torch.from_numpy(acc).cuda(), 400, keep, kept, n_out)
        order = sorted(range(400), key=lambda e: (-int(key[e]), e))[:keep]
        assert kept.cpu().numpy()[0].tolist() == sorted(order) and int(n_out) == keep
