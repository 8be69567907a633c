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


@pytest.mark.parametrize("low,high", [(-70, 60), (-40, 60), (-85, 45), (0, 127), (-90, -89), (-60, 100)])
def test_scales_far_apart(low, high):
    """Entries of scale 2^high among entries of 2^low, a query of zeros: every entry has
    the same weight, whatever its scale.  lse = log n, o = the mean."""
    rng = np.random.default_rng(high - low)
    n = 130
    nib = rng.integers(1, 5, (192, 512)) | rng.integers(0, 2, (192, 512)) << 3
    scales = np.repeat(np.where(np.arange(192) % 2, low, high)[:, None] + 127, 16, 1).astype(np.uint8)
    nib[7] = 0                                     # and one of zeros
    case = LongCase(codes_of(nib), scales, np.arange(3)[None].repeat(2, 0), [n, 1], np.zeros((2, HEADS, 512), np.float32))
    d = case.cuda()
    e = case.keys[:n].mean(0)
    lse = d.lse.cpu().numpy()
    # lse = mu ln 2 + log(sum / 2^mu) with |mu| <= 128: two terms of up to 89 that cancel, ln 2 rounded
    # (2^-24 of 89), the logarithm (2^-23 of it) and the result (2^-24): 4 x 2^-24 x 89 < 2^-15
    assert np.abs(lse[0] - np.log(n)).max() <= 2.0 ** -15 and np.abs(lse[1]).max() <= 2.0 ** -15
    # (equal weights are one power of two in f16)
    o = d.o.float().cpu().numpy().astype(np.float64)
    size = np.abs(case.keys[:n]).mean(0)
    assert (np.abs(o[0] - e) <= 2.0 ** -8 * np.abs(e) + 2.0 ** -14 * size).all()
    # (a single entry is its own output; 2.0 x 2^127 lies beyond fp32 and bf16)
    one = np.where(np.abs(case.keys[0]) < 2.0 ** 128, case.keys[0], np.sign(case.keys[0]) * np.inf)
    finite = np.isfinite(one)
    assert (np.abs(o[1][:, finite] - one[finite]) <= 2.0 ** -8 * np.abs(one[finite])).all()
    assert (o[1][:, ~finite] == one[~finite]).all()


@pytest.mark.parametrize("B,n,nats", [(152, 1 << 17, 17.5), (152, 1 << 20, 17.5), (152, 1 << 20, 16.2), (157, 1 << 18, 19.0),
                                      (152, 1 << 20, 0.3)])
def test_one_entry_above_a_long_rest(B, n, nats):
    """The first entry stands `nats` above all others, which share a mean: together they are up to a tenth
    of the weight, each 2^-23 to 2^-27 of the first's.  A logit is a sum of 64 like terms and smaller ones:
    32 steps lose at most 17 x 2^-23 of 1.2 nats each."""
    rng = np.random.default_rng(int(nats * 10) + n)
    nib = rng.integers(0, 16, (65 * 64, 512))
    nib[:, :64] = 2                                # 1.0 where the query looks
    nib[:, 256:] = rng.integers(4, 8, (65 * 64, 256))
    nib[0, :64] = 7                                # 6.0
    nib[0, 256:] = 11                              # -1.5
    table = repeated_pages(B, n // 64, 64, first=1)
    table[:, 0] = 0
    q = np.zeros((B, HEADS, 512), np.float32)
    q[..., :64] = nats / 5 / 64
    q[..., 64:256] = 0.002 * rng.standard_normal((B, HEADS, 192))
    case = LongCase(codes_of(nib), np.full((65 * 64, 16), 127, np.uint8), table, [n] * B, bf16_values(q))
    d = case.cuda()
    case.check(d, [0, B // 2, B - 1], 32 * 17 * 2.0 ** -23 * 1.2 * nats)


@pytest.mark.parametrize("nq,selected,fmt", [(1, False, 0), (1, False, 1), (2, False, 0), (1, True, 0), (4, True, 1)])
def test_weights_of_a_million_entries(nq, selected, fmt):
    """Three sequences of up to 1,048,576 entries; every entry's weight, or those of 512 a row up to the last."""
    from compressed_sparse_attention_layer_gb300 import csa2
    rng = np.random.default_rng(nq + fmt)
    lens, P = [1 << 20, (1 << 20) - 37, 70], 1 << 14
    nib = rng.integers(0, 16, (48 * 64, 512))
    scales = rng.integers(0x30, 0x3c, (48 * 64, 32)) if fmt else rng.integers(125, 128, (48 * 64, 16))
    case = LongCase(codes_of(nib), scales.astype(np.uint8), repeated_pages(3, P, 48), lens, queries(rng, 3, 1.0), fmt)
    d = case.cuda()
    q = torch.from_numpy(queries(rng, 3 * nq, 1.0)).cuda().to(torch.bfloat16)
    pos = torch.tensor([n - 1 for n in lens for _ in range(nq)], device="cuda")
    batch = csa2.batch_struct(d.n, pos, nq, 1, 1 << 20)
    k = torch.from_numpy(case.keys).cuda()
    l = q.double().view(3, nq * HEADS, 512) @ k.T                              # of the distinct entries
    lse = (torch.logsumexp(l + torch.log(torch.from_numpy(np.stack([case.times(b) for b in range(3)])).cuda())[:, None], 2)
           .view(3 * nq, HEADS).float())
    idx = None
    w = torch.exp(l.view(3, nq, HEADS, -1) - lse.double().view(3, nq, HEADS, 1)).sum(2)        # [3][nq][distinct]
    at = (d.table.long()[:, :, None] * 64 + torch.arange(64, device="cuda")).view(3, -1)       # [3][2^20]
    live = torch.arange(1 << 20, device="cuda") < d.n[:, None]
    if selected:
        idx = torch.full((3 * nq, 512), -1, dtype=torch.int32)
        for r in range(3 * nq):
            n = lens[r // nq]
            e = np.unique(np.concatenate((rng.integers(0, n, 300), [0, n - 1])))
            idx[r, :len(e)] = torch.from_numpy(e)
        idx = idx.cuda()
        want = torch.zeros((3, (1 << 20) + 1), dtype=torch.float64, device="cuda")
        for r in range(3 * nq):
            e = idx[r][idx[r] >= 0].long()
            want[r // nq, e] += w[r // nq, r % nq][at[r // nq, e]]
        want = want[:, :-1]
    else:
        want = torch.where(live, torch.gather(w.sum(1), 1, at), 0.0)
    acc = torch.zeros((3, 1 << 20), device="cuda")
    csa2.csa2_attn_weights(d.cache, batch, q, 1.0, lse, acc, idx=idx)
    # logits of some units: 32 steps of 17 x 2^-23 of up to 4 each, l - lse rounded at 32, the exponential, 64 adds
    tol = want * (32 * 17 * 2.0 ** -23 * 4 + 2.0 ** -18) + nq * 2.0 ** -40
    assert bool(((acc.double() - want).abs() <= tol).all()) and bool((acc[~live] == 0).all())
    assert int(d.status) == 0


@pytest.mark.parametrize("B,fmt", [(152, 0), (100, 1), (190, 0)])
def test_long_rows_repeat_from_any_workspace(B, fmt):
    """Outputs put by on the way through a row, whole or cut: the same bits from a workspace full of NaN, on
    another stream and from a replayed graph."""
    from compressed_sparse_attention_layer_gb300 import csa2
    rng = np.random.default_rng(B)
    nib = rng.integers(0, 16, (64 * 64, 512))
    scales = rng.integers(0x30, 0x3c, (64 * 64, 32)) if fmt else rng.integers(124, 128, (64 * 64, 16))
    lens = [40000 - 61 * (b % 9) for b in range(B)]
    case = LongCase(codes_of(nib), scales.astype(np.uint8), repeated_pages(B, 625, 64), lens, queries(rng, B, 2.0), fmt)
    d = case.cuda()
    # logits of up to some ten units: 32 steps of 17 x 2^-23 of them, in a weight and in the sum
    case.check(d, [0, 1, B // 2, B - 1], 32 * 17 * 2.0 ** -23 * 10)
    first = d.o.clone(), d.lse.clone()
    ws = torch.empty(csa2.csa2_dense_attn_workspace_size(d.batch), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        csa2.csa2_dense_attn(d.cache, d.batch, d.q, 1.0, d.o, d.lse, workspace=ws, stream=stream)

    def same():
        torch.cuda.synchronize()
        assert torch.equal(d.o.view(torch.int16), first[0].view(torch.int16)) and torch.equal(d.lse, first[1])
        d.o.fill_(float("nan"))
        d.lse.fill_(float("nan"))

    for fill in (0xFF, 0x7F, 0):
        ws.fill_(fill)
        call()
        same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for _ in range(3):
        ws.fill_(0xFF)
        g.replay()
        same()
    call(side)
    same()
    assert int(d.status) == 0


@pytest.mark.parametrize("B,n", [(1, 256), (160, 384), (1, 30000), (3, 40001), (152, 20000)])
@pytest.mark.parametrize("low,high,zeros", [(0, 0, True), (-66, 127, False), (0, 127, True), (-40, 100, True), (-90, 64, True)])
def test_scales_far_apart_from_tile_to_tile(B, n, low, high, zeros):
    """A query of zeros over a row whose first half is of one scale (or of zeros) and whose second is of another:
    the reference moves by up to 195 from one tile or one part of the row to the next.  lse = log n all the same."""
    rng = np.random.default_rng(n + high)
    nib = rng.integers(1, 4, (4 * 64, 512))
    scales = np.full((4 * 64, 16), 127 + low, np.uint8)
    scales[128:] = 127 + high
    if zeros:
        nib[:64] = 0
    pages = (n + 63) // 64
    half = pages // 2
    table = np.concatenate((np.arange(half) % (1 if zeros else 2), 2 + np.arange(pages - half) % 2))[None].repeat(B, 0)
    case = LongCase(codes_of(nib), scales, table, [n] * B, np.zeros((B, HEADS, 512), np.float32))
    d = case.cuda()
    # as in test_scales_far_apart, the references of two parts; equal terms add up exactly
    assert np.abs(d.lse.cpu().numpy() - np.log(n)).max() <= 2.0 ** -15
    o, e = d.o[B // 2].float().cpu().numpy().astype(np.float64), case.attention(B // 2)[0]
    assert (np.abs(o - e) <= 2.0 ** -8 * np.abs(e) + 2.0 ** -11 * np.abs(case.keys[128:]).max()).all()
