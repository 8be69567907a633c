"""The operators over the whole FP4 cache where the answer is known to the last bits:
every key counted once, each key found by its own address, a query carried in
full; and the random cases within the bounds of the arithmetic itself."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_layer_gb300 import csa2
from tests.dense_bounds import TightCase, flat_lse
from tests.dense_case import bf16
from tests.dense_long import codes_of
from tests.test_gpu_dense import ATTN, WEIGHTS, some_selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_sparse_attention_layer_gb300 import build
    build.build()
    csa2.load()


def attend(d, case):
    csa2.csa2_dense_attn(d.cache, d.batch, d.q, case.sm_scale, d.o, d.lse, swa=d.swa, evicted=d.evicted)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", list(ATTN))
def test_attention_within_the_arithmetics_bounds(name):
    case = TightCase(500 + list(ATTN).index(name), **ATTN[name])
    d = case.cuda()
    attend(d, case)
    rows = case.B * case.nq
    case.check_attention(d.o, d.lse, rows=sorted({0, rows - 1} | set(range(0, rows, max(1, rows // 24)))))
    assert int(d.status) == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_prompts_within_the_arithmetics_bounds(fmt):
    """A prompt after a prefix, each row of another length; m = 1 and 4."""
    for m, lens, nq in ((1, [700, 150], 140), (4, [300], 257)):
        case = TightCase(540 + fmt, lens, nq=nq, m=m, fmt=fmt, rope_base=10000.0, sink=True)
        d = case.cuda()
        attend(d, case)
        case.check_attention(d.o, d.lse, rows=range(0, case.B * nq, 13))
        assert int(d.status) == 0


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("name", list(WEIGHTS))
def test_weights_within_the_arithmetics_bounds(name, selected):
    case = TightCase(560 + list(WEIGHTS).index(name), **WEIGHTS[name])
    if selected and case.evicted is not None:
        case.evicted = None
        case.q_pos = case.q_pos - 90
    d = case.cuda()
    attend(d, case)
    idx = some_selection(case, 200, case.rng) if selected else None
    acc = torch.zeros((case.B, case.E), device="cuda")
    csa2.csa2_attn_weights(d.cache, d.batch, d.q, case.sm_scale, d.lse, acc,
                           idx=None if idx is None else torch.from_numpy(idx).cuda(), swa=d.swa, evicted=d.evicted)
    want, tol = case.weights(d.lse.cpu().numpy(), idx)
    err = np.abs(acc.cpu().numpy() - want) - tol
    assert err.max() <= 0, (float(err.max()), np.unravel_index(err.argmax(), err.shape))
    assert int(d.status) == 0


FLAT = [dict(lens=[1, 2, 63, 64, 65, 127, 128, 129, 191, 1000]), dict(lens=[70001, 16385, 40000, 5], fmt=1),
        dict(lens=[16384, 16383, 30000]), dict(lens=[300, 17], nq=5, m=2, fmt=1), dict(lens=[260], nq=200),
        dict(lens=[9000, 9001, 1], window=False), dict(lens=[33] * 300), dict(lens=[400], nq=3, evicted=[100])]


@pytest.mark.parametrize("at", range(len(FLAT)))
def test_a_query_of_zeros_counts_every_key_once(at):
    case = TightCase(600 + at, **FLAT[at])
    d = case.cuda()
    d.q.zero_()
    attend(d, case)
    lse = d.lse.cpu().numpy()
    for r in range(case.B * case.nq):
        n = len(case.entries(r // case.nq, r % case.nq)) + len(case.window_tokens(r // case.nq, r % case.nq))
        want, tol = flat_lse(n)
        assert np.abs(lse[r] - want).max() <= tol, (r, n, float(np.abs(lse[r] - want).max()))
    acc = torch.zeros((case.B, case.E), device="cuda")
    csa2.csa2_attn_weights(d.cache, d.batch, d.q, 1.0, torch.zeros_like(d.lse), acc, swa=d.swa, evicted=d.evicted)
    want = np.zeros((case.B, case.E))
    for r in range(case.B * case.nq):              # e^0 of 64 heads each
        want[r // case.nq, case.entries(r // case.nq, r % case.nq)] += 64
    assert np.array_equal(acc.cpu().numpy(), want) and int(d.status) == 0


def addressed(seed, n, fmt, heads):
    """A sequence whose entries hold their index, 16 bits as +-1 in four dims each, before random values, and
    `heads` heads asking for one entry each: its logit is 64 x 5, the next 64 x 5 - 40."""
    case = TightCase(seed, [n], fmt=fmt, nq=(heads + 63) // 64, window=False)
    rng = np.random.default_rng(seed)
    bits = np.where(np.arange(n)[:, None] >> np.arange(16) & 1, 1.0, -1.0).repeat(4, 1)
    nib = rng.integers(0, 16, (n, 512))
    nib[:, :64] = np.where(bits > 0, 2, 10)        # 1.0 and -1.0
    at = case.slots(0, np.arange(n))
    case.kv_codes[at] = codes_of(nib)
    # the address's blocks have the scale 1, the others 2^-4 .. 2^2, or an E4M3 number of that size
    case.kv_scales[at] = rng.integers(0x18, 0x48, case.kv_scales[at].shape) if fmt else rng.integers(123, 130, (n, 16))
    case.kv_scales[at[:, None], np.arange(4 if fmt else 2)] = 0x38 if fmt else 127
    k = case.keys(0, np.arange(n))
    assert np.array_equal(k[:, :64], bits)
    asked = rng.integers(0, n, case.nq * 64) if heads > n else np.concatenate((rng.permutation(n), np.arange(n)))[:case.nq * 64]
    q = np.zeros((case.nq * 64, 512), np.float32)
    q[:, :64] = 5 * bits[asked]
    case.q, case.q_bits = bf16(q.reshape(case.nq, 64, 512))
    case.q_pos = np.full((1, case.nq), n - 1)
    return case, k, asked


@pytest.mark.parametrize("n,fmt", [(64, 0), (129, 1), (700, 0), (1000, 1), (5000, 0), (5000, 1)])
def test_each_key_answers_to_its_address(n, fmt):
    """o is the key itself, bit for bit: its weight is 1 within 2^-11 and the rounding to bf16, whose values the
    keys are, undoes that (but for zeros, which the others' e^-40 remain in).  Its accumulated weight is the number of heads that asked for it."""
    case, k, asked = addressed(700 + n + fmt, n, fmt, n)
    d = case.cuda()
    attend(d, case)
    o, lse = d.o.float().cpu().numpy().reshape(-1, 512), d.lse.cpu().numpy().reshape(-1)
    e = k[asked]
    assert np.array_equal(o[e != 0], e[e != 0].astype(np.float32))
    assert np.abs(o[e == 0]).max() <= n * np.exp(-40) * np.abs(k).max()
    assert np.abs(lse - 320).max() <= 2.0 ** -21 * 320
    idx = np.full((case.nq, 512), -1, np.int32)
    for r in range(case.nq):
        e = np.unique(np.concatenate((asked[64 * r:64 * r + 64], case.rng.integers(0, n, 300))))
        idx[r, :len(e)] = e
    times = np.bincount(asked, minlength=n)
    for it in (None, torch.from_numpy(idx).cuda()):
        acc = torch.zeros((1, n), device="cuda")
        csa2.csa2_attn_weights(d.cache, d.batch, d.q, 1.0, d.lse, acc, idx=it)
        # l - lse: lse's error and the rounding of the product, 2^-21 of 320 in all
        assert np.abs(acc.cpu().numpy()[0] - times).max() <= (2.0 ** -21 * 320 + 2.0 ** -20) * max(1, times.max()), it is None
    assert int(d.status) == 0


@pytest.mark.parametrize("down", [8, 15, 17, 20, 24, 26])
def test_a_query_is_carried_far_below_its_largest_element(down):
    """One element of 1 where the keys are 0, the others 2^-down with seven more bits: the logit of a single key
    is theirs alone."""
    case = TightCase(800 + down, [1] * 20, window=False)
    rng = np.random.default_rng(down)
    import oracle
    x = rng.integers(1, 4, (20, 512)).astype(np.float32)
    x[:, :32] = 0
    at = np.array([case.slots(b, [0])[0] for b in range(20)])
    case.kv_codes[at], case.kv_scales[at] = oracle.KV_FORMATS[0][0](x)
    q = ((1 + rng.integers(0, 128, (20, 64, 512)) / 128) * 2.0 ** -down).astype(np.float32)
    q[:, :, :32] = 0
    q[:, :, 7] = 1.0
    case.q, case.q_bits = bf16(q)
    assert np.array_equal(case.q, q)
    d = case.cuda()
    attend(d, case)
    k = np.stack([case.keys(b, [0])[0] for b in range(20)])
    l = np.einsum("bhd,bd->bh", q.astype(np.float64), k)
    # integers of one scale: every sum is exact; the exponent is held next to Xk and the reference (2^-23 of 4)
    assert np.abs(d.lse.cpu().numpy() - l).max() <= 2.0 ** -21 + 2.0 ** -22 * np.abs(l).max()
    assert np.abs(l).min() > 32 * 2.0 ** -21
    acc = torch.zeros((20, 1), device="cuda")
    csa2.csa2_attn_weights(d.cache, d.batch, d.q, 1.0, torch.zeros_like(d.lse), acc)
    want = np.exp(l).sum(1)
    assert (np.abs(acc.cpu().numpy()[:, 0] - want) <= want * (2.0 ** -20 + 2.0 ** -22 * np.abs(l).max())).all()


# ---------------------------------------------------------------- pages that are not there, entries that no row sees
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("nq", [1, 3, 70])
def test_weights_of_pages_outside_the_cache(nq, fmt):
    """The first, one in the middle and the last page of a sequence name nothing: their entries keep their bits,
    the others get their weight, the status says so, the same bits again."""
    lens = [64 * 5, 64 * 3 + 10, 64 * 4 + 1, 70]
    case = TightCase(830 + nq + fmt, lens, nq=nq, fmt=fmt)
    case.table[0, 0] = -1
    case.table[1, 1] = case.num_pages
    case.table[2, 4] = 1 << 30
    case.table[3, :2] = -5
    d = case.cuda()
    attend(d, case)
    assert int(d.status) == csa2.DEV_BAD_PAGE
    case.check_attention(d.o, d.lse, rows=range(0, 4 * nq, max(1, nq // 5)))
    d.status.zero_()
    start = np.random.default_rng(9).random((4, case.E)).astype(np.float32)
    got = []
    for _ in range(3):
        acc = torch.from_numpy(start.copy()).cuda()
        csa2.csa2_attn_weights(d.cache, d.batch, d.q, case.sm_scale, d.lse, acc, swa=d.swa)
        got.append(acc.cpu().numpy())
    assert int(d.status) == csa2.DEV_BAD_PAGE
    assert all(np.array_equal(g, got[0]) for g in got)
    want, tol = case.weights(d.lse.cpu().numpy())
    assert (np.abs(got[0] - start - want) <= tol + 2.0 ** -23 * (start + want)).all()
    gone = np.zeros((4, case.E), bool)
    gone[0, :64] = gone[1, 64:128] = gone[2, 256:] = gone[3] = True
    for b, n in enumerate(lens):
        gone[b, n:] = True
    assert np.array_equal(got[0][gone], start[gone])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("nq", [1, 2, 5])
def test_weights_beside_garbage_that_no_query_sees(nq, fmt):
    """NaN scales and pages outside the cache behind what the queries see."""
    lens = [300, 128, 90]
    pos = [[150 + i for i in range(nq)], [60 + i for i in range(nq)], [-1 - i for i in range(nq)]]
    case = TightCase(860 + nq + fmt, lens, nq=nq, fmt=fmt, q_pos=pos)
    d = case.cuda()
    attend(d, case)
    want, tol = case.weights(d.lse.cpu().numpy())
    for b, t in enumerate(pos):
        e = np.arange(max(t[-1] + 1, 0), lens[b])
        case.kv_scales[case.slots(b, e)] = 0x7F if fmt else 0xFF
        case.kv_codes[case.slots(b, e)] = 0x77
    case.table[0, 3:] = -3
    case.table[2, :] = case.num_pages + 5
    d.kv_codes.copy_(torch.from_numpy(case.kv_codes))
    d.kv_scales.copy_(torch.from_numpy(case.kv_scales))
    d.table.copy_(torch.from_numpy(case.table))
    acc = torch.full((3, 300), 0.25, device="cuda")
    csa2.csa2_attn_weights(d.cache, d.batch, d.q, case.sm_scale, d.lse, acc, swa=d.swa)
    got = acc.cpu().numpy()
    assert (np.abs(got - 0.25 - want) <= tol + 2.0 ** -23 * (0.25 + want)).all()
    assert (got[want == 0] == 0.25).all()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [2, 130, 3000])
def test_heads_that_lean_on_a_key_of_zeros(n, fmt):
    """The first entry is zeros and every other's logit is -14 to -40: what reaches o are the others' small
    weights alone, and they keep their bits."""
    case = TightCase(880 + n + fmt, [n, n], fmt=fmt, window=False, sink=n == 130)
    rng = np.random.default_rng(n)
    for b in range(2):
        at = case.slots(b, np.arange(n))
        nib = rng.integers(0, 16, (n, 512))
        nib[:, :64] = 2                            # 1.0 where the query looks
        nib[0] = 0
        case.kv_codes[at] = codes_of(nib)
        case.kv_scales[at] = 0x38 if fmt else 127
    q = np.zeros((2, 64, 512), np.float32)
    q[:, :, :64] = -np.linspace(14, 40, 64)[:, None] / 64
    q[:, :, 64:] = 0.002 * rng.standard_normal((2, 64, 448))
    case.q, case.q_bits = bf16(q)
    d = case.cuda()
    attend(d, case)
    case.check_attention(d.o, d.lse)
    assert int(d.status) == 0
