"""Bounds of the operators over the whole FP4 cache from what their arithmetic is:
exact f16 operands, products summed in fp32 by the tensor cores, f16 weights, fp32 sums.
TightCase is DenseCase with these for its own."""
from __future__ import annotations

import numpy as np

import oracle
from tests.dense_case import DenseCase

# One instruction adds 16 products to the accumulator: 17 addends, each cut off below 2^-23 of the largest
# number among them and their sums.
STEP = 17 * 2.0 ** -23


class TightCase(DenseCase):
    def logit_errors(self, q, k, l):
        """Bound of each logit's error [64][keys]: the steps' (the partial sums of 16 dims each), a query
        carried to 2^-38 of its head's largest element, and three roundings of the factors and the product."""
        s = np.abs(self.sm_scale)
        out = 2.0 ** -22 * np.abs(l) + 2.0 ** -38 * s * np.abs(q).max(1)[:, None] * np.abs(k).sum(1)[None]
        acc = np.zeros_like(l)
        for d in range(0, 512, 16):
            new = acc + self.sm_scale * (q[:, d:d + 16] @ k[:, d:d + 16].T)
            top = np.maximum(np.abs(acc), np.abs(new))
            for j in range(d, d + 16):
                np.maximum(top, np.outer(s * np.abs(q[:, j]), np.abs(k[:, j])), out=top)
            out += STEP * top
            acc = new
        return out

    def key_list(self, b, i, entries=None):
        """The keys of a query and 2^Xk of each."""
        e = self.entries(b, i) if entries is None else np.asarray(entries)
        k = self.keys(b, e) if len(e) else np.zeros((0, 512))
        w = np.exp2(12.0 * np.ones(len(e))) if self.fmt else np.maximum(self.weight_unit(b, e), 2.0 ** -66)
        win = self.window_tokens(b, i)
        if len(win):
            rows = np.array(win) % self.ring.shape[1]
            sc = np.abs(self.ring_scales[b, rows].astype(np.float64))
            w = np.concatenate((w, np.exp2(np.maximum(np.floor(np.log2(sc)) + 1, -78) + 12)))
            kw = oracle.dequant_fp8(self.ring[b, rows], self.ring_scales[b, rows]).astype(np.float64).reshape(-1, 512)
            k = np.concatenate((k, kw))
        return k, w

    def attention(self, b, i, entries=None):
        o, lse, _, _ = super().attention(b, i, entries)
        k, w = self.key_list(b, i, entries)
        if not k.shape[0]:
            return o, lse, np.zeros((64, 512)), 2.0 ** -21 * (1 + np.abs(np.where(np.isinf(lse), 0, lse)))
        q = self.q[b * self.nq + i].astype(np.float64)
        l = self.sm_scale * (q @ k.T)
        p = np.exp(l - np.where(np.isinf(lse), np.inf, lse)[:, None])
        # a weight's exponent is held relative to the reference, next to Xk: rounded at the size of both
        # (twice); the exponential to two units
        dl = self.logit_errors(q, k, l) + 2.0 ** -23 * (np.abs(l - l.max(1, keepdims=True)) + np.abs(np.log2(w)) + 16) + 2.0 ** -22
        # a thread adds up a 32nd of the keys; then 160 parts; the logarithm
        n = k.shape[0]
        share = (p * np.expm1(dl)).sum(1)
        tol_lse = share + (n / 32 + 200) * 2.0 ** -24 + 2.0 ** -22 * (2 + np.abs(np.where(np.isinf(lse), 0, lse)))
        size = p @ np.abs(k)
        tiles = n // 128 + 2
        some = (k != 0).any(1)
        # a weight is rounded at 2^-25 where the largest 2^(y - mu) is 2^-1 or more.  Key j's place in the product
        # is |k_j| / w_j; a window row's |k_j| / (w_j f_j), its scale's mantissa f_j in [1/2, 1) being in the weight
        inv = 1.0 / w
        inv[len(w) - len(self.window_tokens(b, i)):] *= 2
        floor = 2.0 ** -24 * (p * (w * some)[None]).max(1)[:, None] * (np.abs(k) * inv[:, None]).sum(0)[None]
        exact = np.abs(p @ k)
        inner = (p * (2.0 ** -11 + np.expm1(dl))) @ np.abs(k) + floor + \
            (tol_lse[:, None] + min(8 * tiles, 1024) * STEP / 2 + 2.0 ** -18) * size
        if self.rope_base > 0:
            # each of the pair's two rounds once to bf16, and takes from both
            inner[:, 448:480] = inner[:, 480:] = inner[:, 448:480] + inner[:, 480:] + \
                2.0 ** -20 * (exact[:, 448:480] + exact[:, 480:])
        return o, lse, 2.0 ** -8 * np.abs(o) + inner + 1e-30, tol_lse

    def weights(self, lse, idx=None):
        out, _ = super().weights(lse, idx)
        tol = np.zeros_like(out)
        for b in range(self.B):
            for i in range(self.nq):
                r = b * self.nq + i
                if idx is None:
                    e = self.entries(b, i)
                else:
                    e = np.asarray(idx[r], np.int64)
                    e = e[(e >= 0) & (e < self.visible(b, i))]
                    win = self.window_tokens(b, i)
                    if self.dedup and self.m == 1 and len(win):
                        e = e[e < win.start]
                    e = e[self.has_page(b, e)] if e.size else e
                if not len(e):
                    continue
                k, q = self.keys(b, e), self.q[r].astype(np.float64)
                l = self.sm_scale * (q @ k.T)
                z = lse[r].astype(np.float64)[:, None]
                w = np.where(np.isinf(z), 0.0, np.exp(l - z))
                # the logit's, l - lse and its product with log2 e rounded, the exponential; 64 heads added
                with np.errstate(invalid="ignore"):
                    rel = self.logit_errors(q, k, l) + 2.0 ** -23 * (np.abs(l) + np.abs(z) + 2)
                np.add.at(tol[b], e, np.where(w > 0, w * np.expm1(rel), 0).sum(0) + 2.0 ** -19 * w.sum(0) + 2.0 ** -40)
        # the rows' sums one after the other
        return out, tol + (self.nq + 2) * 2.0 ** -24 * out


def flat_lse(n):
    """lse of n keys under a query of zeros, and its bound: every term is the same power of two, the sum exact,
    one rounding each in the logarithm, its product and their sum."""
    return float(np.log(n)), 2.0 ** -22 * (1 + float(np.log(n)))
