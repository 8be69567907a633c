"""Long sequences for the operators over the whole FP4 cache: the block tables name
the same few pages over and over, so that a million entries have an expectation in 64
bits at the cost of a few thousand.  Nothing here reads an output of the CUDA path."""
from __future__ import annotations

import numpy as np

import oracle

PAGE, HEADS, DIM = 64, 64, 512


class LongCase:
    """codes, scales: the distinct entries (a multiple of 64 of them); table: page ids [B][P]; n: entries of
    each sequence; q fp32 holding bf16 values [B][64][512], one query a sequence that sees all of it.  No
    window, sink or rotation."""

    def __init__(self, codes, scales, table, n, q, fmt=0):
        self.codes, self.scales, self.fmt = np.ascontiguousarray(codes), np.ascontiguousarray(scales), fmt
        self.table, self.n, self.q = np.ascontiguousarray(table, np.int32), list(n), q
        self.keys = oracle.KV_FORMATS[fmt][1](self.codes, self.scales).astype(np.float64).reshape(-1, DIM)
        s = self.scales.astype(np.int64)
        some = (self.codes.reshape(len(s), 16, 16) & 0x77).any(2)
        self.unit = np.full(len(s), 2.0 ** 12) if fmt else \
            np.exp2(np.where(some, s - 127, -127).max(1).clip(-90).astype(np.float64))

    def times(self, b):
        """How often sequence b holds each distinct entry."""
        n, out = self.n[b], np.zeros(len(self.keys))
        full = n // PAGE
        pages = np.bincount(self.table[b, :full], minlength=len(self.keys) // PAGE)
        out += np.repeat(pages, PAGE)
        if n % PAGE:
            at = int(self.table[b, full]) * PAGE
            out[at:at + n % PAGE] += 1
        return out

    def attention(self, b):
        """o, lse, sum p |k|, the weights p (of all copies of an entry)."""
        k, w = self.keys, self.times(b)
        l = self.q[b].astype(np.float64) @ k.T
        top = np.where(w > 0, l, -np.inf).max(1, keepdims=True)
        p = np.exp(np.minimum(l - top, 0)) * w
        tot = p.sum(1, keepdims=True)
        p /= tot
        return p @ k, np.log(tot[:, 0]) + top[:, 0], p @ np.abs(k), p

    def bounds(self, b, dl):
        """Of o and lse, dl bounding a logit's error: o is rounded to bf16 (2^-8), a weight to f16 (2^-11)
        with a floor of half of f16's smallest step, 2^-25, where the largest is 2^-1 or more for the first
        16,384 entries of each of a row's segments (152 runs cut the rows), 2^7 or more behind them (2^-24 and 2^-32
        of the largest p w, w = 2^Xk; key j takes k_j / w_j times it); 1,024 steps of the accumulator, each with 17
        addends that lose at most 2^-23 of the sum so far, half of the whole on average; twice the logits'
        error and 2^-20 for the exponentials and their sum."""
        o, lse, size, p = self.attention(b)
        t = self.times(b)
        one = np.where(t > 0, p / np.maximum(t, 1), 0.0)                       # a single entry's weight
        small = (2.0 ** -24 * min(self.n[b], (152 // len(self.n) + 3) * 16384) + 2.0 ** -32 * self.n[b]) / self.n[b]
        floor = small * (one * self.unit).max(1)[:, None] * (t[:, None] * np.abs(self.keys) / self.unit[:, None]).sum(0)[None]
        tol_o = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 1024 * 17 * 2.0 ** -24 + 2 * dl + 2.0 ** -20) * size + floor
        return o, lse, tol_o, dl + 2.0 ** -16 + 2.0 ** -20 * np.abs(lse)

    def cuda(self):
        import torch

        from compressed_sparse_attention_layer_gb300 import csa2

        class D:
            pass

        d = D()
        d.codes, d.scales, d.table = (torch.from_numpy(x).cuda() for x in (self.codes, self.scales, self.table))
        d.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        d.n = torch.tensor(self.n, dtype=torch.int64, device="cuda")
        d.pos = d.n - 1
        d.cache = csa2.cache_struct(d.codes, d.scales, d.table, kv_format=self.fmt, status=d.status)
        d.batch = csa2.batch_struct(d.n, d.pos, 1, 1, max(self.n))
        d.q = torch.from_numpy(self.q).cuda().to(torch.bfloat16)
        d.o = torch.full((len(self.n), HEADS, DIM), float("nan"), dtype=torch.bfloat16, device="cuda")
        d.lse = torch.full((len(self.n), HEADS), float("nan"), device="cuda")
        csa2.csa2_dense_attn(d.cache, d.batch, d.q, 1.0, d.o, d.lse)
        torch.cuda.synchronize()
        return d

    def check(self, d, rows, dl):
        for b in rows:
            o, lse, tol_o, tol_l = self.bounds(b, dl)
            x = np.abs(d.o[b].float().cpu().numpy() - o) - tol_o
            assert x.max() <= 0, (b, "o", float(x.max()), np.unravel_index(x.argmax(), x.shape))
            y = np.abs(d.lse[b].cpu().numpy() - lse) - tol_l
            assert y.max() <= 0, (b, "lse", float(y.max()))


def bf16_values(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def codes_of(nibbles):
    """E2M1 codes [N][512] -> bytes [N][256], low nibble first."""
    x = np.asarray(nibbles, np.uint8)
    return x[:, 0::2] | x[:, 1::2] << 4


def repeated_pages(B, pages, distinct, first=0):
    """A table of `pages` ids per sequence, first .. first + distinct - 1 over and over, another start each."""
    return first + (np.arange(pages)[None] + 7 * np.arange(B)[:, None]) % distinct
