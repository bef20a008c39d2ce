"""Random 4-bit caches for the tests: bytes that no token owns hold NaN scales
(0x7F) and the largest codes, so that a read outside the sequences shows."""
from __future__ import annotations

import numpy as np
import torch

from oracle import e2m1

P = 16


class Pool4:
    def __init__(self, blocks, heads, dim, seed):
        self.rng = np.random.default_rng(seed)
        self.blocks, self.H, self.D = blocks, heads, dim
        self.k, self.v = (np.full((blocks, heads, P, dim), 7, np.uint8) for _ in range(2))
        self.ks, self.vs = (np.full((blocks, heads, P, dim // 16), 0x7F, np.uint8) for _ in range(2))
        self.k_scale = (0.0021 + 0.0004 * np.arange(heads)).astype(np.float32)
        self.v_scale = (0.0017 + 0.0003 * np.arange(heads)).astype(np.float32)
        self.order = list(self.rng.permutation(blocks))

    def table(self, lengths, width=None):
        counts = [-(-n // P) for n in lengths]
        t = np.zeros((len(lengths), max([1] + counts) if width is None else width), np.int32)
        for i, (n, c) in enumerate(zip(lengths, counts)):
            t[i, :c] = [self.order.pop() for _ in range(c)]
            if not n:
                continue
            x = self.rng.standard_normal((2, n, self.H, self.D)).astype(np.float32)
            at, off = t[i, np.arange(n) // P], np.arange(n) % P
            self.k[at, :, off], self.ks[at, :, off] = e2m1.quantize(x[0], self.k_scale[None])
            self.v[at, :, off], self.vs[at, :, off] = e2m1.quantize(x[1], self.v_scale[None])
        return t

    def device(self, paired=False):
        kd, vd = (torch.from_numpy(x).cuda() for x in e2m1.pages(self.k, self.ks, self.v, self.vs))
        if paired:
            buf = torch.cat([kd, vd], -1).contiguous()
            return buf, buf.view(-1)[kd.shape[-1]:]
        return kd, vd

    def scales(self):
        return torch.from_numpy(self.k_scale).cuda(), torch.from_numpy(self.v_scale).cuda()

    def query(self, batch, group):
        q = torch.from_numpy(1.5 * self.rng.standard_normal((batch, self.H * group, self.D)).astype(np.float32)).bfloat16()
        return q.cuda(), q.double().numpy()

    def tokens(self, row, lo, hi, h):
        """Values of tokens lo .. hi - 1 of a table row for one head."""
        j = np.arange(lo, hi)
        at, off = row[j // P], j % P
        return (e2m1.dequantize(self.k[at, h, off], self.ks[at, h, off]) * np.float64(self.k_scale[h]),
                e2m1.dequantize(self.v[at, h, off], self.vs[at, h, off]) * np.float64(self.v_scale[h]))

    def attend(self, q, table, lengths, sm_scale, window=-1, bad=()):
        """(out, bound on the kernel's error) of decode; `bad`: (sequence, page) that are masked."""
        B, Hq, D = q.shape
        g = Hq // self.H
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        for b, n in enumerate(lengths):
            lo = max(0, n - window) if window > 0 else 0
            for h in range(self.H):
                k, v = self.tokens(table[b], lo, n, h)
                keep = np.array([(b, t // P) not in bad for t in range(lo, n)], bool)
                k, v = k[keep], v[keep]
                rows = slice(h * g, (h + 1) * g)
                out[b, rows], mag = e2m1.attend(q[b, rows], k, v, sm_scale)
                # half a step of the bf16 output, 2^-8 |out|; of the float16 weight and of its product with the block
                # scale, 2^-11 sum p |v| each, or 2^-25 in absolute terms for those below 2^-14, where the sum of
                # weights is at least 2^4 and the smallest scale here far above 1; 2^-12 sum p |v| for the float32
                # scores and the approximate exponential
                tol[b, rows] = 2.0 ** -8 * np.abs(out[b, rows]) + (2 * 2.0 ** -11 + 2.0 ** -12) * mag + 1e-6
                if len(v):
                    tol[b, rows] += 2.0 ** -28 * np.abs(v).sum(0)
        return out, tol


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def assert_within(got, ref, tol):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    excess = np.abs(got - ref) - tol
    assert excess.max() <= 0, f"error above its bound by {excess.max():.3e} at {np.unravel_index(excess.argmax(), excess.shape)}"
