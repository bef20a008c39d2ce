"""Random paged caches for the serving tests: every slot that no token owns
holds the format's NaN, so that a read outside the sequences shows."""
from __future__ import annotations

import numpy as np
import torch

from oracle import layout
from oracle.kv_cache import BF16, FP8, FP8_E5M2

P = 16
NAN_CODE = {FP8: 0x7F, FP8_E5M2: 0x7F, BF16: 0x7FC0}


class Pool:
    """A cache of `blocks` pages per head handed out in random order."""

    def __init__(self, blocks, heads, dim, dtype, seed, per_token=False):
        self.rng = np.random.default_rng(seed)
        self.dtype, self.H, self.D, self.blocks, self.per_token = dtype, heads, dim, blocks, per_token
        kind = np.uint16 if dtype == BF16 else np.uint8
        self.k = np.full((blocks, heads, P, dim), NAN_CODE[dtype], kind)
        self.v = np.full((blocks, heads, dim, P), NAN_CODE[dtype], kind)
        self.scales = np.full((blocks, heads, 2, P), np.nan, np.float32) if per_token else None
        self.k_scale = (0.02 + 0.005 * np.arange(heads)).astype(np.float32)
        self.v_scale = (0.015 + 0.004 * np.arange(heads)).astype(np.float32)
        if dtype == FP8_E5M2:
            self.k_scale, self.v_scale = self.k_scale / 128, self.v_scale / 128
        self.order = list(self.rng.permutation(blocks))

    def _codes(self, x, scale):
        if self.dtype == BF16:
            return torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
        t = torch.float8_e4m3fn if self.dtype == FP8 else torch.float8_e5m2
        top = 448.0 if self.dtype == FP8 else 57344.0
        return torch.from_numpy((x / scale).clip(-top, top)).to(t).view(torch.uint8).numpy()

    def pages(self, n):
        return [int(self.order.pop()) for _ in range(n)]

    def fill(self, pages, length):
        """Random tokens 0 .. length - 1 in the given pages."""
        H, D, rng = self.H, self.D, self.rng
        x = rng.standard_normal((2, length, H, D)).astype(np.float32)
        for j in range(length):
            blk, off = pages[j // P], j % P
            if self.per_token:
                top = 448.0 if self.dtype == FP8 else 57344.0
                sc = (np.abs(x[:, j]).max(axis=-1) / top * rng.uniform(0.5, 2, (2, H))).astype(np.float32)
                self.scales[blk, :, :, off] = sc.T
                kq, vq = self._codes(x[0, j], sc[0][:, None]), self._codes(x[1, j], sc[1][:, None])
            else:
                kq, vq = self._codes(x[0, j], self.k_scale[:, None]), self._codes(x[1, j], self.v_scale[:, None])
            self.k[blk, :, off], self.v[blk, :, :, off] = kq, vq

    def table(self, lengths, width=None, fill=True):
        """int32 [n][width] block table with fresh pages for each length."""
        counts = [-(-n // P) for n in lengths]
        width = max([1] + counts) if width is None else width
        t = np.zeros((len(lengths), width), np.int32)
        for i, (n, c) in enumerate(zip(lengths, counts)):
            t[i, :c] = self.pages(c)
            if fill:
                self.fill(t[i, :c], n)
        return t

    def device(self, paired=False):
        """(k_cache, v_cache) in the library's page format on the GPU."""
        if paired:
            buf = torch.from_numpy(layout.to_device_format_paired(self.k, self.v, self.scales)).cuda()
            kpage = P * self.D * self.k.dtype.itemsize
            return buf, buf.view(-1)[kpage:]
        if self.per_token:
            kd, vd = layout.to_device_format_per_token(self.k, self.v, self.scales)
        else:
            kd, vd = layout.to_device_format(self.k, self.v)
        return torch.from_numpy(kd).cuda(), torch.from_numpy(vd).cuda()

    def device_scales(self):
        if self.per_token or self.dtype == BF16:
            return None, None
        return torch.from_numpy(self.k_scale).cuda(), torch.from_numpy(self.v_scale).cuda()

    def query(self, batch, group):
        """bf16 queries [batch][H * group][D], and their values."""
        q = torch.from_numpy(1.5 * self.rng.standard_normal((batch, self.H * group, self.D)).astype(np.float32)).bfloat16()
        return q.cuda() if torch.cuda.is_available() else q, q.double().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def output_bound(ref, mag):
    """Half a step of the bf16 output, 2^-8 |out|, and of every float16
    probability, 2^-11 sum p |v|; 2^-12 sum p |v| for the scores (float32 sums
    and the query's two-term FP8 form, 2^-18 of its largest element) and the
    approximate exponential."""
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * mag + 1e-6


def assert_output(got, ref, mag):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    excess = np.abs(got - ref) - output_bound(ref, mag)
    assert excess.max() <= 0, f"error above its bound by {excess.max():.3e} at {np.unravel_index(excess.argmax(), excess.shape)}"
