"""Inputs and error bounds shared by the paged-cache GPU tests."""

from __future__ import annotations

import numpy as np
import torch

BF16, FP16 = torch.bfloat16, torch.float16


def bits64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Cache:
    """A paged cache on the GPU whose slots in use hold Gaussian values and all
    others NaN: what must not be read would show."""

    def __init__(self, B, Hkv, d, ps, lens, dtype, seed, width=None, dev="cuda", nan=True):
        g = torch.Generator().manual_seed(seed)
        need = max(1, max(-(-int(n) // ps) for n in lens))
        width = width or need
        assert width >= need
        pages = B * width + 3
        self.table = torch.randperm(pages, generator=g)[:B * width].to(torch.int32).view(B, width)
        fill = float("nan") if nan else 0.0
        self.k = torch.full((pages, Hkv, ps, d), fill, dtype=dtype)
        self.v = torch.full((pages, Hkv, ps, d), fill, dtype=dtype)
        for b in range(B):
            for p in range(-(-int(lens[b]) // ps)):
                m = min(ps, int(lens[b]) - p * ps)
                page = int(self.table[b, p])
                self.k[page, :, :m] = torch.randn(Hkv, m, d, generator=g).to(dtype)
                self.v[page, :, :m] = torch.randn(Hkv, m, d, generator=g).to(dtype)
        self.B, self.Hkv, self.d, self.ps, self.L = B, Hkv, d, ps, width * ps
        self.lens = torch.tensor([int(n) for n in lens], dtype=torch.int32)
        self.g, self.dtype, self.dev = g, dtype, dev

    def gpu(self):
        return (self.k.to(self.dev), self.v.to(self.dev), self.table.to(self.dev), self.lens.to(self.dev))

    def query(self, Hq, std=1.0):
        return (torch.randn(self.B, Hq, self.d, generator=self.g) * std).to(self.dtype)

    def weights(self):
        return torch.rand(self.B, self.Hkv, self.L, generator=self.g) * 3


def score_error(q, k, scale):
    """Bound on the error of one fp32 score: d products added in fp32, and the
    scaling, each half a step (2^-24) of at most the sum of magnitudes."""
    q, k = np.abs(q), np.abs(k)
    d = q.shape[-1]
    big = float(np.nanmax(q.reshape(-1, d).max(0) @ np.nan_to_num(k.reshape(-1, d)).max(0))) if k.size else 0.0
    return (d + 8) * 2.0 ** -24 * scale * big


def decode_bounds(o_ref, lse_ref, A, ds, n, dtype):
    """(o, lse, relative weight) tolerances. ds: score error; A: sum of p |v|;
    n: slots. p is formed with relative error ds + 2^-22 (exp2) and kept as a
    16-bit value and remainder (2^-16 bf16, 2^-22 fp16); sums of n terms in
    fp32 are off by n half steps; o is rounded once."""
    half = torch.finfo(dtype).eps / 2
    sums = n * 2.0 ** -24
    rel = 2 * ds + 2.0 ** -21 + 2 * sums
    tol_lse = ds + 2.0 ** -21 + sums + 4 * 2.0 ** -24 * np.abs(np.where(np.isfinite(lse_ref), lse_ref, 0.0))
    tol_o = half * np.abs(o_ref) * 1.01 + A * (rel + 2.0 ** -15) + 2.0 ** -25
    return tol_o, tol_lse, rel + float(np.max(tol_lse, initial=0.0)) + 2.0 ** -21
