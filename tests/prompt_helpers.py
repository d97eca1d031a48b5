"""Shared by the tests of the prompt side: random pools and tables, and the error bounds of the kernels.

Bounds (worst cases of the arithmetic, u = 2^-24 the half step of fp32):
- a score of D products: D u |q|.|k| scale on the FMA units; twice that on the
  tensor cores, whose sums may be cut instead of rounded;
- a weight 2^x: ex2.approx 2^-22, and x = s scale log2e - m from at most four
  roundings of numbers up to 2 max|s| log2e, each u relative;
- every weight of a row carries that relative error, the row's sum too, so the
  normalised weights carry twice it; sums over n keys add n u (2 n u on the
  tensor cores), in the numerator and in the denominator; the joining of parts
  adds a weight more: 2 (2^-22 + 4 u X) again;
- bf16: each weight is rounded to bf16 for the product with V, half a step
  2^-8 relative, and the output once, 2^-8 |out|.
An error of the weights moves the output by at most that times sum p|v|."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
LOG2E = 1.4426950408889634


def attention_bounds(ref, bf16: bool):
    out, lse, absv, prod, smax, keys, D = *ref, ref[0].shape[-1]
    mma = 2.0 if bf16 else 1.0
    score = mma * D * U * prod
    weight = score + 2 * (2.0 ** -22 + 4 * U * 2 * smax * LOG2E)
    e = 2 * weight + 2 * mma * keys * U
    tol = absv * (e + (BF16_HALF if bf16 else 0.0))[..., None] + np.abs(out) * (BF16_HALF if bf16 else U) + 1e-30
    lse_tol = weight + mma * keys * U + 4 * U * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return tol, lse_tol


def norm_bounds(ref, mag, bf16: bool):
    """Norm: the sum of squares of D products 14 u (8 of a lane, 4 to 5 exchanges, half of it after the root), rsqrtf
    2 ulp, two products: 13 u. Rotation: the angle's step to fp32 pi/2 u, sincospif 2 ulp, mscale: 6 u, two products
    and a sum 3 u. In all 22 u of |a| + |b|."""
    return 22 * U * mag + np.abs(ref) * (BF16_HALF if bf16 else U) + 1e-30


def pool(rng, B, lens, Hkv, D, page, dtype, extra=2, layout="hnd", device="cpu", std=1.0, cols=None):
    """Random pages for `lens` tokens of each request, in random order: (k, v, table)."""
    held = [-(-int(n) // page) for n in lens]
    total = sum(held) + extra
    ids = rng.permutation(total)
    cols = max([1] + held) if cols is None else cols
    table = np.full((B, cols), -1, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    shape = (total, Hkv, page, D)
    if layout == "nhd":  # rows of a page's token side by side, padded
        k, v = (torch.randn(total, page, Hkv, D + 8, generator=g).mul(std).to(dtype).to(device)[..., :D].transpose(1, 2)
                for _ in range(2))
    else:
        k, v = (torch.randn(shape, generator=g).mul(std).to(dtype).to(device) for _ in range(2))
    return k, v, torch.from_numpy(table).to(device)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()
