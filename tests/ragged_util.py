"""Inputs and tolerances of the ragged-batch tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import ragged as og


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def make_pool(n_pages, H, hd, kind, seed, junk=True):
    """A pool (numpy) with valid codes and scales everywhere, built page by
    page through the definition; the padding holds junk."""
    g = gen(seed)
    amp = torch.ones(hd)
    amp[[7, hd - 5]] = 8.0
    k = (torch.randn(n_pages * 16, H, hd, generator=g) * amp).numpy()
    v = torch.randn(n_pages * 16, H, hd, generator=g).numpy()
    pool = np.full((n_pages, H, og.block_bytes(hd)), 0xA5 if junk else 0, np.uint8)
    og.append(pool, k, v, np.arange(n_pages * 16), kind)
    return pool


def attention_tol(ref, q, pool, kind, hd, n_max, cap, slopes, out_bf16):
    """Bound of |got - exact| per element, from the arithmetic:

    The logit x (base 2) is computed with a relative error of the products of
    2^-21 (the query as the sum of two f16 numbers of 11 bits, scaled so that
    its largest element is in (1/2, 1]) plus hd 2^-24 for the f32 sum, each
    against sum |q||k|; a few f32 roundings (scales, cap, slope) add 2^-21 of
    the largest |x| and of the bias.  exp2 and the weights' two-part f16 form
    add 2^-20.  Weights off by a factor e^dx move the average of values by at
    most 2 dx max|v|.  Sums over the pages add (pages + 32) 2^-24 max|v| each
    for numerator and denominator.  One f16 part instead of two (only with
    bf16 outputs) adds 2^-11 max|v|, and the output's rounding 2^-8 |o|."""
    H = pool.shape[1]
    kv, vv = [], []
    place = og._places(hd)
    for h in range(H):
        for part, acc in ((0, kv), (1, vv)):
            codes = og.decode(pool[:, h][:, place[part]], kind)
            s = pool[:, h, 32 * hd + 4 * part:32 * hd + 4 * part + 4].copy().view(np.float32)[:, 0].astype(np.float64)
            acc.append(np.nanmax(np.abs(codes), axis=(1, 2)) * s)
    kmax, vmax = np.nanmax(np.stack(kv)), np.nanmax(np.stack(vv))
    sum_qk = np.abs(q).sum(-1).max() * kmax * hd ** -0.5
    big = sum_qk if not cap else max(sum_qk, cap)
    bias = 0.0 if slopes is None else float(np.max(np.abs(slopes))) * n_max
    dx = sum_qk * (2.0 ** -21 + hd * 2.0 ** -24) + (big + bias) * 2.0 ** -21 + 2.0 ** -20
    pages = n_max / 16 + 32
    tol = vmax * (2 * dx + 2 * pages * 2.0 ** -24)
    if out_bf16:
        return tol + vmax * 2.0 ** -11 + np.abs(ref) * 2.0 ** -8
    return tol + np.abs(ref) * 2.0 ** -24


def to(dev, x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev)
