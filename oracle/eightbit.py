"""Oracles of the 8-bit projection path -- test infrastructure only.

Plain float64 CPU statements (torch tensors in, torch tensors out) of the
dropout drawn from a counter-based generator, of the norm before a block with
its output in e4m3 and power-of-two scales, of its gradients, of the
quantisation and of the product of quantised matrices.  Only the test-suite
may import this module; it imports nothing from the product.

Parity status: pinned (tests/test_eightbit_oracle_pins.py).
"""
from __future__ import annotations

import numpy as np
import torch

from oracle.training import normalise

GROUP = 128


def _d(t):
    return None if t is None else t.detach().to(torch.float64).cpu()


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
def philox(counter, key):
    """Philox4x32-10 of a counter [..., 4] and a key (two words)."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def keep(shape, p, seed, step, site=0, shared=()):
    """The mask of a [B, I, J, C] tensor, with extent 1 along shared axes."""
    B, I, J, C = (1 if a in shared else n for a, n in enumerate(shape))
    groups = -(-C // 4)
    c = np.zeros((B * I * J, groups, 4), dtype=np.uint64)
    c[..., 0] = np.arange(groups)[None, :]
    c[..., 1] = np.arange(B * I * J)[:, None]
    c[..., 2] = site
    c[..., 3] = step % 2 ** 32
    words = philox(c, (seed % 2 ** 32, (seed >> 32) % 2 ** 32)).reshape(B * I * J, -1)[:, :C]
    threshold = min(int(np.floor(p * 2.0 ** 32 + 0.5)), 2 ** 32 - 1)
    return torch.from_numpy((words >= threshold).reshape(B, I, J, C))


def dropped(u, p=0.0, seed=0, step=0, site=0, shared=()):
    """keep * u / (1 - p)"""
    u = _d(u)
    if p == 0.0:
        return u
    k = keep(u.shape, p, seed, step, site, shared)
    return torch.where(k, u / (1.0 - p), torch.zeros_like(u))


# ---------------------------------------------------------------------------
# codes and scales
# ---------------------------------------------------------------------------
def exponent(amax):
    """k of the smallest 2^k with amax <= 448 2^k (k >= -127; 0 for 0)."""
    amax = _d(amax)
    k = torch.full_like(amax, -127.0)
    for _ in range(256):
        k = torch.where(amax > 448.0 * torch.exp2(k), k + 1, k)
    return torch.where(amax > 0, k, torch.zeros_like(k)).to(torch.int64)


def half_step(x):
    """Half the spacing of e4m3 values around x (normal from 2^-6)."""
    _, e = torch.frexp(_d(x).abs())
    return torch.exp2((e - 1).clamp(-6, 8).double() - 4)


def e4m3(x):
    """x (|x| <= 448) rounded to the nearest e4m3 value, ties to even."""
    x = _d(x)
    step = 2 * half_step(x)
    return torch.round(x / step) * step


def _scaled(x, over):
    """Codes (as values) and scale exponents of groups over the axes `over`."""
    fine = torch.isfinite(x)
    k = exponent(torch.where(fine, x.abs(), torch.zeros_like(x)).amax(over, keepdim=True))
    q = e4m3(torch.where(fine, x * torch.exp2(-k.double()), torch.zeros_like(x)))
    return torch.where(fine, q, torch.full_like(q, float("nan"))), k


def _pad(x, axis):
    n = -x.shape[axis] % GROUP
    shape = list(x.shape)
    shape[axis] = n
    return torch.cat([x, x.new_zeros(shape)], axis)


def quantise(x):
    """Codes and exponents by groups of 128 of the last axis."""
    x = _d(x)
    q, k = _scaled(_pad(x, -1).unflatten(-1, (-1, GROUP)), -1)
    return q.flatten(-2)[..., :x.shape[-1]], k.squeeze(-1)


def quantise_blocks(x):
    """... by 128 x 128 blocks of a matrix."""
    x = _d(x)
    R, K = x.shape
    t = _pad(_pad(x, 0), 1).unflatten(1, (-1, GROUP)).unflatten(0, (-1, GROUP))
    q, k = _scaled(t, (1, 3))
    return q.flatten(2).flatten(0, 1)[:R, :K], k[:, 0, :, 0]


def values(codes, exponents):
    """What codes with scales by row, or by 128 rows, stand for."""
    codes, k = _d(codes), exponents.to(torch.int64).cpu()
    if k.shape[:-1] != codes.shape[:-1]:
        k = k.repeat_interleave(GROUP, 0)[:codes.shape[0]]
    return codes * torch.exp2(k.double()).repeat_interleave(GROUP, -1)[..., :codes.shape[-1]]


def matmul(a, b, add=None):
    """a b^T (+ add) of values, and the sum of the magnitudes of its terms."""
    out, size = a @ b.t(), a.abs() @ b.abs().t()
    if add is not None:
        out, size = out + _d(add), size + _d(add).abs()
    return out, size


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm8(x, u=None, gamma=None, beta=None, rms=False, eps=1e-5, **drop):
    """x1 and y (before its rounding) of evoattn_norm8; drop: the arguments of
    `dropped`."""
    x = _d(x)
    if u is not None:
        x = x + dropped(u, **drop)
    y = normalise(x, rms, eps)[0]
    y = y if gamma is None else y * _d(gamma)
    return x, y if beta is None else y + _d(beta)


def norm8_bwd(dx1, dy, x1, gamma=None, rms=False, eps=1e-5, **drop):
    """Gradients of sum(x1 * dx1) + sum(y * dy): dx, du, dgamma, dbeta."""
    dy, x1 = _d(dy), _d(x1)
    h, r = normalise(x1, rms, eps)
    rows = tuple(range(dy.dim() - 1))
    out = {"dgamma": (dy * h).sum(rows), "dbeta": dy.sum(rows)}
    e = dy if gamma is None else dy * _d(gamma)
    g = e - h * (e * h).mean(-1, keepdim=True)
    if not rms:
        g = g - e.mean(-1, keepdim=True)
    out["dx"] = r * g if dx1 is None else _d(dx1) + r * g
    out["du"] = dropped(out["dx"], **drop) if drop else out["dx"]
    return out
