"""Oracles of the training operators around the blocks -- test infrastructure
only.

Plain float64 CPU statements (torch tensors in, torch float64 out) of the
seam between two blocks (the norm after a block with its gate and residual
scale, the norm before the next one) and its gradients, and of one AdamW step
with 32-bit or 8-bit states.  Only the test-suite may import this module; it
imports nothing from the product.

Parity status: pinned (tests/test_training_oracle_pins.py).
"""
from __future__ import annotations

import torch

BLOCK = 256


def _d(t):
    return None if t is None else t.detach().to(torch.float64).cpu()


def normalise(v, rms, eps):
    """(v - mean) / sqrt(var + eps) over the last axis (rms: v / sqrt(mean v^2
    + eps)); returns it and the factor 1 / sqrt(...)."""
    c = v if rms else v - v.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(c.pow(2).mean(-1, keepdim=True) + eps)
    return c * r, r


def _affine(h, gamma, beta):
    h = h if gamma is None else h * gamma
    return h if beta is None else h + beta


def block_norm(x, u=None, gate=None, scale=None, gamma_post=None, beta_post=None, gamma_pre=None,
               beta_pre=None, rms=False, eps=1e-5, pre=True):
    """(x1, y) of evoattn_block_norm."""
    x, u, gate, scale = _d(x), _d(u), _d(gate), _d(scale)
    if u is not None:
        t = _affine(normalise(u, rms, eps)[0], _d(gamma_post), _d(beta_post))
        if gate is not None:
            t = t * torch.sigmoid(gate)
        x = x + (t if scale is None else t * scale)
    return x, _affine(normalise(x, rms, eps)[0], _d(gamma_pre), _d(beta_pre)) if pre else None


def _through_norm(b, h, r, rms):
    g = b - h * (b * h).mean(-1, keepdim=True)
    return r * (g if rms else g - b.mean(-1, keepdim=True))


def block_norm_bwd(dx1, dy=None, x1=None, u=None, gate=None, scale=None, gamma_post=None,
                   beta_post=None, gamma_pre=None, rms=False, eps=1e-5):
    """Gradients of sum(x1 * dx1) + sum(y * dy) at the given x1 (the norm
    before the next block) and u, gate (the branch): a dict with dx, du, dgate
    (summed over the axes where the gate has extent 1), dscale, dgamma_post,
    dbeta_post, dgamma_pre, dbeta_pre."""
    dy, x1, u, gate = _d(dy), _d(x1), _d(u), _d(gate)
    D = torch.zeros_like(dy) if dx1 is None else _d(dx1)
    rows = tuple(range(D.dim() - 1))
    out = {}
    if dy is not None:
        h, r = normalise(x1, rms, eps)
        out["dgamma_pre"] = (dy * h).sum(rows)
        out["dbeta_pre"] = dy.sum(rows)
        D = D + _through_norm(_affine(dy, _d(gamma_pre), None), h, r, rms)
    out["dx"] = D
    if u is not None:
        h, r = normalise(u, rms, eps)
        w = _affine(h, _d(gamma_post), _d(beta_post))
        q = 1.0 if gate is None else torch.sigmoid(gate)
        e = D if scale is None else D * _d(scale)
        out["dscale"] = (D * q * w).sum(rows)
        if gate is not None:
            dg = e * w * q * (1.0 - q)
            over = [i for i in rows if gate.shape[i] == 1]
            out["dgate"] = dg.sum(over, keepdim=True) if over else dg
        e = e * q
        out["dgamma_post"] = (e * h).sum(rows)
        out["dbeta_post"] = e.sum(rows)
        out["du"] = _through_norm(_affine(e, _d(gamma_post), None), h, r, rms)
    return out


def grad_norm(grads):
    return torch.sqrt(sum(_d(g).pow(2).sum() for g in grads))


def adamw(p, g, m, v, t, lr, betas, eps, weight_decay, clip=1.0):
    """(p, m, v) after step number t (from 1)."""
    p, g, m, v = _d(p), _d(g) * clip, _d(m), _d(v)
    m = betas[0] * m + (1.0 - betas[0]) * g
    v = betas[1] * v + (1.0 - betas[1]) * g * g
    p = p * (1.0 - lr * weight_decay) - lr * (m / (1.0 - betas[0] ** t)) / (
        torch.sqrt(v / (1.0 - betas[1] ** t)) + eps)
    return p, m, v


def block_scales(x):
    """max|x| / 448 of each block of 256 elements of a flat tensor."""
    x = _d(x).reshape(-1)
    x = torch.nn.functional.pad(x, (0, -x.numel() % BLOCK))
    return x.view(-1, BLOCK).abs().amax(1) / 448.0


def e4m3_step(x):
    """The spacing of e4m3 values around x (three bits behind the leading one,
    normal from 2^-6, subnormal spacing 2^-9)."""
    _, e = torch.frexp(_d(x).abs())
    return torch.ldexp(torch.ones_like(_d(x)), (e - 1).clamp(-6, 8) - 3)
