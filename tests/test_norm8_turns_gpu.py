"""The norm with 8-bit output and its gradients where a CTA takes several turns
of rows whose masks are shared: the walk along an axis whose rows have one mask,
beyond the first turn, in either order of the axes in memory.

Tolerances as in test_eightbit_gpu.py; a sum over rows adds u times its depth,
below 1024 here."""
import pytest
import torch

from oracle import eightbit as eb
from protein_folding_attention_gb300 import evoattn
from test_eightbit_gpu import DEV, TYPES, U, check_codes, d, draw, gen, laid, near, params, rng, stored

pytestmark = pytest.mark.gpu

# (147 and 151: no multiple of the rows that a thread holds)
CASES = [((1, 147, 151, 128), (1,)), ((1, 147, 151, 128), (2,)), ((2, 75, 150, 72), (0, 1)),
         ((1, 101, 130, 131), (1,)), ((1, 61, 67, 1032), (1,)), ((3, 21, 41, 4096), (1,)), ((1, 97, 89, 384), (1, 2))]


@pytest.mark.parametrize("shape, shared", CASES)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("how", ["dense", "swapped"])
def test_norm8_bwd_turns_with_shared_masks(shape, shared, types, how):
    res, io = TYPES[types]
    g = gen(31)
    dx1, dy, x1 = draw(shape, res, g), draw(shape, io, g), draw(shape, res, g)
    gamma, beta = params(shape[-1], g, evoattn.NORM_LAYER)
    p, mask = 0.25, dict(site=4, shared=shared)
    got = evoattn.norm8_bwd(laid(dx1, how), laid(dy, how), laid(x1, how), gamma.to(DEV), beta.to(DEV), p=p, rng=rng(), **mask)
    want = eb.norm8_bwd(dx1, dy, x1, gamma, p=p, seed=11, step=5, **mask)
    h, r = eb.normalise(d(x1), False, 1e-5)
    k = d(x1).abs().amax(-1, keepdim=True) * r
    e = (d(dy) * gamma.double()).abs()
    terms = r * (e + h.abs() * (e * h.abs()).mean(-1, keepdim=True) + e.mean(-1, keepdim=True)) + d(dx1).abs()
    err = 128 * U * (1 + k) * terms.amax(-1, keepdim=True)
    stored(got["dx"], want["dx"], err, "dx")
    keep = eb.keep(shape, p, 11, 5, **mask).expand(shape)
    stored(got["du"], want["du"], err / (1 - p) * keep, "du")
    for n, t in (("dgamma", d(dy) * h), ("dbeta", d(dy))):
        near(got[n], want[n], ((1024 + 64 * (1 + k)) * U * t.abs().amax(-1, keepdim=True).maximum(t.abs())).sum((0, 1, 2)), n)


@pytest.mark.parametrize("shape, shared", [((1, 147, 151, 128), (1,)), ((1, 61, 131, 1032), (1,)), ((1, 130, 61, 1030), (2,)),
                                           ((1, 67, 61, 4096), (1,))])
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("how", ["dense", "swapped"])
def test_norm8_turns_with_shared_masks(shape, shared, types, how):
    res, io = TYPES[types]
    g = gen(32)
    x, u = draw(shape, res, g), draw(shape, io, g)
    gamma, beta = params(shape[-1], g, evoattn.NORM_LAYER)
    p, mask = 0.25, dict(site=4, shared=shared)
    got, codes, scales = evoattn.norm8(laid(x, how), laid(u, how), gamma.to(DEV), beta.to(DEV), p=p, rng=rng(), **mask)
    x1, y = eb.norm8(x, u, gamma, beta, p=p, seed=11, step=5, **mask)
    stored(got, x1, 4 * U * (d(x).abs() + eb.dropped(u, p, 11, 5, **mask).abs()), "x1")
    h, r = eb.normalise(x1, False, 1e-5)
    k = x1.abs().amax(-1, keepdim=True) * r
    terms = (h * gamma.double()).abs().amax(-1, keepdim=True) + d(beta).abs().max()
    check_codes(codes, scales, y, 64 * U * (1 + k) * terms)
