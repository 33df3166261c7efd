"""Pins of the 8-bit path's oracle (oracle/eightbit.py) to values worked out
elsewhere: the generator's published answers, torch's own conversion to e4m3,
scales at the borders of a power of two, autograd and differences."""
import numpy as np
import pytest
import torch

from oracle import eightbit as eb


@pytest.mark.parametrize("counter, key, want", [
    # known answers that accompany the generator's publication
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    got = eb.philox(np.array(counter, dtype=np.uint64), key)
    assert tuple(int(v) for v in got) == want


def test_keep_rate_sharing_and_arguments():
    shape = (2, 5, 7, 130)
    k = eb.keep(shape, 0.25, 9, 4, 3)
    assert k.shape == shape
    n = k.numel()
    assert abs(k.double().mean().item() - 0.75) < 5 * (0.75 * 0.25 / n) ** 0.5
    assert eb.keep(shape, 0.25, 9, 4, 3, shared=(1,)).shape == (2, 1, 7, 130)
    # a mask row's index runs over the axes that are not shared
    flat = eb.keep((1, 1, 14, 130), 0.25, 9, 4, 3)
    assert torch.equal(eb.keep(shape, 0.25, 9, 4, 3, shared=(1,)).reshape(14, 130), flat[0, 0])
    for other in ((8, 4, 3), (9, 5, 3), (9, 4, 2), (9 + 2 ** 32, 4, 3)):
        assert not torch.equal(k, eb.keep(shape, 0.25, *other))
    assert torch.equal(k, eb.keep(shape, 0.25, 9, 4 + 2 ** 32, 3))
    assert eb.keep(shape, 0.0, 9, 4).all()
    u = torch.ones(shape)
    d = eb.dropped(u, 0.25, 9, 4, 3)
    assert torch.equal(d != 0, k) and torch.equal(d[k], torch.full((int(k.sum()),), 1 / 0.75, dtype=torch.float64))


def test_e4m3_is_torchs_conversion():
    gen = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=gen) * torch.exp(3 * torch.randn(20000, generator=gen)),
                   torch.arange(-448, 449).float() / 7, torch.tensor([0.0, -0.0, 448.0, 2.0 ** -9, 2.0 ** -10,
                                                                     3 * 2.0 ** -10, 2.0 ** -11])]).clamp(-448, 448)
    assert torch.equal(eb.e4m3(x), x.to(torch.float8_e4m3fn).double())
    assert ((eb.e4m3(x) - x.double()).abs() <= eb.half_step(x)).all()


def test_exponents_at_their_borders():
    for k in (-127, -126, -20, -1, 0, 1, 5, 119):
        top = 448.0 * 2.0 ** k
        a = torch.tensor([top, top * (1 + 2.0 ** -23), top * (1 - 2.0 ** -23)], dtype=torch.float64)
        assert eb.exponent(a).tolist() == [k, k + 1, k]
    assert eb.exponent(torch.tensor([0.0, 1e-45, 3.4028234663852886e38])).tolist() == [0, -127, 120]


def test_quantise_and_values():
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(300, 200, generator=gen) * torch.exp(torch.randn(300, 1, generator=gen))
    q, k = eb.quantise(x)
    assert q.shape == x.shape and k.shape == (300, 2)
    v = eb.values(q, k)
    s = torch.exp2(k.double()).repeat_interleave(128, 1)[:, :200]
    assert ((v - x.double()).abs() <= eb.half_step(x.double() / s) * s).all()
    assert (q.abs().reshape(-1).max() <= 448) and (q.abs()[:, :128].amax(1) > 224 * (1 - 2 ** -4)).all()
    qb, kb = eb.quantise_blocks(x)
    assert kb.shape == (3, 2)
    assert int(kb[2, 1]) == int(eb.exponent(x[256:, 128:].abs().max()))
    vb = eb.values(qb, kb)
    assert ((vb - x.double()).abs() <= 2 ** -4 * x.double().abs() +
            2 ** -10 * torch.exp2(kb.double()).repeat_interleave(128, 0)[:300].repeat_interleave(128, 1)[:, :200]).all()
    # elements that are not finite spoil themselves alone
    x[0, 3], x[1, 5] = float("inf"), float("nan")
    q2, k2 = eb.quantise(x)
    assert torch.isnan(q2[0, 3]) and torch.isnan(q2[1, 5]) and int(torch.isnan(q2).sum()) == 2
    assert torch.equal(q2[2:], q[2:]) and torch.equal(k2[2:], k[2:])


def test_matmul_is_torchs():
    gen = torch.Generator().manual_seed(3)
    a, b, c = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((5, 9), (4, 9), (5, 4)))
    out, size = eb.matmul(a, b, c)
    assert torch.allclose(out, torch.einsum("mk,nk->mn", a, b) + c, rtol=1e-14)
    assert (size >= out.abs() - 1e-12).all()


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_are_autograds_and_differences(rms):
    gen = torch.Generator().manual_seed(4)
    draw = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    x, u, g, b = draw(1, 2, 3, 10), draw(1, 2, 3, 10), 1 + 0.1 * draw(10), draw(10)
    d1, dy = draw(1, 2, 3, 10), draw(1, 2, 3, 10)
    drop = dict(p=0.3, seed=5, step=6, site=7, shared=(1,))

    def loss(x, u, g, b):
        x1, y = eb.norm8(x, u, g, b, rms, **drop)
        return (x1 * d1).sum() + (y * dy).sum()

    x1, y = eb.norm8(x, u, g, b, rms, **drop)
    want = eb.norm8_bwd(d1, dy, x1, g, rms, **drop)
    names = (("dx", x), ("du", u), ("dgamma", g), ("dbeta", b))
    # differences of the loss
    for i, (name, t) in enumerate(names):
        for at in ((0, 0, 0, 1), (0, 1, 2, 7)) if t.dim() == 4 else ((2,), (9,)):
            args = [x, u, g, b]
            sides = []
            for h in (1e-6, -1e-6):
                args[i] = t.clone()
                args[i][at] += h
                sides.append(float(loss(*args)))
            assert abs((sides[0] - sides[1]) / 2e-6 - float(want[name][at])) < 1e-6 * (1 + abs(float(want[name][at])))
    # autograd, through torch's own norm
    xs, us, gs, bs = (t.clone().requires_grad_() for t in (x, u, g, b))
    k = eb.keep(x.shape, 0.3, 5, 6, 7, (1,)).double() / 0.7
    z = xs + us * k
    n = torch.nn.functional.rms_norm(z, (10,), gs, 1e-5) + bs if rms else \
        torch.nn.functional.layer_norm(z, (10,), gs, bs, 1e-5)
    assert torch.allclose(n, y, rtol=1e-12, atol=1e-12)
    ((z * d1).sum() + (n * dy).sum()).backward()
    for (name, _), t in zip(names, (xs, us, gs, bs)):
        assert torch.allclose(t.grad, want[name], rtol=1e-10, atol=1e-12)
