"""Pins of the training oracles (oracle/training.py): closed forms, torch's
autograd in float64 (an independent implementation) and central differences
for every gradient, and a hand-worked AdamW step."""
import math

import pytest
import torch

from oracle import training as tr

F64 = torch.float64


def _inputs(seed, gate_shape=(2, 3, 4, 6)):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)
    return {"x": r(2, 3, 4, 6), "u": r(2, 3, 4, 6) + 0.5, "gate": r(*gate_shape), "scale": r(6),
            "gamma_post": r(6), "beta_post": r(6), "gamma_pre": r(6), "beta_pre": r(6)}


def test_layer_row_by_hand():
    # mean 2.5, variance 1.25
    h, r = tr.normalise(torch.tensor([[1.0, 2.0, 3.0, 4.0]], dtype=F64), False, 0.0)
    s = 1 / math.sqrt(1.25)
    assert torch.allclose(h, torch.tensor([[-1.5 * s, -0.5 * s, 0.5 * s, 1.5 * s]], dtype=F64), atol=1e-14)
    assert r.item() == pytest.approx(s)


def test_rms_row_by_hand():
    h, _ = tr.normalise(torch.tensor([[3.0, 4.0]], dtype=F64), True, 0.0)
    s = 1 / math.sqrt(12.5)
    assert torch.allclose(h, torch.tensor([[3 * s, 4 * s]], dtype=F64), atol=1e-14)


def test_gate_of_zero_halves_and_scale_of_zero_removes_the_branch():
    k = _inputs(0)
    full, _ = tr.block_norm(k["x"], k["u"], None, k["scale"])
    half, _ = tr.block_norm(k["x"], k["u"], torch.zeros_like(k["gate"]), k["scale"])
    assert torch.allclose(half - k["x"], (full - k["x"]) / 2, atol=1e-14)
    none, _ = tr.block_norm(k["x"], k["u"], k["gate"], torch.zeros(6, dtype=F64))
    assert torch.equal(none, k["x"])


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gate_shape", [(2, 3, 4, 6), (2, 3, 1, 6), (2, 1, 1, 6), (1, 3, 1, 6)])
def test_gradients_match_autograd(rms, gate_shape):
    k = _inputs(1, gate_shape)
    gen = torch.Generator().manual_seed(2)
    dx1, dy = (torch.randn(2, 3, 4, 6, generator=gen, dtype=F64) for _ in range(2))

    def sigmoid_free(x, u, gate, scale, g1, b1, g2, b2):
        def norm(v, g, b):
            if rms:
                return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * g + b
            return torch.nn.functional.layer_norm(v, (6,), g, b, 1e-5)
        x1 = x + scale * norm(u, g1, b1) / (1 + torch.exp(-gate))
        return x1, norm(x1, g2, b2)

    leaves = {n: t.clone().requires_grad_() for n, t in k.items()}
    x1, y = sigmoid_free(*leaves.values())
    (x1 * dx1).sum().add((y * dy).sum()).backward()
    ox1, oy = tr.block_norm(**k, rms=rms)
    assert torch.allclose(ox1, x1, atol=1e-12) and torch.allclose(oy, y, atol=1e-12)
    got = tr.block_norm_bwd(dx1, dy, x1, k["u"], k["gate"], k["scale"], k["gamma_post"],
                            k["beta_post"], k["gamma_pre"], rms=rms)
    for n, t in leaves.items():
        assert torch.allclose(got["d" + n], t.grad, atol=1e-11), n


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_match_differences(rms):
    k = _inputs(3, (2, 3, 1, 6))
    gen = torch.Generator().manual_seed(4)
    dx1, dy = (torch.randn(2, 3, 4, 6, generator=gen, dtype=F64) for _ in range(2))

    def loss(**kw):
        x1, y = tr.block_norm(**kw, rms=rms)
        return float((x1 * dx1).sum() + (y * dy).sum())

    x1, _ = tr.block_norm(**k, rms=rms)
    got = tr.block_norm_bwd(dx1, dy, x1, k["u"], k["gate"], k["scale"], k["gamma_post"],
                            k["beta_post"], k["gamma_pre"], rms=rms)
    h = 1e-6
    for n in k:
        way = torch.randn(k[n].shape, generator=gen, dtype=F64)
        diff = (loss(**{**k, n: k[n] + h * way}) - loss(**{**k, n: k[n] - h * way})) / (2 * h)
        want = float((got["d" + n] * way).sum())
        assert diff == pytest.approx(want, rel=1e-6, abs=1e-6), n


def test_norm_before_and_after_alone():
    k = _inputs(5)
    gen = torch.Generator().manual_seed(6)
    d = torch.randn(2, 3, 4, 6, generator=gen, dtype=F64)
    x = k["x"].clone().requires_grad_()
    torch.nn.functional.layer_norm(x, (6,), k["gamma_pre"], None, 1e-5).backward(d)
    got = tr.block_norm_bwd(None, d, k["x"], gamma_pre=k["gamma_pre"])
    assert torch.allclose(got["dx"], x.grad, atol=1e-12) and "du" not in got
    u = k["u"].clone().requires_grad_()
    torch.nn.functional.layer_norm(u, (6,), k["gamma_post"], None, 1e-5).backward(d)
    got = tr.block_norm_bwd(d, u=k["u"], gamma_post=k["gamma_post"])
    assert torch.allclose(got["du"], u.grad, atol=1e-12) and torch.equal(got["dx"], d)


def test_first_adamw_step_moves_by_the_sign():
    """From zero states m / (1 - b1) = g and v / (1 - b2) = g^2: the update is
    lr * g / (|g| + eps), after the decay."""
    p = torch.tensor([1.0, -2.0], dtype=F64)
    g = torch.tensor([0.5, -0.25], dtype=F64)
    z = torch.zeros(2, dtype=F64)
    q, m, v = tr.adamw(p, g, z, z, 1, 0.1, (0.9, 0.999), 1e-12, 0.01)
    assert torch.allclose(q, p * 0.999 - 0.1 * torch.sign(g), atol=1e-9)
    assert torch.allclose(m, 0.1 * g) and torch.allclose(v, 0.001 * g * g)


def test_adamw_matches_torch():
    gen = torch.Generator().manual_seed(7)
    p = torch.randn(50, generator=gen, dtype=F64).requires_grad_()
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-8, weight_decay=0.1)
    q, m, v = p.detach().clone(), torch.zeros(50, dtype=F64), torch.zeros(50, dtype=F64)
    for t in range(1, 6):
        p.grad = torch.randn(50, generator=gen, dtype=F64)
        q, m, v = tr.adamw(q, p.grad, m, v, t, 3e-3, (0.8, 0.95), 1e-8, 0.1)
        opt.step()
        assert torch.allclose(q, p.detach(), atol=1e-12)


def test_e4m3_step_matches_the_format():
    x = torch.linspace(0.001, 447.0, 5000, dtype=F64)
    near = x.float().to(torch.float8_e4m3fn).double()
    assert ((near - x).abs() <= tr.e4m3_step(x) / 2 + 1e-6).all()
    # the two values around 1: spacings 1/16 below and 1/8 above
    assert tr.e4m3_step(torch.tensor([0.99])).item() == 1 / 16
    assert tr.e4m3_step(torch.tensor([1.01])).item() == 1 / 8
    assert tr.e4m3_step(torch.tensor([1e-4])).item() == 2.0 ** -9


def test_norm_and_scales():
    assert tr.grad_norm([torch.tensor([3.0]), torch.tensor([[4.0]])]).item() == 5.0
    x = torch.zeros(300)
    x[5], x[299] = -448.0, 2.0
    assert torch.allclose(tr.block_scales(x), torch.tensor([1.0, 2.0 / 448.0], dtype=F64))
