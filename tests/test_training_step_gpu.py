"""A training step as it is used: the norm before the attention, triangle
attention, the norm after it with its gate and residual scale, the gradients
back through all of them, and one clipped AdamW step of the norms' parameters,
against float64 oracles of every part.

Tolerances: the attention's own parity bar (relative L2 5e-3 forward, 1e-2
for gradients) is what reaches the parameters' gradients; the first AdamW step
from zero states is lr * sign(g) up to eps, so a parameter differs by more
than rounding only where its gradient is within that error of zero."""
import numpy as np
import pytest
import torch

import oracle
from oracle import training as tr
from protein_folding_attention_gb300 import evoattn

from helpers import FWD_REL, GRAD_REL, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_norm_attention_norm_step():
    oracle.build()
    N, H, D = 40, 4, 32
    C = H * D
    gen = torch.Generator().manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)
    x, gate, bias, dx1 = bf(1, N, N, C), bf(1, N, N, C), bf(1, H, N, N), bf(1, N, N, C)
    vec = lambda mean: mean + 0.1 * torch.randn(C, generator=gen)
    prm = {"gamma_pre": vec(1.0), "beta_pre": vec(0.0), "scale": vec(0.5), "gamma_post": vec(1.0),
           "beta_post": vec(0.0)}
    dev = {n: t.to(DEV) for n, t in prm.items()}
    xd, gd, bd, dd = (t.to(DEV) for t in (x, gate, bias, dx1))
    heads = lambda t: t.view(1, N, N, H, D).permute(0, 1, 3, 2, 4)
    rows = lambda t: t.permute(0, 1, 3, 2, 4).reshape(1, N, N, C)

    # forward: q = k = v = the normalised stream
    _, y = evoattn.block_norm(xd, gamma_pre=dev["gamma_pre"], beta_pre=dev["beta_pre"])
    a = heads(y)
    u, lse = evoattn.fwd(a, a, a, bd)
    urows = rows(u).contiguous()
    x1, _ = evoattn.block_norm(xd, urows, gd, dev["scale"], dev["gamma_post"], dev["beta_post"], pre=False)
    # backward
    post = evoattn.block_norm_bwd(dd, u=urows, gate=gd, scale=dev["scale"],
                                  gamma_post=dev["gamma_post"], beta_post=dev["beta_post"])
    du = heads(post["du"]).contiguous()
    att = evoattn.bwd(a, a, a, bd, None, None, u, lse, du)
    dy = rows(att["dq"].float() + att["dk"].float() + att["dv"].float()).to(torch.bfloat16).contiguous()
    pre = evoattn.block_norm_bwd(post["dx"], dy, xd, gamma_pre=dev["gamma_pre"], beta_pre=dev["beta_pre"])
    assert evoattn.device_status() == evoattn.OK

    # the oracles, each fed by the one before
    oy = tr.block_norm(x, gamma_pre=prm["gamma_pre"], beta_pre=prm["beta_pre"])[1]
    on = heads(oy).contiguous().numpy()
    ou, _ = oracle.fwd(on, on, on, bias, None, None)
    ourows = rows(torch.from_numpy(np.asarray(ou)))
    branch = {n: prm[n] for n in ("scale", "gamma_post", "beta_post")}
    ox1 = tr.block_norm(x, ourows, gate, **branch, pre=False)[0]
    opost = tr.block_norm_bwd(dx1, u=ourows, gate=gate, **branch)
    odu = heads(opost["du"]).contiguous().numpy()
    oatt = oracle.bwd(on, on, on, bias, None, None, odu)
    ody = rows(torch.from_numpy(oatt["dq"] + oatt["dk"] + oatt["dv"]))
    opre = tr.block_norm_bwd(opost["dx"], ody, x, gamma_pre=prm["gamma_pre"])
    assert rel_l2(x1, ox1.numpy()) <= FWD_REL
    grads = {"scale": post["dscale"], "gamma_post": post["dgamma_post"], "beta_post": post["dbeta_post"],
             "gamma_pre": pre["dgamma_pre"], "beta_pre": pre["dbeta_pre"]}
    ograds = {n: (opost if n in branch else opre)["d" + n] for n in grads}
    for n in grads:
        assert rel_l2(grads[n], ograds[n].numpy()) <= 2 * GRAD_REL, n
    assert rel_l2(pre["dx"], opre["dx"].numpy()) <= 2 * GRAD_REL

    # the clipped step
    names = list(prm)
    opt = evoattn.AdamW([dev[n] for n in names], [grads[n] for n in names], lr=1e-2, weight_decay=0.1)
    norm = opt.step(max_norm=1.0)
    onorm = float(tr.grad_norm([ograds[n] for n in names]))
    assert float(norm) == pytest.approx(onorm, rel=2 * GRAD_REL)
    for n in names:
        zero = torch.zeros(C, dtype=torch.float64)
        want, _, _ = tr.adamw(prm[n], ograds[n], zero, zero, 1, 1e-2, (0.9, 0.999), 1e-8, 0.1,
                              min(1.0, 1.0 / (onorm + 1e-6)))
        sure = ograds[n].abs() > 10 * GRAD_REL * ograds[n].abs().mean()
        off = (dev[n].double().cpu() - want).abs()
        assert float(off[sure].max()) <= 1e-5 and int(sure.sum()) > C // 2, n
