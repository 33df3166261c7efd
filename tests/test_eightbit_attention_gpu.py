"""From the norm through the 8-bit product into the attention: which layout of
the projection's output the attention takes."""
import pytest
import torch

import oracle
from oracle import eightbit as eb
from protein_folding_attention_gb300 import evoattn

from helpers import FWD_REL, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_projection_into_attention():
    N, H, D, C = 48, 4, 32, 128
    HD, cols = H * D, 4 * H * D + H
    g = torch.Generator().manual_seed(41)
    x = torch.randn(1, N, N, C, generator=g).bfloat16().to(DEV)
    gamma, beta = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    w8, ws = evoattn.quantize8((torch.randn(cols, C, generator=g) / C ** 0.5).to(DEV), blocks=True)
    _, y8, ys = evoattn.norm8(x, None, gamma, beta)

    def heads(h):
        q, k, v, gate = (t.unflatten(-1, (H, D)).permute(0, 1, 3, 2, 4) for t in h[..., :4 * HD].split(HD, -1))
        return q, k, v, gate, h[..., 4 * HD:].permute(0, 3, 1, 2).contiguous()

    # rows that start at multiples of 16 bytes; the bias, whose heads lie innermost, dense
    frame = torch.zeros((1, N, N, cols + 7 & ~7), device=DEV, dtype=torch.bfloat16)
    h = evoattn.matmul8(y8, ys, w8, ws, out=frame[..., :cols])
    y, w = (eb.values(c.double().cpu().flatten(0, -2), s.cpu().view(torch.uint8).flatten(0, -2).long() - 127)
            for c, s in ((y8, ys), (w8, ws)))
    assert rel_l2(h.reshape(N * N, cols), eb.matmul(y, w)[0]) <= 2.0 ** -8
    assert (frame[..., cols:] == 0).all()
    q, k, v, gate, bias = heads(h)
    out, lse = evoattn.fwd(q, k, v, bias, None, gate)
    want, want_lse = oracle.fwd(*(t.cpu() for t in (q, k, v, bias)), None, gate.cpu())
    assert rel_l2(out, want) <= FWD_REL and rel_l2(lse, want_lse) <= FWD_REL
    assert evoattn.device_status() == evoattn.OK
    # the product's own output has rows of 516, of which the attention takes no views
    q, k, v, gate, bias = heads(evoattn.matmul8(y8, ys, w8, ws))
    with pytest.raises(evoattn.EvoAttnError) as refused:
        evoattn.fwd(q, k, v, bias, None, gate)
    assert refused.value.status == evoattn.ERR_ALIGNMENT
