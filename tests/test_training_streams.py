"""What the training calls do for a stream that is handed in: the memory that
their kernels read and write there must not be given away before they are done,
even where the caller drops a tensor right after the call.  Without a GPU the
calls are made on CPU tensors with a library that launches nothing, and the
tensors that are told of the stream are written down; with one, tensors are
dropped behind a busy stream and their memory is filled anew."""
import contextlib

import pytest
import torch

from protein_folding_attention_gb300 import evoattn


class Launches:
    """Stands in for the library: sizes of workspaces, and calls that do nothing."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("_size") else evoattn.OK


class Side:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def told(monkeypatch):
    """Addresses by stream of the tensors that were told of it."""
    told = {}
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, st: told.setdefault(st.cuda_stream, []).append(t.data_ptr()))
    monkeypatch.setattr(evoattn, "load", lambda: Launches())
    monkeypatch.setattr(evoattn, "_on_device", lambda t: t.get_device())
    monkeypatch.setattr(evoattn, "_raw_stream", lambda st, index: 0)
    monkeypatch.setattr(evoattn, "_allocate_on", lambda st: contextlib.nullcontext())
    return told


def addresses(*ts):
    return {t.data_ptr() for t in ts}


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_tells_every_tensor_of_the_stream(told, bits):
    ps = [torch.ones(300), torch.ones(7)]
    cs = [None, torch.ones(7).bfloat16()]
    gs, fresh = [[torch.ones(300), torch.ones(7)] for _ in range(2)]
    lr = torch.tensor(0.1)
    opt = evoattn.AdamW(ps, gs, copies=cs, lr=lr, state_bits=bits)
    opt.step()
    assert not told
    a, b = Side(1), Side(2)
    opt.step(max_norm=1.0, stream=a)
    kept = addresses(*ps, cs[1], opt.exp_avg, opt.exp_avg_sq, opt._state, opt._workspace)
    if bits == 8:
        kept |= addresses(opt.exp_avg_scale, opt.exp_avg_sq_scale)
    assert set(told[1]) == kept | addresses(*gs, lr)
    # new gradients, another stream, and both
    opt.step(grads=fresh, stream=a)
    assert addresses(*fresh) <= set(told[1])
    opt.step(stream=b)
    assert set(told[2]) == kept | addresses(*fresh, lr)
    told.clear()
    opt.step(grads=gs, stream=b)
    assert addresses(*gs) <= set(told[2])
    # a learning rate that takes the place of another
    opt.lr = torch.tensor(0.2)
    opt.step(stream=b)
    assert addresses(opt.lr) <= set(told[2])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_dropped_behind_a_busy_stream(bits):
    """Each step's gradients live until the next step binds others; their memory
    is then filled on the main stream while the side stream has not begun."""
    n, steps = 1 << 20, 4
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    ps = [torch.zeros(n, device="cuda") for _ in range(2)]
    first = torch.zeros(n, device="cuda")
    opt = evoattn.AdamW(ps[:1], [first], lr=0.1, state_bits=bits)
    twin = evoattn.AdamW(ps[1:], [first], lr=0.1, state_bits=bits)
    grads = [torch.full((n,), 1.0 + k, device="cuda") for k in range(steps)]
    torch.cuda.synchronize()
    for g in grads:
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        fresh = g.clone()
        side.wait_stream(main)
        opt.step(max_norm=1.0, grads=[fresh], stream=side)
        del fresh
        junk = [torch.full((n,), -1e3, device="cuda") for _ in range(3)]
        del junk
    for g in grads:
        twin.step(max_norm=1.0, grads=[g])
    torch.cuda.synchronize()
    assert torch.equal(*ps)
