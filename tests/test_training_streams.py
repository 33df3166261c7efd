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


NAMES = ("u", "gate", "scale", "gamma_post", "beta_post", "gamma_pre", "beta_pre")


def seam(device="cpu", rows=6):
    """x, and the block's operands and parameters by name."""
    gen = torch.Generator(device=device).manual_seed(3)
    draw = lambda *shape: torch.randn(shape, generator=gen, device=device)
    k = {"x": draw(1, rows, 4, 64).bfloat16()}
    for n in NAMES[:2]:
        k[n] = draw(1, rows, 4, 64).bfloat16()
    k.update({n: draw(64) for n in NAMES[2:]})
    return k


def test_norms_tell_their_tensors_of_the_stream(told):
    k = seam()
    rows = lambda: torch.empty_like(k["x"])
    evoattn.block_norm(**k)
    evoattn.block_norm_bwd(k["x"], k["x"], k["x"], *[k[n] for n in NAMES])
    evoattn.grad_norm([k["x"]])
    assert not told
    x1, y = rows(), rows()
    evoattn.block_norm(**k, x1=x1, y=y, stream=Side(1))
    assert addresses(x1, y, *k.values()) <= set(told[1])
    shared = k["gate"][:, :, :1].contiguous()   # (expanded to all rows)
    evoattn.block_norm(**{**k, "gate": shared}, stream=Side(2))
    assert addresses(shared) <= set(told[2])
    dx1, dy, dx, ws = rows(), rows(), rows(), torch.empty(64, dtype=torch.uint8)
    evoattn.block_norm_bwd(dx1, dy, x1, *[k[n] for n in NAMES], dx=dx, workspace=ws, stream=Side(3))
    # (beta_pre is not read by any kernel)
    assert addresses(dx1, dy, x1, dx, ws, *[k[n] for n in NAMES[:-1]]) <= set(told[3])
    one = k["gate"][:, :1].contiguous()
    evoattn.block_norm_bwd(dx1, dy, x1, k["u"], one.expand_as(x1), stream=Side(5))   # copied there
    assert addresses(one) <= set(told[5])
    gs = [torch.ones(5), torch.ones(9).bfloat16()]
    evoattn.grad_norm(gs, stream=Side(4))
    assert addresses(*gs) <= set(told[4])


@pytest.mark.gpu
def test_inputs_dropped_behind_a_busy_stream():
    """Operands that nobody holds after the call, their memory filled on the
    main stream while the side stream has not begun."""
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    k = seam("cuda", 512)
    want = evoattn.block_norm(**k)
    back = evoattn.block_norm_bwd(k["x"], k["x"], *want[:1], *[k[n] for n in NAMES])
    norm = evoattn.grad_norm([k["x"]])
    torch.cuda.synchronize()

    def call(run):
        """run(copies of the operands), which are dropped and written over."""
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        copies = {n: t.clone() for n, t in k.items()}
        copies["x1"] = want[0].clone()
        side.wait_stream(main)
        got = run(copies)
        copies.clear()
        junk = [torch.full_like(t, float("nan")) for t in k.values() for _ in range(2)]
        del junk
        torch.cuda.synchronize()
        return got
    got = call(lambda c: evoattn.block_norm(c["x"], *[c[n] for n in NAMES], stream=side))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = call(lambda c: evoattn.block_norm_bwd(c["x"], c["x"], c["x1"], *[c[n] for n in NAMES], stream=side))
    assert all(torch.equal(got[n], back[n]) for n in back)
    assert torch.equal(call(lambda c: evoattn.grad_norm([c["x"]], stream=side)), norm)


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
