"""AdamW over many tensors (32- and 8-bit states), the norm of all gradients
and the clipped step, on the GPU against the float64 oracle
(oracle/training.py).

Tolerances from the arithmetic (u = 2^-24, fp32's half step).  The first
moment is a sum of two products: three roundings of its terms, and the fp32
values of beta, 1 - beta and clip add one u each (the norm, summed in fp64
from short fp32 sums, adds a few): 16 u (|b1 m| + |(1-b1) g'|).  The second
moment likewise, its terms with twice the relative error.  The update
lr (m / c1) / (sqrt(v / c2) + eps) is a quotient of approximate operations of
a few u each: 64 u of its magnitude beside what m's own error (which may be
large against a cancelled m) gives; the parameter is rounded twice.  An 8-bit
value is the nearest e4m3 code: half a step of the format at that magnitude
(in units of the scale) beyond the fp32 error; its scale is max / 448."""
import math

import pytest
import torch

from oracle import training as tr
from protein_folding_attention_gb300 import evoattn

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
SIZES = [1, 3, 4, 255, 256, 257, 511, 2047, 2048, 2049, 5000, 40001]


def close(got, ref, tol, name):
    got = got.detach().double().cpu().reshape(-1)
    off = (got - ref.reshape(-1)).abs() - tol.reshape(-1)
    assert bool((off <= 0).all()), f"{name}: {float(off.max()):.3e} beyond the tolerance"


def make(sizes, seed, grad="bf16", shift=0, decades=1.0):
    """Parameters, gradients and copies; `shift`: elements by which each starts
    behind an aligned address."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cut = lambda n, dt: torch.empty(n + shift, device=DEV, dtype=dt)[shift:]
    ps, gs, cs = [], [], []
    for i, n in enumerate(sizes):
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}.get(grad) or \
            (torch.bfloat16 if i % 2 else torch.float32)
        p, g, c = cut(n, torch.float32), cut(n, dt), cut(n, torch.bfloat16)
        p.normal_(0, 0.02, generator=gen)
        r = torch.randn(n, device=DEV, generator=gen)
        g.copy_(r * torch.exp(decades * torch.randn(n, device=DEV, generator=gen)) * 1e-2)
        ps.append(p)
        gs.append(g)
        cs.append(c)
    return ps, gs, cs


def state_of(opt, i):
    """(m, v) of tensor i as float64, and the tensor's slices of the states."""
    n, at = opt.params[i].numel(), opt.offsets[i]
    m, v = opt.exp_avg[at:at + n].double(), opt.exp_avg_sq[at:at + n].double()
    if opt.state_bits == 8:
        blk = slice(at // 256, at // 256 + -(-n // 256))
        wide = lambda s: s[blk].double().repeat_interleave(256)[:n]
        m, v = m * wide(opt.exp_avg_scale), (v * wide(opt.exp_avg_sq_scale)) ** 2
    return m.cpu(), v.cpu()


def check_step(opt, t, old, clip, decay, lr=None):
    """The state after step t against the oracle's step from `old` (list of
    (p, m, v))."""
    lr = opt.lr if lr is None else lr
    for i, (p0, m0, v0) in enumerate(old):
        g = opt.grads[i].double().cpu().reshape(-1)
        p, m, v = tr.adamw(p0, g, m0, v0, t, lr, opt.betas, opt.eps, decay[i], clip)
        b1, b2 = opt.betas
        gc = g * clip
        em = 16 * U * ((b1 * m0).abs() + ((1 - b1) * gc).abs()) + 1e-37
        ev = 16 * U * (b2 * v0 + 2 * (1 - b2) * gc * gc) + 1e-37
        c1, c2 = 1 - b1 ** t, 1 - b2 ** t
        den = torch.sqrt(v / c2) + opt.eps
        upd = lr * (m / c1).abs() / den
        close(opt.params[i], p, 4 * U * p.abs() + 64 * U * upd + lr * em / c1 / den + 2 * U * p0.abs(),
              f"p {i}")
        if opt.copies[i] is not None:
            assert torch.equal(opt.copies[i], opt.params[i].to(torch.bfloat16))
        n, at = p.numel(), opt.offsets[i]
        if opt.state_bits == 32:
            close(opt.exp_avg[at:at + n], m, em, f"m {i}")
            close(opt.exp_avg_sq[at:at + n], v, ev, f"v {i}")
            continue
        root = torch.sqrt(v)
        for codes, scales, x, err in (
                (opt.exp_avg, opt.exp_avg_scale, m, em),
                (opt.exp_avg_sq, opt.exp_avg_sq_scale, root, ev / (2 * root).clamp_min(1e-30) + U * root)):
            blk = slice(at // 256, at // 256 + -(-n // 256))
            want = tr.block_scales(x)
            got = scales[blk].double().cpu()
            worst = torch.nn.functional.pad(err, (0, -n % 256)).view(-1, 256).amax(1)
            close(got, want, worst / 448 + 4 * U * want, f"scales {i}")
            unit = want.repeat_interleave(256)[:n].clamp_min(1e-300)
            code = codes[at:at + n].double().cpu()
            near = x / unit
            step = torch.maximum(tr.e4m3_step(near), tr.e4m3_step(code))
            slack = err / unit + 16 * U * near.abs()
            low = (x > 0) & (near < 2.0 ** -9) if codes is opt.exp_avg_sq else torch.zeros_like(x, dtype=torch.bool)
            assert bool((code[low] == 2.0 ** -9).all())
            close(code[~low], near[~low], (step / 2 + slack)[~low], f"codes {i}")


def remember(opt):
    return [(p.double().cpu().reshape(-1), *state_of(opt, i)) for i, p in enumerate(opt.params)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad,shift", [("bf16", 0), ("f32", 0), ("both", 0), ("both", 1), ("bf16", 3)])
@pytest.mark.parametrize("max_norm", [None, 0.5])
def test_steps_match_the_oracle(bits, grad, shift, max_norm):
    """Four steps over tensors from one element up, whole and ragged blocks,
    aligned and not, with and without clipping."""
    ps, gs, cs = make(SIZES, 1, grad, shift)
    cs[2] = None
    decay = [0.1 * (i % 3) for i in range(len(ps))]
    opt = evoattn.AdamW(ps, gs, copies=cs, lr=3e-3, betas=(0.9, 0.99), weight_decay=decay,
                        state_bits=bits)
    for t in range(1, 5):
        old = remember(opt)
        norm = opt.step(max_norm=max_norm)
        clip = 1.0
        if max_norm is not None:
            want = float(tr.grad_norm(gs))
            assert float(norm) == pytest.approx(want, rel=1e-6)
            clip = min(1.0, max_norm / (want + 1e-6))
            assert clip < 1.0
        check_step(opt, t, old, clip, decay)
        assert opt.steps_taken() == t
        for i, g in enumerate(gs):
            g.copy_(torch.randn(g.shape, generator=torch.Generator().manual_seed(100 * t + i)) * 0.01)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [1, 32, 33, 416, 417, 536, 537, 1100])
def test_many_tensors(bits, count):
    """Up to three launches, their tensors of 1 to 700 elements."""
    sizes = [(i * 37) % 700 + 1 for i in range(count)]
    ps, gs, cs = make(sizes, 2)
    opt = evoattn.AdamW(ps, gs, copies=cs, weight_decay=0.01, state_bits=bits)
    old = remember(opt)
    norm = opt.step(max_norm=1e-3)
    want = float(tr.grad_norm(gs))
    assert float(norm) == pytest.approx(want, rel=1e-6)
    check_step(opt, 1, old, 1e-3 / (want + 1e-6), [0.01] * count)
    assert opt.steps_taken() == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_empty_tensors_are_passed_over(bits):
    ps, gs, _ = make([0, 10, 0], 3)
    opt = evoattn.AdamW(ps, gs, weight_decay=0.0, state_bits=bits)
    old = remember(opt)
    opt.step(max_norm=100.0)
    check_step(opt, 1, old, 1.0, [0.0] * 3)
    ps, gs, _ = make([0], 3)
    opt = evoattn.AdamW(ps, gs, state_bits=bits)
    assert float(opt.step(max_norm=1.0)) == 0.0 and opt.steps_taken() == 1


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_bad_norm_skips_the_step(bits, bad):
    ps, gs, cs = make([300, 5000], 4)
    opt = evoattn.AdamW(ps, gs, copies=cs, state_bits=bits)
    opt.step(max_norm=1.0)
    keep = [t.clone() for t in ps + cs + [opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8)]]
    good = gs[1][4321].clone()
    gs[1][4321] = bad
    assert not math.isfinite(float(opt.step(max_norm=1.0)))
    now = ps + cs + [opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8)]
    assert all(torch.equal(a, b) for a, b in zip(keep, now)) and opt.steps_taken() == 1
    gs[1][4321] = good
    opt.step(max_norm=1.0)
    assert opt.steps_taken() == 2 and not torch.equal(keep[0], ps[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_only_decay(bits):
    ps, gs, _ = make([700], 5)
    gs[0].zero_()
    opt = evoattn.AdamW(ps, gs, lr=0.1, weight_decay=0.5, state_bits=bits)
    p0 = ps[0].double().cpu()
    opt.step()
    opt.step(max_norm=1.0)
    close(ps[0], p0 * 0.95 * 0.95, 4 * U * p0.abs(), "p")
    assert not bool(opt.exp_avg.float().any()) and not bool(opt.exp_avg_sq.float().any())


@pytest.mark.parametrize("grad,max_norm", [("bf16", None), ("f32", 0.5)])
@pytest.mark.parametrize("sizes", [SIZES, [700000]])
def test_codes_are_those_of_single_operations(grad, max_norm, sizes):
    """8-bit codes and scales are the bits that the formula gives in fp32 with
    every operation rounded by itself.  A root may be off by a last bit once in
    a million; a scale of the roots by that bit.  Zeros, gradients whose squares
    underflow, and large ones occur."""
    ps, gs, _ = make(sizes, 31, grad)
    for i, g in enumerate(gs):
        g.mul_([1.0, 1e-14, 1e5][i % 3])
        g[g.numel() // 2::7] = 0.0
    opt = evoattn.AdamW(ps, gs, lr=1e-3, betas=(0.9, 0.98), state_bits=8)
    ms = [torch.zeros(g.numel(), device=DEV) for g in gs]
    vs = [torch.zeros(g.numel(), device=DEV) for g in gs]
    b1, b2 = opt.betas

    def code(t):
        blocks = torch.nn.functional.pad(t, (0, -t.numel() % 256)).view(-1, 256)
        top = blocks.abs().amax(1, keepdim=True)
        held = top >= 2.0 ** -100
        inverse = torch.where(held, (1.0 / top) * 448.0, torch.zeros_like(top))
        scale = torch.where(held, top * torch.tensor(1 / 448, device=DEV), torch.zeros_like(top))
        return blocks, held, (blocks * inverse).to(torch.float8_e4m3fn).float(), scale

    for step in range(3):
        norm = opt.step(max_norm=max_norm)
        for i, g in enumerate(gs):
            n, at = g.numel(), opt.offsets[i]
            c = g.float()
            if max_norm is not None:
                c = c * torch.clamp(max_norm / (norm + 1e-6), max=1.0)
            m = b1 * ms[i] + (1.0 - b1) * c
            r = torch.sqrt(b2 * (vs[i] * vs[i]) + (1.0 - b2) * (c * c))
            for t, keep, held_in, codes, scales in ((m, ms, False, opt.exp_avg, opt.exp_avg_scale),
                                                    (r, vs, True, opt.exp_avg_sq, opt.exp_avg_sq_scale)):
                blocks, held, want, scale = code(t)
                if held_in:
                    want = torch.where((blocks > 0) & held & (want == 0), torch.full_like(want, 2.0 ** -9), want)
                got = scales[at // 256:at // 256 + scale.numel()].view(-1, 1)
                assert bool(((got - scale).abs() <= (2 * U * scale if held_in else 0 * scale)).all()), (step, i)
                assert torch.equal(codes[at:at + n].float(), want.reshape(-1)[:n]), (step, i)
                keep[i] = (want * got).reshape(-1)[:n]
            g.neg_().mul_(0.75)


def test_wide_range_inside_a_block():
    """Gradients over 12 decades inside a block: the smallest roots take the
    smallest positive code, so no later step divides by eps alone."""
    ps, gs, _ = make([512], 6, "f32")
    gs[0].copy_(10.0 ** torch.linspace(-12, 0, 512))
    opt = evoattn.AdamW(ps, gs, lr=1e-3, weight_decay=0.0, state_bits=8)
    for t in range(1, 4):
        old = remember(opt)
        opt.step()
        check_step(opt, t, old, 1.0, [0.0])
    assert bool((opt.exp_avg_sq.float() > 0).all())
    # the root is never understated, so a step is at most lr times the
    # ratio of corrected moments of a constant gradient, 1, and rounding
    assert float((ps[0].double().cpu() - old[0][0]).abs().max()) <= 1.2e-3


def test_repeats_bit_for_bit_and_leaves_padding_alone():
    out = []
    for _ in range(2):
        ps, gs, cs = make([1000, 30, 70000], 7)
        opt = evoattn.AdamW(ps, gs, copies=cs, state_bits=8)
        pad = torch.ones_like(opt.exp_avg, dtype=torch.bool)
        for p, at in zip(ps, opt.offsets):
            pad[at:at + p.numel()] = False
        mark = opt.exp_avg.view(torch.uint8)
        mark[pad] = 0x38
        for _ in range(3):
            opt.step(max_norm=0.1)
        assert bool((mark[pad] == 0x38).all())
        out.append([t.clone() for t in ps + cs + [mark, opt.exp_avg_sq.view(torch.uint8),
                                                  opt.exp_avg_scale, opt.norm]])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_resumes_from_given_states():
    ps, gs, _ = make([1000, 300], 8)
    a = evoattn.AdamW([p.clone() for p in ps], gs, state_bits=8)
    a.step(), a.step()
    b = evoattn.AdamW([p.clone() for p in a.params], gs, state_bits=8, exp_avg=a.exp_avg.clone(),
                      exp_avg_sq=a.exp_avg_sq.clone(), exp_avg_scale=a.exp_avg_scale.clone(),
                      exp_avg_sq_scale=a.exp_avg_sq_scale.clone(), step=a.steps_taken())
    a.step(), b.step()
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    assert torch.equal(a.exp_avg.view(torch.uint8), b.exp_avg.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_go_on_counting(bits):
    """A captured clipped step replays as the next step, with the step counter
    and the learning rate read on the device."""
    ps, gs, _ = make([3000, 77], 9)
    lr = torch.full((), 1e-2, device=DEV)
    twin = evoattn.AdamW([p.clone() for p in ps], gs, lr=1e-2, state_bits=bits)
    opt = evoattn.AdamW(ps, gs, lr=lr, state_bits=bits)
    twin.step(max_norm=0.3), opt.step(max_norm=0.3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(max_norm=0.3)
    for k in range(3):
        twin.lr = 1e-2 / (k + 1)
        lr.fill_(twin.lr)
        for g in gs:
            g.mul_(1.5)
        graph.replay()
        twin.step(max_norm=0.3)
        assert all(torch.equal(a, b) for a, b in zip(ps, twin.params))
    assert opt.steps_taken() == twin.steps_taken() == 4


def test_new_gradients_and_another_stream():
    ps, gs, _ = make([500, 900], 10)
    other = [g.float() * 2 for g in gs]
    a = evoattn.AdamW([p.clone() for p in ps], gs)
    b = evoattn.AdamW([p.clone() for p in ps], other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(grads=other, max_norm=1.0, stream=side)
    a.step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.step(max_norm=1.0), b.step()
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


def test_many_steps_taken():
    """Bias corrections far into a run, and at beta = 0."""
    for betas, step in (((0.9, 0.999), 999_999), ((0.0, 0.999), 0), ((0.9, 0.0), 3), ((0.99, 0.9999), 12)):
        ps, gs, _ = make([600], 11)
        opt = evoattn.AdamW(ps, gs, betas=betas, step=step)
        old = remember(opt)
        opt.step()
        check_step(opt, step + 1, old, 1.0, [0.01])


def test_more_elements_than_32_bits_count():
    """One tensor of 2^31 + 300 elements in 8-bit states: its last block."""
    n = 2 ** 31 + 300
    p = torch.full((n,), 1.0, device=DEV)
    g = torch.full((n,), 0.5, device=DEV, dtype=torch.bfloat16)
    g[-3:] = -0.25
    opt = evoattn.AdamW([p], [g], lr=0.125, weight_decay=0.0, state_bits=8)
    norm = opt.step(max_norm=math.inf)
    assert float(norm) == pytest.approx(math.sqrt(0.25 * (n - 3) + 3 / 16), rel=1e-6)
    want = torch.full((300,), 0.875)
    want[-3:] = 1.125
    close(p[-300:], want.double(), torch.full((300,), 1e-5, dtype=torch.float64), "p")
    assert float(p[:2 ** 20].double().sub(0.875).abs().max()) < 1e-5
    assert float(p[2 ** 31 - 5:2 ** 31 + 5].double().sub(0.875).abs().max()) < 1e-5


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_alone(grad, shift):
    for sizes in ([1], [8192], [8191, 3, 100000], [5] * 900, [3] * 1408, [3] * 1409, [3_000_001]):
        _, gs, _ = make(sizes, 12, grad, shift)
        got = evoattn.grad_norm(gs)
        assert float(got) == pytest.approx(float(tr.grad_norm(gs)), rel=1e-6)
        assert torch.equal(got, evoattn.grad_norm(gs))


def test_python_refusals():
    ps, gs, cs = make([100, 200], 13)
    ok = lambda **kw: evoattn.AdamW(**{**dict(params=ps, grads=gs), **kw})
    ok()
    for bad in (dict(params=[]), dict(grads=gs[:1]), dict(copies=cs[:1]), dict(weight_decay=[0.1]),
                dict(state_bits=16), dict(params=[ps[0].half(), ps[1]]), dict(params=[ps[0], ps[0][:200]]),
                dict(params=[ps[0], ps[0]], grads=[gs[0], gs[0]]), dict(grads=[gs[0].half(), gs[1]]),
                dict(grads=[gs[1], gs[0]]), dict(copies=[cs[0].float(), None]),
                dict(exp_avg=torch.zeros(511, device=DEV)), dict(exp_avg_scale=torch.zeros(2, device=DEV)),
                dict(params=[p.expand(2, -1) for p in ps], grads=[g.expand(2, -1) for g in gs]),
                dict(params=[torch.zeros(200, device=DEV)[::2], ps[1]]),
                dict(grads=[ps[0], gs[1]]), dict(grads=[gs[0], cs[1]], copies=cs)):
        with pytest.raises(ValueError):
            ok(**bad)
    opt = ok()
    with pytest.raises(ValueError):
        opt.step(grads=gs[:1])
    with pytest.raises(evoattn.EvoAttnError):
        opt.step(max_norm=0.0)
    opt.lr = float("nan")
    with pytest.raises(evoattn.EvoAttnError):
        opt.step()
    with pytest.raises(ValueError):
        evoattn.grad_norm([gs[0].half()])


def test_refused_gradients_leave_the_old_ones_bound():
    """New gradients of which a later one is refused replace none."""
    ps, gs, _ = make([300, 500], 21)
    other = [p.clone() for p in ps]
    a, b = evoattn.AdamW(ps, gs), evoattn.AdamW(other, gs)
    fresh = [torch.ones_like(gs[0]), torch.ones(499, device=DEV)]
    with pytest.raises(ValueError):
        a.step(grads=fresh)
    a.step(), b.step()
    assert all(torch.equal(x, y) for x, y in zip(ps, other))
    assert a.grads[0] is gs[0] and a.steps_taken() == 1


def test_roots_are_rounded_to_nearest_beside_any_values():
    """The scale of a block's roots is its largest root / 448: for roots of
    every exponent from 2^-50 to 2^50 and 80,000 mantissas, beside values as
    large, zeros, and values outside the range of the step's own root, it is
    the bits that the correctly rounded root gives."""
    n, b2 = 80_000, 0.9
    gen = torch.Generator().manual_seed(42)
    top = ((1.0 + torch.rand(n, generator=gen)) * 2.0 ** (torch.arange(n) % 101 - 50).float()).to(DEV)
    beside = torch.tensor([0.5, 0.0, 2.0 ** -60, 1.0], device=DEV)[torch.arange(n, device=DEV) // 101 % 4]
    g = (top * beside)[:, None].repeat(1, 256)
    g[:, 5] = top
    opt = evoattn.AdamW([torch.zeros(n, 256, device=DEV)], [g], betas=(0.9, b2), state_bits=8)
    opt.step()
    f = lambda x: torch.tensor(x, dtype=torch.float32, device=DEV)
    v = f(1.0 - b2) * (top * top)     # in fp32, the old v being zero
    root = torch.sqrt(v.double()).float()   # (53 bits are enough to round a root of 24 bits right)
    assert torch.equal(opt.exp_avg_sq_scale, root * f(1 / 448))


@pytest.mark.parametrize("bits", [32, 8])
def test_second_moments_below_the_normal_range(bits):
    """An eps that is small against the root of a subnormal v: the root is not
    taken as zero (the quotient would be m / eps).  v = (1 - beta2) g^2 is off
    by half a unit 2^-149 for each of its two products, the quotient by half of
    that relatively, beside its own 64 u."""
    n = 1000
    gen = torch.Generator().manual_seed(41)
    g = ((1.0 + 3.0 * torch.rand(n, generator=gen)) * 1e-19 *
         (1 - 2 * torch.randint(0, 2, (n,), generator=gen))).to(DEV)
    p = torch.zeros(n, device=DEV)
    opt = evoattn.AdamW([p], [g], lr=1e-3, betas=(0.9, 0.999), eps=1e-30, weight_decay=0.0, state_bits=bits)
    opt.step()
    zero = torch.zeros(n, dtype=torch.float64)
    want, _, v = tr.adamw(zero, g, zero, zero, 1, 1e-3, (0.9, 0.999), 1e-30, 0.0)
    assert float(v.max()) < 2.0 ** -126
    close(p, want, (64 * U + 2.0 ** -149 / v) * want.abs(), "p")
