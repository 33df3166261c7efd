"""The 8-bit projection path on the GPU against the float64 oracle
(oracle/eightbit.py).

Tolerances, per element, from the arithmetic (u = 2^-24, the half step of
fp32).  What is stored in bf16 is off by half a step, 2^-8 of its magnitude
(taken at the exact value plus the fp32 error before it).
Dropout: one multiplication by a factor that is itself rounded and one
addition: 4 u of the terms.  Norm: a row's sums are trees of depth below 32 and
the centred values are off by 32 u k, k = max|v| / sqrt(var + eps); with the
root, the affine map and the division 64 u (1 + k) of the largest terms of a row,
twice that where two normalised quantities are multiplied (gradients).  A code
is off by half a step of e4m3 in units of the scale, and a scale's exponent
differs only where the maximum is that near to the border.  A sum over rows
adds u times its depth, below 512 here.  Product: each MMA adds 32 exact products
to an fp32 sum, at worst truncating each to the largest term's last bit:
K 2^-23 of the sum of the magnitudes, and one more per piece of the sum and for
the addend."""
import pytest
import torch

from oracle import eightbit as eb
from protein_folding_attention_gb300 import evoattn

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": (torch.bfloat16, torch.bfloat16), "mixed": (torch.float32, torch.bfloat16),
         "f32": (torch.float32, torch.float32)}


def half(dtype):
    return torch.finfo(dtype).eps / 2


def d(t):
    return t.detach().double().cpu()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def draw(shape, dtype, g):
    C = shape[-1]
    return (torch.randn(shape, generator=g) * (0.5 + torch.rand(C, generator=g)) + torch.randn(C, generator=g)).to(dtype)


def laid(t, how):
    """The tensor on the device in another layout: dense, with the middle row
    axes swapped in memory, in rows wider than it, or at an odd address."""
    if how == "dense":
        return t.to(DEV)
    if how == "swapped":
        return t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    if how == "wide":
        full = torch.full((*t.shape[:-1], t.shape[-1] + 11), 7.0, dtype=t.dtype, device=DEV)
        full[..., 3:3 + t.shape[-1]] = t.to(DEV)
        return full[..., 3:3 + t.shape[-1]]
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)
    flat[1:] = t.reshape(-1).to(DEV)
    return flat[1:].view(t.shape)


def near(got, want, tol, what=""):
    off = (d(got) - want).abs()
    assert torch.isfinite(d(got)).all(), what
    worst = (off - tol).max()
    assert worst <= 0, f"{what}: beyond the tolerance by {float(worst):.3g} at {int((off - tol).argmax())}"


def stored(got, want, err, what=""):
    near(got, want, half(got.dtype) * (want.abs() + err) + err, what)


def rng(seed=11, step=5):
    return torch.tensor([seed, step], dtype=torch.int64, device=DEV)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
DROP = [((1, 1, 1, 1), (), "dense"), ((1, 1, 1, 128), (), "dense"), ((2, 3, 5, 8), (1,), "swapped"),
        ((1, 7, 9, 128), (1,), "dense"), ((1, 7, 9, 128), (2,), "swapped"), ((2, 4, 6, 99), (0, 2), "dense"),
        ((2, 4, 6, 99), (1,), "wide"), ((1, 3, 4, 200), (), "odd"), ((3, 2, 5, 1024), (0,), "dense"),
        ((1, 5, 1, 333), (0, 1, 2), "dense"), ((1, 2, 3, 4096), (), "dense"), ((1, 2, 300, 4), (2,), "dense"),
        ((2, 1, 130, 127), (1,), "swapped")]


@pytest.mark.parametrize("shape, shared, how", DROP)
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32, None])
@pytest.mark.parametrize("ut", [torch.bfloat16, torch.float32])
def test_dropout_add(shape, shared, how, xt, ut):
    g = gen(1)
    u = draw(shape, ut, g)
    x = None if xt is None else draw(shape, xt, g)
    mask = dict(p=0.3, seed=11, step=5, site=2, shared=shared)
    want = eb.dropped(u, **mask)
    size = want.abs()
    if x is not None:
        want, size = want + d(x), size + d(x).abs()
    got = evoattn.dropout_add(laid(u, how), 0.3, rng(), x=None if x is None else laid(x, how), site=2, shared=shared)
    assert got.dtype == (xt or ut)
    stored(got, want, 4 * U * size)
    if x is None:  # what is dropped is zero, and nothing else
        k = eb.keep(shape, 0.3, 11, 5, 2, shared).expand(shape)
        assert torch.equal(d(got) != 0, k & (d(u) != 0))


@pytest.mark.parametrize("seed, step, site", [(0, 0, 0), (-1, 2 ** 32 - 1, 2 ** 32 - 1), (2 ** 62 + 5, 2 ** 40 + 7, 1)])
def test_dropout_numbers(seed, step, site):
    shape = (1, 4, 5, 132)
    got = evoattn.dropout_add(torch.ones(shape, device=DEV), 0.5, rng(seed, step), site=site)
    assert torch.equal(d(got) != 0, eb.keep(shape, 0.5, seed, step, site))


@pytest.mark.parametrize("p", [0.0, 1e-12, 2.0 ** -32, 0.1, 0.999, 1 - 2.0 ** -40])
def test_dropout_probabilities(p):
    shape = (1, 4, 50, 264)
    u = torch.full(shape, 3.0, device=DEV)
    got = evoattn.dropout_add(u, p, rng() if p else None)
    want = eb.dropped(torch.full(shape, 3.0), p, 11, 5)
    near(got, want, 4 * U * want.abs())


def test_dropout_gradient_and_in_place():
    shape, mask = (2, 6, 7, 128), dict(site=9, shared=(1,))
    g = gen(2)
    u, x, dout = draw(shape, torch.bfloat16, g), draw(shape, torch.float32, g), draw(shape, torch.float32, g)
    out = evoattn.dropout_add(u.to(DEV), 0.25, rng(), x=x.to(DEV), **mask)
    # the gradient of the branch, in the branch's type: <dout, out(u) - x> = <du, u>
    du = evoattn.dropout_add(dout.to(DEV), 0.25, rng(), out_dtype=torch.bfloat16, **mask)
    want = eb.dropped(dout, 0.25, 11, 5, **mask)
    assert du.dtype is torch.bfloat16
    stored(du, want, 4 * U * want.abs())
    h = 2.0 ** -10  # the map is linear in u: a difference of any width is its derivative
    moved = d(evoattn.dropout_add((d(u) + h).to(DEV, torch.float32), 0.25, rng(), x=x.to(DEV), **mask))
    same = d(evoattn.dropout_add(d(u).to(DEV, torch.float32), 0.25, rng(), x=x.to(DEV), **mask))
    k = eb.keep(shape, 0.25, 11, 5, **mask).double() / 0.75
    assert ((moved - same - h * k).abs() <= 16 * U * (d(x).abs() + 2 * d(u).abs() + 1)).all()
    xd = x.to(DEV)
    assert evoattn.dropout_add(u.to(DEV), 0.25, rng(), x=xd, out=xd, **mask) is xd
    assert torch.equal(xd, out)
    ud = dout.to(DEV)
    evoattn.dropout_add(ud, 0.25, rng(), out=ud, **mask)
    stored(ud, want, 4 * U * want.abs())


def test_dropout_not_finite():
    u = torch.tensor([float("inf"), float("-inf"), float("nan"), 1.0] * 64, device=DEV).view(1, 1, 2, 128)
    got = evoattn.dropout_add(u, 0.5, rng())
    k = eb.keep((1, 1, 2, 128), 0.5, 11, 5)
    assert (d(got)[~k] == 0).all()
    assert torch.equal(torch.isnan(d(got)[k]), torch.isnan(d(u)[k]))


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------
def bits(t):
    return t.view(torch.uint8).cpu()


def same_codes(codes, want, what=""):
    """Codes against their values, a NaN code where the value is one."""
    got = d(codes)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got.nan_to_num(), want.nan_to_num()), what


def same_scales(scales, k, what=""):
    assert torch.equal(bits(scales).to(torch.int64) - 127, k), what


SIZES = [(1, 1), (1, 128), (3, 129), (128, 128), (129, 256), (200, 333), (5, 1000), (1000, 5), (257, 96), (64, 4104)]


@pytest.mark.parametrize("R, K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("how", ["dense", "wide", "odd"])
def test_quantize8(R, K, dtype, blocks, how):
    g = gen(R + K)
    x = (torch.randn(R, K, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))).to(dtype)
    xd = laid(x, how)
    q, s, qt, st = evoattn.quantize8(xd, cols=True, blocks=blocks)
    if blocks:
        want, k = eb.quantise_blocks(x)
        want_t, kt = want.t(), k.t()
    else:
        (want, k), (want_t, kt) = eb.quantise(x), eb.quantise(x.t())
    same_codes(q, want)
    same_codes(qt, want_t)
    same_scales(s, k)
    same_scales(st, kt)
    # one of the two alone
    for a, b in zip((*evoattn.quantize8(xd, blocks=blocks), *evoattn.quantize8(xd, rows=False, cols=True, blocks=blocks)),
                    (q, s, qt, st)):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("R, K", [(5000, 2000), (39000, 130), (130, 39000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize8_more_tiles_than_places(R, K, dtype):
    x = torch.randn(R, K, generator=gen(4)).to(dtype)
    x[R // 2, K - 1], x[R - 1, 0] = float("inf"), float("nan")
    for blocks in (False, True):
        q, s, qt, st = evoattn.quantize8(x.to(DEV), cols=True, blocks=blocks)
        want, k = eb.quantise_blocks(x) if blocks else eb.quantise(x)
        same_codes(q, want)
        same_scales(s, k)
        want, k = (want.t(), k.t()) if blocks else eb.quantise(x.t())
        same_codes(qt, want)
        same_scales(st, k)


def test_quantize8_values_at_the_edges():
    x = torch.zeros(16, 256)
    x[0, 0], x[0, 1] = 448.0, 2.0 ** -10                    # 2^-10 is a tie with zero
    x[1, 0], x[1, 1] = 448.0 * (1 + 2.0 ** -23), 3 * 2.0 ** -10
    x[2, 0], x[2, 1], x[2, 130] = float("inf"), 1.0, float("nan")
    x[3, :128] = float("nan")
    x[4, 0], x[4, 1] = 3.4028234663852886e38, -1.0
    x[5, 0], x[5, 1] = 1e-45, -1e-40                        # subnormal in fp32
    x[6, 0] = -0.0
    x[7, :128] = torch.linspace(-448, 448, 128)
    x[8, :128] = 2.0 ** -127 * 448 * (1 + 2.0 ** -10)
    x[9, 5], x[9, 200] = -7.0, -float("inf")
    for t in (x, x.bfloat16()):
        q, s, qt, st = evoattn.quantize8(t.to(DEV), cols=True)
        want, k = eb.quantise(t)
        same_codes(q, want)
        same_scales(s, k)
        want, k = eb.quantise(t.t())
        same_codes(qt, want)
        same_scales(st, k)
        q, s = evoattn.quantize8(t.to(DEV), blocks=True)
        want, k = eb.quantise_blocks(t)
        same_codes(q, want)
        same_scales(s, k)


def test_quantize8_leaves_what_is_not_its_own():
    """Bytes behind a row's end and behind the last row keep their values."""
    R, K = 131, 77
    x = torch.randn(R, K, generator=gen(3)).to(DEV)
    q, qt = (torch.full(n, 99, dtype=torch.uint8, device=DEV) for n in ((R + 2, 96), (K + 2, 160)))
    s, st = (torch.full(n, 55, dtype=torch.uint8, device=DEV) for n in ((3, R + 5), (3, K + 5)))
    lib = evoattn.load()
    assert lib.evoattn_quantize8(evoattn._PACK_QUANTIZE8(
        x.data_ptr(), R, K, K, evoattn.F32, 0, q.data_ptr(), 96, s.data_ptr(), 1, R + 5, qt.data_ptr(), 160,
        st.data_ptr(), 1, K + 5), torch.cuda.current_stream().cuda_stream) == evoattn.OK
    a, ka = eb.quantise(x)
    b, kb = eb.quantise(x.t())
    same_codes(q[:R, :K].view(torch.float8_e4m3fn), a)
    same_codes(qt[:K, :R].view(torch.float8_e4m3fn), b)
    assert (q[R:] == 99).all() and (q[:, K:] == 99).all() and (qt[K:] == 99).all() and (qt[:, R:] == 99).all()
    assert torch.equal(s[0, :R].cpu().long() - 127, ka[:, 0]) and torch.equal(st[:2, :K].t().cpu().long() - 127, kb)
    assert (s[:, R:] == 55).all() and (s[1:] == 55).all() and (st[:, K:] == 55).all() and (st[2:] == 55).all()


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
NORM = [((1, 1, 1, 1), "dense", ()), ((1, 1, 1, 128), "dense", ()), ((1, 3, 5, 64), "swapped", (1,)),
        ((2, 3, 5, 72), "dense", (2,)), ((1, 9, 8, 128), "swapped", (1,)), ((1, 5, 4, 130), "dense", ()),
        ((1, 5, 4, 99), "odd", (0,)), ((1, 6, 7, 256), "wide", (1, 2)), ((1, 6, 7, 384), "dense", ()),
        ((2, 2, 9, 513), "dense", (1,)), ((1, 3, 3, 768), "swapped", ()), ((1, 1, 37, 1000), "dense", ()),
        ((1, 2, 3, 1025), "dense", (2,)), ((1, 4, 5, 2048), "dense", ()), ((1, 2, 9, 4096), "dense", (1,)),
        ((1, 2, 3, 4093), "dense", ()), ((1, 1, 300, 8), "dense", (2,)), ((1, 1, 2, 3), "dense", ())]


def params(C, g, kind):
    gamma = 1.0 + 0.2 * torch.randn(C, generator=g)
    return gamma, (0.3 * torch.randn(C, generator=g) if kind == evoattn.NORM_LAYER else None)


def check_codes(codes, scales, y, err):
    """Codes and scales against y, which the kernel knows to within err."""
    s = torch.exp2((bits(scales).to(torch.int64) - 127).double())
    groups = eb._pad(y.abs(), -1).unflatten(-1, (-1, 128)).amax(-1)
    e = err.expand_as(y)[..., :1]
    k = bits(scales).to(torch.int64) - 127
    assert (eb.exponent((groups - e).clamp_min(0)) <= torch.where(groups > e, k, k.clamp_min(0))).all()
    assert (k <= eb.exponent(groups + e).clamp_min(0 if bool((groups <= e).any()) else -127)).all()
    s = s.repeat_interleave(128, -1)[..., :y.shape[-1]]
    near(d(codes) * s, y, eb.half_step((y.abs() + err) / s) * s + err, "codes")


@pytest.mark.parametrize("shape, how, shared", NORM)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("kind", [evoattn.NORM_LAYER, evoattn.NORM_RMS])
@pytest.mark.parametrize("branch", ["drop", "add", "none"])
def test_norm8(shape, how, shared, types, kind, branch):
    res, io = TYPES[types]
    g = gen(sum(shape))
    x, u = draw(shape, res, g), draw(shape, io, g)
    gamma, beta = params(shape[-1], g, kind)
    rms, p = kind == evoattn.NORM_RMS, 0.2 if branch == "drop" else 0.0
    mask = dict(p=p, seed=11, step=5, site=2, shared=shared)
    x1, y = eb.norm8(x, None if branch == "none" else u, gamma, beta, rms, **mask)
    xd = laid(x, how)
    got, codes, scales = evoattn.norm8(xd, None if branch == "none" else laid(u, how), gamma.to(DEV),
                                       None if beta is None else beta.to(DEV), kind=kind, p=p,
                                       rng=rng() if p else None, site=2, shared=shared if p else ())
    if branch == "none":
        assert got is xd
    else:
        stored(got, x1, 4 * U * (d(x).abs() + eb.dropped(u, **mask).abs()), "x1")
    h, r = eb.normalise(x1, rms, 1e-5)
    k = x1.abs().amax(-1, keepdim=True) * r
    terms = (h * gamma.double()).abs().amax(-1, keepdim=True) + (0 if beta is None else d(beta).abs().max())
    check_codes(codes, scales, y, 64 * U * (1 + k) * terms)


@pytest.mark.parametrize("shape", [(1, 1, 8000, 1032), (1, 1, 8000, 1030), (1, 1, 4200, 4096), (1, 70, 300, 128)])
@pytest.mark.parametrize("types", list(TYPES))
def test_norm8_many_rows(shape, types):
    """More rows than the kernel has places for: a sample of them."""
    res, io = TYPES[types]
    g = gen(12)
    x, u = draw(shape, res, g), draw(shape, io, g)
    gamma, beta = params(shape[-1], g, evoattn.NORM_LAYER)
    got, codes, scales = evoattn.norm8(x.to(DEV), u.to(DEV), gamma.to(DEV), beta.to(DEV))
    n = shape[1] * shape[2]
    rows = torch.cat([torch.arange(0, n, 41), torch.arange(n - 40, n)])
    pick = lambda t: t.reshape(1, 1, n, -1)[:, :, rows.to(t.device)]
    x1, y = eb.norm8(pick(x), pick(u), gamma, beta)
    stored(pick(got), x1, 4 * U * (d(pick(x)).abs() + d(pick(u)).abs()), "x1")
    h, r = eb.normalise(x1, False, 1e-5)
    k = x1.abs().amax(-1, keepdim=True) * r
    terms = (h * gamma.double()).abs().amax(-1, keepdim=True) + d(beta).abs().max()
    check_codes(pick(codes.view(torch.uint8)).view(torch.float8_e4m3fn),
                pick(scales.view(torch.uint8)).contiguous().view(torch.float8_e8m0fnu), y, 64 * U * (1 + k) * terms)


def test_norm8_without_parameters_and_in_place():
    g = gen(6)
    x, u = draw((1, 4, 5, 128), torch.float32, g), draw((1, 4, 5, 128), torch.bfloat16, g)
    x1, y = eb.norm8(x, u)
    xd = x.to(DEV)
    got, codes, scales = evoattn.norm8(xd, u.to(DEV), x1=xd)
    assert got is xd
    stored(xd, x1, 4 * U * (d(x).abs() + d(u).abs()))
    check_codes(codes, scales, y, 64 * U * (1 + y.abs().amax(-1, keepdim=True)) * y.abs().amax(-1, keepdim=True) * 2)


def test_norm8_rows_that_are_not_finite_spoil_themselves_alone():
    x = draw((1, 1, 6, 256), torch.float32, gen(7))
    clean = evoattn.norm8(x.to(DEV), kind=evoattn.NORM_RMS)
    x[0, 0, 1, 3], x[0, 0, 4, 200] = float("nan"), float("inf")
    _, codes, scales = evoattn.norm8(x.to(DEV), kind=evoattn.NORM_RMS)
    rows = [0, 2, 3, 5]
    assert torch.equal(bits(codes)[:, :, rows], bits(clean[1])[:, :, rows])
    assert torch.equal(bits(scales)[:, :, rows], bits(clean[2])[:, :, rows])
    assert torch.isnan(d(codes)[0, 0, 1]).all() and torch.isnan(d(codes)[0, 0, 4, 200])
    # constant rows: layer norm leaves beta
    _, codes, scales = evoattn.norm8(torch.full((1, 1, 3, 128), 5.0, device=DEV), beta=torch.full((128,), 2.0, device=DEV))
    assert (d(codes) * torch.exp2(bits(scales).double() - 127) == 2.0).all()


@pytest.mark.parametrize("shape, how, shared", NORM)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("kind", [evoattn.NORM_LAYER, evoattn.NORM_RMS])
@pytest.mark.parametrize("branch", ["drop", "add", "none"])
def test_norm8_bwd(shape, how, shared, types, kind, branch):
    res, io = TYPES[types]
    g = gen(sum(shape) + 1)
    dx1, dy, x1 = draw(shape, res, g), draw(shape, io, g), draw(shape, res, g)
    gamma, beta = params(shape[-1], g, kind)
    rms, p = kind == evoattn.NORM_RMS, 0.2 if branch == "drop" else 0.0
    mask = dict(p=p, seed=11, step=5, site=2, shared=shared)
    if branch == "add" and shape[-1] % 2:
        dx1 = None
    want = eb.norm8_bwd(dx1, dy, x1, gamma, rms, **mask)
    got = evoattn.norm8_bwd(None if dx1 is None else laid(dx1, how), laid(dy, how), laid(x1, how), gamma.to(DEV),
                            None if beta is None else beta.to(DEV), kind=kind, p=p, rng=rng() if p else None, site=2,
                            shared=shared if p else (), branch=branch != "none")
    assert set(got) == {"dx", "dgamma"} | ({"du"} if branch != "none" else set()) | ({"dbeta"} if beta is not None else set())
    h, r = eb.normalise(d(x1), rms, 1e-5)
    k = d(x1).abs().amax(-1, keepdim=True) * r
    e = (d(dy) * gamma.double()).abs()
    terms = r * (e + h.abs() * (e * h.abs()).mean(-1, keepdim=True) + e.mean(-1, keepdim=True))
    terms = (terms + (0 if dx1 is None else d(dx1).abs())).amax(-1, keepdim=True)
    err = 128 * U * (1 + k) * terms
    stored(got["dx"], want["dx"], err, "dx")
    if branch != "none":
        stored(got["du"], want["du"], err / (1 - p) * (want["du"] != 0), "du")
    rows = (0, 1, 2)
    near(got["dgamma"], want["dgamma"], ((512 + 64 * (1 + k)) * U * (d(dy) * h).abs().amax(-1, keepdim=True)
                                         .maximum((d(dy) * h).abs())).sum(rows), "dgamma")
    if beta is not None:
        near(got["dbeta"], want["dbeta"], 512 * U * d(dy).abs().sum(rows), "dbeta")


@pytest.mark.parametrize("shape", [(1, 130, 150, 128), (1, 100, 130, 131), (1, 40, 60, 1032), (1, 30, 30, 4093)])
@pytest.mark.parametrize("types", list(TYPES))
def test_norm8_bwd_many_rows_in_place_and_again(shape, types):
    """More rows than the kernel has places for; the same bits every time."""
    res, io = TYPES[types]
    g = gen(8)
    dx1, dy, x1 = draw(shape, res, g), draw(shape, io, g), draw(shape, res, g)
    gamma, beta = params(shape[-1], g, evoattn.NORM_LAYER)
    want = eb.norm8_bwd(dx1, dy, x1, gamma)
    args = dy.to(DEV), x1.to(DEV), gamma.to(DEV), beta.to(DEV)
    ws = torch.full((evoattn.load().evoattn_norm8_bwd_workspace_size(shape[-1]),), 255, dtype=torch.uint8, device=DEV)
    a = evoattn.norm8_bwd(dx1.to(DEV), *args)
    dd = dx1.to(DEV)
    b = evoattn.norm8_bwd(dd, *args, dx=dd, workspace=ws)
    assert b["dx"] is dd
    for n in a:
        assert torch.equal(a[n], b[n]), n
    h, r = eb.normalise(d(x1), False, 1e-5)
    k = d(x1).abs().amax(-1, keepdim=True) * r
    e = (d(dy) * gamma.double()).abs()
    terms = r * (e + h.abs() * (e * h.abs()).mean(-1, keepdim=True) + e.mean(-1, keepdim=True)) + d(dx1).abs()
    err = 128 * U * (1 + k) * terms.amax(-1, keepdim=True)
    stored(a["dx"], want["dx"], err, "dx")
    stored(a["du"], want["dx"], err, "du")
    for n, t in (("dgamma", d(dy) * h), ("dbeta", d(dy))):
        near(a[n], want[n], 1024 * U * t.abs().sum((0, 1, 2)), n)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------
def operand(R, K, seed, blocks=False, spread=2.0):
    """Codes and scales on the CPU, and what they stand for."""
    g = gen(seed)
    x = torch.randn(R, K, generator=g) * torch.exp(spread * torch.randn(R, 1, generator=g)) / K ** 0.5
    q, k = (eb.quantise_blocks if blocks else eb.quantise)(x)
    return q.to(torch.float8_e4m3fn), (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu), eb.values(q, k)


def codes_on_device(q, extra=0):
    R, K = q.shape
    full = torch.full((R, -(-K // 16) * 16 + extra), 0x7F, dtype=torch.uint8, device=DEV)  # NaN beside the rows
    full[:, :K] = q.view(torch.uint8).to(DEV)
    return full.view(torch.float8_e4m3fn)[:, :K]


def check_product(got, a, b, add=None):
    want, size = eb.matmul(a, b, add)
    stored(got, want, (a.shape[1] + 64) * 2.0 ** -23 * size)


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 700, 300), (3, 5, 16), (16, 129, 127), (17, 100, 129), (31, 516, 128),
          (33, 64, 1000), (64, 200, 640), (65, 256, 250), (128, 128, 4096), (129, 130, 131), (300, 516, 128),
          (513, 1, 300), (1000, 300, 72), (2, 3, 5000), (500, 8, 33), (300, 140, 256), (3000, 272, 700), (700, 257, 1024), (20, 300, 2100), (90, 260, 2176), (5, 40, 2048)]


@pytest.mark.parametrize("M, N, K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("blocks", [False, True])
def test_matmul8(M, N, K, dtype, blocks):
    qa, sa, a = operand(M, K, 1)
    qb, sb, b = operand(N, K, 2, blocks)
    got = evoattn.matmul8(codes_on_device(qa), sa.to(DEV), codes_on_device(qb, 32), sb.to(DEV), dtype)
    assert got.shape == (M, N) and got.dtype == dtype
    assert evoattn.device_status() == evoattn.OK
    check_product(got, a, b)


@pytest.mark.parametrize("M, N, K", [(4097, 1500, 1100), (2500, 1999, 1290), (3840, 1152, 1157), (20000, 240, 1281)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("extra", ["none", "blocks", "add"])
def test_matmul8_wide(M, N, K, dtype, extra):
    """Sizes that pairs of CTAs share, ragged in every direction: the values of a
    sample of rows (every row of the last tiles among them), and nothing beyond."""
    qa, sa, a = operand(M, K, 1)
    qb, sb, b = operand(N, K, 2, extra == "blocks")
    add = torch.randn(M, N, generator=gen(3)).to(dtype) if extra == "add" else None
    frame = torch.full((M + 1, N + 3), 5.0, dtype=dtype, device=DEV)
    out = frame[:M, :N]
    evoattn.matmul8(codes_on_device(qa), sa.to(DEV), codes_on_device(qb), sb.to(DEV), dtype,
                    add=None if add is None else add.to(DEV), out=out)
    assert evoattn.device_status() == evoattn.OK
    rows = torch.cat([torch.arange(0, M, 37), torch.arange(max(0, M - 260), M)])
    check_product(out[rows.to(DEV)], a[rows], b, None if add is None else add[rows])
    assert not torch.isnan(out).any()
    frame[:M, :N] = 5.0
    assert (frame == 5.0).all()


@pytest.mark.parametrize("M, N, K", [(1, 300, 500), (40, 129, 4000), (200, 516, 256), (700, 33, 100)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["full", "row", "in place", "wide"])
def test_matmul8_add_and_strides(M, N, K, dtype, kind):
    qa, sa, a = operand(M, K, 3, blocks=M % 2 == 0)
    qb, sb, b = operand(N, K, 4)
    add = torch.randn((N,) if kind == "row" else (M, N), generator=gen(5)).to(dtype)
    # scales whose rows are contiguous, and every second of a wider tensor
    sad = sa.view(torch.uint8).to(DEV).repeat_interleave(2, 1)[:, ::2].view(torch.float8_e8m0fnu)
    addd = add.to(DEV)
    out = None
    frame = torch.full((M + 2, N + 7), 5.0, dtype=dtype, device=DEV)
    if kind == "in place":
        out = addd
    elif kind == "wide":
        out = frame[1:M + 1, 3:N + 3]
        addd = torch.zeros((M, N + 5), dtype=dtype, device=DEV)[:, 1:N + 1].copy_(addd)
    got = evoattn.matmul8(codes_on_device(qa, 16), sad, codes_on_device(qb), sb.to(DEV), dtype, add=addd, out=out)
    assert out is None or got is out
    check_product(got, a, b, add)
    frame[1:M + 1, 3:N + 3] = 5.0
    assert (frame == 5.0).all()


def test_matmul8_leading_axes():
    x1, q, s = evoattn.norm8(torch.randn(2, 5, 7, 200, generator=gen(9)).to(DEV))
    qb, sb, b = operand(96, 200, 10)
    got = evoattn.matmul8(q, s, codes_on_device(qb), sb.to(DEV), torch.float32)
    assert got.shape == (2, 5, 7, 96)
    a = d(q) * torch.exp2(bits(s).double() - 127).repeat_interleave(128, -1)[..., :200]
    check_product(got.view(70, 96), a.reshape(70, 200), b)


def test_matmul8_values_at_the_edges():
    K = 256
    a = torch.zeros(20, K)
    a[0, 0], a[1, 200], a[2] = 448.0, -448.0, 2.0 ** -9
    a[4] = 448.0
    qa = a.to(torch.float8_e4m3fn)
    b = torch.zeros(130, K)
    b[0], b[1, 0], b[129] = 448.0, 2.0 ** -9, 448.0
    qb = b.to(torch.float8_e4m3fn)
    one = lambda R: torch.full((R, 2), 127, dtype=torch.uint8)
    run = lambda qa, sa, qb, sb: d(evoattn.matmul8(codes_on_device(qa), sa.view(torch.float8_e8m0fnu).to(DEV),
                                                   codes_on_device(qb), sb.view(torch.float8_e8m0fnu).to(DEV),
                                                   torch.float32))
    assert torch.equal(run(qa, one(20), qb, one(130)), a.double() @ b.double().t())   # every sum is exact
    # scales far apart, whose products are in range
    sa, sb = one(20), one(130)
    sa[0], sb[1], sb[0] = 254, 20, 10
    sa[1], sb[129] = 1, 200
    want = (a.double() * torch.exp2(sa[:, :1].double() - 127)) @ (b.double() * torch.exp2(sb[:, :1].double() - 127)).t()
    got = run(qa, sa, qb, sb)
    fits = want.abs() < 3.4e38
    assert ((got - want).abs()[fits] <= 2.0 ** -22 * want.abs()[fits] + 2.0 ** -126).all()
    # a NaN code or scale spoils its row or column alone
    bad = qa.view(torch.uint8).clone()
    bad[3, 7] = 0x7F
    got = run(bad.view(torch.float8_e4m3fn), one(20), qb, one(130))
    assert torch.isnan(got[3]).all() and int(torch.isnan(got).sum()) == 130
    sb = one(130)
    sb[5, 1] = 255
    got = run(qa, one(20), qb, sb)
    assert torch.isnan(got[:, 5]).all() and int(torch.isnan(got).sum()) == 20


@pytest.mark.parametrize("M, N, K", [(4, 300, 3000), (600, 200, 256), (64, 64, 20000), (2900, 1500, 1100)])
def test_matmul8_same_bits_and_streams(M, N, K):
    """Repeated, on two streams at once with workspaces of their own, and captured."""
    qa, sa, a = operand(M, K, 11)
    qb, sb, b = operand(N, K, 12)
    args = codes_on_device(qa), sa.to(DEV), codes_on_device(qb), sb.to(DEV), torch.float32
    want = evoattn.matmul8(*args)
    check_product(want, a, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[evoattn.matmul8(*args, stream=st) for st in streams] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for pair in outs for o in pair)
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(evoattn.matmul8(*args))
    for o in outs:
        o.zero_()
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert evoattn.device_status() == evoattn.OK


def test_matmul8_workspace():
    M, N, K = 4, 300, 3000
    need = evoattn.matmul8_workspace_size(M, N, K)
    assert need > 0 and evoattn.matmul8_workspace_size(4096, 4096, 128) == 0
    qa, sa, a = operand(M, K, 13)
    qb, sb, b = operand(N, K, 14)
    args = codes_on_device(qa), sa.to(DEV), codes_on_device(qb), sb.to(DEV), torch.float32
    for size in (need, need + 1000):
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        check_product(evoattn.matmul8(*args, workspace=ws), a, b)
    with pytest.raises(evoattn.EvoAttnError):
        evoattn.matmul8(*args, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(evoattn.EvoAttnError):  # rows of codes that do not start at 16 bytes
        evoattn.matmul8(args[0].contiguous()[:, :2990], args[1], args[2][:, :2990], args[3], torch.float32)


def test_matmul8_gives_up_and_recovers():
    """A wait that nothing ends: every CTA gives up, and the next call is right."""
    for M, N, K in ((300, 300, 700), (4, 300, 3000), (4097, 1200, 1300)):
        qa, sa, a = operand(M, K, 15)
        qb, sb, b = operand(N, K, 16)
        args = codes_on_device(qa), sa.to(DEV), codes_on_device(qb), sb.to(DEV), torch.float32
        assert evoattn.device_status() == evoattn.OK
        evoattn.debug_set_wait(50_000, stall=True)
        try:
            evoattn.matmul8(*args)
            status = evoattn.device_status()
        finally:
            evoattn.debug_set_wait(0, stall=False)
        assert status == evoattn.ERR_TIMEOUT
        check_product(evoattn.matmul8(*args), a, b)
        assert evoattn.device_status() == evoattn.OK


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def layer_step(x, u, gamma, beta, w, dout, state, p, shared):
    """A pre-norm layer in 8 bits, forwards and backwards, as a training step
    runs it: (x1, h) and the gradients of x, u, gamma, beta and w."""
    w8, ws, w8t, wst = evoattn.quantize8(w, cols=True, blocks=True)
    x1, y8, ys = evoattn.norm8(x, u, gamma, beta, p=p, rng=state, site=1, shared=shared)
    h = evoattn.matmul8(y8, ys, w8, ws)
    g8, gs, g8t, gst = evoattn.quantize8(dout, cols=True)
    dy = evoattn.matmul8(g8, gs, w8t, wst)
    _, y = evoattn.block_norm(x1, gamma_pre=gamma, beta_pre=beta)  # y again, along the other axis
    y8t, yst = evoattn.quantize8(y, rows=False, cols=True)
    dw = evoattn.matmul8(g8t, gst, y8t, yst, torch.float32)
    grads = evoattn.norm8_bwd(None, dy, x1, gamma, beta, p=p, rng=state, site=1, shared=shared)
    return x1, h, {**grads, "dw": dw}


def test_a_layer_as_it_is_used():
    """Against the formula in 64 bits: a relative error of the sums of the sizes
    that the roundings to e4m3 give.  A code is off by 2^-4 of itself at most,
    uniform within its step by 2^-4 / sqrt(3) at the bottom of a binade and half
    that at its top: below 0.027 in the root mean square.  h and dw have two factors
    rounded, the gradients behind the input's product three roundings at most:
    sqrt(3) * 0.027 = 0.047 where the errors do not cancel with the terms; dgamma
    multiplies by the norm's output, which x1's rounding to bf16 moves too."""
    g = gen(20)
    shape, N, p, shared = (1, 24, 40, 128), 192, 0.25, (1,)
    x, u = draw(shape, torch.bfloat16, g), draw(shape, torch.bfloat16, g)
    gamma, beta = params(128, g, evoattn.NORM_LAYER)
    w = torch.randn(N, 128, generator=g) / 128 ** 0.5
    dout = torch.randn(*shape[:3], N, generator=g).bfloat16()
    dev = [t.to(DEV) for t in (x, u, gamma, beta, w, dout)]
    state = rng()
    x1, h, got = layer_step(*dev, state, p, shared)
    mask = dict(p=p, seed=11, step=5, site=1, shared=shared)
    wx1, y = eb.norm8(x, u, gamma, beta, **mask)
    want_h = y @ w.double().t()
    dy = d(dout) @ w.double()
    want = eb.norm8_bwd(None, dy, wx1, gamma, **mask)
    want["dw"] = torch.einsum("bijn,bijc->nc", d(dout), y)
    rel = lambda a, b: float((d(a) - b).norm() / b.norm())
    assert rel(h, want_h) < 0.047
    for n in got:
        assert rel(got[n], want[n]) < 0.06, n
    # captured: the state on the device moves on between replays
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cx1, ch, cgot = layer_step(*dev, state, p, shared)
        state[1] += 1
    for step in (5, 6):
        graph.replay()
        torch.cuda.synchronize()
        ref = layer_step(*dev, rng(11, step), p, shared)
        assert torch.equal(cx1, ref[0]) and torch.equal(ch, ref[1])
        for n in got:
            assert torch.equal(cgot[n], ref[2][n]), n


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows against a call on them alone."""
    rows, C = (1 << 31) // 128 + 1000, 128
    u = torch.zeros((1, 1, rows, C), dtype=torch.bfloat16, device=DEV)
    tail = draw((1, 1, 600, C), torch.bfloat16, gen(21)).to(DEV)
    u[:, :, -600:] = tail
    out = evoattn.dropout_add(u, 0.25, rng(), out=torch.full_like(u, 3.0))
    first = rows - 600
    k = eb.philox(_counters(first, 600, C), (11, 0)).reshape(600, C)
    keep = torch.from_numpy(k >= 2 ** 30)
    want = torch.where(keep, d(tail[0, 0]) / 0.75, torch.zeros(1, dtype=torch.float64))
    stored(out[0, 0, -600:], want, 4 * U * want.abs())
    assert (out[0, 0, :1000] == 0).all()
    del out
    _, codes, scales = evoattn.norm8(u)
    alone = evoattn.norm8(tail.contiguous())
    assert torch.equal(bits(codes[0, 0, -600:]), bits(alone[1][0, 0])) and \
        torch.equal(bits(scales[0, 0, -600:]), bits(alone[2][0, 0]))
    q, s = evoattn.quantize8(u)
    ref = evoattn.quantize8(tail.contiguous())
    assert torch.equal(bits(q[0, 0, -600:]), bits(ref[0][0, 0])) and torch.equal(bits(s[0, 0, -600:]), bits(ref[1][0, 0]))
    qb, sb, b = operand(132, C, 22)
    w = codes_on_device(qb), sb.to(DEV)
    got = evoattn.matmul8(q, s, *w)
    want = evoattn.matmul8(ref[0], ref[1], *w)
    assert torch.equal(got[0, 0, -600:], want[0, 0])
    del got, q, s, codes, scales
    dx = evoattn.norm8_bwd(None, u, u, branch=False)["dx"]
    alone = evoattn.norm8_bwd(None, tail.contiguous(), tail.contiguous(), branch=False)["dx"]
    assert torch.equal(dx[0, 0, -600:], alone[0, 0])
    assert evoattn.device_status() == evoattn.OK


def _counters(first, rows, C):
    import numpy as np
    c = np.zeros((rows, C // 4, 4), dtype=np.uint64)
    c[..., 0] = np.arange(C // 4)[None]
    c[..., 1] = first + np.arange(rows)[:, None]
    c[..., 3] = 5
    return c
