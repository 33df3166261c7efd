"""The block norm and its gradients (evoattn_block_norm, _bwd) on the GPU
against the float64 oracle (oracle/training.py).

Tolerances, per element, from the arithmetic (u = 2^-24, the half step of
fp32): a stored bf16 value is off by half a step, 2^-8 of its magnitude, and
before it is rounded by the fp32 arithmetic.  A row's mean is a sum in a tree
of depth at most 8 + 5 + 16 additions (a thread's channels, a warp, the warps
of a row), so it is off by 29 u max|v|, which after the division by the
standard deviation is 29 u k with k = max|v| rstd; the variance, its root, the
affine map and the sigmoid add a few u each.  64 u (1 + k) times the largest
magnitude of the terms that are added bounds all of it, and a gradient, which
multiplies two normalised quantities, takes twice that.  A sum over rows adds
u times its depth (rows of a thread, groups of a CTA, CTAs: below 256 here)
times the sum of the magnitudes."""
import itertools

import pytest
import torch

from oracle import training as tr
from protein_folding_attention_gb300 import evoattn

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": (torch.bfloat16, torch.bfloat16), "mixed": (torch.float32, torch.bfloat16),
         "f32": (torch.float32, torch.float32)}
PARAMS = ("scale", "gamma_post", "beta_post", "gamma_pre", "beta_pre")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def draw(shape, types, gate="full", post=True, pre=True, params=PARAMS, seed=0, backward=False):
    """Seeded CPU inputs: channels with an offset and a scale of their own."""
    res, io = TYPES[types]
    gen = torch.Generator().manual_seed(seed)
    C = shape[3]
    rows = lambda dt: (torch.randn(shape, generator=gen) * (0.5 + torch.rand(C, generator=gen)) +
                       torch.randn(C, generator=gen)).to(dt)
    vec = lambda mean: mean + 0.2 * torch.randn(C, generator=gen)
    k = {"u": None, "gate": None}
    if post:
        k["u"] = rows(io)
        if gate != "none":
            b, i, j, _ = shape
            gs = {"full": shape, "row": (b, i, 1, C), "batch": (b, 1, 1, C), "all": (1, 1, 1, C),
                  "middle": (b, 1, j, C), "column": (1, i, j, C)}[gate]
            k["gate"] = torch.randn(gs, generator=gen).to(io)
    for name, mean in zip(PARAMS, (0.5, 1.0, 0.0, 1.0, 0.0)):
        on = (post if name in PARAMS[:3] else pre) and name in params
        k[name] = vec(mean) if on else None
    if backward:
        k["dx1"] = rows(res)
        k["dy"] = rows(io) if pre else None
        k["x1"] = rows(res) if pre else None
    else:
        k["x"] = rows(res)
    return k


def to_gpu(k):
    return {n: (None if t is None else t.to(DEV)) for n, t in k.items()}


def kappa(v, rms, eps=1e-5):
    v = v.double()
    return float((v.abs().amax(-1, keepdim=True) * tr.normalise(v, rms, eps)[1]).max())


def close(got, ref, tol, name):
    got = got.detach().double().cpu()
    off = ((got - ref).abs() - tol)
    assert got.shape == ref.shape and bool((off <= 0).all()), \
        f"{name}: {float((got - ref).abs().max()):.3e} off, {float(off.max()):.3e} beyond the tolerance"


def amax(*ts):
    return max([1.0] + [float(t.abs().max()) for t in ts if t is not None])


def check_fwd(k, x1, y, rms):
    rx1, ry = tr.block_norm(**{n: k[n] for n in ("x", "u", "gate") + PARAMS}, rms=rms,
                            pre=y is not None)
    kx = 1.0
    if k["u"] is not None:
        kx += kappa(k["u"], rms)
    branch = 64 * U * kx * kx * amax(k["scale"]) * (amax(k["gamma_post"]) + amax(k["beta_post"]))
    if k["u"] is not None:
        close(x1, rx1, half(x1.dtype) * rx1.abs() + branch + 4 * U * rx1.abs(), "x1")
    if y is not None:
        r = tr.normalise(rx1, rms, 1e-5)[1]
        ky = kappa(rx1, rms)
        tol = 64 * U * (1 + ky) ** 2 * amax(k["gamma_pre"]) + 2 * (branch if k["u"] is not None else 0) * (
            1 + ky) * float(r.max()) * amax(k["gamma_pre"])
        close(y, ry, half(y.dtype) * ry.abs() + tol + 4 * U * amax(k["beta_pre"]), "y")


def check_bwd(k, got, rms):
    names = ("dx1", "dy", "x1", "u", "gate", "scale", "gamma_post", "beta_post", "gamma_pre")
    ref = tr.block_norm_bwd(**{n: k[n] for n in names}, rms=rms)
    rows = tuple(range(3))
    D = ref["dx"]
    err_D = torch.zeros_like(D)
    if k["dy"] is not None:
        h, r = tr.normalise(k["x1"].double(), rms, 1e-5)
        kx = 1 + kappa(k["x1"], rms)
        a = k["dy"].double().abs() * (1.0 if k["gamma_pre"] is None else k["gamma_pre"].double().abs())
        size = r * (a.amax(-1, keepdim=True) * (1 + h.abs().amax(-1, keepdim=True) ** 2))
        err_D = 128 * U * kx * size + 4 * U * D.abs()
        close(got["dx"], D, half(got["dx"].dtype) * D.abs() + err_D, "dx")
        dy = k["dy"].double()
        if k["gamma_pre"] is not None:
            mass = (dy * h).abs().sum(rows)
            close(got["dgamma_pre"], ref["dgamma_pre"],
                  U * (256 * mass + 64 * kx * dy.abs().sum(rows) * (1 + h.abs().amax())), "dgamma_pre")
        if k["beta_pre"] is not None:
            close(got["dbeta_pre"], ref["dbeta_pre"], 256 * U * dy.abs().sum(rows) + 1e-30, "dbeta_pre")
    if k["u"] is None:
        return
    h, r = tr.normalise(k["u"].double(), rms, 1e-5)
    ku = 1 + kappa(k["u"], rms)
    one = torch.ones(k["u"].shape[-1], dtype=torch.float64)
    s = one if k["scale"] is None else k["scale"].double()
    g1 = one if k["gamma_post"] is None else k["gamma_post"].double()
    b1 = 0 * one if k["beta_post"] is None else k["beta_post"].double()
    w = h * g1 + b1
    werr = 64 * U * ku * (1 + h.abs()) * g1.abs() + 4 * U * b1.abs()
    q = torch.ones_like(h) if k["gate"] is None else torch.sigmoid(k["gate"].double()).expand_as(h)
    dabs = D.abs()
    if k["scale"] is not None:
        term = (D * q * w).abs()
        close(got["dscale"], ref["dscale"],
              (256 * U * term + err_D * (q * w).abs() + dabs * q * (werr + 64 * U * w.abs())).sum(rows) + 1e-30,
              "dscale")
    e = dabs * s.abs() * q
    err_e = err_D * s.abs() * q + 64 * U * e
    if k["gate"] is not None:
        term = e * w.abs() * (1 - q)
        err = err_e * w.abs() * (1 - q) + e * werr * (1 - q) + 64 * U * e * w.abs()
        if k["gate"].shape != k["u"].shape:
            over = [i for i in rows if k["gate"].shape[i] == 1]
            term, err = term.sum(over, keepdim=True), err.sum(over, keepdim=True)
        close(got["dgate"], ref["dgate"],
              half(got["dgate"].dtype) * ref["dgate"].abs() + err + 256 * U * term + 1e-30, "dgate")
    if k["gamma_post"] is not None:
        close(got["dgamma_post"], ref["dgamma_post"],
              (256 * U * e * h.abs() + err_e * h.abs() + 64 * U * ku * e * (1 + h.abs())).sum(rows) + 1e-30,
              "dgamma_post")
    if k["beta_post"] is not None:
        close(got["dbeta_post"], ref["dbeta_post"], (256 * U * e + err_e).sum(rows) + 1e-30, "dbeta_post")
    b, err_b = e * g1.abs(), err_e * g1.abs()
    big = lambda t: t.amax(-1, keepdim=True)
    size = r * big(b) * (1 + big(h.abs()) ** 2)
    err = r * big(err_b) * (1 + big(h.abs()) ** 2) + 128 * U * ku * size
    close(got["du"], ref["du"], half(got["du"].dtype) * ref["du"].abs() + err, "du")


BWD_ARGS = ("dx1", "dy", "x1", "u", "gate") + PARAMS


def run_fwd(k, rms, **kw):
    g = to_gpu(k)
    return evoattn.block_norm(g["x"], *[g[n] for n in ("u", "gate") + PARAMS],
                              kind=evoattn.NORM_RMS if rms else evoattn.NORM_LAYER, **kw)


def run_bwd(k, rms, **kw):
    g = to_gpu(k)
    return evoattn.block_norm_bwd(*[g[n] for n in BWD_ARGS],
                                  kind=evoattn.NORM_RMS if rms else evoattn.NORM_LAYER, **kw)


WIDTHS = [1, 2, 7, 8, 31, 32, 33, 64, 72, 99, 128, 200, 256, 257, 264, 384, 500, 509, 768, 1000, 1001, 1024, 1032, 1600,
          2048, 2056, 3000, 4000, 4095, 4096]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("types,rms", [("bf16", False), ("bf16", True), ("mixed", False), ("f32", True)])
def test_widths(C, types, rms):
    """Every way a row is laid over threads, whole and ragged."""
    shape = (1, 3, 11, C)
    k = draw(shape, types, seed=C)
    x1, y = run_fwd(k, rms)
    check_fwd(k, x1, y, rms)
    k = draw(shape, types, seed=C + 1, backward=True)
    check_bwd(k, run_bwd(k, rms), rms)


@pytest.mark.parametrize("shape", [(1, 1, 1, 128), (1, 1, 2, 128), (3, 5, 7, 64), (2, 67, 129, 40),
                                   (1, 150, 150, 128), (2, 1, 513, 384), (1, 40, 1, 1000)])
@pytest.mark.parametrize("gate", ["none", "full", "row", "batch", "all", "middle", "column"])
def test_shapes_and_shared_gates(shape, gate):
    """One row to several per group of threads; gates shared along any axes."""
    k = draw(shape, "bf16", gate, seed=7)
    x1, y = run_fwd(k, False)
    check_fwd(k, x1, y, False)
    k = draw(shape, "bf16", gate, seed=8, backward=True)
    check_bwd(k, run_bwd(k, False), False)


@pytest.mark.parametrize("C", [8, 33, 99, 136, 256, 300, 384, 511, 520, 777, 1096, 2056, 4088])
@pytest.mark.parametrize("types,gate", [("bf16", "row"), ("mixed", "batch"), ("f32", "middle"),
                                        ("f32", "row"), ("mixed", "none")])
def test_widths_with_shared_gates(C, types, gate):
    """Every way a row is laid over threads, gate rows shared by a few rows (a
    group walks them) and by many (spread over a CTA)."""
    for shape in ((2, 3, 5, C), (1, 2, 75, C)):
        k = draw(shape, types, gate, seed=C)
        x1, y = run_fwd(k, C % 2 == 0)
        check_fwd(k, x1, y, C % 2 == 0)
        k = draw(shape, types, gate, seed=C + 1, backward=True)
        check_bwd(k, run_bwd(k, C % 2 == 0), C % 2 == 0)


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("post,pre", [(True, False), (False, True)])
@pytest.mark.parametrize("C,gate", [(128, "full"), (50, "row"), (512, "none"), (300, "batch")])
def test_one_norm_alone(types, post, pre, C, gate):
    shape = (2, 9, 5, C)
    k = draw(shape, types, gate, post, pre, seed=1)
    kw = {} if post else {"y_dtype": TYPES[types][1]}
    x1, y = run_fwd(k, True, pre=pre, **kw)
    assert (y is None) == (not pre)
    check_fwd(k, x1, y, True)
    k = draw(shape, types, gate, post, pre, seed=2, backward=True)
    got = run_bwd(k, True)
    check_bwd(k, got, True)
    if not pre:
        assert torch.equal(got["dx"].cpu(), k["dx1"])


@pytest.mark.parametrize("keep", [s for r in range(3) for s in itertools.combinations(PARAMS, r)])
def test_absent_parameters(keep):
    shape = (1, 4, 9, 96)
    k = draw(shape, "mixed", "row", params=keep, seed=3)
    x1, y = run_fwd(k, False)
    check_fwd(k, x1, y, False)
    k = draw(shape, "mixed", "row", params=keep, seed=4, backward=True)
    got = run_bwd(k, False)
    check_bwd(k, got, False)
    assert set(got) == {"dx", "du", "dgate"} | {"d" + n for n in keep}


def test_no_gradient_on_the_stream():
    k = draw((1, 6, 10, 128), "bf16", seed=5, backward=True)
    k["dx1"] = None
    check_bwd(k, run_bwd(k, False), False)


def _views(k):
    """The same values as views: (i, j) transposed, channels cut from wider
    rows at an offset that is not 16-byte aligned, every second row."""
    def transposed(t):
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    def cut(t):
        wide = torch.zeros(*t.shape[:3], t.shape[3] + 5, dtype=t.dtype)
        wide[..., 3:3 + t.shape[3]] = t
        return wide[..., 3:3 + t.shape[3]]

    def sparse(t):
        wide = torch.zeros(t.shape[0], t.shape[1], 2 * t.shape[2], t.shape[3], dtype=t.dtype)
        wide[:, :, ::2] = t
        return wide[:, :, ::2]
    return [transposed, cut, sparse]


@pytest.mark.parametrize("C", [128, 384])
@pytest.mark.parametrize("gate", ["full", "row"])
def test_strides(C, gate):
    """Operands in different layouts, each against the same values."""
    shape = (2, 10, 6, C)
    for seed, order in enumerate(itertools.permutations(_views(None))):
        move = lambda t, f: f(t).to(DEV) if f is order[0] else _keep(f(t))
        k = draw(shape, "bf16", gate, seed=20 + seed)
        g = to_gpu(k)
        g["x"], g["u"] = move(k["x"], order[0]), move(k["u"], order[1])
        if gate == "full":
            g["gate"] = move(k["gate"], order[2])
        x1, y = evoattn.block_norm(g["x"], *[g[n] for n in ("u", "gate") + PARAMS])
        check_fwd(k, x1, y, False)
        k = draw(shape, "bf16", gate, seed=40 + seed, backward=True)
        g = to_gpu(k)
        for n, f in zip(("dx1", "dy", "x1", "u"), order + (order[0],)):
            g[n] = move(k[n], f)
        check_bwd(k, evoattn.block_norm_bwd(*[g[n] for n in BWD_ARGS]), False)


def _keep(t):
    """The view on the GPU with the same strides and the same offset."""
    base = t if t._base is None else t._base
    return base.to(DEV).as_strided(t.size(), t.stride(), t.storage_offset())


def test_outputs_as_views_leave_the_rest_alone():
    shape = (1, 5, 7, 64)
    k = draw(shape, "bf16", seed=9)
    g = to_gpu(k)
    wide = torch.full((1, 5, 9, 80), 7.0, device=DEV, dtype=torch.bfloat16)
    both = torch.full((2, 1, 5, 7, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    x1, y = evoattn.block_norm(g["x"], *[g[n] for n in ("u", "gate") + PARAMS],
                               x1=wide[:, :, 1:8, 8:72], y=both[1])
    check_fwd(k, x1, y, False)
    assert bool((both[0] == 7).all())
    wide[:, :, 1:8, 8:72] = 7.0
    assert bool((wide == 7).all())


def test_repeated_input_rows():
    """Inputs whose rows repeat by a stride of 0 (a broadcast stream)."""
    k = draw((2, 1, 1, 128), "bf16", "none", seed=10)
    big = draw((2, 6, 5, 128), "bf16", "full", seed=11)
    big["x"] = k["x"].expand(2, 6, 5, 128)
    g = to_gpu(big)
    g["x"] = k["x"].to(DEV).expand(2, 6, 5, 128)
    x1, y = evoattn.block_norm(g["x"], *[g[n] for n in ("u", "gate") + PARAMS])
    check_fwd(big, x1, y, False)
    b = draw((2, 6, 5, 128), "bf16", "full", seed=12, backward=True)
    b["dx1"] = k["x"].expand(2, 6, 5, 128)
    b["gate"] = k["x"].expand(2, 6, 5, 128)
    g = to_gpu(b)
    g["dx1"] = k["x"].to(DEV).expand(2, 6, 5, 128)
    g["gate"] = g["dx1"]
    got = evoattn.block_norm_bwd(*[g[n] for n in BWD_ARGS])
    assert got["dgate"].shape == (2, 6, 5, 128)   # an expanded gate: each row's own gradient
    check_bwd(b, got, False)
    # a gate shared along j that is itself expanded along b
    b["gate"] = b["gate"][:1, :, :1].contiguous().expand(2, 6, 1, 128)
    g["gate"] = b["gate"][:1].to(DEV).expand(2, 6, 1, 128)
    got = evoattn.block_norm_bwd(*[g[n] for n in BWD_ARGS])
    check_bwd(b, got, False)


def test_in_place_gives_the_same_bits():
    for types in TYPES:
        k = draw((2, 30, 41, 128), types, seed=13)
        x1, y = run_fwd(k, False)
        g = to_gpu(k)
        z1, z = evoattn.block_norm(g["x"], *[g[n] for n in ("u", "gate") + PARAMS], x1=g["x"])
        assert z1 is g["x"] and torch.equal(z1, x1) and torch.equal(z, y)
        k = draw((2, 30, 41, 128), types, seed=14, backward=True)
        want = run_bwd(k, False)
        g = to_gpu(k)
        got = evoattn.block_norm_bwd(*[g[n] for n in BWD_ARGS], dx=g["dx1"])
        assert got["dx"] is g["dx1"]
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("gate", ["full", "row", "batch"])
def test_repeats_bit_for_bit(gate):
    k = draw((1, 150, 150, 128), "bf16", gate, seed=15, backward=True)
    a = run_bwd(k, False)
    for _ in range(3):
        b = run_bwd(k, False)
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_full_size_sampled():
    """The pair representation of the N = 384 workload: a sample of rows, and
    the parameter gradients of all of them against float64 on the GPU."""
    shape = (1, 384, 384, 128)
    k = draw(shape, "bf16", seed=16)
    x1, y = run_fwd(k, False)
    gen = torch.Generator().manual_seed(1)
    i, j = torch.randint(0, 384, (60,), generator=gen), torch.randint(0, 384, (60,), generator=gen)
    pick = lambda t: t[:, i, j].reshape(1, 6, 10, 128)
    small = {n: (pick(t) if t is not None and t.dim() == 4 else t) for n, t in k.items()}
    check_fwd(small, pick(x1.cpu()), pick(y.cpu()), False)
    k = draw(shape, "bf16", seed=17, backward=True)
    got = run_bwd(k, False)
    small = {n: (pick(t) if t is not None and t.dim() == 4 else t) for n, t in k.items()}
    rows = {n: (pick(t.cpu()) if t.dim() == 4 else None) for n, t in got.items()}
    ref = tr.block_norm_bwd(**{n: small[n] for n in BWD_ARGS[:-1]})
    for n in ("dx", "du", "dgate"):
        lim = half(torch.bfloat16) * ref[n].abs() + 2.0 ** -12
        close(rows[n], ref[n], lim, n)
    full = tr.block_norm_bwd(**{n: k[n] for n in BWD_ARGS[:-1]})
    for n in ("dscale", "dgamma_post", "dbeta_post", "dgamma_pre", "dbeta_pre"):
        # 147,456 rows of random sign: a relative error of the norm of the vector
        off = (got[n].double().cpu() - full[n]).norm() / full[n].norm()
        assert float(off) <= 1e-5, (n, float(off))


def test_offsets_beyond_32_bits():
    """Rows 2.2 GB apart: byte offsets pass 2^32, element offsets 2^31."""
    n, gap, C = 3, 1_100_000_008, 64
    k = draw((1, 1, n, C), "bf16", seed=18)
    base = torch.empty(gap * (n - 1) + C, device=DEV, dtype=torch.bfloat16)
    view = base.as_strided((1, 1, n, C), (gap * n, gap * n, gap, 1))
    g = to_gpu(k)
    view.copy_(g["x"])
    x1, y = evoattn.block_norm(view, *[g[n_] for n_ in ("u", "gate") + PARAMS], x1=view)
    check_fwd(k, x1.contiguous(), y, False)


def test_a_bad_row_stays_its_own():
    """Infinities and NaN reach their own rows and the sums over rows only."""
    k = draw((1, 8, 8, 128), "bf16", seed=19)
    clean = run_fwd(k, False)
    k["u"][0, 2, 3, 5], k["x"][0, 4, 1, 0], k["gate"][0, 6, 6, 7] = float("inf"), float("nan"), float("nan")
    x1, y = run_fwd(k, False)
    bad = torch.zeros(1, 8, 8, dtype=torch.bool)
    bad[0, 2, 3] = bad[0, 4, 1] = bad[0, 6, 6] = True
    for got, want in ((x1, clean[0]), (y, clean[1])):
        got, want = got.cpu(), want.cpu()
        assert torch.equal(got[~bad], want[~bad])
        assert not bool(torch.isfinite(got[bad]).all(-1).any())
    k = draw((1, 8, 8, 128), "bf16", seed=20, backward=True)
    clean = run_bwd(k, False)
    k["dy"][0, 2, 3, 5] = float("nan")
    got = run_bwd(k, False)
    bad[:] = False
    bad[0, 2, 3] = True
    for n in ("dx", "du", "dgate"):
        assert torch.equal(got[n].cpu()[~bad], clean[n].cpu()[~bad]), n
    assert bool(torch.isnan(got["dx"].cpu()[bad]).all())


def test_extreme_magnitudes():
    """Rows whose squares are near the limits of fp32, a constant row (variance
    0) and a row of zeros."""
    k = draw((1, 1, 6, 128), "f32", "none", seed=21)
    k["x"][0, 0, 0] *= 1e17
    k["u"][0, 0, 1] *= 1e-18
    k["u"][0, 0, 2] = 3.0
    k["u"][0, 0, 3] = 0.0
    k["x"][0, 0, 4] = 0.0
    for rms in (False, True):
        x1, y = run_fwd(k, rms)
        rx1, ry = tr.block_norm(**{n: k[n] for n in ("x", "u", "gate") + PARAMS}, rms=rms)
        assert bool(torch.isfinite(x1).all()) and bool(torch.isfinite(y).all())
        close(x1, rx1, 1e-4 + 2 * U * rx1.abs(), "x1")
        # row 0: x1 is 1e17 times unit values, normalised again
        close(y[0, 0, 0], ry[0, 0, 0], 1e-4 * torch.ones(128, dtype=torch.float64), "y")


def test_gradients_match_differences_of_the_forward():
    """The fp32 kernels' own outputs, differenced in a random direction.  The
    step 2^-7 leaves a truncation error of h^2 times a third derivative of
    order one per term, and the outputs' rounding divided by the step."""
    k = draw((1, 4, 5, 64), "f32", seed=22)
    gen = torch.Generator().manual_seed(23)
    dx1, dy = (torch.randn(1, 4, 5, 64, generator=gen) for _ in range(2))
    x1, _ = run_fwd(k, False)
    b = dict(k, dx1=dx1, dy=dy, x1=x1.cpu())
    got = run_bwd(b, False)
    h = 2.0 ** -7
    for n in ("x", "u", "gate") + PARAMS:
        way = torch.randn(k[n].shape, generator=gen)
        way /= way.norm()

        def loss(sign):
            p, q = run_fwd(dict(k, **{n: k[n] + sign * h * way}), False)
            return float((p.double().cpu() * dx1.double()).sum() + (q.double().cpu() * dy.double()).sum())
        diff = (loss(1) - loss(-1)) / (2 * h)
        want = float((got["d" + n].double().cpu() * way.double()).sum())
        grad = float(got["d" + n].double().norm())
        # unit direction: the derivative along it is at most the gradient's
        # norm; truncation h^2 = 6e-5 of it times a constant of order ten
        assert abs(diff - want) <= 1e-3 * max(grad, 1.0), (n, diff, want)


def test_capture_and_other_streams():
    """A captured forward and backward replayed on new inputs, and calls on a
    stream of their own, give the eager call's bits."""
    k = draw((1, 64, 33, 128), "bf16", "row", seed=24, backward=True)
    f = draw((1, 64, 33, 128), "bf16", "row", seed=25)
    k2 = draw((1, 64, 33, 128), "bf16", "row", seed=26, backward=True)
    f2 = draw((1, 64, 33, 128), "bf16", "row", seed=27)
    g, gf = to_gpu(k), to_gpu(f)
    side = torch.cuda.Stream()
    fargs = [gf[n] for n in ("x", "u", "gate") + PARAMS]
    bargs = [g[n] for n in BWD_ARGS]
    side.wait_stream(torch.cuda.current_stream())
    a = evoattn.block_norm(*fargs, stream=side)
    b = evoattn.block_norm_bwd(*bargs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = run_fwd(f, False), run_bwd(k, False)
    assert torch.equal(a[0], want[0][0]) and torch.equal(a[1], want[0][1])
    for n in b:
        assert torch.equal(b[n], want[1][n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = evoattn.block_norm(*fargs)
        b = evoattn.block_norm_bwd(*bargs)
    for new, old in ((f2, gf), (k2, g)):
        for n, t in new.items():
            old[n].copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    want = run_fwd(f2, False), run_bwd(k2, False)
    assert torch.equal(a[0], want[0][0]) and torch.equal(a[1], want[0][1])
    for n in b:
        assert torch.equal(b[n], want[1][n]), n


@pytest.mark.parametrize("gate", ["none", "full", "row"])
def test_flat_and_packed_calls_agree(gate):
    """The two forms of the C entry points give the same bits."""
    import ctypes
    lib = evoattn.load()
    shape = (2, 5, 7, 72)
    S4 = ctypes.c_int64 * 4
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda t: None if t is None else t.data_ptr()
    s = lambda t: None if t is None else S4(*t.stride())
    ps = lambda t: (p(t), s(t))
    wide = lambda t: None if t is None else t.expand(shape)
    k = to_gpu(draw(shape, "mixed", gate, seed=30))
    x1, y = evoattn.block_norm(*[k[n] for n in ("x", "u", "gate") + PARAMS])
    a, b = torch.empty_like(x1), torch.empty_like(y)
    assert lib.evoattn_block_norm(*ps(k["x"]), *ps(k["u"]), *ps(wide(k["gate"])), *[p(k[n]) for n in PARAMS],
                                  *ps(a), *ps(b), *shape, evoattn.F32, evoattn.BF16, 0, 1e-5, stream) == 0
    assert torch.equal(a, x1) and torch.equal(b, y)
    k = to_gpu(draw(shape, "mixed", gate, seed=31, backward=True))
    want = evoattn.block_norm_bwd(*[k[n] for n in BWD_ARGS])
    got = {n: torch.empty_like(t) for n, t in want.items()}
    ws = torch.empty(lib.evoattn_block_norm_bwd_workspace_size(72), device=DEV, dtype=torch.uint8)
    assert lib.evoattn_block_norm_bwd(
        *[v for n in ("dx1", "dy", "x1", "u") for v in ps(k[n])], *ps(wide(k["gate"])),
        *[p(k[n]) for n in PARAMS[:4]], *ps(got["dx"]), *ps(got["du"]), *ps(wide(got.get("dgate"))),
        *[p(got["d" + n]) for n in PARAMS], *shape, evoattn.F32, evoattn.BF16, 0, 1e-5, ws.data_ptr(),
        ws.numel(), stream) == 0
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_first_call_under_capture():
    """A fresh process whose first calls of the library are captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from protein_folding_attention_gb300 import evoattn
x, v = torch.randn(1, 7, 9, 128, device="cuda").bfloat16(), torch.ones(128, device="cuda")
p, g = torch.ones(1000, device="cuda"), torch.ones(1000, device="cuda")
opt = evoattn.AdamW([p], [g], lr=0.5, weight_decay=0.0, state_bits=8)
evoattn.load()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    x1, y = evoattn.block_norm(x, x, x, v, v, v, v, v)
    d = evoattn.block_norm_bwd(x, x, x1, x, x, v, v, v, v, v)
    opt.step(max_norm=1.0)
assert bool((p == 1).all())
graph.replay()
torch.cuda.synchronize()
a, b = evoattn.block_norm(x, x, x, v, v, v, v, v)
e = evoattn.block_norm_bwd(x, x, a, x, x, v, v, v, v, v)
assert torch.equal(a, x1) and torch.equal(b, y) and all(torch.equal(d[k], e[k]) for k in e)
assert abs(float(p[5]) - 0.5) < 1e-5 and opt.steps_taken() == 1
print("done")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr


def test_two_streams_at_once():
    """Calls on two streams that overlap, each with a workspace of its own."""
    ks = [draw((1, 200, 150, 128), "bf16", "row", seed=50 + i, backward=True) for i in range(2)]
    want = [run_bwd(k, False) for k in ks]
    gs = [to_gpu(k) for k in ks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ks]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            got[i] = evoattn.block_norm_bwd(*[gs[i][n] for n in BWD_ARGS], stream=st)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for n in b:
            assert torch.equal(a[n], b[n]), n


def test_python_refusals():
    k = draw((1, 2, 3, 16), "bf16", seed=28)
    g = to_gpu(k)
    call = lambda **kw: evoattn.block_norm(**{**{"x": g["x"], "u": g["u"], "gate": g["gate"]}, **kw})
    for bad in (dict(u=g["u"][:, :1]), dict(u=g["u"].half()), dict(u=g["u"].float()),
                dict(gate=g["gate"][..., :8]), dict(gate=g["gate"][:, :, :2]), dict(gate=g["gate"].cpu()),
                dict(gate=g["gate"].float()), dict(scale=g["scale"][:8]), dict(scale=g["scale"].bfloat16()),
                dict(gamma_pre=torch.ones(32, device=DEV)[::2]), dict(y_dtype=torch.float32),
                dict(pre=False, y=torch.empty_like(g["x"])), dict(x=g["x"][0]),
                dict(u=None, gate=None, x1=torch.empty_like(g["x"]))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        evoattn.block_norm(g["x"].half())
    with pytest.raises(evoattn.EvoAttnError):
        evoattn.block_norm(torch.zeros(1, 1, 1, 4104, device=DEV))
    with pytest.raises(evoattn.EvoAttnError):
        call(x=g["x"].transpose(2, 3).contiguous().transpose(2, 3))   # channels not contiguous
    with pytest.raises(evoattn.EvoAttnError):
        call(x1=g["x"][:, :1].expand(1, 2, 3, 16))                    # overlapping output rows
    b = to_gpu(draw((1, 2, 3, 16), "bf16", seed=29, backward=True))
    for bad in (dict(dx1=None, dy=None), dict(x1=None), dict(u=None, dy=None), dict(x1=b["x1"].float()),
                dict(beta_pre=b["beta_pre"][:3]), dict(dx1=b["dx1"][0]),
                dict(dy=None, gamma_pre=None, beta_pre=None, dx=torch.empty_like(b["dx1"]))):
        with pytest.raises(ValueError):
            evoattn.block_norm_bwd(**{**{n: b[n] for n in BWD_ARGS}, **bad})
    with pytest.raises(evoattn.EvoAttnError):
        evoattn.block_norm_bwd(*[b[n] for n in BWD_ARGS],
                               workspace=torch.empty(256, device=DEV, dtype=torch.uint8))


def test_workspaces_that_the_kernels_cannot_use_are_refused():
    b = to_gpu(draw((1, 2, 3, 16), "bf16", seed=29, backward=True))
    n = evoattn.load().evoattn_block_norm_bwd_workspace_size(16)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, device=DEV, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            evoattn.block_norm_bwd(*[b[k] for k in BWD_ARGS], workspace=ws)


@pytest.mark.parametrize("C", [16, 24, 32, 40, 48, 72, 80])
@pytest.mark.parametrize("gate", ["none", "full", "row", "batch"])
def test_narrow_rows_that_share_a_warp(C, gate):
    """Groups of as many lanes as a row has parts, lanes left over or not: one
    row, part of a turn, and several turns."""
    for shape in ((1, 1, 1, C), (2, 3, 17, C), (2, 40, 301, C)):
        k = draw(shape, "bf16", gate, seed=C)
        x1, y = run_fwd(k, C % 16 == 0)
        check_fwd(k, x1, y, C % 16 == 0)
        k = draw(shape, "bf16", gate, seed=C + 1, backward=True)
        check_bwd(k, run_bwd(k, C % 16 == 0), C % 16 == 0)


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 400, 300, 24), (1, 400, 300, 37), (2, 3, 7000, 61), (1, 350, 64, 131),
                                   (1, 5, 900, 301)])
def test_gate_rows_cut_into_pieces(types, shape):
    """More gate rows than CTAs, and few long ones: pieces of a gate row's rows
    whose sums a second kernel joins, rows copied one by one or a turn at once."""
    k = draw(shape, types, "row", seed=shape[3], backward=True)
    got = run_bwd(k, False)
    check_bwd(k, got, False)
    again = run_bwd(k, False)
    assert all(torch.equal(got[n], again[n]) for n in got)


def _check_dgate(k, got, most=0.0):
    """dgate against float64 with a tolerance that shrinks with q (1 - q).
    q = 1 / (1 + t), t = exp(-g): the exponent is off by 2 u |g|, and with it q
    and 1 - q = t q by that relatively, beside a few roundings and the two
    approximate operations: (64 + 4 |g|) u of q (1 - q).  `most`: what may be
    lost where q or t leaves the range of fp32."""
    rows = tuple(range(3))
    h, _ = tr.normalise(k["u"].double(), False, 1e-5)
    ku = 1 + kappa(k["u"], False)
    s, g1, b1 = (k[n].double() for n in ("scale", "gamma_post", "beta_post"))
    w = h * g1 + b1
    werr = 64 * U * ku * (1 + h.abs()) * g1.abs() + 4 * U * b1.abs()
    v = k["gate"].double().expand_as(h)
    e = k["dx1"].double() * s
    f = torch.sigmoid(v) * torch.sigmoid(-v)
    ref, term = e * w * f, (e * w * f).abs()
    err = (e * f).abs() * werr + (256 + 64 + 4 * v.abs().clamp_max(200)) * U * term + most * (e * w).abs()
    over = [i for i in rows if k["gate"].shape[i] == 1]
    if over:
        ref, err = ref.sum(over, keepdim=True), err.sum(over, keepdim=True)
    dtype = got["dgate"].dtype  # (the half step of a subnormal value is that of the smallest normal one)
    close(got["dgate"], ref, half(dtype) * ref.abs().clamp_min(torch.finfo(dtype).tiny) + err, "dgate")


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("gate", ["full", "row", "batch"])
@pytest.mark.parametrize("C", [40, 64, 99, 384, 1000])
def test_gradients_of_gates_far_from_zero(types, gate, C):
    """1 - q is taken without cancellation: gates from 5 to 30 and -5 to -30,
    of each row and shared by a few rows and by many."""
    for shape in ((2, 6, 40, C), (2, 5, 3, C)):
        k = draw(shape, types, gate, pre=False, seed=60 + C, backward=True)
        gen = torch.Generator().manual_seed(61)
        values = torch.tensor([5.0, 8.0, 13.0, 17.0, 23.0, 30.0])
        values = torch.cat([values, -values])
        k["gate"] = values[torch.randint(0, 12, k["gate"].shape, generator=gen)].to(k["gate"].dtype)
        _check_dgate(k, run_bwd(k, False))


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("gate", ["full", "row"])
def test_gradients_of_gates_at_the_ends(types, gate):
    """Gates whose sigmoid, or whose distance from 1, underflows: no NaN from
    an exponential that overflows.  (Below 2^-126 fp32 and bf16 results may be
    flushed to zero.)"""
    k = draw((1, 6, 24, 64), types, gate, pre=False, seed=62, backward=True)
    values = torch.tensor([float("inf"), 3e38, 100.0, 88.5, 88.0, 87.5, 87.0, 80.0])
    values = torch.cat([values, -values])
    gen = torch.Generator().manual_seed(63)
    k["gate"] = values[torch.randint(0, 16, k["gate"].shape, generator=gen)].to(k["gate"].dtype)
    got = run_bwd(k, False)
    assert all(bool(torch.isfinite(t).all()) for t in got.values())
    _check_dgate(k, got, most=2.0 ** -125)


def test_sums_do_not_depend_on_earlier_calls():
    """A process whose first call has other rows, of which fewer CTAs fit on an
    SM, gives the same bits: fp32 rows of 1001 after rows of 2047 and the other
    way round (both 256 threads, the latter with more shared memory)."""
    import os
    import subprocess
    import sys
    code = """
import hashlib, sys, torch
from protein_folding_attention_gb300 import evoattn
for C in map(int, sys.argv[1:]):
    gen = torch.Generator(device="cuda").manual_seed(C)
    dx1, dy, x1, u = (torch.randn(1, 1, 4000, C, device="cuda", generator=gen) for _ in range(4))
    v = 1.0 + 0.1 * torch.randn(C, device="cuda", generator=gen)
    out = evoattn.block_norm_bwd(dx1, dy, x1, u, None, v, v, v, v, v)
print("bits", hashlib.sha256(b"".join(out[n].cpu().numpy().tobytes() for n in sorted(out))).hexdigest())
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

    def bits(*widths):
        r = subprocess.run([sys.executable, "-c", code, *map(str, widths)], cwd=root, capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.split("bits")[1].strip()
    assert bits(2047, 1001) == bits(1001)
    assert bits(1001, 2047) == bits(2047)
