"""Refusals of the 8-bit path's entry points without a GPU: each bad argument
gives the documented status, or the binding's error, before anything touches
the device (the pointers are never dereferenced); and what the calls do for a
stream that is handed in."""
import contextlib
import math

import pytest
import torch

from protein_folding_attention_gb300 import build_lib, evoattn

FAKE = 1 << 20
BF16, F32 = evoattn.BF16, evoattn.F32
I, U, A, W = (evoattn.ERR_INVALID_ARG, evoattn.ERR_UNSUPPORTED, evoattn.ERR_ALIGNMENT,
              evoattn.ERR_WORKSPACE)
SHAPE = (2, 3, 4, 16)
NONE = (0, 0, 0, 0, 0)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return evoattn.load()


def dense(B, I_, J, C):
    return I_ * J * C, J * C, C, 1


def rows(p=FAKE, s=None, shape=SHAPE):
    return (p, *(s or dense(*shape))) if p else NONE


def drop(p=0.25, rng=FAKE, site=0, shared=0):
    return rng, p, site, shared


def dropout(lib, *, x=None, u=None, out=None, d=None, shape=SHAPE, sd=BF16, io=BF16):
    pick = lambda r: rows(shape=shape) if r is None else r
    return lib.evoattn_dropout_add(evoattn._PACK_DROPOUT(*pick(x), *pick(u), *pick(out), *(d or drop()), *shape, sd, io),
                                   None)


def norm(lib, *, x=None, u=None, x1=None, codes=None, scales=None, g=FAKE, b=FAKE, d=None, eps=1e-5, shape=SHAPE,
         sd=BF16, io=BF16, kind=0):
    pick = lambda r: rows(shape=shape) if r is None else r
    sc = rows(s=dense(*shape[:3], -(-shape[3] // 128))) if scales is None else scales
    return lib.evoattn_norm8(evoattn._PACK_NORM8(*pick(x), *pick(u), *pick(x1), *pick(codes), *sc, g, b, *(d or drop()),
                                                 eps, *shape, sd, io, kind), None)


def norm_bwd(lib, *, dx1=None, dy=None, x1=None, dx=None, du=None, g=FAKE, dg=FAKE, db=FAKE, d=None, eps=1e-5,
             shape=SHAPE, sd=BF16, io=BF16, kind=0, ws=FAKE, size=1 << 40):
    pick = lambda r: rows(shape=shape) if r is None else r
    return lib.evoattn_norm8_bwd(
        evoattn._PACK_NORM8_BWD(*pick(dx1), *pick(dy), *pick(x1), *pick(dx), *pick(du), g, dg, db, *(d or drop()),
                                eps, *shape, sd, io, kind, ws, size), None)


def test_null_structs(lib):
    for name in ("dropout_add", "norm8", "norm8_bwd", "quantize8", "matmul8"):
        assert getattr(lib, "evoattn_" + name)(None, None) == I


@pytest.mark.parametrize("call", [dropout, norm, norm_bwd])
def test_dropout_arguments(lib, call):
    for p in (-0.1, 1.0, 1.5, math.nan, math.inf):
        assert call(lib, d=drop(p=p)) == I
    assert call(lib, d=drop(rng=0)) == I
    assert call(lib, d=drop(rng=FAKE + 4)) == A
    for site in (-1, 2 ** 32):
        assert call(lib, d=drop(site=site)) == I
    for shared in (-1, 8):
        assert call(lib, d=drop(shared=shared)) == I


@pytest.mark.parametrize("call, out", [(dropout, "out"), (norm, "x1"), (norm, "codes"), (norm_bwd, "dx"), (norm_bwd, "du")])
def test_row_operands(lib, call, out):
    for k in range(4):
        assert call(lib, shape=tuple(0 if i == k else n for i, n in enumerate(SHAPE))) == I
        assert call(lib, shape=tuple(-1 if i == k else n for i, n in enumerate(SHAPE))) == I
    assert call(lib, shape=(1, 1, 1, 4097)) == U
    assert call(lib, shape=(1, 46341, 46341, 8)) == U
    assert call(lib, shape=(2 ** 40, 1, 1, 8)) == U
    assert call(lib, shape=(2, 2 ** 40, 1, 8)) == U
    assert call(lib, sd=7) == U and call(lib, io=-1) == U
    for s in ((192, 64, 0, 1), (192, 64, 15, 1), (192, 63, 16, 1), (-192, 64, 16, 1), (2 ** 62, 64, 16, 1)):
        assert call(lib, **{out: rows(s=s)}) == I
    assert call(lib, **{out: rows(s=(384, 128, 32, 2))}) == A
    if out != "codes":
        assert call(lib, **{out: rows(FAKE + 1)}) == A


def test_dropout_add_rejects(lib):
    assert dropout(lib, u=NONE) == I
    assert dropout(lib, out=NONE) == I
    assert dropout(lib, shape=(1, 2 ** 12, 2 ** 11, 4096)) == U   # 2^32 parts of eight channels
    assert dropout(lib, sd=F32, x=rows(FAKE + 2)) == A
    assert dropout(lib, io=F32, u=rows(FAKE + 2)) == A


def test_norm8_rejects(lib):
    for k in ("x", "codes", "scales"):
        assert norm(lib, **{k: NONE}) == I
    assert norm(lib, u=NONE) == I and norm(lib, x1=NONE) == I
    assert norm(lib, u=NONE, x1=NONE) == I                  # dropout of nothing
    assert norm(lib, sd=BF16, io=F32) == U
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert norm(lib, eps=eps) == I
    assert norm(lib, kind=2) == I
    assert norm(lib, g=FAKE + 2) == A and norm(lib, b=FAKE + 1) == A
    wide = (2, 3, 4, 256)
    for s in ((24, 8, 2, 0), (24, 8, 1, 1), (0, 8, 2, 1), (24, -8, 2, 1), (2 ** 60, 8, 2, 1)):
        assert norm(lib, shape=wide, scales=rows(s=s)) == I


def test_norm8_bwd_rejects(lib):
    for k in ("dy", "x1", "dx"):
        assert norm_bwd(lib, **{k: NONE}) == I
    assert norm_bwd(lib, du=NONE) == I                      # dropout of nothing
    assert norm_bwd(lib, sd=BF16, io=F32) == U
    assert norm_bwd(lib, kind=-1) == I and norm_bwd(lib, eps=0.0) == I
    for k in ("g", "dg", "db"):
        assert norm_bwd(lib, **{k: FAKE + 2}) == A
    need = lib.evoattn_norm8_bwd_workspace_size(16)
    assert need > 0
    assert norm_bwd(lib, ws=0) == W and norm_bwd(lib, size=need - 1) == W and norm_bwd(lib, ws=FAKE + 16) == W
    assert norm_bwd(lib, size=-1) == W
    assert [lib.evoattn_norm8_bwd_workspace_size(c) for c in (0, -1, 4097)] == [0, 0, 0]


def quant(lib, *, x=FAKE, R=10, K=300, ld=300, dt=BF16, blocks=0, q=(FAKE, 304), s=(FAKE, 1, 10), qt=(FAKE, 16),
          st=(FAKE, 1, 300)):
    return lib.evoattn_quantize8(evoattn._PACK_QUANTIZE8(x, R, K, ld, dt, blocks, *q, *s, *qt, *st), None)


def test_quantize8_rejects(lib):
    no2, no3 = (0, 0), (0, 0, 0)
    assert quant(lib, x=0) == I
    assert quant(lib, q=no2, s=no3, qt=no2, st=no3) == I
    assert quant(lib, s=no3) == I and quant(lib, st=no3) == I
    assert quant(lib, q=no2) == I and quant(lib, qt=no2) == I
    assert quant(lib, blocks=1) == I                         # scales_t with blocks
    assert quant(lib, blocks=1, s=no3, st=no3) == I
    for k in ("R", "K"):
        assert quant(lib, **{k: 0}) == I and quant(lib, **{k: -5}) == I
    assert quant(lib, dt=2) == U
    assert quant(lib, R=2 ** 39, K=2 ** 39) == U
    assert quant(lib, R=2 ** 22, K=2 ** 22) == U
    assert quant(lib, ld=-300) == I and quant(lib, ld=2 ** 60) == I
    assert quant(lib, q=(FAKE, 299)) == I and quant(lib, qt=(FAKE, 9)) == I
    assert quant(lib, q=(FAKE, 312)) == A and quant(lib, q=(FAKE + 8, 304)) == A
    assert quant(lib, qt=(FAKE, 24)) == A and quant(lib, qt=(FAKE + 1, 16)) == A
    assert quant(lib, x=FAKE + 1) == A and quant(lib, dt=F32, x=FAKE + 2) == A
    for s in ((FAKE, 0, 10), (FAKE, 1, 9), (FAKE, 1, 0), (FAKE, -1, 10), (FAKE, 2, 1), (FAKE, 2 ** 60, 1)):
        assert quant(lib, s=s) == I


def product(lib, *, a=None, b=None, M=5, N=7, K=300, out=FAKE, ld=7, add=0, ld_add=0, dt=BF16, ws=FAKE, size=1 << 40):
    a = a or (FAKE, 304, FAKE, 1, 5, 1)
    b = b or (FAKE, 304, FAKE, 1, 7, 1)
    return lib.evoattn_matmul8(evoattn._PACK_MATMUL8(*a, *b, M, N, K, out, ld, add, ld_add, dt, ws, size), None)


def test_matmul8_rejects(lib):
    for k in "MNK":
        assert product(lib, **{k: 0}) == I and product(lib, **{k: -1}) == I
        assert product(lib, **{k: 2 ** 31}) == U
    assert product(lib, out=0) == I
    for k in "ab":
        good = (FAKE, 304, FAKE, 1, 7, 1)
        bad = lambda i, v: {k: good[:i] + (v,) + good[i + 1:]}
        assert product(lib, **bad(0, 0)) == I and product(lib, **bad(2, 0)) == I
        assert product(lib, **bad(1, 299)) == I
        assert product(lib, **bad(1, 312)) == A and product(lib, **bad(0, FAKE + 8)) == A
        assert product(lib, **bad(1, 2 ** 40)) == I
        for per in (0, 2, 127, -1):
            assert product(lib, **bad(5, per)) == I
        for i in (3, 4):
            assert product(lib, **bad(i, -1)) == I and product(lib, **bad(i, 2 ** 60)) == I
    assert product(lib, ld=6) == I and product(lib, ld=2 ** 60) == I
    assert product(lib, add=FAKE, ld_add=6) == I and product(lib, add=FAKE, ld_add=-1) == I
    assert product(lib, dt=5) == U
    assert product(lib, out=FAKE + 1) == A and product(lib, dt=F32, out=FAKE + 2) == A
    assert product(lib, add=FAKE + 1, ld_add=7) == A
    assert [lib.evoattn_matmul8_workspace_size(*n) for n in ((0, 1, 1), (1, -1, 1), (1, 1, 0))] == [0, 0, 0]


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
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
    caches = evoattn._matmul8_workspace, evoattn._norm8_bwd_workspace
    for c in caches:
        c.cache_clear()
    yield told
    for c in caches:
        c.cache_clear()


def addresses(*ts):
    return {t.data_ptr() for t in ts}


def test_calls_tell_their_tensors_of_the_stream(told):
    r = lambda: torch.randn(1, 3, 4, 24)
    x, u, g, b = r(), r(), torch.ones(24), torch.zeros(24)
    rng = torch.tensor([1, 2])
    evoattn.dropout_add(u, 0.1, rng, x=x)
    assert not told
    out = evoattn.dropout_add(u, 0.1, rng, x=x, stream=Side(1))
    assert addresses(x, u, rng, out) <= set(told[1])
    x1, q, s = evoattn.norm8(x, u, g, b, p=0.1, rng=rng, stream=Side(2))
    assert addresses(x, u, g, b, rng, x1) <= set(told[2])
    evoattn.norm8_bwd(x, u, x1, g, b, p=0.1, rng=rng, stream=Side(3))
    assert addresses(x, u, x1, g, rng) <= set(told[3])
    evoattn.quantize8(x, stream=Side(4))
    assert addresses(x) <= set(told[4])
    w, ws = evoattn.quantize8(torch.randn(8, 24))
    add, ws8 = torch.zeros(1, 3, 4, 8), torch.empty(64, dtype=torch.uint8)
    o = evoattn.matmul8(q, s, w, ws, torch.float32, add=add, workspace=ws8, stream=Side(5))
    assert o.shape == (1, 3, 4, 8)
    assert addresses(q, s, w, ws, add, o, ws8) <= set(told[5])


def test_layouts(told):
    q, s, qt, st = evoattn.quantize8(torch.randn(5, 3, 200), cols=True)
    assert q.shape == (5, 3, 200) and q.stride() == (624, 208, 1) and s.shape == (5, 3, 2) and s.stride() == (3, 1, 15)
    assert qt.shape == (200, 15) and qt.stride() == (16, 1) and st.shape == (200, 1)
    q, s, qt, st = evoattn.quantize8(torch.randn(300, 200), cols=True, blocks=True)
    assert s.shape == (3, 2) and st.shape == (2, 3) and st.data_ptr() == s.data_ptr()
    assert len(evoattn.quantize8(torch.randn(300, 200), rows=False, cols=True)) == 2
    x1, q, s = evoattn.norm8(torch.randn(2, 3, 4, 130))
    assert q.shape == (2, 3, 4, 130) and q.stride(2) == 144 and s.shape == (2, 3, 4, 2) and s.stride() == (12, 4, 1, 24)


def test_binding_refuses(told):
    r = lambda *shape: torch.randn(*(shape or (1, 3, 4, 24)))
    rng = torch.tensor([1, 2])
    for wrong in (None, rng.int(), torch.tensor([1, 2, 3]), torch.tensor([1, 0, 2, 0])[::2]):
        with pytest.raises(ValueError):
            evoattn.dropout_add(r(), 0.1, wrong)
    with pytest.raises(ValueError):
        evoattn.dropout_add(r(), 0.1, rng, shared=(3,))
    with pytest.raises(ValueError):
        evoattn.dropout_add(r(4, 24), 0.1, rng)
    with pytest.raises(ValueError):
        evoattn.dropout_add(r(), 0.1, rng, x=r(1, 3, 5, 24))
    with pytest.raises(ValueError):
        evoattn.dropout_add(r(), 0.1, rng, x=r(), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        evoattn.norm8(r(), x1=r())
    with pytest.raises(ValueError):
        evoattn.norm8(r(), r(), torch.ones(23))
    with pytest.raises(ValueError):
        evoattn.norm8_bwd(r(), r(), r(), torch.ones(24), torch.ones(25))
    with pytest.raises(ValueError):
        evoattn.norm8_bwd(r(), r().bfloat16(), r(), dx=r().bfloat16())
    with pytest.raises(ValueError):
        evoattn.quantize8(r(), rows=False)
    with pytest.raises(ValueError):
        evoattn.quantize8(r().transpose(1, 2))               # rows that are no matrix
    with pytest.raises(ValueError):
        evoattn.quantize8(r(30, 20).t())                     # columns not contiguous
    with pytest.raises(TypeError):
        evoattn.quantize8(r().half())
    q, s = evoattn.quantize8(r(6, 24))
    w, ws = evoattn.quantize8(r(8, 24))
    evoattn.matmul8(q, s, w, ws)
    for wrong in ((q.float(), s, w, ws), (q, s.float(), w, ws), (q[:5], s, w, ws), (q, s, w[:, :20], ws),
                  (q, s, w, ws[:3])):
        with pytest.raises(ValueError):
            evoattn.matmul8(*wrong)
    for k in (dict(out_dtype=torch.float16), dict(add=r(6, 8)), dict(out=torch.empty(6, 9).bfloat16()),
              dict(out_dtype=torch.float32, add=r(7)), dict(out_dtype=torch.float32, out=torch.empty(8, 6).t())):
        with pytest.raises(ValueError):
            evoattn.matmul8(q, s, w, ws, **k)


def test_tensors_of_the_cpu_are_refused():
    x = torch.randn(1, 2, 3, 16)
    q, s = torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.ones(4, 1).to(torch.float8_e8m0fnu)
    for call in (lambda: evoattn.dropout_add(x, 0.0, None), lambda: evoattn.norm8(x), lambda: evoattn.norm8_bwd(x, x, x),
                 lambda: evoattn.quantize8(x), lambda: evoattn.matmul8(q, s, q, s)):
        with pytest.raises((ValueError, RuntimeError, AttributeError)):
            call()
