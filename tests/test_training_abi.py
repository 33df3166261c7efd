"""Refusals of the training entry points (block norm, gradient norm, AdamW)
without a GPU: each bad argument gives the documented status before anything
touches the device (the pointers are never dereferenced)."""
import ctypes
import math

import pytest

from protein_folding_attention_gb300 import build_lib, evoattn

FAKE = 1 << 20
S4 = ctypes.c_int64 * 4
BF16, F32 = evoattn.BF16, evoattn.F32


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return evoattn.load()


def dense(B, I, J, C):
    return S4(I * J * C, J * C, C, 1)


SHAPE = (2, 3, 4, 16)


def fwd(lib, *, x=FAKE, xs=None, u=FAKE, us=None, gate=FAKE, gs=None, scale=FAKE, g1=FAKE, b1=FAKE,
        g2=FAKE, b2=FAKE, x1=FAKE, x1s=None, y=FAKE, ys=None, shape=SHAPE, sd=BF16, d=BF16, kind=0,
        eps=1e-5):
    s = dense(*shape)
    return lib.evoattn_block_norm(x, xs or s, u, us or s, gate, gs or s, scale, g1, b1, g2, b2, x1,
                                  x1s or s, y, ys or s, *shape, sd, d, kind, eps, None)


def test_block_norm_rejects_bad_arguments(lib):
    I, U, A = evoattn.ERR_INVALID_ARG, evoattn.ERR_UNSUPPORTED, evoattn.ERR_ALIGNMENT
    none = dict(u=None, x1=None, gate=None, scale=None, g1=None, b1=None)
    assert fwd(lib, x=None) == I
    assert fwd(lib, x1=None) == I                          # u without x1
    assert fwd(lib, u=None) == I                           # x1 without u
    for k in ("gate", "scale", "g1", "b1"):                # branch parameters without u
        assert fwd(lib, **{**none, k: FAKE}) == I
    assert fwd(lib, y=None) == I                           # gamma_pre without y
    assert fwd(lib, y=None, g2=None, b2=None, **none) == I  # nothing to do
    for k in range(4):
        assert fwd(lib, shape=tuple(0 if i == k else n for i, n in enumerate(SHAPE))) == I
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert fwd(lib, eps=eps) == I
    assert fwd(lib, kind=2) == I
    assert fwd(lib, shape=(1, 1, 1, 4097)) == U
    assert fwd(lib, shape=(1, 46341, 46341, 8)) == U       # 2^31 rows
    assert fwd(lib, shape=(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 8)) == U
    assert fwd(lib, sd=BF16, d=F32) == U
    assert fwd(lib, sd=7) == U
    assert fwd(lib, x=FAKE + 1) == A
    assert fwd(lib, scale=FAKE + 2) == A
    assert fwd(lib, sd=F32, x=FAKE + 2) == A
    assert fwd(lib, xs=S4(384, 128, 32, 2)) == A            # channels not contiguous
    assert fwd(lib, xs=S4(-192, 64, 16, 1)) == I
    assert fwd(lib, xs=S4(2 ** 62, 64, 16, 1)) == I         # an address beyond 64 bits
    for k in ("x1s", "ys"):                                 # overlapping output rows
        assert fwd(lib, **{k: S4(192, 64, 0, 1)}) == I
        assert fwd(lib, **{k: S4(192, 64, 15, 1)}) == I
        assert fwd(lib, **{k: S4(192, 63, 16, 1)}) == I


def bwd(lib, *, dx1=FAKE, dy=FAKE, x1=FAKE, u=FAKE, gate=FAKE, gs=None, scale=FAKE, g1=FAKE, b1=FAKE,
        g2=FAKE, dx=FAKE, dxs=None, du=FAKE, dgate=FAKE, dgs=None, grads=(FAKE,) * 5, shape=SHAPE,
        ws=FAKE, ws_bytes=1 << 40, sd=BF16, d=BF16, kind=0, eps=1e-5):
    s = dense(*shape)
    return lib.evoattn_block_norm_bwd(dx1, s, dy, s, x1, s, u, s, gate, gs or s, scale, g1, b1, g2,
                                      dx, dxs or s, du, s, dgate, dgs or s, *grads, *shape, sd, d,
                                      kind, eps, ws, ws_bytes, None)


def test_block_norm_bwd_rejects_bad_arguments(lib):
    I, U, A, W = (evoattn.ERR_INVALID_ARG, evoattn.ERR_UNSUPPORTED, evoattn.ERR_ALIGNMENT,
                  evoattn.ERR_WORKSPACE)
    no_branch = dict(u=None, du=None, gate=None, dgate=None, scale=None, g1=None, b1=None)
    assert bwd(lib, dx1=None, dy=None, x1=None, dx=None, g2=None, grads=(None,) * 5) == I
    assert bwd(lib, x1=None) == I
    assert bwd(lib, dx=None) == I
    assert bwd(lib, dy=None, x1=None, dx=None) == I          # gamma_pre without dy
    assert bwd(lib, dy=None, x1=None, dx=None, g2=None) == I  # its gradient without dy
    assert bwd(lib, du=None) == I
    assert bwd(lib, dgate=None) == I
    assert bwd(lib, gate=None) == I
    assert bwd(lib, **no_branch) == I                         # branch gradients without u
    assert bwd(lib, **{**no_branch, "scale": FAKE}, grads=(None,) * 5) == I
    assert bwd(lib, shape=(1, 1, 1, 5000)) == U
    assert bwd(lib, sd=BF16, d=F32) == U
    assert bwd(lib, kind=-1) == I
    assert bwd(lib, dx=FAKE + 1) == A
    assert bwd(lib, grads=(FAKE + 1,) * 5) == A
    assert bwd(lib, dxs=S4(0, 64, 16, 1)) == I
    shared = S4(64, 0, 0, 1)
    assert bwd(lib, gs=shared) == I                           # dgate does not share the gate's rows
    assert bwd(lib, dgs=shared) == I
    assert bwd(lib, gs=shared, dgs=shared, ws=None) == W      # (every other check passed)
    need = evoattn.load().evoattn_block_norm_bwd_workspace_size(16)
    assert need > 0 and lib.evoattn_block_norm_bwd_workspace_size(0) == 0
    assert lib.evoattn_block_norm_bwd_workspace_size(4097) == 0
    assert bwd(lib, ws_bytes=need - 1) == W
    assert bwd(lib, ws=FAKE + 128) == W


def tensors(count=2, **kw):
    t = (evoattn.AdamwTensor * count)()
    for row in t:
        row.param = row.grad = row.exp_avg = row.exp_avg_sq = row.copy = FAKE
        row.n, row.weight_decay, row.grad_dtype = 100, 0.01, BF16
    for k, v in kw.items():
        setattr(t[count - 1], k, v)
    return t


def step(lib, t, *, count=None, lr=1e-3, lr_dev=None, b1=0.9, b2=0.999, eps=1e-8, bits=32, flags=0,
         state=FAKE):
    return lib.evoattn_adamw(t, len(t) if count is None else count, lr, lr_dev, b1, b2, eps, bits,
                             flags, state, None)


def test_adamw_rejects_bad_arguments(lib):
    I, U, A = evoattn.ERR_INVALID_ARG, evoattn.ERR_UNSUPPORTED, evoattn.ERR_ALIGNMENT
    assert step(lib, None, count=1) == I
    assert step(lib, tensors(), count=0) == I
    assert step(lib, tensors(), state=None) == I
    assert step(lib, tensors(), state=FAKE + 4) == A
    for k in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert step(lib, tensors(**{k: None})) == I
        if k != "grad":
            assert step(lib, tensors(**{k: FAKE + 2})) == A
    assert step(lib, tensors(grad=FAKE + 1)) == A
    assert step(lib, tensors(grad=FAKE + 2, grad_dtype=F32)) == A
    assert step(lib, tensors(copy=FAKE + 1)) == A
    assert step(lib, tensors(n=-1)) == I
    assert step(lib, tensors(n=1 << 50)) == U
    assert step(lib, tensors(grad_dtype=5)) == U
    assert step(lib, tensors(weight_decay=-1.0)) == I
    assert step(lib, tensors(weight_decay=math.nan)) == I
    for lr in (-1.0, math.nan, math.inf):
        assert step(lib, tensors(), lr=lr) == I
    for b in (-0.1, 1.0, math.nan):
        assert step(lib, tensors(), b1=b) == I
        assert step(lib, tensors(), b2=b) == I
    for eps in (0.0, 1e-40, math.nan, math.inf):
        assert step(lib, tensors(), eps=eps) == I
    assert step(lib, tensors(), bits=16) == U
    assert step(lib, tensors(), flags=2) == I
    assert step(lib, tensors(), lr_dev=FAKE + 2) == A
    assert step(lib, tensors(exp_avg_scale=FAKE)) == I       # scales with 32-bit states
    assert step(lib, tensors(), bits=8) == I                 # 8-bit states without scales


def norm(lib, t, *, count=None, max_norm=1.0, state=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return lib.evoattn_grad_norm(t, len(t) if count is None else count, max_norm, state, ws,
                                 ws_bytes, None)


def test_grad_norm_rejects_bad_arguments(lib):
    I, W = evoattn.ERR_INVALID_ARG, evoattn.ERR_WORKSPACE
    assert norm(lib, None, count=1) == I
    assert norm(lib, tensors(), count=0) == I
    assert norm(lib, tensors(), state=None) == I
    for m in (0.0, -1.0, math.nan):
        assert norm(lib, tensors(), max_norm=m) == I
    assert norm(lib, tensors(), ws=None) == W
    assert norm(lib, tensors(), ws=FAKE + 8) == W
    need = lib.evoattn_grad_norm_workspace_size(2)
    assert need > 0 and lib.evoattn_grad_norm_workspace_size(0) == 0
    assert norm(lib, tensors(), ws_bytes=need - 1) == W
    assert lib.evoattn_grad_norm_workspace_size(10_000) > need


def test_python_refuses_tensors_that_are_not_on_the_current_gpu():
    import torch
    x = torch.zeros(1, 1, 1, 8)
    with pytest.raises(ValueError):
        evoattn.block_norm(x)
    with pytest.raises(ValueError):
        evoattn.block_norm_bwd(x, x, x)
    with pytest.raises(ValueError):
        evoattn.AdamW([torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError):
        evoattn.grad_norm([torch.zeros(4)])
    with pytest.raises(ValueError):
        evoattn.grad_norm([])


def test_a_negative_number_of_steps_taken_is_refused():
    """(At step -1 the first bias correction would divide by zero.)"""
    import torch
    with pytest.raises(ValueError, match="steps already taken"):
        evoattn.AdamW([torch.ones(3)], [torch.ones(3)], step=-1)
