"""The training operators around the pair-stack blocks, as cases to measure.

* ``norm_fwd`` / ``norm_bwd``: the seam between two blocks.  The block's
  output u is normalised, gated and scaled into the residual stream x, and the
  stream is normalised again for the next block:

      x1 = x + scale * sigmoid(gate) * norm(u; gamma_post, beta_post)
      y  = norm(x1; gamma_pre, beta_pre)

  and the gradients of x, u, gate, scale and the four norm parameters.
* ``adamw``: one AdamW step over the parameters of a whole stack of blocks
  (fp32 master weights, the bf16 copies that the projections read, states in
  32 or 8 bits), optionally after clipping by the norm of all gradients.

``run`` computes the plain form in elementary torch operations unless ``own``
is set, where it calls the library.
"""
import math

import torch

own = False

QBLOCK = 256      # elements that share a scale in the 8-bit states
FP8_MAX = 448.0   # largest e4m3 value
FP8_MIN = 2.0 ** -9   # smallest positive e4m3 value
EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY, MAX_NORM = 1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, op, B, I, J, C, types="bf16", kind="layer", gate="full", post=True, pre=True,
          transposed=False):
    return {"name": name, "op": op, "B": B, "I": I, "J": J, "C": C, "types": types,
            "kind": kind, "gate": gate, "post": post, "pre": pre, "transposed": transposed}


def _adamw(name, layers, width, bits, grads, clip):
    return {"name": name, "op": "adamw", "layers": layers, "width": width, "bits": bits,
            "grads": grads, "clip": clip}


def listed():
    return [
        # one token of a stream: what a launch costs
        _norm("fwd_one_row", "norm_fwd", 1, 1, 1, 128),
        # the pair representation of the N = 384 and N = 768 workloads
        _norm("fwd_pair_n384", "norm_fwd", 1, 384, 384, 128),
        _norm("fwd_pair_n768_row_gate", "norm_fwd", 1, 768, 768, 128, gate="row"),
        # a ragged MSA crop with a channel count that fits no vector
        _norm("fwd_msa_odd_f32", "norm_fwd", 1, 127, 193, 99, types="f32", kind="rms", gate="none"),
        # the single representation of an N = 384 crop, fp32
        _norm("bwd_single_n384", "norm_bwd", 1, 1, 384, 384, types="f32"),
        _norm("bwd_pair_n384", "norm_bwd", 1, 384, 384, 128),
        # the ending node's transposed views, the residual stream in fp32
        _norm("bwd_pair_n768_ending", "norm_bwd", 1, 768, 768, 128, types="mixed",
              transposed=True),
        # an MSA crop gated by one vector per batch entry (conditioning)
        _norm("bwd_msa_batch_gate", "norm_bwd", 2, 255, 383, 72, kind="rms", gate="batch"),
        # the parameters of one block: launch cost
        _adamw("adamw_one_block", 1, 128, 32, "f32", False),
        # a 48-block stack, 528 tensors, clipped
        _adamw("adamw_stack48_clip", 48, 128, 32, "bf16", True),
        # an odd width: tensors that end inside a block of the 8-bit states
        _adamw("adamw8_odd_clip", 12, 101, 8, "f32", True),
        # a wide stack, where only the memory rate counts
        _adamw("adamw8_wide", 6, 1024, 8, "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "adamw"])
    if op == "adamw":
        bits = rng.choice([32, 8])
        width = _log(rng, 8, 700)
        most = max(1, min(60, int(60e6 / (17 * width * width))))
        return {k: v for k, v in _adamw("", _log(rng, 1, most), width, bits,
                                        rng.choice(["bf16", "f32"]), rng.random() < 0.5).items()
                if k != "name"}
    C = rng.choice([_log(rng, 32, 1500), 8 * _log(rng, 4, 190), 64, 128, 256, 384])
    rows = _log(rng, 1, max(2, int(4.0e7 / C)))
    B = rng.choice([1, 1, 2, 3])
    I = max(1, min(_log(rng, 1, 768), rows // B))
    J = max(1, rows // (B * I))
    post = rng.random() < 0.85
    return {k: v for k, v in _norm("", op, B, I, J, C, types=rng.choice(["bf16", "bf16", "mixed", "f32"]),
                                   kind=rng.choice(["layer", "rms"]),
                                   gate=rng.choice(["full", "row", "batch", "none"]) if post else "none",
                                   post=post, pre=(not post) or rng.random() < 0.8,
                                   transposed=rng.random() < 0.3).items() if k != "name"}


def _block_shapes(C):
    """The parameter tensors of one pair-stack block of C channels (H = 4)."""
    return [(4 * C + 4, C), (C,), (C,),          # LayerNorm + projection: w, gamma, beta
            (C, C),                              # output projection
            (8 * C, C), (C, 4 * C), (C,), (C,),  # transition: w1, w2, gamma, beta
            (C,), (C,), (C,)]                    # post-norm gamma and beta, residual scale


def _n_norm(case):
    return case["B"] * case["I"] * case["J"], case["C"]


def work(case):
    if case["op"] == "adamw":
        n = case["layers"] * sum(math.prod(s) for s in _block_shapes(case["width"]))
        state = 16 if case["bits"] == 32 else 4 + 16 / QBLOCK
        grad = 2 if case["grads"] == "bf16" else 4
        return {"bytes": n * (8 + grad + state + 2), "flops": n * (16 + (2 if case["clip"] else 0))}
    rows, C = _n_norm(case)
    res = 2 if case["types"] == "bf16" else 4
    io = 4 if case["types"] == "f32" else 2
    gates = {"full": rows, "row": case["B"] * case["I"], "batch": case["B"], "none": 0}[case["gate"]]
    post, pre = case["post"], case["pre"]
    if case["op"] == "norm_fwd":
        per = res + (io + res if post else 0) + (io if pre else 0)
        return {"bytes": rows * C * per + gates * C * io, "flops": rows * C * (8 * post + 8 * pre + 4)}
    per = res + (res + io if pre else 0) + res + (2 * io if post else 0)
    return {"bytes": rows * C * per + 2 * gates * C * io, "flops": rows * C * (24 * post + 16 * pre)}


# ---------------------------------------------------------------------------
# what a user's program has in hand
# ---------------------------------------------------------------------------
def _prepare_norm(case, gen):
    B, I, J, C = case["B"], case["I"], case["J"], case["C"]
    res = torch.bfloat16 if case["types"] == "bf16" else torch.float32
    io = torch.float32 if case["types"] == "f32" else torch.bfloat16
    f32 = {"device": "cuda", "dtype": torch.float32}

    def rows(dtype, spread=False):
        shape = (B, J, I, C) if case["transposed"] else (B, I, J, C)
        t = torch.randn(shape, generator=gen, **f32)
        if spread:  # channels with an offset and a scale of their own
            t = t * (torch.rand(C, generator=gen, **f32) * 1.5 + 0.5) + torch.randn(C, generator=gen, **f32)
        t = t.to(dtype)
        return t.transpose(1, 2) if case["transposed"] else t

    def vector(mean, spread):
        return mean + spread * torch.randn(C, generator=gen, **f32)

    s = {"op": case["op"], "kind": case["kind"], "post": case["post"], "pre": case["pre"],
         "u": None, "gate": None, "scale": None, "gamma_post": None, "beta_post": None,
         "gamma_pre": None, "beta_pre": None, "dy": None, "y_dtype": io}
    layer = case["kind"] == "layer"
    if case["op"] == "norm_fwd":
        s["x"] = rows(res, True)
    else:
        s["x1"] = rows(res, True) if case["pre"] else None
        s["dx1"] = rows(res)
        s["dy"] = rows(io) if case["pre"] else None
    if case["post"]:
        s["u"] = rows(io, True)
        s["scale"], s["gamma_post"] = vector(0.5, 0.1), vector(1.0, 0.1)
        s["beta_post"] = vector(0.0, 0.1) if layer else None
        if case["gate"] == "full":
            s["gate"] = rows(io)
        elif case["gate"] != "none":
            shape = (B, I, 1, C) if case["gate"] == "row" else (B, 1, 1, C)
            s["gate"] = torch.randn(shape, generator=gen, **f32).to(io)
    if case["pre"]:
        s["gamma_pre"] = vector(1.0, 0.1)
        s["beta_pre"] = vector(0.0, 0.1) if layer else None
    return s


def _prepare_adamw(case, gen):
    """Parameters, their bf16 copies and the states lie in flat buffers, each
    tensor at a multiple of QBLOCK elements with zeros behind it; gradients are
    tensors of their own, which the backward pass fills anew for every step."""
    shapes = _block_shapes(case["width"]) * case["layers"]
    sizes = [math.prod(s) for s in shapes]
    padded = [-(-n // QBLOCK) * QBLOCK for n in sizes]
    starts = [0]
    for n in padded:
        starts.append(starts[-1] + n)
    total = starts[-1]
    f32 = {"device": "cuda", "dtype": torch.float32}
    real = torch.zeros(total, **f32)
    for a, n in zip(starts, sizes):
        real[a:a + n] = 1.0
    p = 0.02 * torch.randn(total, generator=gen, **f32) * real
    # second moments that spread over a few decades inside a block, first
    # moments below their square root, gradients of the same size
    r = 1e-3 * torch.exp(1.5 * torch.randn(total, generator=gen, **f32)) * real
    m = 0.3 * r * torch.randn(total, generator=gen, **f32)
    g = r * torch.randn(total, generator=gen, **f32)
    dtype = torch.bfloat16 if case["grads"] == "bf16" else torch.float32
    grads = [g[a:a + n].view(shape).to(dtype, copy=True) for a, n, shape in zip(starts, sizes, shapes)]

    def parts(flat):
        return [flat[a:a + n].view(shape) for a, n, shape in zip(starts, sizes, shapes)]

    s = {"op": "adamw", "bits": case["bits"], "p": p, "copy": p.to(torch.bfloat16), "grads": grads,
         "decay": [DECAY if len(shape) > 1 else 0.0 for shape in shapes], "padded": padded,
         "pads": [torch.zeros(b - n, **f32) for n, b in zip(sizes, padded)],
         "max_norm": MAX_NORM if case["clip"] else None,
         "step": torch.full((), 100, device="cuda", dtype=torch.int64)}
    if case["bits"] == 32:
        s["m"], s["v"] = m, r * r
    else:
        for name, t in (("m", m), ("v", r)):
            t = t.view(-1, QBLOCK)
            a = t.abs().amax(1, keepdim=True)
            s[name] = (t * (FP8_MAX / a)).to(torch.float8_e4m3fn).view(-1)
            s[name + "_scale"] = (a / FP8_MAX).view(-1).contiguous()
        # a positive root has a positive code
        low = torch.full((), FP8_MIN, **f32).to(torch.float8_e4m3fn)
        flat = s["v"].view(torch.uint8)
        flat[(flat == 0) & (real > 0)] = low.view(torch.uint8)
    if own:  # the optimizer object that a training program keeps
        from protein_folding_attention_gb300 import evoattn
        s["opt"] = evoattn.AdamW(
            parts(p), grads, copies=parts(s["copy"]), lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS,
            weight_decay=s["decay"], state_bits=case["bits"], exp_avg=s["m"], exp_avg_sq=s["v"],
            exp_avg_scale=s.get("m_scale"), exp_avg_sq_scale=s.get("v_scale"), step=100)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return (_prepare_adamw if case["op"] == "adamw" else _prepare_norm)(case, gen)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _standardise(v, kind):
    """(v - mean) * rstd (or v * rstd) over the channels, and rstd."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * rstd, rstd


def _affine(h, gamma, beta):
    h = h * gamma
    return h if beta is None else h + beta


def _plain_norm_fwd(s):
    x1 = s["x"].float()
    if s["post"]:
        h, _ = _standardise(s["u"].float(), s["kind"])
        t = s["scale"] * _affine(h, s["gamma_post"], s["beta_post"])
        if s["gate"] is not None:
            t = t / (1.0 + torch.exp(-s["gate"].float()))
        x1 = x1 + t
    y = None
    if s["pre"]:
        h, _ = _standardise(x1, s["kind"])
        y = _affine(h, s["gamma_pre"], s["beta_pre"]).to(s["y_dtype"])
    return {"x1": x1.to(s["x"].dtype) if s["post"] else None, "y": y}


def _standardise_grad(d, h, rstd, kind):
    d = d - h * (d * h).mean(-1, keepdim=True) - (d.mean(-1, keepdim=True) if kind == "layer" else 0.0)
    return d * rstd


def _plain_norm_bwd(s):
    out = {}
    D = s["dx1"].float()
    if s["pre"]:
        dy = s["dy"].float()
        h, rstd = _standardise(s["x1"].float(), s["kind"])
        out["dgamma_pre"] = (dy * h).sum((0, 1, 2))
        if s["beta_pre"] is not None:
            out["dbeta_pre"] = dy.sum((0, 1, 2))
        D = D + _standardise_grad(dy * s["gamma_pre"], h, rstd, s["kind"])
    out["dx"] = D.to(s["dx1"].dtype)
    if s["post"]:
        h, rstd = _standardise(s["u"].float(), s["kind"])
        w = _affine(h, s["gamma_post"], s["beta_post"])
        e = D * s["scale"]
        if s["gate"] is None:
            out["dscale"] = (D * w).sum((0, 1, 2))
        else:
            q = 1.0 / (1.0 + torch.exp(-s["gate"].float()))
            out["dscale"] = (D * q * w).sum((0, 1, 2))
            dg = e * w * (q * (1.0 - q))
            over = [i for i in range(3) if s["gate"].shape[i] == 1]
            out["dgate"] = (dg.sum(over, keepdim=True) if over else dg).to(s["gate"].dtype)
            e = e * q
        out["dgamma_post"] = (e * h).sum((0, 1, 2))
        if s["beta_post"] is not None:
            out["dbeta_post"] = e.sum((0, 1, 2))
        out["du"] = _standardise_grad(e * s["gamma_post"], h, rstd, s["kind"]).to(s["u"].dtype)
    return out


def _quantise(t, keep_positive):
    """Codes and scales of one 8-bit state."""
    t = t.view(-1, QBLOCK)
    a = t.abs().amax(1, keepdim=True)
    held = a >= 2.0 ** -100
    inverse = torch.where(held, FP8_MAX / a, torch.zeros_like(a))
    code = (t * inverse).to(torch.float8_e4m3fn).float()
    if keep_positive:
        code = torch.where((t > 0) & held & (code == 0), torch.full_like(code, FP8_MIN), code)
    return code.to(torch.float8_e4m3fn).view(-1), torch.where(held, a / FP8_MAX, torch.zeros_like(a)).view(-1)


def _plain_adamw(s):
    g = torch.cat([piece for g, pad in zip(s["grads"], s["pads"]) for piece in (g.reshape(-1).float(), pad)])
    step = s["step"].add_(1)
    norm = None
    if s["max_norm"] is not None:
        norm = torch.sqrt((g * g).sum(dtype=torch.float64)).float()
        g = g * torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    if s["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, QBLOCK) * s["m_scale"][:, None]).view(-1)
        r = (s["v"].float().view(-1, QBLOCK) * s["v_scale"][:, None]).view(-1)
        v = r * r
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    powers = torch.tensor([BETA1, BETA2], dtype=torch.float64, device=g.device) ** step
    correct = (1.0 - powers).float()
    decay = torch.repeat_interleave(torch.tensor(s["decay"], device=g.device),
                                    torch.tensor(s["padded"], device=g.device))
    update = (m / correct[0]) / (torch.sqrt(v / correct[1]) + ADAM_EPS)
    s["p"].copy_(s["p"] * (1.0 - LR * decay) - LR * update)
    s["copy"].copy_(s["p"])
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for name, t, keep in (("m", m, False), ("v", torch.sqrt(v), True)):
            code, scale = _quantise(t, keep)
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
    return norm


def _adamw_outputs(s, norm):
    return {"p": s["p"], "copy": s["copy"], "m": s["m"], "v": s["v"], "m_scale": s.get("m_scale"),
            "v_scale": s.get("v_scale"), "norm": norm}


def run(s):
    if s["op"] == "adamw":
        norm = s["opt"].step(max_norm=s["max_norm"]) if own else _plain_adamw(s)
        return _adamw_outputs(s, norm)
    if own:
        from protein_folding_attention_gb300 import evoattn
        kind = evoattn.NORM_LAYER if s["kind"] == "layer" else evoattn.NORM_RMS
        if s["op"] == "norm_fwd":
            x1, y = evoattn.block_norm(s["x"], s["u"], s["gate"], s["scale"], s["gamma_post"],
                                       s["beta_post"], s["gamma_pre"], s["beta_pre"], kind=kind,
                                       eps=EPS, pre=s["pre"], y_dtype=s["y_dtype"])
            return {"x1": x1 if s["post"] else None, "y": y}
        return evoattn.block_norm_bwd(s["dx1"], s["dy"], s["x1"], s["u"], s["gate"], s["scale"],
                                      s["gamma_post"], s["beta_post"], s["gamma_pre"],
                                      s["beta_pre"], kind=kind, eps=EPS)
    return (_plain_norm_fwd if s["op"] == "norm_fwd" else _plain_norm_bwd)(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_seam(x, u, gate, scale, g1, b1, g2, b2, kind):
    """x1 and y, through torch's differentiable operations in 64 bits."""
    def norm(v, gamma, beta):
        c = v.mean(dim=-1, keepdim=True) if kind == "layer" else 0.0
        var = v.var(dim=-1, keepdim=True, unbiased=False) if kind == "layer" else v.pow(2).mean(dim=-1, keepdim=True)
        n = (v - c) * (var + EPS).rsqrt() * gamma
        return n if beta is None else n + beta
    x1 = x
    if u is not None:
        t = norm(u, g1, b1) * scale
        x1 = x + (t if gate is None else t * gate.sigmoid())
    return x1, (None if g2 is None else norm(x1, g2, b2))


def _exact_norm(case, seed):
    s = prepare(case, seed)
    wide = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    names = ["u", "gate", "scale", "gamma_post", "beta_post", "gamma_pre", "beta_pre"]
    if case["op"] == "norm_fwd":
        x1, y = _exact_seam(wide["x"], *[wide[k] for k in names], case["kind"])
        return {"x1": x1 if case["post"] else None, "y": y}
    # y's gradient is taken at the stored x1, the branch's at u and the gate
    grads = {}
    D = wide["dx1"]
    if case["pre"]:
        at = [wide["x1"].requires_grad_(), wide["gamma_pre"].requires_grad_()]
        at += [] if wide["beta_pre"] is None else [wide["beta_pre"].requires_grad_()]
        _, y = _exact_seam(wide["x1"], None, None, None, None, None, wide["gamma_pre"], wide["beta_pre"], case["kind"])
        got = torch.autograd.grad(y, at, wide["dy"])
        D = D + got[0]
        grads["dgamma_pre"] = got[1]
        if wide["beta_pre"] is not None:
            grads["dbeta_pre"] = got[2]
    grads["dx"] = D
    if case["post"]:
        at = {k: wide[k].requires_grad_() for k in names[:5] if wide[k] is not None}
        x1, _ = _exact_seam(torch.zeros_like(D), *[wide[k] for k in names[:5]], None, None, case["kind"])
        for k, v in zip(at, torch.autograd.grad(x1, list(at.values()), D)):
            grads["d" + k] = v
    return {k: v.detach() for k, v in grads.items()}


def _exact_adamw(case, seed):
    s = prepare(case, seed)
    sizes = [g.numel() for g in s["grads"]]
    total = sum(s["padded"])
    real = torch.zeros(total, dtype=torch.float64, device="cuda")
    decay = torch.zeros_like(real)
    at = 0
    for g, wd, n, b in zip(s["grads"], s["decay"], sizes, s["padded"]):
        real[at:at + n] = g.double().reshape(-1)
        decay[at:at + b] = wd
        at += b
    norm = None
    if s["max_norm"] is not None:
        norm = torch.linalg.vector_norm(real)
        real *= min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    old_m, old_v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        old_m = old_m * s["m_scale"].double().repeat_interleave(QBLOCK)
        old_v = (old_v * s["v_scale"].double().repeat_interleave(QBLOCK)).square()
    m = torch.lerp(real, old_m, BETA1)
    v = torch.lerp(real.square(), old_v, BETA2)
    t = 101
    p = s["p"].double()
    p = p - LR * decay * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    out = {"p": p, "copy": p, "m": m, "v": v, "m_scale": None, "v_scale": None, "norm": norm}
    if case["bits"] == 8:
        for name, x in (("m", m), ("v", v.sqrt())):
            scale = x.abs().view(-1, QBLOCK).amax(1) / FP8_MAX
            x = x / scale.repeat_interleave(QBLOCK).clamp_min(1e-300)
            # e4m3: three bits behind the leading one, exponents from -6 (subnormal below)
            _, e = torch.frexp(x)
            ulp = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(-6) - 3)
            x = torch.round(x / ulp) * ulp
            if name == "v":
                x = torch.where((v > 0) & (x == 0), FP8_MIN, x)
            out[name], out[name + "_scale"] = x, scale
    return out


def exact(case, seed):
    return (_exact_adamw if case["op"] == "adamw" else _exact_norm)(case, seed)
