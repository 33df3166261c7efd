"""The 8-bit projection path around a block, as cases to measure.

* ``dropout``: out = x + keep * u / (1 - p), the residual add with a dropout
  whose mask is drawn from a counter-based generator and never stored; the mask
  may be shared along row axes (the row- and column-wise dropout of a pair
  stack).  Its gradient is the same call without x.
* ``norm8_fwd`` / ``norm8_bwd``: x1 = x + keep * u / (1 - p), y = norm(x1), y in
  e4m3 with a power-of-two scale for each 128 channels; and the gradients.
* ``quantize8``: a matrix in e4m3 with a scale for each 128 elements of a row,
  of a column (stored transposed), both in one pass, or for each 128 x 128 block.
* ``matmul8``: a b^T of two such matrices, in bf16 or fp32.

``run`` computes the plain form in elementary torch operations unless ``own``
is set, where it calls the library.
"""
import functools
import math

import torch

own = False

GROUP = 128       # elements that share a scale
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rows(name, op, B, I, J, C, types="bf16", kind="layer", branch=True, p=0.25, shared="none",
          transposed=False):
    return {"name": name, "op": op, "B": B, "I": I, "J": J, "C": C, "types": types, "kind": kind,
            "branch": branch, "p": p, "shared": shared, "transposed": transposed}


def _quantize(name, R, K, types, out):
    return {"name": name, "op": "quantize8", "R": R, "K": K, "types": types, "out": out}


def _matmul(name, M, N, K, scales="blocks", out="bf16", add=False):
    return {"name": name, "op": "matmul8", "M": M, "N": N, "K": K, "scales": scales, "out": out, "add": add}


def listed():
    return [
        # the residual add after triangle attention on the N = 384 pair tensor,
        # one mask for all rows i (row-wise dropout)
        _rows("dropout_pair_n384_shared", "dropout", 1, 384, 384, 128, shared="i"),
        # a ragged MSA crop with a channel count that fits no vector, every
        # element with its own random number
        _rows("dropout_msa_odd_f32", "dropout", 1, 127, 193, 99, types="f32", p=0.15),
        # one token of a stream: what a launch costs
        _rows("norm8_one_row", "norm8_fwd", 1, 1, 1, 128, kind="rms", p=0.0),
        # between two blocks of the N = 768 workload
        _rows("norm8_pair_n768", "norm8_fwd", 1, 768, 768, 128, shared="i"),
        # the same seam backwards, N = 384, ending node (transposed views)
        _rows("norm8_bwd_pair_n384", "norm8_bwd", 1, 384, 384, 128, shared="j", transposed=True),
        # two MSA crops with an fp32 stream and an odd width
        _rows("norm8_bwd_msa_mixed", "norm8_bwd", 2, 255, 383, 72, types="mixed", kind="rms", p=0.15),
        # a gradient of the transition's hidden layer (N = 384, F = 512): rows
        # for the input's gradient, columns for the weight's
        _quantize("quantize8_hidden_both", 147456, 512, "bf16", "both"),
        # an fp32 weight of odd sizes in 128 x 128 blocks
        _quantize("quantize8_weight_odd", 1001, 333, "f32", "blocks"),
        # one token through a wide layer: the weight is read once
        _matmul("matmul8_one_token", 1, 4096, 1536),
        # q, k, v, gate and pair bias of the N = 768 pair tensor (4 * 128 + 4 columns)
        _matmul("matmul8_pair_proj_n768", 589824, 516, 128),
        # the gradient of a 512 x 128 weight over the N = 384 pair tensor's rows
        _matmul("matmul8_weight_grad", 512, 128, 147456, scales="rows", out="f32", add=True),
        # a wide layer, where the tensor cores count
        _matmul("matmul8_wide", 8192, 4096, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _draw_rows(rng, op):
    C = rng.choice([_log(rng, 32, 1500), 8 * _log(rng, 4, 190), 64, 128, 256, 384])
    rows = _log(rng, 1, max(2, int(4.0e7 / C)))
    B = rng.choice([1, 1, 2, 3])
    I = max(1, min(_log(rng, 1, 768), rows // B))
    J = max(1, rows // (B * I))
    branch = op == "dropout" or rng.random() < 0.8
    return _rows("", op, B, I, J, C, types=rng.choice(["bf16", "bf16", "mixed", "f32"]),
                 kind=rng.choice(["layer", "rms"]), branch=branch,
                 p=rng.choice([0.0, 0.1, 0.15, 0.25]) if branch and op != "dropout" else 0.25 if branch else 0.0,
                 shared=rng.choice(["none", "i", "j"]) if branch else "none",
                 transposed=rng.random() < 0.3)


def _draw_matmul(rng):
    if rng.random() < 0.25:  # a few tokens
        M, N, K = _log(rng, 1, 128), _log(rng, 64, 8000), _log(rng, 64, 8000)
        return _matmul("", M, N, K, out=rng.choice(["bf16", "f32"]))
    if rng.random() < 0.33:  # a long sum and a small result
        M, N = _log(rng, 32, 1024), _log(rng, 32, 1024)
        K = _log(rng, 2000, min(3.0e5, 2.0e8 / max(M, N), 3.0e10 / (M * N)))
        return _matmul("", M, N, K, scales="rows", out="f32", add=rng.random() < 0.5)
    N, K = _log(rng, 32, 4096), _log(rng, 32, 4096)
    M = _log(rng, 64, min(6.0e5, 2.0e8 / max(N, K), 1.0e11 / (N * K)))
    return _matmul("", M, N, K, scales=rng.choice(["blocks", "rows"]), out=rng.choice(["bf16", "bf16", "f32"]),
                   add=rng.random() < 0.25)


def draw(rng):
    op = rng.choice(["dropout", "norm8_fwd", "norm8_bwd", "quantize8", "matmul8", "matmul8"])
    if op == "matmul8":
        case = _draw_matmul(rng)
    elif op == "quantize8":
        K = rng.choice([_log(rng, 16, 4096), 128 * _log(rng, 1, 32)])
        case = _quantize("", _log(rng, 1, 7.0e7 / K), K, rng.choice(["bf16", "f32"]),
                         rng.choice(["rows", "cols", "both", "blocks"]))
    else:
        case = _draw_rows(rng, op)
    return {k: v for k, v in case.items() if k != "name"}


def _types(case):
    """Types of the residual stream and of the block's tensors."""
    return (torch.bfloat16 if case["types"] == "bf16" else torch.float32,
            torch.float32 if case["types"] == "f32" else torch.bfloat16)


def work(case):
    if case["op"] == "matmul8":
        M, N, K = case["M"], case["N"], case["K"]
        groups = -(-K // GROUP)
        wide = 2 if case["out"] == "bf16" else 4
        b_scales = (N if case["scales"] == "rows" else -(-N // GROUP)) * groups
        return {"bytes": (M + N) * K + M * groups + b_scales + M * N * wide * (2 if case["add"] else 1),
                "flops": 2 * M * N * K}
    if case["op"] == "quantize8":
        n = case["R"] * case["K"]
        copies = {"rows": 1, "cols": 1, "both": 2, "blocks": 2}[case["out"]]
        return {"bytes": n * ((2 if case["types"] == "bf16" else 4) + copies * (1 + 1 / GROUP)), "flops": 4 * n}
    n = case["B"] * case["I"] * case["J"] * case["C"]
    res, io = (t.itemsize for t in _types(case))
    if case["op"] == "dropout":
        return {"bytes": n * (2 * res + io), "flops": 4 * n}
    if case["op"] == "norm8_fwd":
        return {"bytes": n * (res + (io + res if case["branch"] else 0) + 1 + 1 / GROUP), "flops": 12 * n}
    return {"bytes": n * (3 * res + io + (io if case["branch"] else 0)), "flops": 20 * n}


# ---------------------------------------------------------------------------
# what a user's program has in hand
# ---------------------------------------------------------------------------
def _exponents(amax):
    """k of the smallest power of two 2^k >= amax / 448 (0 for amax = 0, -127 at least)."""
    m, e = torch.frexp(amax)
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-127)
    return torch.where(amax > 0, k, torch.zeros_like(k))


def _codes(t, k):
    return torch.ldexp(t, -k).to(torch.float8_e4m3fn)


def _e8m0(k):
    return (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _groups(t):
    """The last axis in groups of 128, the last one filled up with zeros."""
    return torch.nn.functional.pad(t, (0, -t.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP))


def _quantise_rows(t):
    """Codes and scales of groups along the last axis of an fp32 tensor."""
    g = _groups(t)
    k = _exponents(g.abs().amax(-1))
    return _codes(g, k.unsqueeze(-1)).flatten(-2)[..., :t.shape[-1]], _e8m0(k)


def _quantise_blocks(t):
    R, K = t.shape
    g = _groups(torch.nn.functional.pad(t, (0, 0, 0, -R % GROUP))).unflatten(0, (-1, GROUP))
    k = _exponents(g.abs().amax((1, 3)))
    return _codes(g, k[:, None, :, None]).flatten(2).flatten(0, 1)[:R, :K], _e8m0(k)


def _operand(t, blocks):
    """An operand of the product as the library keeps it: rows of codes at a
    multiple of 16 bytes, scales with the rows innermost."""
    q, s = (_quantise_blocks if blocks else _quantise_rows)(t)
    R, K = t.shape
    codes = torch.zeros((R, -(-K // 16) * 16), device="cuda", dtype=torch.float8_e4m3fn)
    codes[:, :K] = q
    scales = s.view(torch.uint8).t().contiguous().t().view(torch.float8_e8m0fnu)
    return codes[:, :K], scales


def _prepare_matmul(case, gen):
    M, N, K = case["M"], case["N"], case["K"]
    f32 = {"device": "cuda", "dtype": torch.float32}
    # activations whose rows and channels have a size of their own, weights of variance 1 / K
    a = torch.randn((M, K), generator=gen, **f32)
    a *= torch.exp(0.7 * torch.randn((M, 1), generator=gen, **f32))
    a *= 0.5 + torch.rand(K, generator=gen, **f32)
    b = torch.randn((N, K), generator=gen, **f32) * K ** -0.5
    s = {"op": "matmul8", "dtype": torch.bfloat16 if case["out"] == "bf16" else torch.float32}
    s["a"], s["a_scale"] = _operand(a, False)
    s["b"], s["b_scale"] = _operand(b, case["scales"] == "blocks")
    s["add"] = torch.randn((M, N), generator=gen, **f32).to(s["dtype"]) if case["add"] else None
    return s


def _prepare_rows(case, gen):
    B, I, J, C = case["B"], case["I"], case["J"], case["C"]
    res, io = _types(case)
    f32 = {"device": "cuda", "dtype": torch.float32}

    def rows(dtype, spread=False):
        shape = (B, J, I, C) if case["transposed"] else (B, I, J, C)
        t = torch.randn(shape, generator=gen, **f32)
        if spread:  # channels with an offset and a scale of their own
            t = t * (torch.rand(C, generator=gen, **f32) * 1.5 + 0.5) + torch.randn(C, generator=gen, **f32)
        t = t.to(dtype)
        return t.transpose(1, 2) if case["transposed"] else t

    s = {"op": case["op"], "kind": case["kind"], "p": case["p"], "branch": case["branch"],
         "shared": {"none": (), "i": (1,), "j": (2,)}[case["shared"]], "site": 3, "io": io,
         # the generator's state as a training program holds it: seed and step
         "rng": torch.randint(1 << 40, (2,), generator=gen, device="cuda")}
    if case["op"] == "norm8_bwd":
        s["x1"], s["dx1"], s["dy"] = rows(res, True), rows(res), rows(io)
    else:
        s["x"], s["u"] = rows(res, True), rows(io, True) if case["branch"] else None
    if case["op"] != "dropout":
        s["gamma"] = 1.0 + 0.1 * torch.randn(C, generator=gen, **f32)
        s["beta"] = 0.1 * torch.randn(C, generator=gen, **f32) if case["kind"] == "layer" else None
    return s


def _prepare_quantize(case, gen):
    R, K = case["R"], case["K"]
    f32 = {"device": "cuda", "dtype": torch.float32}
    t = torch.randn((R, K), generator=gen, **f32) * torch.exp(torch.randn((R, 1), generator=gen, **f32))
    return {"op": "quantize8", "out": case["out"],
            "x": t.to(torch.bfloat16 if case["types"] == "bf16" else torch.float32)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    make = {"matmul8": _prepare_matmul, "quantize8": _prepare_quantize}.get(case["op"], _prepare_rows)
    return make(case, gen)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
LOW32 = 0xFFFFFFFF


def _philox_round(state, r):
    """One of the ten rounds of Philox4x32 (Salmon et al., 2011)."""
    c0, c1, c2, c3, k0, k1 = state
    p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57   # 64-bit products, wrapped: the bits are right
    return ((p1 >> 32 & LOW32) ^ c1 ^ k0, p1 & LOW32, (p0 >> 32 & LOW32) ^ c3 ^ k1, p0 & LOW32,
            k0 + 0x9E3779B9 & LOW32, k1 + 0xBB67AE85 & LOW32)


def _keep(s, shape):
    """The mask: channel c of a mask row takes word c % 4 of the block with the
    counter (c / 4, row, site, step) and the key seed."""
    C = shape[3]
    lead = [1 if i in s["shared"] else n for i, n in enumerate(shape[:3])]
    dev = s["rng"].device
    row = torch.arange(math.prod(lead), device=dev).view(-1, 1)
    group = torch.arange(-(-C // 4), device=dev).view(1, -1)
    seed, step = s["rng"][0], s["rng"][1]
    zero = row * 0 + group * 0
    start = (zero + group, zero + row, zero + s["site"], zero + (step & LOW32),
             zero + (seed & LOW32), zero + (seed >> 32 & LOW32))
    words = torch.stack(functools.reduce(_philox_round, range(10), start)[:4], -1)
    threshold = min(int(math.floor(s["p"] * 2.0 ** 32 + 0.5)), LOW32)
    return (words >= threshold).flatten(-2)[:, :C].reshape(*lead, C)


def _dropped(s, t):
    """keep * t / (1 - p)"""
    if s["p"] == 0.0:
        return t
    return torch.where(_keep(s, t.shape), t * (1.0 / (1.0 - s["p"])), torch.zeros_like(t))


def _standardise(v, kind):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * rstd, rstd


def _plain_norm8(s):
    x1 = s["x"].float()
    if s["branch"]:
        x1 = x1 + _dropped(s, s["u"].float())
    h, _ = _standardise(x1, s["kind"])
    y = h * s["gamma"]
    q, scale = _quantise_rows(y if s["beta"] is None else y + s["beta"])
    return {"x1": x1.to(s["x"].dtype) if s["branch"] else None, "y": q, "scale": scale}


def _plain_norm8_bwd(s):
    dy = s["dy"].float()
    h, rstd = _standardise(s["x1"].float(), s["kind"])
    out = {"dgamma": (dy * h).sum((0, 1, 2))}
    if s["beta"] is not None:
        out["dbeta"] = dy.sum((0, 1, 2))
    d = dy * s["gamma"]
    g = d - h * (d * h).mean(-1, keepdim=True) - (d.mean(-1, keepdim=True) if s["kind"] == "layer" else 0.0)
    D = s["dx1"].float() + g * rstd
    out["dx"] = D.to(s["dx1"].dtype)
    if s["branch"]:
        out["du"] = _dropped(s, D).to(s["io"])
    return out


def _plain_quantize(s):
    x, out = s["x"].float(), s["out"]
    if out == "blocks":
        q, k = _quantise_blocks(x)
        return {"codes": q, "scales": k, "codes_t": q.t().contiguous(), "scales_t": k.t()}
    r = {}
    if out != "cols":
        r["codes"], r["scales"] = _quantise_rows(x)
    if out != "rows":
        r["codes_t"], r["scales_t"] = _quantise_rows(x.t())
    return r


def _values(codes, scales):
    """What codes stand for, in 32 bits."""
    R, K = codes.shape
    s = scales.float()
    if s.shape[0] != R:
        s = s.repeat_interleave(GROUP, 0)[:R]
    return codes.float() * s.repeat_interleave(GROUP, 1)[:, :K]


def _plain_matmul(s):
    out = _values(s["a"], s["a_scale"]) @ _values(s["b"], s["b_scale"]).t()
    if s["add"] is not None:
        out = out + s["add"].float()
    return out.to(s["dtype"])


def _plain(s):
    if s["op"] == "dropout":
        return (s["x"].float() + _dropped(s, s["u"].float())).to(s["x"].dtype)
    return {"norm8_fwd": _plain_norm8, "norm8_bwd": _plain_norm8_bwd, "quantize8": _plain_quantize,
            "matmul8": _plain_matmul}[s["op"]](s)


def _own(s):
    from protein_folding_attention_gb300 import evoattn
    op = s["op"]
    if op == "matmul8":
        return evoattn.matmul8(s["a"], s["a_scale"], s["b"], s["b_scale"], add=s["add"], out_dtype=s["dtype"])
    if op == "quantize8":
        out = s["out"]
        if out == "blocks":
            r = evoattn.quantize8(s["x"], cols=True, blocks=True)
        else:
            r = evoattn.quantize8(s["x"], rows=out != "cols", cols=out != "rows")
        return dict(zip([n for n in ("codes", "scales", "codes_t", "scales_t")
                         if out in ("both", "blocks") or n.endswith("_t") == (out == "cols")], r))
    mask = {"p": s["p"], "rng": s["rng"], "site": s["site"], "shared": s["shared"]}
    if op == "dropout":
        return evoattn.dropout_add(s["u"], x=s["x"], **mask)
    kind = evoattn.NORM_LAYER if s["kind"] == "layer" else evoattn.NORM_RMS
    if op == "norm8_fwd":
        x1, y, scale = evoattn.norm8(s["x"], s["u"], s["gamma"], s["beta"], kind=kind, eps=EPS, **mask)
        return {"x1": x1 if s["branch"] else None, "y": y, "scale": scale}
    return evoattn.norm8_bwd(s["dx1"], s["dy"], s["x1"], s["gamma"], s["beta"], kind=kind, eps=EPS,
                             branch=s["branch"], **mask)


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _mulhilo(a, m):
    """High and low half of a 32 x 32 bit product, from 16-bit halves."""
    lo, hi = a & 0xFFFF, a >> 16
    x, y = lo * (m & 0xFFFF), hi * (m & 0xFFFF)
    z, w = lo * (m >> 16), hi * (m >> 16)
    mid = (x >> 16) + (y & 0xFFFF) + (z & 0xFFFF)
    return w + (y >> 16) + (z >> 16) + (mid >> 16), (x & 0xFFFF) | (mid & 0xFFFF) << 16


def _exact_mask(s, shape):
    """keep / (1 - p), in 64 bits, over `shape` (1 along shared axes)."""
    B, I, J, C = (1 if i in s["shared"] else n for i, n in enumerate(shape))
    seed, step = (int(v) for v in s["rng"].tolist())
    flat = torch.arange(B * I * J, device=s["rng"].device)
    c = [torch.arange((C + 3) // 4, device=flat.device).repeat(B * I * J, 1),
         flat[:, None].repeat(1, (C + 3) // 4)]
    c += [torch.full_like(c[0], s["site"]), torch.full_like(c[0], step % 2 ** 32)]
    key = [seed % 2 ** 32, (seed >> 32) % 2 ** 32]
    for _ in range(10):
        h0, l0 = _mulhilo(c[0], 0xD2511F53)
        h1, l1 = _mulhilo(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    r = torch.empty((B * I * J, 4 * c[0].shape[1]), dtype=torch.int64, device=flat.device)
    for w in range(4):
        r[:, w::4] = c[w]
    # a word at or above p 2^32 (to the nearest whole number) keeps its element
    kept = r[:, :C] >= min(round(s["p"] * 2 ** 32), 2 ** 32 - 1)
    return kept.view(B, I, J, C).double() / (1.0 - s["p"])


def _exact_norm(v, gamma, beta, kind):
    c = v.mean(dim=-1, keepdim=True) if kind == "layer" else 0.0
    var = v.var(dim=-1, keepdim=True, unbiased=False) if kind == "layer" else v.pow(2).mean(dim=-1, keepdim=True)
    n = (v - c) * (var + EPS).rsqrt() * gamma
    return n if beta is None else n + beta


def _exact_codes(t, over):
    """Codes (as their values) and the exponents of groups over the axes `over`."""
    a = t.abs().amax(over, keepdim=True)
    k = torch.ceil(torch.log2(a.clamp_min(1e-300) / 448.0))
    k = torch.where(torch.exp2(k - 1) * 448.0 >= a, k - 1, k)  # a rounded logarithm
    k = torch.where(torch.exp2(k) * 448.0 < a, k + 1, k)
    k = torch.where(a > 0, k.clamp_min(-127), torch.zeros_like(k))
    x = t / torch.exp2(k)
    # e4m3: three bits behind the leading one, exponents from -6 (subnormal below)
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20)))
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e)
    ulp = torch.exp2(e.clamp_min(-6) - 3)
    return torch.round(x / ulp) * ulp, torch.exp2(k)


def _exact_rows8(t):
    lead, C = t.shape[:-1], t.shape[-1]
    full = t.new_zeros(*lead, (C + GROUP - 1) // GROUP * GROUP)
    full[..., :C] = t
    q, k = _exact_codes(full.view(*lead, -1, GROUP), -1)
    return q.reshape(*lead, -1)[..., :C], k.squeeze(-1)


def _exact_blocks8(t):
    R, K = t.shape
    full = t.new_zeros((R + GROUP - 1) // GROUP * GROUP, (K + GROUP - 1) // GROUP * GROUP)
    full[:R, :K] = t
    q, k = _exact_codes(full.view(full.shape[0] // GROUP, GROUP, -1, GROUP), (1, 3))
    return q.reshape(full.shape)[:R, :K], k.view(k.shape[0], k.shape[2])


def _exact_values(codes, scales):
    full = scales.view(torch.uint8).to(torch.int32) - 127
    R, K = codes.shape
    r = torch.arange(R, device="cuda") // (1 if full.shape[0] == R else GROUP)
    return codes.double() * torch.exp2(full.double())[r][:, torch.arange(K, device="cuda") // GROUP]


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() if isinstance(v, torch.Tensor) and v.dtype in (torch.bfloat16, torch.float32) else v
            for k, v in s.items()}
    if case["op"] == "matmul8":
        out = torch.einsum("mk,nk->mn", _exact_values(s["a"], s["a_scale"]), _exact_values(s["b"], s["b_scale"]))
        return out if s["add"] is None else out + wide["add"]
    if case["op"] == "quantize8":
        if case["out"] == "blocks":
            q, k = _exact_blocks8(wide["x"])
            return {"codes": q, "scales": k, "codes_t": q.t(), "scales_t": k.t()}
        out = {}
        if case["out"] != "cols":
            out["codes"], out["scales"] = _exact_rows8(wide["x"])
        if case["out"] != "rows":
            out["codes_t"], out["scales_t"] = _exact_rows8(wide["x"].t())
        return out
    if case["op"] == "dropout":
        return wide["x"] + wide["u"] * _exact_mask(s, s["u"].shape)
    if case["op"] == "norm8_fwd":
        x1 = wide["x"]
        if s["branch"]:
            x1 = x1 + (wide["u"] * _exact_mask(s, x1.shape) if s["p"] else wide["u"])
        q, k = _exact_rows8(_exact_norm(x1, wide["gamma"], wide["beta"], case["kind"]))
        return {"x1": x1 if s["branch"] else None, "y": q, "scale": k}
    # y's gradient passes through its rounding
    at = [wide["x1"].requires_grad_(), wide["gamma"].requires_grad_()]
    at += [] if wide["beta"] is None else [wide["beta"].requires_grad_()]
    y = _exact_norm(wide["x1"], wide["gamma"], wide["beta"], case["kind"])
    got = torch.autograd.grad(y, at, wide["dy"])
    D = wide["dx1"] + got[0]
    out = {"dgamma": got[1], "dx": D}
    if wide["beta"] is not None:
        out["dbeta"] = got[2]
    if s["branch"]:
        out["du"] = D * _exact_mask(s, D.shape) if s["p"] else D
    return out
