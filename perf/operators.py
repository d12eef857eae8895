"""Cases, plain forms and definitions of the operators of a gated FP8 MLP half.

Three operators, each with the ranges it is used at:
  norm   root-mean-square norm of the residual stream with the residual's
         addition, its output quantized to E4M3 in 1x128 blocks (rowwise, and
         transposed for training), and the backward pass;
  gated  gated feed-forward H = act(X Wg^T) * (X Wu^T) on FP8 operands
         (tensorwise or block scaling), and the backward pass;
  clip   global gradient norm over many tensors, and clipping.

own = False: elementary torch operations in fp32.  own = True: the calls that
a user makes of the framework.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX, E5M2_MAX = 448.0, 57344.0
EPS = 1e-6


def listed():
    return [
        # one token of a d = 4096 model being decoded: pure latency
        dict(name="norm token", op="norm", train=False, R=1, C=4096, residual=True),
        # a ragged prefill batch of a wide model, serving (no transposed copy)
        dict(name="norm prefill", op="norm", train=False, R=1999, C=8192, residual=True),
        # the d = 512 model's microbatch (64 x 2048 tokens), forward and backward
        dict(name="norm train 512", op="norm", train=True, R=131072, C=512, residual=True),
        # the large MLP's microbatch with a ragged token count, forward and backward
        dict(name="norm train 4096", op="norm", train=True, R=16379, C=4096, residual=True),
        # one token through the large MLP: the weights stream once
        dict(name="gated token", op="gated", train=False, N=1, K=4096, F=14336, recipe="block", act="silu"),
        # a decode batch of the small model, tensorwise
        dict(name="gated decode 37", op="gated", train=False, N=37, K=512, F=2048, recipe="tensorwise", act="silu"),
        # a prefill of the large MLP with an odd token count
        dict(name="gated prefill", op="gated", train=False, N=2049, K=4096, F=14336, recipe="block", act="silu"),
        # the small model's microbatch: tensorwise recipe, forward and backward
        dict(name="gated train 512", op="gated", train=True, N=131072, K=512, F=2048, recipe="tensorwise",
             act="silu"),
        # the large MLP's microbatch: block recipe, forward and backward
        dict(name="gated train 4096", op="gated", train=True, N=16384, K=4096, F=14336, recipe="block", act="gelu"),
        # the vectors of one layer (norm weights, biases): latency
        dict(name="clip vectors", op="clip", tensors=9, numel=515, bf16=False, max_norm=1.0),
        # the 8-layer d = 512 stack's fp32 gradient accumulators
        dict(name="clip stack", op="clip", tensors=16, numel=512 * 2048, bf16=False, max_norm=1.0),
        # the large MLP's bf16 weight gradients
        dict(name="clip large", op="clip", tensors=7, numel=4096 * 14336, bf16=True, max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gated", "gated", "clip"])
    if op == "norm":
        train = rng.random() < 0.6
        C = 16 * _log(rng, 8, 512)
        R = _log(rng, 1, min(131072, 16384 * 4096 // C))
        return dict(op="norm", train=train, R=R, C=C, residual=rng.random() < 0.7)
    if op == "gated":
        train = rng.random() < 0.5
        recipe = rng.choice(["tensorwise", "block"])
        K = 16 * _log(rng, 8, 256)
        F = 128 * _log(rng, 2, 112) if recipe == "block" else 16 * _log(rng, 16, 896)
        most = max(1, min(131072, 16384 * 4096 * 14336 // (K * F)))
        N = _log(rng, 1, most if train or rng.random() < 0.5 else min(most, 300))
        return dict(op="gated", train=train, N=N, K=K, F=F, recipe=recipe, act=rng.choice(["silu", "gelu"]))
    numel = _log(rng, 100, 4096 * 14336)
    tensors = rng.randint(1, max(1, min(40, 7 * 4096 * 14336 // (2 * numel))))
    return dict(op="clip", tensors=tensors, numel=numel, bf16=rng.random() < 0.5,
                max_norm=rng.choice([0.5, 1.0, 1e9]))


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, sigma, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(sigma).to(dtype)


def _stream(gen, R, C):
    """A residual stream: unit normal, with a few channels twenty times larger."""
    x = torch.randn((R, C), generator=gen, device="cuda", dtype=torch.float32)
    big = torch.randint(0, C, (max(1, C // 256),), generator=gen, device="cuda")
    x[:, big] *= 20.0
    return x.to(torch.bfloat16)


def _sizes(case):
    """Element counts of the gradients: the named size, and smaller odd ones."""
    n = case["numel"]
    return [n if i % 2 == 0 else n // 2 + (i * 37) % 101 + 1 for i in range(case["tensors"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        R, C = case["R"], case["C"]
        s["x"] = _stream(gen, R, C)
        s["res"] = _normal(gen, (R, C), 1.0) if case["residual"] else None
        s["w"] = (1.0 + 0.1 * torch.randn(C, generator=gen, device="cuda")).float()
        if case["train"]:
            s["dy"] = _normal(gen, (R, C), 1e-3)
            s["dr"] = _normal(gen, (R, C), 1e-3)
        if own:
            import fp8_mixed_precision_gb300 as fp
            s["out"] = fp.rmsnorm_buffers(R, C, "cuda", residual=case["residual"], colwise=case["train"])
            if case["train"]:
                s["ws"] = fp.rmsnorm_workspace(R, C, "cuda")
                s["dx"] = torch.empty((R, C), dtype=torch.bfloat16, device="cuda")
                s["dw"] = torch.empty(C, dtype=torch.float32, device="cuda")
    elif case["op"] == "gated":
        N, K, F = case["N"], case["K"], case["F"]
        s["x"] = _normal(gen, (N, K), 1.0)
        w = _normal(gen, (2 * F, K), 0.02)
        if case["train"]:
            s["dh"] = _normal(gen, (N, F), 1e-3)
        if own:
            import fp8_mixed_precision_gb300 as fp
            s["cache"] = fp.WeightCache()
            s["h"] = s["cache"].register(w, case["recipe"])
            s["cache"].begin_cycle()
            s["cache"].get(s["h"])
            s["ws"] = fp.gated_workspace(case["recipe"], N, K, F, "cuda", train=case["train"])
            s["y"] = torch.empty((N, F), dtype=torch.bfloat16, device="cuda")
            if case["train"]:
                s["ctx"] = fp.gated_context(case["recipe"], N, K, F, "cuda")
                s["dx"] = torch.empty((N, K), dtype=torch.bfloat16, device="cuda")
                s["dw"] = torch.empty((2 * F, K), dtype=torch.bfloat16, device="cuda")
        else:  # the FP8 weight that a program keeps for all microbatches of a cycle
            s["wq"] = _weight_values(w, case["recipe"])
    else:
        dtype = torch.bfloat16 if case["bf16"] else torch.float32
        s["grads"] = [_normal(gen, (n,), 1e-2, dtype) for n in _sizes(case)]
        if own:
            import fp8_mixed_precision_gb300 as fp
            s["clip"] = fp.GradClip(s["grads"], [torch.empty_like(g) for g in s["grads"]])
    return s


# ---------------------------------------------------------------- plain forms
def _scales(amax, fmax):
    """scale = fp32(fmax / amax) and its reciprocal; 1 where nothing is there."""
    scale = torch.where(amax == 0, torch.ones_like(amax), torch.full_like(amax, fmax) / amax)  # one division
    scale = scale.clamp(max=torch.finfo(torch.float32).max)
    return scale, torch.ones_like(scale) / scale


def _cast(v, scale, fmax):
    fmt = torch.float8_e4m3fn if fmax == E4M3_MAX else torch.float8_e5m2
    return (v * scale).clamp(-fmax, fmax).to(fmt)


def _blocks(v, fmax):
    """1x128 blocks along the last axis: (codes, scale_inv)."""
    R, C = v.shape
    nb = -(-C // 128)
    p = torch.nn.functional.pad(v, (0, nb * 128 - C)).view(R, nb, 128)
    scale, inv = _scales(p.abs().amax(-1), fmax)
    return _cast(p, scale[..., None], fmax).view(R, nb * 128)[:, :C], inv


def _values(q, inv):
    """What codes in 1x128 blocks along the last axis stand for."""
    return q.float() * inv.repeat_interleave(128, 1)[:, : q.shape[1]]


def _tensor_values(v, fmax):
    scale, inv = _scales(v.abs().amax(), fmax)
    return _cast(v, scale, fmax).float() * inv


def _weight_values(w, recipe):
    v = w.float()
    if recipe == "tensorwise":
        return _tensor_values(v, E4M3_MAX)
    O, K = v.shape
    a, b = -(-O // 128), -(-K // 128)
    p = torch.nn.functional.pad(v, (0, b * 128 - K, 0, a * 128 - O)).view(a, 128, b, 128)
    scale, inv = _scales(p.abs().amax((1, 3)), E4M3_MAX)
    q = _cast(p, scale[:, None, :, None], E4M3_MAX).float() * inv[:, None, :, None]
    return q.view(a * 128, b * 128)[:O, :K].contiguous()


def _plain_norm(s):
    r = (s["x"].float() + s["res"].float()).to(torch.bfloat16) if s["residual"] else s["x"]
    rf = r.float()
    rstd = torch.rsqrt((rf * rf).mean(-1) + EPS)
    y = rf * rstd[:, None] * s["w"]
    row, row_inv = _blocks(y, E4M3_MAX)
    out = dict(r=r, rstd=rstd, row=row, row_scale_inv=row_inv)
    if s["train"]:
        # the transposed copy is padded with zeros to a multiple of 16 tokens
        yt = torch.nn.functional.pad(y.t(), (0, -s["R"] % 16))
        out["col"], out["col_scale_inv"] = _blocks(yt, E4M3_MAX)
        dy = s["dy"].float()
        g = dy * s["w"]
        c = (g * rf).mean(-1) * rstd * rstd * rstd
        out["dx"] = (s["dr"].float() + g * rstd[:, None] - rf * c[:, None]).to(torch.bfloat16)
        out["dw"] = (dy * rf * rstd[:, None]).sum(0)
    return out


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    phi = 0.5 * torch.erfc(-g * math.sqrt(0.5))
    return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_gated(s):
    block, F, wq = s["recipe"] == "block", s["F"], s["wq"]
    x = s["x"].float()
    xq = _values(*_blocks(x, E4M3_MAX)) if block else _tensor_values(x, E4M3_MAX)
    gu = xq @ wq.t()
    h = (_act(gu[:, :F], s["act"])[0] * gu[:, F:]).to(torch.bfloat16)
    if not s["train"]:
        return dict(h=h)
    # the backward pass reads both projections as the forward pass kept them, in bf16
    kept = gu.to(torch.bfloat16).float()
    a, da = _act(kept[:, :F], s["act"])
    dh = s["dh"].float()
    dgu = torch.cat([dh * kept[:, F:] * da, dh * a], 1)
    if block:  # each layout has its own blocks along its own contiguous axis
        drow = _values(*_blocks(dgu, E5M2_MAX))
        dcol = _values(*_blocks(dgu.t(), E5M2_MAX))
        xcol = _values(*_blocks(x.t(), E4M3_MAX))
    else:
        drow = _tensor_values(dgu, E5M2_MAX)
        dcol, xcol = drow.t(), xq.t()
    return dict(h=h, dx=(drow @ wq).to(torch.bfloat16), dw=(dcol @ xcol.t()).to(torch.bfloat16))


def _plain_clip(s):
    flat = torch.cat(s["grads"]).float()
    norm = (flat * flat).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    out = (flat * coef).to(s["grads"][0].dtype)
    return dict(norm=norm.reshape(1), grads=list(out.split(_sizes(s))))


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "gated": _plain_gated, "clip": _plain_clip}[s["op"]](s)
    import fp8_mixed_precision_gb300 as fp
    if s["op"] == "norm":
        o = fp.fp8_rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS, colwise=s["train"], out=s["out"])
        out = dict(r=o["r"], rstd=o["rstd"], row=o["row"].view(torch.float8_e4m3fn), row_scale_inv=o["row_scale_inv"])
        if s["train"]:
            out["col"], out["col_scale_inv"] = o["col"].view(torch.float8_e4m3fn), o["col_scale_inv"]
            out["dx"], out["dw"] = fp.fp8_rmsnorm_bwd(s["dy"], o["r"], o["rstd"], s["w"], dr=s["dr"], dx=s["dx"],
                                                      dw=s["dw"], ws=s["ws"])
        return out
    if s["op"] == "gated":
        if not s["train"]:
            h, _ = fp.fp8_gated_fwd(s["x"], s["cache"], s["h"], s["recipe"], act=s["act"], train=False, ws=s["ws"],
                                    y=s["y"])
            return dict(h=h)
        h, ctx = fp.fp8_gated_fwd(s["x"], s["cache"], s["h"], s["recipe"], act=s["act"], ws=s["ws"], y=s["y"],
                                  ctx=s["ctx"])
        dx, dw = fp.fp8_gated_bwd(s["dh"], ctx, s["cache"], s["h"], s["recipe"], ws=s["ws"], dx=s["dx"], dw=s["dw"])
        return dict(h=h, dx=dx, dw=dw)
    norm, grads = s["clip"].clip(s["max_norm"])
    return dict(norm=norm, grads=list(grads))


def work(case):
    if case["op"] == "norm":
        R, C = case["R"], case["C"]
        nb, rb = -(-C // 128), -(-R // 128)
        # x (and the residual) read, the stream written when it is new, FP8 rows and scales
        b = R * C * (2 + (4 if case["residual"] else 0) + 1) + 4 * R * (nb + 1) + 4 * C
        flops = 6 * R * C
        if case["train"]:  # transposed FP8 and scales; dy, dr, r read, dx written
            b += R * C + 4 * C * rb + 8 * R * C + 4 * R + 4 * C
            flops += 12 * R * C
        return dict(bytes=b, flops=flops)
    if case["op"] == "gated":
        N, K, F = case["N"], case["K"], case["F"]
        b = 2 * N * K + 2 * F * K + 2 * N * F
        flops = 4 * N * K * F
        if case["train"]:
            b += 2 * N * F + 2 * N * K + 4 * F * K
            flops *= 3
        return dict(bytes=b, flops=flops)
    n = sum(_sizes(case))
    return dict(bytes=2 * n * (2 if case["bf16"] else 4), flops=3 * n)


# ---------------------------------------------------------------- definitions in 64 bits
def _round_fp8(v, fmax):
    """Nearest value (ties to even) with 3 (E4M3) or 2 (E5M2) mantissa bits, saturating, in float64."""
    mant, emin = (3, -6) if fmax == E4M3_MAX else (2, -14)
    e = torch.frexp(v)[1].to(torch.float64) - 1.0
    step = torch.exp2(torch.clamp(e, min=emin) - mant)
    return torch.clamp(torch.round(v / step) * step, -fmax, fmax)


def _f32(v):
    return v.to(torch.float32).to(torch.float64)


def _exact_group(v, dims, fmax):
    """Codes and scale_inv of groups spanning `dims` of v; the definition has the scale, the value and their product
    in fp32 (in 64 bits, the exact ties that bf16 inputs have against their block's maximum would fall elsewhere)."""
    v = _f32(v)
    amax = v.abs().amax(dims, keepdim=True)
    scale = _f32(torch.where(amax > 0, fmax / torch.where(amax > 0, amax, torch.ones_like(amax)),
                             torch.ones_like(amax)))
    return _round_fp8(_f32(v * scale), fmax), _f32(1.0 / scale)


def _padded(v, a, b):
    p = torch.zeros((-(-v.shape[0] // a) * a, -(-v.shape[1] // b) * b), dtype=torch.float64, device=v.device)
    p[: v.shape[0], : v.shape[1]] = v
    return p


def _exact_quantized(v, a, b, fmax):
    """Codes [R, C] and scale_inv [R/a, C/b] of a x b blocks (a = b = 0: the whole tensor)."""
    R, C = v.shape
    if a == 0:
        q, inv = _exact_group(v, (0, 1), fmax)
        return q, inv
    p = _padded(v, a, b)
    q, inv = _exact_group(p.view(p.shape[0] // a, a, p.shape[1] // b, b), (1, 3), fmax)
    return q.view(p.shape)[:R, :C], inv[:, 0, :, 0]


def _exact_values(v, a, b, fmax):
    q, inv = _exact_quantized(v, a, b, fmax)
    if a == 0:
        return q * inv
    return q * inv.repeat_interleave(a, 0).repeat_interleave(b, 1)[: v.shape[0], : v.shape[1]]


def _exact_norm(s):
    x, w = s["x"].double(), s["w"].double()
    r = (x + s["res"].double()).to(torch.bfloat16).double() if s["residual"] else x
    rstd = (r.square().mean(1) + EPS) ** -0.5
    y = r * rstd.unsqueeze(1) * w
    q, inv = _exact_quantized(y, 1, 128, E4M3_MAX)
    out = dict(r=r, rstd=rstd, row=q, row_scale_inv=inv)
    if s["train"]:
        out["col"], out["col_scale_inv"] = _exact_quantized(_padded(y, 16, 1).t().contiguous(), 1, 128, E4M3_MAX)
        xhat = r * rstd.unsqueeze(1)
        dy = s["dy"].double()
        dxhat = dy * w
        out["dx"] = s["dr"].double() + rstd.unsqueeze(1) * (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True))
        out["dw"] = (dy * xhat).sum(0)
    return out


def _exact_act(g, act):
    if act == "silu":
        sg = torch.sigmoid(g)
        return g * sg, sg + g * sg * (1 - sg)
    phi = torch.special.erfc(-g / math.sqrt(2)) / 2
    return g * phi, phi + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)


def _exact_gated(case, seed):
    N, K, F = case["N"], case["K"], case["F"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = _normal(gen, (N, K), 1.0).double()
    w = _normal(gen, (2 * F, K), 0.02).double()
    dh = _normal(gen, (N, F), 1e-3).double() if case["train"] else None
    row, tile = ((1, 128), (128, 128)) if case["recipe"] == "block" else ((0, 0), (0, 0))
    wq = _exact_values(w, *tile, E4M3_MAX)
    del w
    gu = _exact_values(x, *row, E4M3_MAX) @ wq.t()
    out = dict(h=_exact_act(gu[:, :F], case["act"])[0] * gu[:, F:])
    if case["train"]:
        gu = gu.to(torch.bfloat16).double()  # as the forward pass keeps them
        a, da = _exact_act(gu[:, :F], case["act"])
        dgu = torch.cat([dh * gu[:, F:] * da, dh * a], 1)
        del gu, a, da
        out["dx"] = _exact_values(dgu, *row, E5M2_MAX) @ wq
        out["dw"] = _exact_values(dgu.t().contiguous(), *row, E5M2_MAX) @ _exact_values(x.t().contiguous(), *row,
                                                                                       E4M3_MAX).t()
    return out


def exact(case, seed):
    if case["op"] == "gated":
        return _exact_gated(case, seed)
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    total = sum(float(np.square(g.double().cpu().numpy()).sum()) for g in s["grads"]) if sum(_sizes(case)) < 1 << 20 \
        else float(sum(g.double().square().sum() for g in s["grads"]))
    norm = math.sqrt(total)
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return dict(norm=torch.tensor([norm], dtype=torch.float64), grads=[g.double() * coef for g in s["grads"]])
