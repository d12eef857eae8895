"""Cases, plain forms and definitions of the operators of an MLP half with experts.

Four operators, each with the ranges it is used at:
  route    scores of each token for all experts, the choice of k of them (bias,
           groups), their weights, and the backward pass;
  rows     token rows brought into the experts' order, the experts' output rows
           weighted and summed per token, and both backward passes;
  w4       products with 4-bit weights in groups along K, as a linear layer and
           as the gated feed-forward, for few tokens;
  experts  the gated MLP of each token's experts on 4-bit weights.

own = False: elementary torch operations.  own = True: the calls that a user
makes of the framework.
"""
import math

import torch

own = False


def listed():
    return [
        # one token of a model being decoded: pure latency
        dict(name="route token", op="route", train=False, T=1, E=64, k=8, score="softmax", f32=True, bias=False,
             groups=1, kept=1, top=1, renorm=True, scale=1.0, pad=0),
        # a decode batch, sigmoid scores, the balance bias and groups
        dict(name="route decode 61", op="route", train=False, T=61, E=256, k=8, score="sigmoid", f32=True, bias=True,
             groups=8, kept=4, top=2, renorm=True, scale=2.0, pad=3),
        # the microbatch of 64 x 2048 tokens, forward and backward
        dict(name="route train", op="route", train=True, T=131072, E=128, k=8, score="softmax", f32=False, bias=False,
             groups=1, kept=1, top=1, renorm=False, scale=1.0, pad=0),
        # a ragged microbatch with padding, groups and a bias, forward and backward
        dict(name="route train groups", op="route", train=True, T=16379, E=256, k=6, score="sigmoid", f32=True,
             bias=True, groups=8, kept=3, top=2, renorm=True, scale=1.5, pad=128),
        # a decode batch of the large model: the order, the rows there and back
        dict(name="rows decode 37", op="rows", train=False, T=37, E=32, k=4, C=4096, pad=2),
        # the d = 512 model's microbatch, forward and backward
        dict(name="rows train 512", op="rows", train=True, T=131072, E=16, k=2, C=512, pad=0),
        # the large model's microbatch with a ragged token count and padding, forward and backward
        dict(name="rows train 4096", op="rows", train=True, T=16379, E=64, k=4, C=4096, pad=100),
        # one token through the large MLP's gate and up projections: the weights stream once
        dict(name="w4 gated token", op="w4", gated=True, T=1, N=14336, K=4096, group=128, zero=False, act="silu"),
        # a small decode batch through its down projection, codes with zero points
        dict(name="w4 down 7", op="w4", gated=False, T=7, N=4096, K=14336, group=64, zero=True, act="silu"),
        # a decode batch of the small model
        dict(name="w4 decode 37", op="w4", gated=False, T=37, N=2048, K=512, group=32, zero=False, act="silu"),
        # one token through its experts of the large MLP's size
        dict(name="experts token", op="experts", T=1, E=8, k=2, K=4096, F=14336, group=128, zero=False, act="silu",
             pad=0),
        # a decode batch over many small experts, some of its slots empty
        dict(name="experts decode 64", op="experts", T=64, E=32, k=4, K=4096, F=2048, group=64, zero=True, act="silu",
             pad=2),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "rows", "w4", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        kept = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(12, E // groups * kept))
        T = _log(rng, 1, min(131072, 131072 * 128 // E))
        return dict(op="route", train=rng.random() < 0.6, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    f32=rng.random() < 0.5, bias=rng.random() < 0.5, groups=groups, kept=kept, top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.5, 2.0]), pad=rng.choice([0, T // 10]))
    if op == "rows":
        E = _log(rng, 2, 256)
        k, C = rng.randint(1, min(8, E)), 16 * _log(rng, 8, 512)
        T = _log(rng, 1, max(1, min(131072, 16379 * 4 * 4096 // (k * C))))
        return dict(op="rows", train=rng.random() < 0.6, T=T, E=E, k=k, C=C, pad=rng.choice([0, T // 10]))
    group, zero, act = rng.choice([32, 64, 128]), rng.random() < 0.5, rng.choice(["silu", "gelu"])
    if op == "w4":
        N, K = 16 * _log(rng, 8, 896), 32 * _log(rng, 4, 448)
        K = max(32, min(K, 14336 * 4096 // N // 32 * 32))
        return dict(op="w4", gated=rng.random() < 0.5, T=_log(rng, 1, 64), N=N, K=K, group=group, zero=zero, act=act)
    E = _log(rng, 2, 64)
    k, K, F = rng.randint(1, min(8, E)), 32 * _log(rng, 8, 128), 32 * _log(rng, 8, 448)
    F = max(32, min(F, 2 * 4096 * 14336 // (E * K) // 32 * 32))
    T = _log(rng, 1, 96)
    return dict(op="experts", T=T, E=E, k=k, K=K, F=F, group=group, zero=zero, act=act, pad=rng.choice([0, T // 10]))


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, sigma, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(sigma).to(dtype)


def _choice(gen, T, E, k, pad, skew):
    """k distinct experts of each token, some experts taken more often than others; the last `pad` tokens have none."""
    p = torch.rand((T, E), generator=gen, device="cuda") + skew * torch.rand(E, generator=gen, device="cuda")
    e = p.topk(k, 1).indices.to(torch.int32)
    e[T - pad:] = -1
    w = torch.rand((T, k), generator=gen, device="cuda") + 0.1
    w = w / w.sum(1, keepdim=True)
    w[T - pad:] = 0.0
    return e, w


def _codes(gen, shape, group, zero):
    """4-bit weights [..., K]: two codes a byte (the even k in the low four bits), scales, zero points."""
    K = shape[-1]
    nb = -(-K // group)
    codes = torch.randint(0, 256, shape[:-1] + (K // 2,), generator=gen, device="cuda", dtype=torch.uint8)
    scale = (0.003 + 0.003 * torch.rand(shape[:-1] + (nb,), generator=gen, device="cuda")).to(torch.bfloat16)
    z = torch.randint(5, 11, shape[:-1] + (nb,), generator=gen, device="cuda", dtype=torch.uint8) if zero else None
    return codes, scale, z


def _rows(T, k, E):
    """Rows of a buffer in the experts' order, each expert's rows beginning at a multiple of 16."""
    return (T * k + 15 * min(E, T * k) + 15) // 16 * 16


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _normal(gen, (T, E), 1.0, torch.float32 if case["f32"] else torch.bfloat16)
        s["logits"][T - case["pad"]:] = -math.inf  # tokens that no expert takes
        s["b"] = _normal(gen, (E,), 0.05, torch.float32) if case["bias"] else None
        s["dw"] = _normal(gen, (T, k), 1e-2, torch.float32) if case["train"] else None
    elif case["op"] == "rows":
        T, E, k, C = case["T"], case["E"], case["k"], case["C"]
        s["e"], s["w"] = _choice(gen, T, E, k, case["pad"], 0.5)
        s["x"] = _normal(gen, (T, C), 1.0)
        R = _rows(T, k, E)
        s["z"] = _normal(gen, (R, C), 1.0)
        # the experts' input rows and the gradient of their output rows: buffers that a program keeps
        s["xs"] = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
        if case["train"]:
            s["dy"] = _normal(gen, (T, C), 1e-3)
            s["dxs"] = _normal(gen, (R, C), 1e-3)
            s["dz"] = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "w4":
        N, K = case["N"] * (2 if case["gated"] else 1), case["K"]
        s["x"] = _normal(gen, (case["T"], K), 1.0)
        s["W"] = _codes(gen, (N, K), case["group"], case["zero"])
    else:
        T, E, k, K, F = (case[n] for n in ("T", "E", "k", "K", "F"))
        s["x"] = _normal(gen, (T, K), 1.0)
        s["e"], s["w"] = _choice(gen, T, E, k, case["pad"], 0.0)
        s["Wgu"] = _codes(gen, (E, 2 * F, K), case["group"], case["zero"])
        s["Wd"] = _codes(gen, (E, K, F), case["group"], case["zero"])
    return s


# ---------------------------------------------------------------- plain forms
def _plain_choice(s):
    """Chosen experts [T, k], -1 where there is none.  In 64 bits: what a rounding to 32 would tie or swap is decided
    by the scores themselves."""
    T, E, G = s["T"], s["E"], s["groups"]
    l = s["logits"].double()
    masked = l == -math.inf
    if s["score"] == "sigmoid":
        c = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True)
        p = torch.where(masked, 0.0, torch.exp(l - m))
        c = p / p.sum(1, keepdim=True)
    if s["bias"]:
        c = c + s["b"].double()
    c = torch.where(masked, -math.inf, c)
    if G > 1:
        g = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, : s["top"]]
        none = g[:, :, 0] == -math.inf
        score = torch.where(none, -math.inf, torch.where(g == -math.inf, 0.0, g).sum(2))
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, : s["kept"]]
        out = torch.ones((T, G), dtype=torch.bool, device=c.device).scatter_(1, kept, False)
        c = torch.where(out.repeat_interleave(E // G, 1), -math.inf, c)
    v, e = c.sort(dim=1, descending=True, stable=True)
    v, e = v[:, : s["k"]], e[:, : s["k"]]
    return torch.where(v == -math.inf, -1, e).to(torch.int32)


def _plain_route(s):
    e = _plain_choice(s)
    at, none = e.clamp(min=0).long(), e < 0
    l = s["logits"].float()
    if s["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
        p = p / p.sum(1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
    chosen = torch.where(none, 0.0, p.gather(1, at))
    total = chosen.sum(1, keepdim=True)
    w = chosen / torch.where(total > 0, total, 1.0) if s["renorm"] else chosen
    out = dict(weights=w * s["scale"], experts=e)
    if s["train"]:
        # gradient of log s at the chosen experts, then of the logits
        g = s["dw"] * w * s["scale"]
        a = g - w * g.sum(1, keepdim=True) if s["renorm"] else g
        a = torch.where(none, 0.0, a)
        if s["score"] == "sigmoid":
            a = a * (1.0 - p.gather(1, at))
        d = torch.zeros_like(p).scatter_add_(1, at, a)
        if s["score"] == "softmax" and not s["renorm"]:
            d = d - p * a.sum(1, keepdim=True)
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_order(e, E):
    """Rows of each expert, where they begin (multiples of 16), and each slot's row."""
    flat = e.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    count = torch.bincount(key, minlength=E + 1)
    start = torch.zeros(E + 1, dtype=torch.int64, device=e.device)
    start[1:] = ((count[:E] + 15) // 16 * 16).cumsum(0)
    first = count.cumsum(0) - count  # without the gaps
    order = key.sort(stable=True).indices
    sorted_key = key[order]
    row = start[sorted_key] + torch.arange(flat.numel(), device=e.device) - first[sorted_key]
    position = torch.empty_like(flat)
    position[order] = torch.where(sorted_key < E, row, -1)
    return position.view(e.shape), start, count[:E]


def _plain_rows(s):
    position, start, count = _plain_order(s["e"], s["E"])
    at, some = position.clamp(min=0), position >= 0
    t = torch.arange(s["T"], device=at.device)[:, None].expand_as(at)
    xs = s["xs"]
    xs[position[some]] = s["x"][t[some]]
    w = torch.where(some, s["w"], 0.0)[:, :, None]
    z = s["z"][at].float()
    out = dict(position=position.to(torch.int32), offsets=start.to(torch.int32), counts=count.to(torch.int32), xs=xs,
               y=(z * w).sum(1).to(torch.bfloat16))
    if s["train"]:
        dy = s["dy"].float()[:, None]
        dz = s["dz"]
        dz[position[some]] = (dy * w).to(torch.bfloat16)[some]
        dweights = torch.where(some, (dy * z).sum(2), 0.0)
        dx = torch.where(some[:, :, None], s["dxs"][at].float(), 0.0).sum(1).to(torch.bfloat16)
        out.update(dz=dz, dweights=dweights, dx=dx)
    return out


def _values(W, group):
    """What 4-bit weights stand for, in fp32."""
    codes, scale, zero = W
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    K = q.shape[-1]
    z = 8.0 if zero is None else zero.float().repeat_interleave(group, -1)[..., :K]
    return (q - z) * scale.float().repeat_interleave(group, -1)[..., :K]


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * torch.erfc(-g * math.sqrt(0.5))


def _plain_w4(s):
    y = s["x"].float() @ _values(s["W"], s["group"]).t()
    if s["gated"]:
        y = _act(y[:, : s["N"]], s["act"]) * y[:, s["N"]:]
    return dict(y=y.to(torch.bfloat16))


def _plain_experts(s):
    e, F, T = s["e"], s["F"], s["T"]
    used = torch.unique(e[e >= 0]).long()  # the experts that have a token
    part = lambda W: tuple(None if t is None else t[used] for t in W)  # noqa: E731
    # each used expert on all tokens; a token's weight for an expert that it has not chosen is 0
    gu = s["x"].float() @ _values(part(s["Wgu"]), s["group"]).transpose(1, 2)
    h = _act(gu[..., :F], s["act"]) * gu[..., F:]
    share = ((e.long()[None] == used[:, None, None]) * s["w"]).sum(2)  # [used, T]
    z = h @ _values(part(s["Wd"]), s["group"]).transpose(1, 2)
    return dict(y=(z * share[:, :, None]).sum(0).to(torch.bfloat16))


# ---------------------------------------------------------------- one pass
def _own_route(s):
    import fp8_mixed_precision_gb300 as fp
    kw = dict(score=s["score"], renormalize=s["renorm"], scale=s["scale"])
    w, e = fp.fp8_route_fwd(s["logits"], s["k"], bias=s["b"], groups=s["groups"], groups_kept=s["kept"],
                            group_top=s["top"], **kw)
    out = dict(weights=w, experts=e)
    if s["train"]:
        out["dlogits"] = fp.fp8_route_bwd(s["dw"], s["logits"], w, e, **kw)
    return out


def _own_rows(s):
    import fp8_mixed_precision_gb300 as fp
    o = fp.fp8_expert_order(s["e"], s["E"], align=16)
    xs = fp.fp8_expert_gather(s["x"], o, out=s["xs"])
    out = dict(position=o.position, offsets=o.offsets, counts=o.counts, xs=xs,
               y=fp.fp8_expert_combine(s["z"], o, s["w"]))
    if s["train"]:
        out["dz"], out["dweights"] = fp.fp8_expert_combine_bwd(s["dy"], s["z"], o, s["w"], dz=s["dz"])
        out["dx"] = fp.fp8_expert_combine(s["dxs"], o)
    return out


def _own_w4(s):
    import fp8_mixed_precision_gb300 as fp
    W = fp.W4Weight(*s["W"], s["group"])
    return dict(y=fp.fp8_w4_gated(s["x"], W, act=s["act"]) if s["gated"] else fp.fp8_w4_linear(s["x"], W))


def _own_experts(s):
    import fp8_mixed_precision_gb300 as fp
    gu, d = fp.W4Weight(*s["Wgu"], s["group"]), fp.W4Weight(*s["Wd"], s["group"])
    return dict(y=fp.fp8_w4_experts(s["x"], s["w"], s["e"], gu, d, act=s["act"]))


def run(state):
    s = state
    if own:
        return {"route": _own_route, "rows": _own_rows, "w4": _own_w4, "experts": _own_experts}[s["op"]](s)
    return {"route": _plain_route, "rows": _plain_rows, "w4": _plain_w4, "experts": _plain_experts}[s["op"]](s)


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["f32"] else 2
        b = T * E * size + 8 * T * k + (4 * E if case["bias"] else 0)
        flops = 4 * T * E
        if case["train"]:  # the gradient of the weights read, that of the logits written
            b += 4 * T * k + T * E * size
            flops += 2 * T * E
        return dict(bytes=b, flops=flops)
    if case["op"] == "rows":
        T, k, C = case["T"] - case["pad"], case["k"], case["C"]
        b = 2 * C * T * (1 + k) * 2 + 4 * case["T"] * k * 3
        flops = 2 * T * k * C
        if case["train"]:  # dy and z read, dz written; dxs read, dx written
            b += 2 * C * T * (1 + 2 * k) + 2 * C * T * (1 + k) + 4 * T * k
            flops += 4 * T * k * C
        return dict(bytes=b, flops=flops)
    per = 0.5 + (3 if case["zero"] else 2) / case["group"]  # bytes of a weight
    if case["op"] == "w4":
        T, N, K = case["T"], case["N"], case["K"]
        n = N * K * (2 if case["gated"] else 1)
        return dict(bytes=int(n * per) + 2 * T * (K + N), flops=2 * T * n)
    T, E, k, K, F = case["T"] - case["pad"], case["E"], case["k"], case["K"], case["F"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # expected number of experts that have a token
    return dict(bytes=int(used * 3 * K * F * per) + 4 * T * K + 8 * T * k, flops=6 * T * k * K * F)


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_route(s):
    l, k, scale = s["logits"].double(), s["k"], s["scale"]
    logp = torch.nn.functional.logsigmoid(l) if s["score"] == "sigmoid" else torch.log_softmax(l, 1)
    p = torch.nan_to_num(logp.exp())
    c = torch.where(torch.isinf(l), -1e300, p + s["b"].double() if s["bias"] else p)
    if s["groups"] > 1:
        per = s["E"] // s["groups"]
        score = c.view(-1, s["groups"], per).topk(min(s["top"], per), 2).values.sum(2)
        first = torch.sort(score, dim=1, descending=True, stable=True).indices[:, : s["kept"]]
        kept = torch.zeros_like(score).scatter_(1, first, 1.0)
        c = torch.where(kept.repeat_interleave(per, 1) > 0, c, -1e300)
    v, e = torch.sort(c, dim=1, descending=True, stable=True)  # bf16 logits tie: the lowest index first
    v, e = v[:, :k], e[:, :k]
    some = (v > -1e299).double()
    pc = p.gather(1, e) * some
    if s["renorm"]:
        total = pc.sum(1, keepdim=True)
        u = pc / (total + (total == 0))
    else:
        u = pc
    out = dict(weights=scale * u, experts=None)
    if s["train"]:
        g = s["dw"].double() * scale
        # through the weights to the scores, then through the scores to the logits
        dp = (g - (g * u).sum(1, keepdim=True)) / (total + (total == 0)) if s["renorm"] else g
        full = torch.zeros_like(p).scatter_(1, e, dp * some)
        d = full * p * (1 - p) if s["score"] == "sigmoid" else p * (full - (full * p).sum(1, keepdim=True))
        out["dlogits"] = d
    return out


def _exact_rows(s):
    T, k, C, E = s["T"], s["k"], s["C"], s["E"]
    at, tt, jj, start = [], [], [], 0
    for i in range(E):
        t, j = (s["e"] == i).nonzero(as_tuple=True)  # in the order of the slots
        at.append(start + torch.arange(t.numel(), device="cuda"))
        tt.append(t)
        jj.append(j)
        start += (t.numel() + 15) // 16 * 16
    at, tt, jj = torch.cat(at), torch.cat(tt), torch.cat(jj)
    xs = s["xs"].double()
    xs[at] = s["x"].double()[tt]
    wz = s["z"].double()[at] * s["w"].double()[tt, jj][:, None]
    y = torch.zeros((T, C), dtype=torch.float64, device="cuda").index_add_(0, tt, wz)
    out = dict(position=None, offsets=None, counts=None, xs=xs, y=y)
    if s["train"]:
        del wz
        dyr = s["dy"].double()[tt]
        out["dz"] = s["dz"].double()
        out["dz"][at] = dyr * s["w"].double()[tt, jj][:, None]
        out["dweights"] = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        out["dweights"][tt, jj] = (dyr * s["z"].double()[at]).sum(1)
        del dyr
        out["dx"] = torch.zeros((T, C), dtype=torch.float64, device="cuda").index_add_(0, tt, s["dxs"].double()[at])
    return out


def _exact_weight(W, group):
    codes, scale, zero = W
    N, half = codes.shape
    q = torch.empty((N, 2 * half), dtype=torch.float64, device=codes.device)
    q[:, 0::2], q[:, 1::2] = (codes % 16).double(), (codes // 16).double()
    g = torch.arange(2 * half, device=codes.device) // group
    return (q - (8.0 if zero is None else zero.double()[:, g])) * scale.double()[:, g]


def _exact_gate(gu, act):
    g, u = gu.chunk(2, 1)
    return (g * torch.sigmoid(g) if act == "silu" else g * torch.special.erfc(-g / math.sqrt(2.0)) / 2.0) * u


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "rows":
        return _exact_rows(s)
    if case["op"] == "w4":
        y = s["x"].double() @ _exact_weight(s["W"], s["group"]).t()
        return dict(y=_exact_gate(y, s["act"]) if s["gated"] else y)
    y = torch.zeros((s["T"], s["K"]), dtype=torch.float64, device="cuda")
    for i in torch.unique(s["e"]).tolist():
        if i >= 0:
            t, j = (s["e"] == i).nonzero(as_tuple=True)
            gu, d = (tuple(None if v is None else v[i] for v in s[n]) for n in ("Wgu", "Wd"))
            h = _exact_gate(s["x"][t].double() @ _exact_weight(gu, s["group"]).t(), s["act"])
            y.index_add_(0, t, (h @ _exact_weight(d, s["group"]).t()) * s["w"][t, j].double()[:, None])
    return dict(y=y)
