"""FP8 MLP stack with experts over the C ABI (marshalling only): the gated MLP
stack whose every layer sends a token through top_k of n_experts gated MLPs.

One layer, on a residual stream s and the branch b that the layer before it
left:  s = s + b;  Xn = norm(s) w;  logits = Xn Wr^T (an FP8 linear);
(weights, experts) = route(logits);  b[t] = sum_j weights[t, j] mlp_e(Xn[t]) with
e = experts[t, j] and mlp_e(x) = (act(x Wg_e^T) * (x Wu_e^T)) Wd_e^T.
After the last layer a final norm of s + b gives the output.

Training brings the tokens' rows into the experts' order, each expert's rows a
multiple of 16, and runs the FP8 gated feed-forward and linear on each expert's
rows; where they begin is read on the host, once per layer and microbatch.
Decoding runs the experts on 4-bit weights, without the host.
"""
from __future__ import annotations

import torch

import fp8_mixed_precision_gb300 as fp
from fp8_mixed_precision_gb300 import synthetic as syn


class FP8ExpertMLPStack:
    """n_tokens: tokens per microbatch of step(), a multiple of 16; n_experts a
    multiple of 16 (the rules of the FP8 linear); decode() takes any number of tokens."""

    def __init__(self, d: int, ffn: int, n_layers: int, n_tokens: int, n_experts: int, top_k: int,
                 recipe: str = "block", act: str = "silu", score: str = "softmax", max_norm: float = 1.0,
                 device="cuda", seed: int = 43):
        self.d, self.F, self.L, self.N, self.E, self.k = d, ffn, n_layers, n_tokens, n_experts, top_k
        self.recipe, self.act, self.score, self.max_norm = recipe, act, score, max_norm
        dev = self.dev = torch.device(device)
        self.cache = fp.WeightCache()
        layers, experts = range(n_layers), range(n_experts)
        self.wr = [syn.bf16_normal((n_experts, d), 0.05, seed + 7 * l, device=dev) for l in layers]
        # the experts' weights as one stack a layer, each expert's part registered by itself
        self.wgu = [syn.bf16_normal((n_experts, 2 * ffn, d), 0.02, seed + 7 * l + 1, device=dev) for l in layers]
        self.wd = [syn.bf16_normal((n_experts, d, ffn), 0.02, seed + 7 * l + 2, device=dev) for l in layers]
        self.hr = [self.cache.register(w, recipe) for w in self.wr]
        self.hgu = [[self.cache.register(w[e], recipe) for e in experts] for w in self.wgu]
        self.hd = [[self.cache.register(w[e], recipe) for e in experts] for w in self.wd]
        self.wn = [torch.ones(d, dtype=torch.float32, device=dev) for _ in range(n_layers + 1)]
        # added to the scores for the choice of experts alone; balance() moves it
        self.bias = [torch.zeros(n_experts, dtype=torch.float32, device=dev) for _ in layers]
        self.counts = [torch.zeros(n_experts, dtype=torch.int32, device=dev) for _ in layers]
        f32 = dict(dtype=torch.float32, device=dev)
        self.dwr = [torch.zeros((n_experts, d), **f32) for _ in layers]
        self.dwgu = [torch.zeros((n_experts, 2 * ffn, d), **f32) for _ in layers]
        self.dwd = [torch.zeros((n_experts, d, ffn), **f32) for _ in layers]
        self.dwn = [torch.zeros(d, **f32) for _ in range(n_layers + 1)]
        self.grads = self.dwr + self.dwgu + self.dwd + self.dwn
        self.clipper = fp.GradClip(self.grads)
        self.version = 0
        self.w4 = None

    # ------------------------------------------------------------ training
    def _experts_fwd(self, l, xs, spans, use_cache):
        """Every expert's gated MLP on its rows of xs: (output rows, what the backward pass needs)."""
        r, c = self.recipe, self.cache
        z, kept = torch.empty_like(xs), {}
        for e, (r0, r1) in spans.items():
            c.get(self.hgu[l][e], self.version, use_cache)
            c.get(self.hd[l][e], self.version, use_cache)
            h, ctx = fp.fp8_gated_fwd(xs[r0:r1], c, self.hgu[l][e], r, self.act)
            _, lin = fp.fp8_linear_fwd(h, c, self.hd[l][e], r, y=z[r0:r1])
            kept[e] = (ctx, lin)
        return z, kept

    def _experts_bwd(self, l, dz, spans, kept):
        r, c = self.recipe, self.cache
        dxs = torch.empty_like(dz)
        for e, (r0, r1) in spans.items():
            ctx, lin = kept[e]
            dh, dwd = fp.fp8_linear_bwd(dz[r0:r1], lin, c, self.hd[l][e], r)
            fp.fp8_grad_accumulate(self.dwd[l][e], dwd)
            _, dwgu = fp.fp8_gated_bwd(dh, ctx, c, self.hgu[l][e], r, dx=dxs[r0:r1])
            fp.fp8_grad_accumulate(self.dwgu[l][e], dwgu)
        return dxs

    def microbatch(self, x: torch.Tensor, dy: torch.Tensor, use_cache: bool = True):
        """Forward and backward of one microbatch: x [N, d] enters the stream, dy
        is the gradient of the output.  Returns (output, dx, experts of each
        layer), new tensors; weight gradients accumulate."""
        r, c = self.recipe, self.cache
        norm = dict(rowwise=False, colwise=False, bf16=True)
        layers, stream, branch = [], None, x
        for l in range(self.L):
            o = fp.fp8_rmsnorm_fwd(branch, self.wn[l], residual=stream, **norm)
            c.get(self.hr[l], self.version, use_cache)
            logits, rctx = fp.fp8_linear_fwd(o["y"], c, self.hr[l], r)
            weights, experts = fp.fp8_route_fwd(logits, self.k, self.score, bias=self.bias[l])
            order = fp.fp8_expert_order(experts, self.E, align=16)
            xs = fp.fp8_expert_gather(o["y"], order)
            ends = order.offsets.tolist()  # the host waits here
            spans = {e: (ends[e], ends[e + 1]) for e in range(self.E) if ends[e + 1] > ends[e]}
            z, kept = self._experts_fwd(l, xs, spans, use_cache)
            self.counts[l].add_(order.counts)
            layers.append((o, logits, rctx, weights, experts, order, spans, z, kept))
            stream, branch = o["r"], fp.fp8_expert_combine(z, order, weights)
        f = fp.fp8_rmsnorm_fwd(branch, self.wn[self.L], residual=stream, **norm)
        g, dwn = fp.fp8_rmsnorm_bwd(dy, f["r"], f["rstd"], self.wn[self.L])
        self.dwn[self.L].add_(dwn)
        for l in reversed(range(self.L)):
            o, logits, rctx, weights, experts, order, spans, z, kept = layers[l]
            # the stream's gradient g is also the branch's
            dz, dweights = fp.fp8_expert_combine_bwd(g, z, order, weights)
            dxn = fp.fp8_expert_combine(self._experts_bwd(l, dz, spans, kept), order)
            dlogits = fp.fp8_route_bwd(dweights, logits, weights, experts, self.score)
            dxr, dwr = fp.fp8_linear_bwd(dlogits, rctx, c, self.hr[l], r)
            fp.fp8_grad_accumulate(self.dwr[l], dwr)
            g, dwn = fp.fp8_rmsnorm_bwd(dxn.add_(dxr), o["r"], o["rstd"], self.wn[l], dr=g)
            self.dwn[l].add_(dwn)
        return f["y"], g, [t[4] for t in layers]

    def step(self, xs, dys, use_cache: bool = True):
        """One gradient-accumulation cycle, then clipping.  Returns (global norm
        before clipping as a new device tensor, the clipped gradients, which are
        the accumulators that the next step clears)."""
        self.cache.begin_cycle()
        self.version += 1
        for g in self.grads + self.counts:
            g.zero_()
        for x, dy in zip(xs, dys):
            self.microbatch(x, dy, use_cache)
        return self.clipper.clip(self.max_norm)

    def balance(self, rate: float = 1e-3):
        """Moves each layer's bias by `rate` towards even counts of the last step."""
        for b, n in zip(self.bias, self.counts):
            n = n.float()
            b.add_(torch.sign(n.mean() - n), alpha=rate)

    # ------------------------------------------------------------ serving
    def load(self, group: int = 128, zero: bool = False):
        """Make the router's FP8 weights and the experts' 4-bit weights current for decode()."""
        self.cache.begin_cycle()
        self.version += 1
        for h in self.hr:
            self.cache.get(h, self.version)
        self.w4 = [(fp.fp8_w4_quantize(gu, group, zero), fp.fp8_w4_quantize(d, group, zero))
                   for gu, d in zip(self.wgu, self.wd)]

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """Output for any number of tokens x [n, d], one included."""
        n = x.shape[0]
        norm = dict(rowwise=False, colwise=False, bf16=True)
        padded = torch.zeros((-(-n // 16) * 16, self.d), dtype=torch.bfloat16, device=self.dev)
        stream, branch = None, x
        for l in range(self.L):
            o = fp.fp8_rmsnorm_fwd(branch, self.wn[l], residual=stream, **norm)
            padded[:n] = o["y"]  # the FP8 linear takes multiples of 16 tokens
            logits, _ = fp.fp8_linear_fwd(padded, self.cache, self.hr[l], self.recipe)
            weights, experts = fp.fp8_route_fwd(logits[:n], self.k, self.score, bias=self.bias[l])
            gate_up, down = self.w4[l]
            stream, branch = o["r"], fp.fp8_w4_experts(o["y"], weights, experts, gate_up, down, self.act)
        return fp.fp8_rmsnorm_fwd(branch, self.wn[self.L], residual=stream, **norm)["y"]


def main():
    """A training step and a decoded token on synthetic inputs."""
    torch.cuda.set_device(0)
    d, ffn, layers, n, experts, k = 512, 512, 2, 2048, 16, 2
    m = FP8ExpertMLPStack(d, ffn, layers, n, experts, k)
    xs = [syn.bf16_normal((n, d), 1.0, 42 + i, device="cuda") for i in range(2)]
    dys = [syn.bf16_normal((n, d), 1e-3, 44 + i, device="cuda") for i in range(2)]
    norm, grads = m.step(xs, dys)
    print(f"gradient norm {float(norm):.4f} over {len(grads)} tensors, "
          f"{int(m.counts[0].min())} to {int(m.counts[0].max())} tokens an expert")
    m.balance()
    m.load()
    y = m.decode(xs[0][:1])
    print(f"one token: output norm {float(y.float().norm()):.3f}")


if __name__ == "__main__":
    main()
