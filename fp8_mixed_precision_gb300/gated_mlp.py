"""FP8 gated MLP stack over the C ABI (marshalling only): the RMS norm with the
residual's addition, the gated feed-forward and gradient clipping together
with the FP8 linear that closes the block.

One layer, on a residual stream s and the branch b that the layer before it
left:  s = s + b;  H = act(Xn Wg^T) * (Xn Wu^T) with Xn = norm(s) w;  b = H Wd^T.
After the last layer a final norm of s + b gives the output.  Under the block
recipe the norm writes its FP8 output and, for training, the transposed copy
straight into the gated feed-forward's context; under the tensorwise recipe
the norm's bf16 output is quantized by the gated call.

A training step is a gradient-accumulation cycle over microbatches (weights
through the weight cache, as FP8MLPStack); at its end all accumulated
gradients are clipped to one global norm.
"""
from __future__ import annotations

import torch

import fp8_mixed_precision_gb300 as fp
from fp8_mixed_precision_gb300 import synthetic as syn


class FP8GatedMLPStack:
    """n_tokens: tokens per microbatch of step() (a multiple of 16, the rule of
    the FP8 linear); decode() takes any number."""

    def __init__(self, d: int, ffn: int, n_layers: int, n_tokens: int, recipe: str = "block",
                 act: str = "silu", max_norm: float = 1.0, device="cuda", seed: int = 43):
        self.d, self.F, self.L, self.N = d, ffn, n_layers, n_tokens
        self.recipe, self.act, self.max_norm = recipe, act, max_norm
        dev = self.dev = torch.device(device)
        self.cache = fp.WeightCache()
        self.wgu = [syn.bf16_normal((2 * ffn, d), 0.02, seed + 2 * l, device=dev)
                    for l in range(n_layers)]
        self.wd = [syn.bf16_normal((d, ffn), 0.02, seed + 2 * l + 1, device=dev)
                   for l in range(n_layers)]
        self.hgu = [self.cache.register(w, recipe) for w in self.wgu]
        self.hd = [self.cache.register(w, recipe) for w in self.wd]
        # norm weights: one per layer and the final one
        self.wn = [torch.ones(d, dtype=torch.float32, device=dev) for _ in range(n_layers + 1)]
        f32 = dict(dtype=torch.float32, device=dev)
        self.dwgu = [torch.zeros((2 * ffn, d), **f32) for _ in range(n_layers)]
        self.dwd = [torch.zeros((d, ffn), **f32) for _ in range(n_layers)]
        self.dwn = [torch.zeros(d, **f32) for _ in range(n_layers + 1)]
        self.grads = self.dwgu + self.dwd + self.dwn
        self.clipper = fp.GradClip(self.grads)
        self.version = 0
        self._train = None

    # ------------------------------------------------------------ training
    def _buffers(self):
        """Buffers of one microbatch in flight, made on the first one."""
        if self._train is not None:
            return self._train
        N, d, F, r, dev = self.N, self.d, self.F, self.recipe, self.dev
        bf16 = dict(dtype=torch.bfloat16, device=dev)
        block = r == "block"
        b = dict(layers=[])
        for _ in range(self.L):
            ctx = fp.gated_context(r, N, d, F, dev)
            norm = fp.rmsnorm_buffers(N, d, dev, rowwise=block, colwise=False, bf16=not block)
            if block:
                norm.update(fp.gated_norm_columns(r, ctx))
                norm["rstd_lo"] = torch.empty(N, dtype=torch.float32, device=dev)
            b["layers"].append(dict(
                ctx=ctx, norm=norm, H=torch.empty((N, F), **bf16), Y=torch.empty((N, d), **bf16),
                lin=fp.LinearContext(fp._empty_bytes(fp._ctx_bytes(r, N, F), dev), N, F)))
        b["final"] = fp.rmsnorm_buffers(N, d, dev, rowwise=False, colwise=False, bf16=True)
        b["ws"] = max(fp.gated_workspace(r, N, d, F, dev), fp.linear_workspace(r, N, F, d, dev),
                      fp.rmsnorm_workspace(N, d, dev), key=lambda t: t.numel())
        b["dH"] = torch.empty((N, F), **bf16)
        b["g"] = [torch.empty((N, d), **bf16) for _ in range(2)]
        b["dXn"] = torch.empty((N, d), **bf16)
        b["dwgu"] = torch.empty((2 * F, d), **bf16)
        b["dwd"] = torch.empty((d, F), **bf16)
        b["dwn"] = torch.empty(d, dtype=torch.float32, device=dev)
        self._train = b
        return b

    def microbatch(self, x: torch.Tensor, dy: torch.Tensor, use_cache: bool = True):
        """Forward and backward of one microbatch: x [N, d] enters the stream, dy
        is the gradient of the output.  Returns (output, dx), new tensors; weight
        gradients accumulate."""
        b, r, c, block = self._buffers(), self.recipe, self.cache, self.recipe == "block"
        b["final"]["y"] = torch.empty((self.N, self.d), dtype=torch.bfloat16, device=self.dev)
        # the stream's gradient: two buffers in turn, the last one returned
        grad = [torch.empty_like(b["final"]["y"])] + [b["g"][l % 2] for l in range(self.L)]
        stream, branch = None, x
        for l, t in enumerate(b["layers"]):
            c.get(self.hgu[l], self.version, use_cache)
            c.get(self.hd[l], self.version, use_cache)
            o = fp.fp8_rmsnorm_fwd(branch, self.wn[l], residual=stream, rowwise=block,
                                   colwise=block, bf16=not block, out=t["norm"])
            t["r"], t["rstd"] = o["r"], o["rstd"]
            if block:
                fp.fp8_gated_fwd_quantized(o["row"], o["row_scale_inv"], c, self.hgu[l], r,
                                           self.act, y=t["H"], ctx=t["ctx"])
            else:
                fp.fp8_gated_fwd(o["y"], c, self.hgu[l], r, self.act, ws=b["ws"], y=t["H"],
                                 ctx=t["ctx"])
            fp.fp8_linear_fwd(t["H"], c, self.hd[l], r, ws=b["ws"], y=t["Y"], ctx=t["lin"])
            stream, branch = o["r"], t["Y"]
        f = fp.fp8_rmsnorm_fwd(branch, self.wn[self.L], residual=stream, rowwise=False,
                               colwise=False, bf16=True, out=b["final"])
        g, _ = fp.fp8_rmsnorm_bwd(dy, f["r"], f["rstd"], self.wn[self.L], dx=grad[self.L],
                                  dw=b["dwn"], ws=b["ws"])
        self.dwn[self.L].add_(b["dwn"])
        for l in reversed(range(self.L)):
            t = b["layers"][l]
            # the stream's gradient g is also the branch's
            fp.fp8_linear_bwd(g, t["lin"], c, self.hd[l], r, ws=b["ws"], dx=b["dH"], dw=b["dwd"])
            fp.fp8_grad_accumulate(self.dwd[l], b["dwd"])
            fp.fp8_gated_bwd(b["dH"], t["ctx"], c, self.hgu[l], r, ws=b["ws"], dx=b["dXn"],
                             dw=b["dwgu"])
            fp.fp8_grad_accumulate(self.dwgu[l], b["dwgu"])
            g, _ = fp.fp8_rmsnorm_bwd(b["dXn"], t["r"], t["rstd"], self.wn[l], dr=g,
                                      dx=grad[l], dw=b["dwn"], ws=b["ws"])
            self.dwn[l].add_(b["dwn"])
        return f["y"], g

    def step(self, xs, dys, use_cache: bool = True):
        """One gradient-accumulation cycle, then clipping.  Returns (global norm
        before clipping as a new device tensor, the clipped gradients, which are
        the accumulators that the next step clears)."""
        self.cache.begin_cycle()
        self.version += 1
        for g in self.grads:
            g.zero_()
        for x, dy in zip(xs, dys):
            self.microbatch(x, dy, use_cache)
        return self.clipper.clip(self.max_norm)

    # ------------------------------------------------------------ serving
    def load(self):
        """Make the FP8 weights current for decode()."""
        self.cache.begin_cycle()
        self.version += 1
        for h in self.hgu + self.hd:
            self.cache.get(h, self.version)

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """Output for any number of tokens x [n, d], one included."""
        r, c, block = self.recipe, self.cache, self.recipe == "block"
        n = x.shape[0]
        npad = -(-n // 16) * 16  # the closing linear takes multiples of 16 tokens
        H = torch.zeros((npad, self.F), dtype=torch.bfloat16, device=self.dev)
        stream, branch = None, x
        for l in range(self.L):
            o = fp.fp8_rmsnorm_fwd(branch, self.wn[l], residual=stream, rowwise=block,
                                   colwise=False, bf16=not block)
            if block:
                fp.fp8_gated_fwd_quantized(o["row"], o["row_scale_inv"], c, self.hgu[l], r,
                                           self.act, y=H[:n])
            else:
                fp.fp8_gated_fwd(o["y"], c, self.hgu[l], r, self.act, train=False, y=H[:n])
            y, _ = fp.fp8_linear_fwd(H, c, self.hd[l], r)
            stream, branch = o["r"], y[:n]
        return fp.fp8_rmsnorm_fwd(branch, self.wn[self.L], residual=stream, rowwise=False,
                                  colwise=False, bf16=True)["y"]


def main():
    """A training step and a decoded token on synthetic inputs."""
    torch.cuda.set_device(0)
    d, ffn, layers, n = 512, 2048, 4, 2048
    m = FP8GatedMLPStack(d, ffn, layers, n)
    xs = [syn.bf16_normal((n, d), 1.0, 42 + i, device="cuda") for i in range(2)]
    dys = [syn.bf16_normal((n, d), 1e-3, 44 + i, device="cuda") for i in range(2)]
    norm, grads = m.step(xs, dys)
    print(f"gradient norm {float(norm):.4f} over {len(grads)} tensors")
    m.load()
    y = m.decode(xs[0][:1])
    print(f"one token: output norm {float(y.float().norm()):.3f}")


if __name__ == "__main__":
    main()
