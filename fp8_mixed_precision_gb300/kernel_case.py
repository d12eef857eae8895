"""Runs one library kernel on one synthetic case a few times, for profiling
single launches (e.g. under ncu) and timing them with CUDA events.

    python -m fp8_mixed_precision_gb300.kernel_case gemm --M 131072 --N 8192 --K 512 \
        --scaling tensor --reps 3
    python -m fp8_mixed_precision_gb300.kernel_case quantize --M 131072 --N 2048 \
        --recipe tensorwise --role act --reps 3
    python -m fp8_mixed_precision_gb300.kernel_case gelu_bwd --M 131072 --N 2048 --reps 7
    python -m fp8_mixed_precision_gb300.kernel_case norm --M 65536 --N 512
    python -m fp8_mixed_precision_gb300.kernel_case gated_bwd --M 2048 --N 14336 --K 4096 --recipe block
    python -m fp8_mixed_precision_gb300.kernel_case clip --M 8 --N 8388608

norm, norm_bwd: M rows of N columns; gated, gated_bwd: M tokens, N outputs, K
inputs (forward with what training keeps; gated_bwd the whole backward pass);
clip: M bf16 gradients of N elements.
"""
from __future__ import annotations

import argparse
import json

import torch

import fp8_mixed_precision_gb300 as fp
from fp8_mixed_precision_gb300 import synthetic as syn


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("kind", choices=["gemm", "quantize", "gelu", "gelu_bwd", "gelu_quant",
                                     "gelu_bwd_quant", "norm", "norm_bwd", "gated", "gated_bwd",
                                     "clip"])
    ap.add_argument("--M", type=int, required=True)
    ap.add_argument("--N", type=int, required=True)
    ap.add_argument("--K", type=int, default=512)
    ap.add_argument("--scaling", default="tensor", choices=list(fp.SCALING))
    ap.add_argument("--recipe", default="tensorwise", choices=list(fp.RECIPE))
    ap.add_argument("--role", default="act", choices=list(fp.ROLE))
    ap.add_argument("--afmt", default="e4m3", choices=list(fp.FORMAT))
    ap.add_argument("--bfmt", default="e4m3", choices=list(fp.FORMAT))
    ap.add_argument("--act", default="silu", choices=list(fp.ACTIVATION))
    ap.add_argument("--infer", action="store_true", help="gated: keep nothing for a backward pass")
    ap.add_argument("--reps", type=int, default=3)
    a = ap.parse_args(argv)
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    if a.kind == "gemm":
        # random FP8 codes from a normal draw (valid, finite codes only)
        A = syn.bf16_normal((a.M, a.K), 1.0, 1, device=dev).float().to(torch.float8_e4m3fn)
        B = syn.bf16_normal((a.N, a.K), 1.0, 2, device=dev).float().to(torch.float8_e4m3fn)
        A, B = A.view(torch.uint8), B.view(torch.uint8)
        kb = -(-a.K // 128)
        if a.scaling == "tensor":
            sa, sb = torch.full((1,), 0.01, device=dev), torch.full((1,), 0.02, device=dev)
        elif a.scaling == "1x128_128x128":
            sa = torch.rand((a.M, kb), generator=g, device=dev) * 0.01 + 1e-3
            sb = torch.rand((-(-a.N // 128), kb), generator=g, device=dev) * 0.01 + 1e-3
        else:
            sa = torch.rand((a.M, kb), generator=g, device=dev) * 0.01 + 1e-3
            sb = torch.rand((a.N, kb), generator=g, device=dev) * 0.01 + 1e-3
        C = torch.empty((a.M, a.N), dtype=torch.bfloat16, device=dev)
        run = lambda: fp.fp8_gemm(A, a.afmt, sa, B, a.bfmt, sb, a.scaling, out=C)
        flops = 2.0 * a.M * a.N * a.K
        nbytes = a.M * a.K + a.N * a.K + 2.0 * a.M * a.N
    elif a.kind == "quantize":
        x = syn.bf16_normal((a.M, a.N), 1.0, 3, device=dev)
        run = lambda: fp.fp8_quantize(x, a.recipe, a.role)
        flops = 0.0
        nbytes = (6.0 if a.recipe == "tensorwise" else 4.125) * a.M * a.N
    elif a.kind == "gelu":
        h = syn.bf16_normal((a.M, a.N), 1.0, 4, device=dev)
        out = torch.empty_like(h)
        run = lambda: fp.fp8_gelu_fwd(h, out=out)
        flops = 0.0
        nbytes = 4.0 * a.M * a.N
    elif a.kind == "gelu_bwd":
        h = syn.bf16_normal((a.M, a.N), 1.0, 4, device=dev)
        da = syn.bf16_normal((a.M, a.N), 1.0, 5, device=dev)
        out = torch.empty_like(h)
        run = lambda: fp.fp8_gelu_bwd(da, h, out=out)
        flops = 0.0
        nbytes = 6.0 * a.M * a.N
    elif a.kind in ("norm", "norm_bwd"):
        x = syn.bf16_normal((a.M, a.N), 1.0, 6, device=dev)
        y = syn.bf16_normal((a.M, a.N), 1.0, 7, device=dev)
        w = torch.ones(a.N, dtype=torch.float32, device=dev)
        out = fp.rmsnorm_buffers(a.M, a.N, dev)
        flops = 0.0
        if a.kind == "norm":
            run = lambda: fp.fp8_rmsnorm_fwd(x, w, residual=y, out=out)
            nbytes = 8.125 * a.M * a.N
        else:
            o = fp.fp8_rmsnorm_fwd(x, w, residual=y, out=out)
            dx, dw = torch.empty_like(x), torch.empty_like(w)
            ws = fp.rmsnorm_workspace(a.M, a.N, dev)
            run = lambda: fp.fp8_rmsnorm_bwd(y, o["r"], o["rstd"], w, dr=x, dx=dx, dw=dw, ws=ws)
            nbytes = 8.0 * a.M * a.N
    elif a.kind in ("gated", "gated_bwd"):
        x = syn.bf16_normal((a.M, a.K), 1.0, 8, device=dev)
        w = syn.bf16_normal((2 * a.N, a.K), 0.02, 9, device=dev)
        cache = fp.WeightCache()
        h = cache.register(w, a.recipe)
        cache.begin_cycle()
        cache.get(h)
        ws = fp.gated_workspace(a.recipe, a.M, a.K, a.N, dev)
        ctx = None if a.infer else fp.gated_context(a.recipe, a.M, a.K, a.N, dev)
        y = torch.empty((a.M, a.N), dtype=torch.bfloat16, device=dev)
        fwd = lambda: fp.fp8_gated_fwd(x, cache, h, a.recipe, a.act, train=not a.infer, ws=ws, y=y,
                                       ctx=ctx)
        flops = 4.0 * a.M * a.N * a.K
        nbytes = 2.0 * a.M * a.K + 2.0 * a.N * a.K + (2.0 if a.infer else 6.0) * a.M * a.N
        run = fwd
        if a.kind == "gated_bwd":
            fwd()
            dh = syn.bf16_normal((a.M, a.N), 1e-3, 10, device=dev)
            dx = torch.empty_like(x)
            dw = torch.empty_like(w)
            run = lambda: fp.fp8_gated_bwd(dh, ctx, cache, h, a.recipe, ws=ws, dx=dx, dw=dw)
            flops *= 2
            nbytes = 6.0 * a.M * a.N + 4.0 * a.M * a.K + 6.0 * a.N * a.K
    elif a.kind == "clip":
        grads = [syn.bf16_normal((a.N,), 1e-2, 11 + i, device=dev) for i in range(a.M)]
        clip = fp.GradClip(grads, [torch.empty_like(t) for t in grads])
        run = lambda: clip.clip(1.0)
        flops = 3.0 * a.M * a.N
        nbytes = 4.0 * a.M * a.N
    else:  # fused GELU (backward) + 1x128 quantization, both layouts
        h = syn.bf16_normal((a.M, a.N), 1.0, 4, device=dev)
        if a.kind == "gelu_quant":
            q = fp.QuantizedTensor(a.M, a.N, "act", dev)
            run = lambda: fp.fp8_gelu_quantize(h, q)
            nbytes = 4.125 * a.M * a.N
        else:
            da = syn.bf16_normal((a.M, a.N), 1.0, 5, device=dev)
            q = fp.QuantizedTensor(a.M, a.N, "grad", dev)
            run = lambda: fp.fp8_gelu_bwd_quantize(da, h, q)
            nbytes = 6.125 * a.M * a.N
        flops = 0.0
    run()
    torch.cuda.synchronize()
    ts = []
    for _ in range(a.reps):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        run()
        e1.record()
        torch.cuda.synchronize()
        ts.append(e0.elapsed_time(e1))
    st = fp.fp8_get_device_status()
    ms = min(ts)
    print(json.dumps({"kind": a.kind, "M": a.M, "N": a.N, "K": a.K, "ms_min": ms,
                      "GB/s": nbytes / ms / 1e6, "TFLOP/s": flops / ms / 1e9, "status": st}))
    return 0 if st == 0 else 1


if __name__ == "__main__":
    raise SystemExit(main())
