"""The Python calls run on the host: CPU tensors that claim to be CUDA ones, and
a library whose launching functions are recorded instead of called (its sizes,
layouts, plans and weight caches are the real ones)."""
import contextlib
import ctypes

import torch

# functions that enqueue work: recorded with their arguments, answered with 0
LAUNCHING = ("fp8_rmsnorm_fwd", "fp8_rmsnorm_bwd", "fp8_gated_fwd", "fp8_gated_fwd_quantized", "fp8_gated_bwd",
             "fp8_grad_clip_run", "fp8_grad_norm", "fp8_weight_cache_get", "fp8_linear_fwd", "fp8_linear_bwd",
             "fp8_grad_accumulate", "fp8_quantize", "fp8_quantize_delayed", "fp8_gemm", "fp8_gelu_fwd", "fp8_gelu_bwd")


class Dev(torch.Tensor):
    """A host tensor that passes for a CUDA one."""
    is_cuda = property(lambda self: True)
    device_index, recorded = 0, None

    def get_device(self):
        return self.device_index

    def record_stream(self, stream):
        self.recorded = (self.recorded or []) + [stream.cuda_stream]


class FakeStream:
    def __init__(self, raw):
        self.cuda_stream = raw


def dev(t, index=0):
    t = t.as_subclass(Dev)
    t.device_index = index
    return t


class Host:
    """calls: (name, arguments, stream the allocator was on) of every launch;
    made: (tensor, stream the allocator was on) of every torch.empty."""

    def __init__(self, fp, monkeypatch):
        self.calls, self.made, self.on = [], [], []
        self.current = 0
        real, host = fp.lib(), self

        class Lib:
            def __getattr__(self, name):
                if name not in LAUNCHING:
                    return getattr(real, name)

                def launch(*args):
                    host.calls.append((name, args))
                    return 0
                return launch

        fake = Lib()
        monkeypatch.setattr(fp, "lib", lambda: fake)
        monkeypatch.setattr(fp, "_stream", lambda s=None: host.at() if s is None else s.cuda_stream)
        empty, empty_like = torch.empty, torch.empty_like

        def made(t):
            host.made.append((t, host.at()))
            return t

        def fake_empty(*a, **kw):
            if kw.pop("device", None) is None:
                return empty(*a, **kw)
            return made(dev(empty(*a, **kw)))

        monkeypatch.setattr(torch, "empty", fake_empty)
        monkeypatch.setattr(torch, "empty_like", lambda t, **kw: made(dev(empty_like(t, **kw))))
        to = torch.Tensor.to

        def fake_to(t, *a, **kw):
            if a and str(a[0]) in ("cpu", "cuda"):  # the upload of a plan's table
                return made(dev(t.clone()))
            return to(t, *a, **kw)

        monkeypatch.setattr(torch.Tensor, "to", fake_to)

        @contextlib.contextmanager
        def stream(s):
            host.on.append(s.cuda_stream)
            yield
            host.on.pop()

        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(host.at()))

    def at(self):
        return self.on[-1] if self.on else self.current

    def launches(self, name):
        return [a for n, a in self.calls if n == name]


def bf16(*shape):
    return dev(torch.zeros(shape, dtype=torch.bfloat16))


def f32(*shape):
    return dev(torch.zeros(shape, dtype=torch.float32))


def value(p):
    """The integer of a pointer argument."""
    return p.value if isinstance(p, ctypes.c_void_p) else p
