"""A GPU that is not there, for tests of the binding's host side: which stream
device memory is taken on, filled on, read on and recorded on.  Tensors are
CPU ones that say they are on cuda:0; the library's calls are noted and launch
nothing."""
import contextlib

import torch

import fsdp_sharded_state_amd as fs


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, torch.device("cuda", 0)

    def __eq__(self, other):
        return isinstance(other, Stream) and other.cuda_stream == self.cuda_stream

    __hash__ = None


class GpuTensor(torch.Tensor):
    """`pool`: handle of the stream it was allocated on; `recorded`: handles that record_stream was called with."""

    @staticmethod
    def of(t, pool):
        t = t.as_subclass(GpuTensor)
        t.pool, t.recorded = pool, []
        return t

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func == torch.Tensor.get_device:
            return 0
        if func == torch.Tensor.is_cuda.__get__:
            return True
        if func == torch.Tensor.device.__get__:
            return torch.device("cuda", 0)
        return super().__torch_function__(func, types, args, kwargs or {})


class FakeGpu:
    """`current`: the current stream.  `calls`: (name, arguments) of every library call on a device."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.calls, self.during = Stream(0), False, [], {}
        empty, tensor, real, patch = torch.empty, torch.tensor, fs.lib(), monkeypatch.setattr
        on_gpu = (lambda device: device is not None and torch.device("cuda" if isinstance(device, int) else device).type == "cuda")

        def make(f):
            def made(*args, device=None, **kw):
                return GpuTensor.of(f(*args, **kw), self.current.cuda_stream) if on_gpu(device) else f(*args, device=device, **kw)
            return made

        patch(torch, "empty", make(empty))
        patch(torch, "tensor", make(tensor))
        patch(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
        patch(torch._C, "_cuda_getCurrentRawStream", lambda index: self.current.cuda_stream, raising=False)
        patch(torch.cuda, "current_device", lambda: 0)
        patch(torch.cuda, "current_stream", lambda device=None: self.current)
        patch(torch.cuda, "default_stream", lambda device=None: Stream(0))
        patch(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        patch(torch.cuda, "Stream", Stream)
        patch(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
        patch(torch.cuda, "stream", self.on)
        gpu = self

        class Library:
            def __getattr__(self, name):
                if not name.endswith("_upload") and name not in DEVICE_CALLS:
                    return getattr(real, name)

                def call(*args):
                    gpu.calls.append((name, args))
                    gpu.during.get(name, lambda *a: None)(*args)
                    return 0
                return call

        patch(fs, "lib", Library)

    @contextlib.contextmanager
    def on(self, stream):
        before, self.current = self.current, stream
        try:
            yield
        finally:
            self.current = before

    def empty(self, *shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")


DEVICE_CALLS = {"fs_pack", "fs_pack_cast", "fs_unpack", "fs_load_local", "fs_reshard", "fs_pack_mx4", "fs_unpack_mx4",
                "fs_reduce_shard_mx4"}
