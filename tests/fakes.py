"""CUDA tensors that are none, for tests of what the Python calls check and pass
on before the library is reached."""
import torch


class Fake(torch.Tensor):
    """A tensor of any size on any device, without memory."""

    @staticmethod
    def __new__(cls, *shape, dtype=torch.bfloat16, device="cuda:0"):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    def data_ptr(self):
        return 1 << 40

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(str(func))


class Library:
    """Stands for the loaded library: notes each call, returns success."""

    def __init__(self, on_call=lambda name, args: None):
        self.calls, self.on_call = [], on_call

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            self.on_call(name, args)
            return 0
        return call
