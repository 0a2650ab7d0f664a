"""Stand-ins for CUDA tensors and for the library, for the Python form of the calls without a GPU: the tensors have types,
shapes, strides, a device and an address, and nothing behind it."""
import torch

import quantized_moe_expert_routed_gb300 as M

BF16, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, device=0, stride=None, address=1 << 20):
        like = torch.empty(shape, dtype=dtype, device="meta")
        self.like = like if stride is None else like.as_strided(shape, stride)
        self.index, self.address = device, address
        self.dtype, self.shape = dtype, self.like.shape

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.address

    def __getattr__(self, name):  # dim, stride, numel, element_size, is_contiguous
        return getattr(self.like, name)


class Library:
    """Takes every call, launches nothing, and says how often it was called; sizes come from the real one."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


def install(monkeypatch, device=0):
    lib = Library(M.load())
    M._load_calls()
    monkeypatch.setattr(M, "load", lambda: lib)
    monkeypatch.setattr(M, "_current_device", lambda: device)
    monkeypatch.setattr(M, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(M, "_scratch", lambda n, t, stream, handle: (1 << 24, None))
    return lib


def arguments(name):
    """Every tensor argument of a call, and the others."""
    cache = dict(k_cache=Tensor((5, 2, 16, 64), U8), v_cache=Tensor((5, 2, 16, 64), U8), k_scale=Tensor((5, 2, 16, 8), U8),
                 v_scale=Tensor((5, 2, 16, 8), U8), block_table=Tensor((3, 4), I32), cache_lens=Tensor((3,), I32),
                 q_start=Tensor((4,), I32), err=Tensor((1,), I32))
    if name == "mnw_kv_append":
        return dict(q=Tensor((6, 4, 128), BF16), k=Tensor((6, 2, 128), BF16), v=Tensor((6, 2, 128), BF16),
                    inv_freq=Tensor((64,), F32), q_out=Tensor((6, 4, 128), BF16), **cache), {}
    if name == "mnw_attn_paged":
        n = M.mnw_attn_paged_workspace_size(3, 6, 4, 2, 128)
        return dict(q=Tensor((6, 4, 128), BF16), out=Tensor((6, 4, 128), BF16), lse=Tensor((6, 4), F32), ws=Tensor((n,), U8), **cache), \
            dict(blk=1, scale=0.1)
    if name == "mnw_kv_values":
        return dict(cache=Tensor((5, 2, 16, 64), U8), scale=Tensor((5, 2, 16, 8), U8), out=Tensor((5, 2, 16, 128), BF16)), {}
    assert name == "mnw_lora_add"
    return dict(y=Tensor((1100, 64), BF16), x=Tensor((1100, 32), BF16), a=Tensor((3, 16, 32), BF16), b=Tensor((3, 64, 16), BF16),
                adapter=Tensor((1100,), I32), scale=Tensor((3,), F32), ranks=Tensor((3,), I32), out=Tensor((1100, 64), BF16),
                ws=Tensor((M.mnw_lora_workspace_size(1100, 32, 16, 3),), U8), err=Tensor((1,), I32)), {}


CALLS = ["mnw_kv_append", "mnw_attn_paged", "mnw_kv_values", "mnw_lora_add"]
# the tensor whose device the others are compared with
FIRST = {"mnw_kv_append": "k", "mnw_attn_paged": "q", "mnw_kv_values": "cache", "mnw_lora_add": "y"}
