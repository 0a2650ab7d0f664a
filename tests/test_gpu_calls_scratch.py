"""A call whose arguments are refused keeps none of the memory that it took."""
import ctypes
import gc

import pytest
import torch

import int4_util as U4
from test_gpu_decode_ops import M, _randn

pytestmark = pytest.mark.gpu


def allocated():
    """Bytes held, without what earlier tests left for the collector (it would go at any time)."""
    torch.cuda.synchronize()
    gc.collect()
    return torch.cuda.memory_allocated()


def test_refused_arguments_leave_no_memory_behind():
    m = M()
    c = U4.Cache([500], 16, 1, 64, 51)
    kw = dict(k_scale=c.ks, v_scale=c.vs)
    q = _randn((1, 4, 64), 52)
    y, x, a, b = _randn((1100, 64), 53), _randn((1100, 64), 54), _randn((1, 8, 64), 55), _randn((1, 64, 8), 56)
    ids = torch.zeros(1100, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    here = torch.cuda.current_stream()
    calls = [lambda blk=1, scale=0.1, **s: m.mnw_attn_paged(q, c.k, c.v, c.table, c.cache_lens, blk, scale, out=out, **kw, **s)]
    for call in calls:
        call()
        call(stream=here)
        memory = allocated()
        for bad in (dict(blk=32.0), dict(blk="x"), dict(scale="x"), dict(blk=0)):
            for s in ({}, dict(stream=here)):
                with pytest.raises((m.MnwError, ctypes.ArgumentError, TypeError)):
                    call(**bad, **s)
                assert allocated() == memory, (bad, s)
    held = allocated()
    for s in ({}, dict(stream=here)):
        with pytest.raises(m.MnwError):
            m.mnw_lora_add(y, x, a, b, ids, out=x, **s)  # refused by the library, behind the scratch's allocation
        assert allocated() == held
