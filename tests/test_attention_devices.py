"""Every streaming-attention call runs on its tensors' device, whichever is current, and on that device's stream: the C
library is replaced by one that notes what is current when it is called (no GPU)."""

import contextlib

import pytest
import torch

import residual_vector_quantization_amd as rvq
from residual_vector_quantization_amd import attention

CURRENT, OWN = 0, 1


class There(torch.Tensor):
    """A CPU tensor that says it is on the second GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", OWN))


def there(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(There)


class Library:
    def __init__(self):
        self.current, self.calls = CURRENT, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 64
            self.calls.append((name, self.current, args[-1]))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()

    @contextlib.contextmanager
    def device(d):
        was, lib.current = lib.current, d.index
        yield
        lib.current = was

    monkeypatch.setattr(attention, "_ready", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: lib.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    return lib


def heads(n, h):
    return there(n, h, 64, dtype=torch.bfloat16)


Q, K, CU = heads(6, 4), heads(6, 2), there(3)
POOL, TABLE, LENS, REFS = there(5, 2, 16, 64, dtype=torch.bfloat16), there(2, 3), there(2), there(5)
ONE_Q, ONE_K, LSE, F = heads(2, 4), heads(2, 2), there(4, 6, dtype=torch.float32), there(32, dtype=torch.float64)

CALLS = {
    "rvq_window_attention": lambda: rvq.rvq_window_attention(Q, K, K, CU),
    "rvq_window_attention_backward": lambda: rvq.rvq_window_attention_backward(Q, Q, K, K, Q, LSE, CU),
    "rvq_cross_attention": lambda: rvq.rvq_cross_attention(Q, K, K, CU, CU),
    "rvq_cross_attention_backward": lambda: rvq.rvq_cross_attention_backward(Q, Q, K, K, Q, LSE, CU, CU),
    "rvq_cache_append": lambda: rvq.rvq_cache_append(K, K, POOL, POOL, TABLE, LENS, CU),
    "rvq_cache_attention": lambda: rvq.rvq_cache_attention(ONE_Q, POOL, POOL, TABLE, LENS),
    "rvq_cache_chunk_attention": lambda: rvq.rvq_cache_chunk_attention(Q, POOL, POOL, TABLE, LENS, CU),
    "rvq_rotary": lambda: rvq.rvq_rotary(Q, K, F, cu=CU),
    "rvq_rotary_append": lambda: rvq.rvq_rotary_append(Q, K, K, F, POOL, POOL, TABLE, LENS, CU),
    "rvq_cache_reserve": lambda: rvq.rvq_cache_reserve(TABLE, LENS, LENS, REFS, 16),
    "rvq_cache_fork": lambda: rvq.rvq_cache_fork(TABLE, LENS, REFS, there(1), there(1), POOL, POOL),
    "rvq_cache_free": lambda: rvq.rvq_cache_free(TABLE, LENS, REFS, 16),
    "rvq_cache_compact": lambda: rvq.rvq_cache_compact(TABLE, REFS, POOL, POOL),
    "rvq_cache_copy": lambda: rvq.rvq_cache_copy(there(1), there(1), POOL, POOL),
}


def test_all_calls_are_here():
    device = {n for n in attention.EXPORTED_ATTENTION if not n.endswith("_bytes") and n != "rvq_rotary_frequencies"}
    assert device == set(CALLS)


@pytest.mark.parametrize("name", list(CALLS))
def test_calls_run_on_their_tensors_device(lib, name):
    CALLS[name]()
    assert lib.calls == [(name, OWN, 1000 + OWN)]
    assert lib.current == CURRENT
