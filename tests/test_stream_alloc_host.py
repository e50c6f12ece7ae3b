"""CPU side of calls on a given stream: what a call allocates (outputs and workspaces) is
allocated with that stream current. The caching allocator hands out a block that was
freed on the current stream at once, while kernels queued there may still use it, and
nothing orders another stream behind those. The streams and the library here are fakes;
the allocations are seen by a dispatch mode."""
import contextlib
import types

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from learned_token_pruning_gemm_b200 import api

STREAM = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 0))
CALLER = types.SimpleNamespace(cuda_stream=1)


class Allocations(TorchDispatchMode):
    """The stream that was current at each allocation."""

    def __init__(self, current):
        super().__init__()
        self.current, self.seen = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if "empty" in func.__name__ or "zeros" in func.__name__:
            self.seen.append(self.current[-1])
        return func(*args, **(kwargs or {}))


@pytest.fixture
def fakes(monkeypatch):
    current, calls, recorded = [CALLER], [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *a: 4096

            def entry(*a):
                calls.append(a[-1])
                return 0
            return entry
    monkeypatch.setattr(api._lib, "load", lambda *a: Lib())
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: {5: STREAM}[handle])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: CALLER)
    monkeypatch.setattr(api, "_call", lambda fn, what, stream, tensors, args:
                        fn(*args, (stream or CALLER).cuda_stream))
    monkeypatch.setattr(api, "_cuda", lambda t, name, dtype=None: t.data_ptr())
    monkeypatch.setattr(api, "_stream", lambda stream=None: (stream or CALLER).cuda_stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: recorded.append((self.data_ptr(), s.cuda_stream)),
                        raising=False)
    return current, calls, recorded


I32, BF = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
Z = torch.zeros


def _norm():
    return Z(5, 4, 64), Z(5, 2, 64), Z(64), Z(64), Z(5, **I32)


def _norm_bwd():
    return (*_norm(), Z(5, 4, 64), Z(5, 2, 64))


def _read():
    kc, sc = Z(2, 9, 2, 64, dtype=torch.int8), Z(2, 9, 2)
    return kc, kc, sc, sc, Z(2, 9), Z(2, **I32), Z(3, **I32), 7


def _tree():
    d, c = Z(2, 3, 2, 64, **BF), Z(2, 9, 2, 64, **BF)
    return (Z(2, 3, 4, 64, **BF), d, d, Z(2, 3), Z(2, 3, dtype=torch.int64), c, c, Z(2, 9), Z(2, **I32), Z(4), Z(4), 9)


def _attn():
    return Z(5, 4, 64), Z(5, 2, 64), Z(5, 2, 64)


def _attn_bwd():
    q, k, v = _attn()
    return q, k, v, q, q, Z(4, 5), Z(5), Z(4), Z(4), Z(2, **I32), 5


def _decode():
    c = Z(2, 9, 2, 64, **BF)
    return Z(2, 4, 64, **BF), c, c, Z(2, 9), Z(2, **I32), Z(4), Z(4), 9


OLDER = {
    "gate_score": (api.gate_score, lambda: (Z(5, 8), Z(4, 8), Z(4), Z(4), 0.0), 1),
    "select_topk": (lambda *a, **kw: api.select_topk(*a, want_pos=True, **kw),
                    lambda: (Z(5), Z(2, **I32), Z(1, **I32), Z(1, **I32), Z(1, **I32), 3, 5), 4),
    "compact_rows": (lambda *a, **kw: tuple(api.compact_rows(*a, **kw)), lambda: ([Z(5, 8), Z(5, 4)], Z(3, **I32)), 2),
    "gated_attention": (api.gated_attention, lambda: (*_attn(), Z(5), Z(4), Z(4), Z(2, **I32), 5), 1),
    "gated_attention_bwd": (api.gated_attention_bwd, _attn_bwd, 7),
    "gated_delta_rule": (api.gated_delta_rule, lambda: (*(Z(5, 2, 64, **BF) for _ in range(3)), Z(5, 2), Z(5, 2),
                                                        Z(2, **I32), 5), 2),
    "qkv_rope": (api.qkv_rope, lambda: (Z(5, 8, **BF), Z(64, 8, **BF), 2, 1, Z(5, **I32)), 3),
    "compact_qkv_rope": (api.compact_qkv_rope, lambda: (Z(9, 8, **BF), Z(5, **I32), Z(64, 8, **BF), 2, 1, Z(5, **I32)), 4),
    "gated_decode": (api.gated_decode, _decode, 2),
}
CASES = {   # (call, its inputs, allocations)
    "qk_norm_rope": (api.qk_norm_rope, _norm, 2),
    "qk_norm_rope_bwd": (api.qk_norm_rope_bwd, _norm_bwd, 5),
    "quant_cache_read": (api.quant_cache_read, _read, 3),
    "tree_attention": (api.tree_attention, _tree, 2),
}


CASES.update(OLDER)


@pytest.mark.parametrize("name", sorted(CASES))
def test_a_call_allocates_on_its_stream(fakes, name):
    current, calls, recorded = fakes
    fn, inputs, n = CASES[name]
    args = inputs()
    for stream in (None, STREAM):
        with Allocations(current) as a:
            out = fn(*args, **({} if stream is None else dict(stream=stream)))
        assert a.seen == [stream or CALLER] * n
        assert current == [CALLER] and calls[-1] == (stream or CALLER).cuda_stream
        if stream is None:
            assert not recorded
    outputs = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    assert sorted(recorded) == sorted((t.data_ptr(), CALLER.cuda_stream) for t in outputs), "kept for the caller's stream"
