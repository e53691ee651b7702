"""What the binding of the layer operators hands to the library, seen by a stand-in for it, without a GPU."""
from __future__ import annotations


import pytest
import torch

import mixed_precision_partial_amd as ar


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = True


def on_device(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


class Recorder:
    """Stands for the library: records the last argument of each call, its stream."""

    def __init__(self):
        self.streams = {}

    def __getattr__(self, name):
        def call(*args):
            self.streams[name] = args[-1]
            return ar.AR_OK
        return call


def layer_calls(stream):
    q, k, table, pos = on_device(4, 2, 64), on_device(4, 1, 64), on_device(9, 64, dtype=torch.float32), on_device(4, dtype=torch.int64)
    ar.ar_qk_norm_rope(None, q, k, None, None, table, pos, stream=stream)
    ar.ar_attention(None, torch.empty_like(q), q, k, k, on_device(2, dtype=torch.int32), on_device(1, dtype=torch.int64),
                    on_device(1, dtype=torch.int32), 4, 4, stream=stream)
    codes, scales = on_device(4, 128, dtype=torch.uint8), on_device(4, 1, dtype=torch.float32)
    ar.ar_fp8_quantize(None, codes, scales, q.view(4, 128), stream=stream)
    ar.ar_fp8_matmul(None, on_device(4, 4, dtype=torch.float32), codes, scales, codes, on_device(1, 1, dtype=torch.float32),
                     stream=stream)


@pytest.mark.parametrize("given", [None, 0, 0x7000])
def test_calls_without_a_stream_go_to_the_current_one(monkeypatch, given):
    """torch's current stream of the tensors' device unless a stream is given; 0 is the null stream."""
    current = 0x5000
    seen = Recorder()
    monkeypatch.setattr(ar, "load_library", lambda: seen)
    monkeypatch.setattr(ar, "_layouts", {})     # the stand-in's answers are not kept
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: current)
    layer_calls(given)
    want = current if given is None else given
    for name in ("ar_qk_norm_rope", "ar_attention", "ar_fp8_quantize", "ar_fp8_matmul"):
        assert seen.streams[name] == want, name


def attention_shapes(tokens, rows, heads_q=16, heads_kv=2, dim=128):
    """out, q, k, v of a call by their sizes alone."""
    q = torch.empty(tokens, heads_q, dim, dtype=torch.bfloat16, device="meta")
    k = torch.empty(rows, heads_kv, dim, dtype=torch.bfloat16, device="meta")
    return q, q, k, k


@pytest.mark.parametrize("bound", [(1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 5, 1 << 70])
def test_bounds_of_keys_past_32_bits_hold(bound):
    """Any bound of the lengths holds that is not below them; a larger one is no smaller for the library."""
    need = ar.ar_attention_workspace(*attention_shapes(1, 131072), 1, 1, 131072)
    assert need > 0
    assert ar.ar_attention_workspace(*attention_shapes(1, 131072), 1, 1, bound) == need


@pytest.mark.parametrize("bounds", [(-1, 4), (4, -1), (-(1 << 32), 4), (4, -(1 << 32) + 3), (1 << 32, 4)], ids=str)
def test_bounds_outside_the_limits_are_refused(bounds):
    with pytest.raises(ar.ArError):
        ar.ar_attention_workspace(*attention_shapes(4, 100), 1, *bounds)


@pytest.mark.parametrize("make", [lambda n: torch.zeros(2 * n, dtype=torch.uint8)[::2], lambda n: torch.zeros(n, 2, dtype=torch.uint8)[:, :1],
                                  lambda n: torch.zeros(1, dtype=torch.uint8).expand(n)], ids=["every second", "a column", "expanded"])
def test_workspaces_with_gaps_are_refused(monkeypatch, make):
    """A call writes the bytes that follow the workspace's first: they have to be the workspace's own."""
    class Needs(Recorder):
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_workspace"):
                    args[-1]._obj.value = 4096
                    return ar.AR_OK
                raise AssertionError(f"{name} was called")
            return call
    monkeypatch.setattr(ar, "load_library", Needs)
    monkeypatch.setattr(ar, "_layouts", {})     # the stand-in's answers are not kept
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="workspace"):
        ar.ar_attention(None, torch.empty_like(q), q, k, k, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64),
                        torch.zeros(1, dtype=torch.int32), 4, 4, workspace=make(4096))
    codes = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        ar.ar_fp8_matmul(None, torch.zeros(4, 4), codes, torch.zeros(4, 1), codes, torch.zeros(1, 1), workspace=make(4096))


def test_single_rows_of_head_major_buffers():
    """The one token of a [heads, tokens, head_dim] buffer: a single row's distance to the next is no limit."""
    q = torch.empty(32, 8192, 128, dtype=torch.bfloat16, device="meta")[:, 5:6].transpose(0, 1)
    k = torch.empty(8, 1 << 20, 128, dtype=torch.bfloat16, device="meta").transpose(0, 1)
    assert ar.ar_attention_workspace(q, q, k, k, 1, 1, 131072) > 0
    one = k[7:8]
    assert ar.ar_attention_workspace(q, q, one, one, 1, 1, 1) == 0
