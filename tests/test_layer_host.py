"""MoELayer on the host: refusals before anything is launched, and the stream that workspaces are allocated on (runs
without a GPU)."""
import contextlib
import types

import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib
from moe_expert_layer_renorm_b200.build import build
from moe_expert_layer_renorm_b200.layer import MoELayer


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.fixture
def launched(monkeypatch):
    calls = []
    for name in ("route", "permute", "route_permute", "ffn_nvfp4", "ffn_fp8", "layer_nvfp4", "combine", "combine_bf16"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: calls.append(name))
    monkeypatch.setattr("moe_expert_layer_renorm_b200.layer._stream", lambda s: 0)
    return calls


@pytest.mark.parametrize("fmt", [_lib.FT_SCALE_NVFP4, _lib.FT_SCALE_MXFP4])
def test_whole_layer_call_writes_fp32_expert_outputs_only(launched, fmt):
    T, E, k, H, I = 4, 8, 2, 256, 512
    pool = types.SimpleNamespace(fmt=fmt, ptr=0, layout=_lib.slot_layout(H, I, E, fmt))
    args = (torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, E), torch.zeros(E, dtype=torch.int32), pool)
    lay = MoELayer(T, E, k, H, I, device="cpu", whole=True, out_dtype=torch.bfloat16)
    for call in (lay.forward, lay.layer):
        with pytest.raises(AssertionError, match="bf16 expert outputs"):
            call(*args)
    assert not launched
    MoELayer(T, E, k, H, I, device="cpu", whole=True).forward(*args)
    assert launched == ["layer_nvfp4"]


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("fmt,whole,front,made", [
    (_lib.FT_SCALE_NVFP4, False, False, {"perm_ws", "ffn_ws"}), (_lib.FT_SCALE_NVFP4, False, True, {"perm_ws", "ffn_ws"}),
    (_lib.FT_SCALE_NVFP4, True, False, {"layer_ws"}), (_lib.FT_SCALE_FP8, False, False, {"perm_ws", "fp8_ws"})])
def test_workspaces_are_allocated_on_the_calls_stream(launched, monkeypatch, fmt, whole, front, made, given):
    """Memory that the current stream's allocator hands out may still be written by kernels queued there."""
    T, E, k, H, I = 4, 8, 2, 256, 512
    pool = types.SimpleNamespace(fmt=fmt, ptr=0, layout=_lib.slot_layout(H, I, E, fmt))
    lay = MoELayer(T, E, k, H, I, device="cpu", whole=whole, fused_front=front)
    current, where = ["the current stream"], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "zeros"):
        def wrapped(*a, plain=getattr(torch, name), **kw):
            where.append(current[0])
            return plain(*a, **kw)
        monkeypatch.setattr(torch, name, wrapped)
    args = [torch.ones(T, H, dtype=torch.bfloat16), torch.ones(T, E), torch.ones(E, dtype=torch.int32), pool]
    lay.forward(*args, stream="a stream" if given else None)
    assert where == ["a stream" if given else "the current stream"] * len(made)
    assert {n for n in ("perm_ws", "ffn_ws", "fp8_ws", "layer_ws") if getattr(lay, "_" + n) is not None} == made
    lay.forward(*args, stream="another")
    assert len(where) == len(made)
