"""MoELayer refuses combinations of buffers and pools before anything is launched (runs without a GPU)."""
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
