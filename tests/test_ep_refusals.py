"""ExpertParallelMoE refuses a pool that it cannot run before any collective (runs without a GPU)."""
import types

import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib
from moe_expert_layer_renorm_b200.build import build
from moe_expert_layer_renorm_b200.ep import ExpertParallelMoE


class NoExchange:
    """Two ranks whose collectives are only counted."""

    world_size = 2

    def __init__(self, rank):
        self.rank, self.calls = rank, 0

    def gather_offsets(self, offsets):
        self.calls += 1
        raise RuntimeError("a collective")

    rows = gather_offsets


@pytest.mark.parametrize("rank", [0, 1])
def test_fp8_pool_is_refused_on_every_rank_before_the_first_collective(monkeypatch, rank):
    build()
    launched = []
    for name in ("route", "permute", "gather_rows", "ffn_nvfp4", "combine"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: launched.append(name))
    for module in ("layer", "ep"):
        monkeypatch.setattr(f"moe_expert_layer_renorm_b200.{module}._stream", lambda s: 0)
    T, E, k, H, I = 4, 8, 2, 256, 512
    ex = NoExchange(rank)
    ep = ExpertParallelMoE(T, E, k, H, I, exchange=ex, device="cpu")
    x, logits = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, E)
    table = torch.zeros(E // 2, dtype=torch.int32)
    pool = lambda fmt: types.SimpleNamespace(fmt=fmt, ptr=0, layout=_lib.slot_layout(H, I, E // 2, fmt))  # noqa: E731
    with pytest.raises(AssertionError, match="NVFP4 and MXFP4"):
        ep.forward(x, logits, table, pool(_lib.FT_SCALE_FP8))
    assert ex.calls == 0 and not launched
    with pytest.raises(RuntimeError, match="a collective"):
        ep.forward(x, logits, table, pool(_lib.FT_SCALE_MXFP4))
    assert ex.calls == 1
