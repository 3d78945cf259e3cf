"""h = silu(G) U of the FP8 expert FFN and its codes, on weights that let single values of it through to the output."""
import numpy as np
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib
from moe_expert_layer_renorm_b200.layer import ExpertPool, MoELayer
from oracle import fp8 as F

pytestmark = pytest.mark.gpu

H = I = 256


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    _lib.device_status(clear=True)
    yield
    assert _lib.device_status(clear=True) == _lib.FT_DEV_OK


def _one_expert(x, gate, up):
    """Outputs of one expert whose down weight is 448 times the identity (codes 448, scales 1): 448 h as FP8 holds it."""
    pool = ExpertPool(H, I, 1, fmt=_lib.FT_SCALE_FP8)
    for mat, w in enumerate((gate, up, 448.0 * torch.eye(H))):
        pool.pack_into(0, mat, w.cuda())
    T = x.shape[0]
    lay = MoELayer(T, 1, 1, H, I)
    lay.perm_src.copy_(torch.arange(T))
    lay.offsets.copy_(torch.tensor([0, T]))
    lay.ffn(x.bfloat16().cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), pool)
    return lay.out_perm.double().cpu().numpy()


def _as_codes(n, places):
    """A whole number as a sum of E4M3 values."""
    out = []
    for _ in range(places):
        v = F.TABLE[:127][F.TABLE[:127] <= n].max()
        out.append(v)
        n -= v
    assert n == 0
    return torch.tensor(out)


@pytest.mark.parametrize("T", [3, 20, 45, 90, 200])
@pytest.mark.parametrize("js", [(36, 28), (17, 42)])
def test_ties_of_h_go_to_the_even_code(js, T):
    """G = 32, so silu(G) = G in fp32, and U is a whole number: h = 32 U exactly.  With 28 j the largest U of a block,
    U = q j / 16 has the quotient q = 448 h / m for every j, and q is taken halfway between two codes."""
    x = torch.zeros(T, H)
    x[:, :9], x[:, 101] = 1.0, 448.0                      # scale 1
    gate, up = torch.zeros(I, H), torch.zeros(I, H)
    want = np.zeros(H)
    ties = 0
    for b, j in enumerate(js):
        qs = [2.0 ** e * (1 + (o + 0.5) / 8) for e in range(3, 9) for o in range(8)]
        qs = [448.0] + [q for q in qs if q < 448 and (q * j / 16).is_integer()]
        for i, q in enumerate(qs):
            f = b * 128 + i
            gate[f, 8], up[f, :8] = 32.0, _as_codes(q * j / 16, 8)
            want[f] = F.decode(F.encode(np.array(q))) * 448 * 2 * j        # scale of h: 32 * 28 j / 448
        ties += len(qs) - 1
        gate[b * 128, 100] = up[b * 128, 100] = 448.0     # scale 1; x has a zero there
    assert ties >= 12
    out = _one_expert(x, gate, up)
    assert np.array_equal(out, np.broadcast_to(want, out.shape))
