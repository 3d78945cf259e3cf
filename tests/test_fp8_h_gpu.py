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


@pytest.mark.parametrize("at_once", [11, 22, 60, 66])
def test_silu_to_a_few_fp32_steps(at_once):
    """One h alone in each block of 128 is the block's largest, and the output 448 h.

    G and U are exact.  In units of 2^-24: the exponential 4 (two steps), 1 + e one, the quotient two, its product with
    G one (with U, a power of two, none), the scale one, the output one: 10, and 12 with the products of these.  Where
    e^-|G| is subnormal it is held to 2^-149."""
    U = 2.0 ** 30
    x0 = np.array([s * m / 8 * 2.0 ** e for e in range(-3, 1) for m in range(8, 16) for s in (1, -1)] + [2.0, -2.0])
    x = torch.zeros(len(x0), H)
    x[:, 0], x[:, 1], x[:, 101] = torch.from_numpy(x0), 1.0, 448.0
    gate, up = torch.zeros(I, H), torch.zeros(I, H)
    wg = np.array([4.0, 44.0])
    for b in range(2):
        gate[b * 128, 0], up[b * 128, 1] = wg[b], U
        gate[b * 128, 100], up[b * 128, 100] = 448.0, 448.0 * U
    out = np.concatenate([_one_expert(x[i:i + at_once], gate, up) for i in range(0, len(x0), at_once)])
    G = x0[:, None] * wg
    h = G * U / (1 + np.exp(-G))
    got = out[:, [0, 128]] / 448
    assert np.all(np.abs(got - h) <= 12 * 2.0 ** -24 * np.abs(h) + np.abs(G) * U * 2.0 ** -149)
    rest = np.ones(H, bool)
    rest[[0, 128]] = False
    assert not out[:, rest].any()
