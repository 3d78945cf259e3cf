"""The balance loss and its gradient to single fp32 steps, on rows of two experts with the others masked out."""
import numpy as np
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib
from moe_expert_layer_renorm_b200.balance import RouterBalance
from oracle import fp8 as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24      # half a step of fp32, relative
# logits on a grid, so that their differences are exact; e^-d down to 2^-124
D = np.arange(8, 86 * 64, 131) / 64.0
EXPERTS = [2, 40, 64, 100, 128, 256, 512, 700, 1023, 1024]


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    _lib.device_status(clear=True)
    yield
    assert _lib.device_status(clear=True) == _lib.FT_DEV_OK


def _rows(E):
    l = torch.full((len(D), E), float("-inf"))
    l[:, 0], l[:, E - 1] = 1.5, torch.from_numpy(1.5 - D).float()
    return l.cuda()


@pytest.mark.parametrize("E", EXPERTS)
def test_gradient_of_an_unlikely_expert(E):
    """All tokens chose expert 0: dlogits of the last one is -f p (T p_0), and no sum here has more than two terms.

    In U: the exponential 4 (two steps); z, its reciprocal and f = scale / z 3; scale 6 (its products and quotient);
    the mean 3 and z again 2; the difference, product and store 2: 20."""
    l, T = _rows(E), len(D)
    b = RouterBalance(T, E, 1, 0.25)
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    b.forward(l, ids)
    d = b.backward(l, ids).double().cpu().numpy()
    p = np.exp(-D) / (1 + np.exp(-D))
    ref = 0.25 * E / T ** 2 * p * T * (1 - p)
    assert np.all(np.abs(d[:, E - 1] + ref) <= 20 * U * ref)
    assert np.all(np.abs(d[:, 0] - ref) <= 2 ** -20 * 0.25 * E / T)      # its c - mean cancels
    assert not d[:, 1:E - 1].any()


@pytest.mark.parametrize("E", EXPERTS)
def test_loss_of_an_unlikely_choice(E):
    """One token whose choice has the probability p: coef E p.

    In U: the exponential 4; z, its reciprocal and p 3; count times p one; coef E, the quotient and the product 3: 11,
    and 12 with the products of these."""
    l = _rows(E)
    b = RouterBalance(1, E, 1, 0.3)
    ids = torch.full((1, 1), E - 1, dtype=torch.int32, device="cuda")
    got = np.array([float(b.forward(l[i:i + 1], ids)) for i in range(len(D))])
    ref = float(np.float32(0.3)) * E * np.exp(-D) / (1 + np.exp(-D))
    assert np.all(np.abs(got - ref) <= 12 * U * ref)


@pytest.mark.parametrize("T,E,k", [(8192, 512, 10), (5000, 1024, 8), (257, 100, 4), (256, 128, 8), (3000, 33, 2), (20000, 8, 2)])
def test_loss_and_gradient_of_many_tokens(T, E, k):
    """In U.  A probability: its argument |l - m|, the exponential 4, at most 32 places a lane and 5 exchanges in its
    sum, the reciprocal and its product 2.  A sum over the tokens adds no more terms in a chain than a warp takes tokens
    (all warps: 8 x 8 up to 256 tokens, else at least 8 x 16 of each of two clusters), then 16 warps, 8 CTAs and the
    clusters, 18 on this device and 32 at most; the loss a product, one chain of at most 32 + 5 + 32 experts' terms and
    6 for its factor.  All terms are positive."""
    g = torch.Generator().manual_seed(T + E)
    l = (torch.randn(T, E, generator=g) * 2.0 + torch.randn(E, generator=g)).cuda()
    ids = l.topk(k, dim=-1).indices.int()
    b = RouterBalance(T, E, k, 0.3)
    loss = float(b.forward(l, ids))
    d = b.backward(l, ids).double().cpu().numpy()
    ln, coef = l.double().cpu().numpy(), float(np.float32(0.3))
    counts, ref, dref = F.balance(ln, ids.cpu().numpy(), np.ones(T, bool), coef)
    assert np.array_equal(b.counts.cpu().numpy(), counts)
    spread = ln.max(1) - ln.min(1)
    p_err = spread.max() + 4 + 32 + 5 + 2
    tokens = T / (8 * 8 if T <= 256 else 2 * 8 * 16)
    assert abs(loss - ref) <= 1.01 * (p_err + tokens + 1 + 16 + 8 + 32 + 1 + 32 + 5 + 32 + 6) * U * ref
    # f p (c - mean): p and mean as above (the mean one product a place more), f six, the difference and products 4;
    # the difference may cancel, so its errors are those of c + mean
    p = np.exp(ln - ln.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    mean = (p * counts).sum(1, keepdims=True)
    scale = coef * E / (float(T) ** 2 * k)
    tol = 1.01 * U * scale * p * ((p_err + 10) * np.abs(counts - mean) + 4 * counts + (2 * p_err + 4) * mean)
    assert np.all(np.abs(d - dref) <= tol)
