"""Balance loss, per-expert counts and the router's gradient on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib
from moe_expert_layer_renorm_b200.balance import RouterBalance
from oracle import fp8 as F

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    _lib.device_status(clear=True)
    yield
    assert _lib.device_status(clear=True) == _lib.FT_DEV_OK


def _batch(T, E, k, seed, spread=1.0, pitch=None):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(T, pitch or E, generator=g) * spread
    l = wide.cuda()[:, :E]
    top = l.topk(k, dim=-1)
    w = torch.softmax(top.values, -1)
    dw = torch.randn(T, k, generator=g).cuda()
    return l, top.indices.int(), w, dw


# fp32 against 64 bits.  A probability: the exponential's argument l - m loses 2^-24 |l - m| <= 2^-19 for the spreads
# here, exp and the division a few steps: 2^-18 of p.  A sum of T of them, added in chains of at most T / 8 terms a
# warp, 8 warps and the blocks: (T + 200) 2^-24 more of the sum.
def _p_error(T):
    return 2.0 ** -18 + (T + 200) * 2.0 ** -24


SHAPES = [(1, 1, 1), (1, 2, 1), (1, 128, 8), (7, 5, 3), (64, 128, 8), (300, 512, 10), (129, 33, 4), (1000, 1024, 32),
          (4096, 64, 6), (50, 100, 2), (9, 1023, 7), (2500, 256, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("padded", [False, True])
def test_balance_and_its_gradient(T, E, k, padded):
    l, ids, w, dw = _batch(T, E, k, T + E, spread=2.0, pitch=E + (3 if padded else 0))
    valid = None
    v = np.ones(T, bool)
    if padded:
        v = np.random.default_rng(T).random(T) < 0.8
        valid = torch.from_numpy(v).cuda()
        ids[~valid] = -1                                  # ids of padding are not read
        l[~valid] = float("nan")                         # nor its logits
        w[~valid], dw[~valid] = float("nan"), float("nan")
    b = RouterBalance(T, E, k, 0.37)
    b._ws.fill_(0xFF)
    loss = b.forward(l, ids, valid=valid)
    idn = ids.cpu().numpy()
    ln = l.double().cpu().numpy()
    counts, ref, dref = F.balance(ln, idn, v, 0.37)
    assert np.array_equal(b.counts.cpu().numpy(), counts) and int(b.n_valid) == v.sum()
    assert abs(float(loss) - ref) <= (_p_error(T) + 2.0 ** -20) * ref      # all terms are positive
    dloss = torch.tensor([1.7], device="cuda")
    b.dlogits.fill_(float("nan"))
    d = b.backward(l, ids, dloss=dloss, valid=valid).double().cpu().numpy()
    dl = float(dloss)
    # p (c - sum p c): the factor loses at most 2^-18 of the largest count, the product a few steps
    scale = dl * 0.37 * E / (max(1, v.sum()) ** 2 * k)
    p = np.zeros((T, E))
    p[v] = torch.softmax(l.double(), -1).cpu().numpy()[v]
    tol = 2.0 ** -17 * np.abs(dl * dref) + scale * p * counts.max() * 2.0 ** -16 + 1e-30
    assert np.all(np.abs(d - dl * dref) <= tol)
    assert not d[~v].any()
    # with the weights' gradient in the same pass, and alone
    wref = np.zeros((T, E))
    wn, dwn = w.double().cpu().numpy(), dw.double().cpu().numpy()
    wref[v] = F.weights_grad(idn[v], wn[v], dwn[v], E)
    wtol = 2.0 ** -20 * (np.abs(wref) + (np.abs(dwn).max(1, initial=0, where=~np.isnan(dwn)) * 1.0)[:, None])
    both = b.backward(l, ids, dloss=dloss, w=w, dw=dw, valid=valid).double().cpu().numpy()
    assert np.all(np.abs(both - dl * dref - wref) <= tol + wtol)
    alone = torch.full((T, E), float("nan"), device="cuda")
    _lib.route_backward(0, 0, ids.data_ptr(), w.data_ptr(), dw.data_ptr(), 0 if valid is None else valid.data_ptr(), T, E, k,
                        0.0, 0, 0, 0, alone.data_ptr(), E, torch.cuda.current_stream().cuda_stream)
    assert np.all(np.abs(alone.double().cpu().numpy() - wref) <= wtol)


def test_no_tokens_and_no_valid_tokens():
    b = RouterBalance(0, 16, 2, 0.1)
    b.loss.fill_(9)
    b.counts.fill_(9)
    e = torch.empty
    b.forward(e(0, 16, device="cuda"), e(0, 2, dtype=torch.int32, device="cuda"))
    assert float(b.loss) == 0 and not b.counts.any() and int(b.n_valid) == 0
    l, ids, w, dw = _batch(5, 16, 2, 1)
    b = RouterBalance(5, 16, 2, 0.1)
    none = torch.zeros(5, dtype=torch.bool, device="cuda")
    assert float(b.forward(l, ids, valid=none)) == 0 and not b.counts.any()
    b.dlogits.fill_(7)
    assert not b.backward(l, ids, w=w, dw=dw, valid=none).any()


def test_masked_experts_empty_rows_and_non_finite_logits():
    l, ids, _, _ = _batch(6, 40, 3, 2)
    l[:, 7] = float("-inf")                # an expert nobody may use
    ids = l.topk(3, dim=-1).indices.int()
    b = RouterBalance(6, 40, 3, 0.5)
    loss = float(b.forward(l, ids))
    counts, ref, dref = F.balance(l.double().cpu().numpy(), ids.cpu().numpy(), np.ones(6, bool), 0.5)
    assert loss == pytest.approx(ref, rel=1e-5) and int(b.counts[7]) == 0
    d = b.backward(l, ids)
    assert not d[:, 7].any() and torch.isfinite(d).all()
    l[3] = float("-inf")                   # a row without probabilities
    loss = float(b.forward(l, ids))
    _, ref, _ = F.balance(l.double().cpu().numpy(), ids.cpu().numpy(), np.ones(6, bool), 0.5)
    assert loss == pytest.approx(ref, rel=1e-5)
    d = b.backward(l, ids)
    assert not d[3].any() and torch.isfinite(d).all()
    l[4, 0] = float("nan")
    assert torch.isnan(b.forward(l, ids)).all()
    d = b.backward(l, ids)
    assert torch.isnan(d[4]).all() and torch.isfinite(d[:4]).all() and torch.isfinite(d[5]).all()


def test_repeated_and_bad_ids():
    l, ids, w, dw = _batch(4, 16, 3, 5)
    ids[0] = ids[0, 0]                      # one expert three times
    b = RouterBalance(4, 16, 3, 1.0)
    b.forward(l, ids)
    idn = ids.cpu().numpy()
    assert np.array_equal(b.counts.cpu().numpy(), np.bincount(idn.reshape(-1), minlength=16))
    d = b.backward(l, ids, w=w, dw=dw).double().cpu().numpy()
    ref = F.balance(l.double().cpu().numpy(), idn, np.ones(4, bool), 1.0)[2] + F.weights_grad(
        idn, w.double().cpu().numpy(), dw.double().cpu().numpy(), 16)
    assert np.all(np.abs(d - ref) <= 1e-5)   # values of order 1, a few dozen fp32 steps of 6e-8
    ids[2, 1] = 16
    b.forward(l, ids)
    assert _lib.device_status(clear=True) == _lib.FT_DEV_BAD_INDEX
    assert int(b.counts.sum()) == 11
    b.backward(l, ids, w=w, dw=dw)
    assert _lib.device_status(clear=True) == _lib.FT_DEV_BAD_INDEX


@pytest.mark.parametrize("T,E,k", [(64, 128, 8), (5000, 100, 4)])
def test_same_bits_eager_again_and_in_a_graph(T, E, k):
    l, ids, w, dw = _batch(T, E, k, 8)
    b = RouterBalance(T, E, k, 0.01)
    loss, d = b.forward(l, ids).clone(), b.backward(l, ids, w=w, dw=dw).clone()
    assert torch.equal(loss, b.forward(l, ids)) and torch.equal(d, b.backward(l, ids, w=w, dw=dw))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(l, ids)
        b.backward(l, ids, w=w, dw=dw)
    for _ in range(3):
        b.loss.zero_(), b.dlogits.zero_(), b.counts.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, b.loss) and torch.equal(d, b.dlogits) and int(b.counts.sum()) == T * k


def test_router_step_lowers_a_skewed_loss_with_the_router_kernel():
    """route, balance and gradient together: the gradient agrees with differences of the GPU's own loss."""
    T, E, k = 256, 32, 4
    l, _, _, _ = _batch(T, E, k, 3)
    l = l.contiguous()
    l[:, :4] += 1.0
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    _lib.route(l.data_ptr(), T, E, k, 0, ids.data_ptr(), w.data_ptr(), s)
    b = RouterBalance(T, E, k, 1.0)
    b.forward(l, ids)
    d = b.backward(l, ids).clone()
    step = torch.randn(T, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) * 0.05
    up, down = float(b.forward(l + step, ids)), float(b.forward(l - step, ids))
    # the third-order term of a step of 0.05 is a few 1e-3 of the first; the loss itself is good to 1e-6
    assert (up - down) / 2 == pytest.approx(float((d * step).sum()), rel=2e-2, abs=2e-6)


def test_tensors_of_another_device_are_refused():
    b = RouterBalance(4, 8, 2, 0.01)
    logits, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    valid, one = torch.ones(4, dtype=torch.bool), torch.ones(1)
    L, I, W = logits.cuda(), ids.cuda(), w.cuda()
    for call in (lambda: b.forward(logits, I), lambda: b.forward(L, ids), lambda: b.forward(L, I, valid),
                 lambda: b.backward(L, I, dloss=one), lambda: b.backward(L, I, w=w, dw=W),
                 lambda: b.backward(L, I, w=W, dw=w)):
        with pytest.raises(AssertionError):
            call()
