"""Pins of the FP8 and balance oracle: closed forms, hand-worked blocks, differences (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8 as F


def test_e4m3_codes_against_the_published_format():
    assert F.e4m3_value(0x7E) == 448.0 and F.e4m3_value(0x08) == 2.0 ** -6 and F.e4m3_value(0x01) == 2.0 ** -9
    assert F.e4m3_value(0x38) == 1.0 and F.e4m3_value(0xB8) == -1.0 and math.isnan(F.e4m3_value(0xFF))
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(F.TABLE)) and np.array_equal(t[~np.isnan(t)], F.TABLE[~np.isnan(t)])


def test_encode_is_nearest_even_and_the_inverse_of_decode():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    assert np.array_equal(F.encode(F.decode(codes)), codes)
    mid = (F.TABLE[:126] + F.TABLE[1:127]) / 2           # ties: to the even code
    assert np.array_equal(F.encode(mid), np.array([c if c % 2 == 0 else c + 1 for c in range(126)], np.uint8))
    assert np.array_equal(F.encode(mid * (1 + 1e-12)), np.arange(1, 127, dtype=np.uint8))
    assert np.array_equal(F.encode(mid * (1 - 1e-12)), np.arange(126, dtype=np.uint8))
    assert F.encode(np.array([1e9, -1e9, np.nan])).tolist() == [0x7E, 0xFE, 0x7F]


def test_hand_worked_group():
    x = np.zeros((1, 130))
    x[0, :3] = [2.0, -1.0, 2.0 / 448]       # m = 2: 448, -224, 1
    x[0, 128] = 448 * 2.0 ** -110            # a group below the floor: 448 * 448 * 2^-10 = 196 -> 192 (tie-free)
    codes, scales, q = F.quant_rows(x)
    assert F.decode(codes)[0, :3].tolist() == [448.0, -224.0, 1.0]
    assert scales[0].tolist() == [2.0 / 448, 2.0 ** -100 / 448]
    assert q[0, 128] == 196.0 and F.decode(codes)[0, 128] == 192.0 and codes[0, 129] == 0


def test_ffn_bound_covers_a_perturbed_evaluation():
    g = np.random.default_rng(0)
    H, I = 256, 320
    w = [F.pack(g.standard_normal(s) * 0.02) for s in ((I, H), (I, H), (H, I))]
    x = g.standard_normal((5, H))
    out, bound = F.ffn_rows(x, *w)
    assert np.all(bound < 0.2 * np.sqrt(np.mean(out ** 2)))     # the bound says something
    cx, sx, _ = F.quant_rows(x)
    xv = F.rows_value(cx, sx).astype(np.float32)
    G, U, D = (F.weight_value(*t).astype(np.float32) for t in w)
    gg, uu = xv @ G.T, xv @ U.T
    h = gg / (1 + np.exp(-gg)) * uu
    ch, sh, _ = F.quant_rows(h)
    got = F.rows_value(ch, sh.astype(np.float32)).astype(np.float32) @ D.T
    assert np.all(np.abs(got - out) <= bound)


@pytest.mark.parametrize("T,E,k", [(5, 6, 2), (7, 3, 3), (1, 4, 1)])
def test_balance_gradient_is_the_difference_quotient(T, E, k):
    g = np.random.default_rng(T)
    l = g.standard_normal((T, E))
    ids = np.argsort(-l, axis=1)[:, :k]
    valid = np.ones(T, bool)
    valid[-1] = T == 1
    counts, loss, d = F.balance(l, ids, valid, 0.3)
    for t in range(T):
        for e in range(E):
            a, b = l.copy(), l.copy()
            a[t, e] += 1e-5
            b[t, e] -= 1e-5
            diff = (F.balance(a, ids, valid, 0.3)[1] - F.balance(b, ids, valid, 0.3)[1]) / 2e-5
            assert abs(diff - d[t, e]) < 1e-9        # the third derivative times 1e-10
    assert counts.sum() == k * valid.sum()


def test_balance_of_an_even_spread_is_the_coefficient():
    T, E, k = 12, 4, 2
    ids = np.array([[t % E, (t + 1) % E] for t in range(T)])
    counts, loss, d = F.balance(np.zeros((T, E)), ids, np.ones(T, bool), 0.01)
    assert counts.tolist() == [6] * 4 and loss == pytest.approx(0.01, rel=1e-15) and not d.any()
    assert F.balance(np.zeros((T, E)), ids, np.zeros(T, bool), 0.01)[1] == 0.0


def test_weights_gradient_is_the_difference_quotient():
    g = np.random.default_rng(3)
    l, dw = g.standard_normal((4, 6)), g.standard_normal((4, 3))
    ids = np.argsort(-l, axis=1)[:, :3]

    def f(l):
        s = np.take_along_axis(l, ids, 1)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        return w, float((w * dw).sum())

    d = F.weights_grad(ids, f(l)[0], dw, 6)
    for t in range(4):
        for e in range(6):
            a, b = l.copy(), l.copy()
            a[t, e] += 1e-5
            b[t, e] -= 1e-5
            assert abs((f(a)[1] - f(b)[1]) / 2e-5 - d[t, e]) < 1e-9
