"""The FP8 and balance entry points refuse bad arguments before they touch the GPU (runs without a GPU)."""
import ctypes

import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib, fp8
from moe_expert_layer_renorm_b200.build import build

INVALID = _lib.FT_ERR_INVALID_ARG
A = 1 << 20      # an address that is aligned and never read


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


@pytest.mark.parametrize("H,I", [(256, 512), (2048, 768), (2880, 2880), (320, 448)])
def test_fp8_layout_rules(L, H, I):
    lay = _lib.slot_layout(H, I, 3, _lib.FT_SCALE_FP8)
    rows, ks, end = (I, I, H), (H, H, I), 0
    assert (lay.scale_format, lay.tiled, lay.num_slots) == (_lib.FT_SCALE_FP8, 0, 3)
    for m in range(3):
        nb, kb = (rows[m] + 127) // 128, (ks[m] + 127) // 128
        assert lay.ld_scale[m] % 16 == 0 and lay.ld_scale[m] >= 4 * kb
        assert lay.codes_off[m] % 256 == 0 and lay.codes_off[m] >= end
        assert lay.scales_off[m] % 256 == 0 and lay.scales_off[m] >= lay.codes_off[m] + rows[m] * ks[m]
        end = lay.scales_off[m] + nb * lay.ld_scale[m]
    assert lay.slot_bytes % 256 == 0 and lay.slot_bytes >= end + 12


def test_fp8_layout_refusals(L):
    lay = _lib.SlotLayout()
    for H, I, n in ((100, 512, 1), (256, 500, 1), (256, 512, 0), (0, 512, 1)):
        assert L.ft_fp8_slot_layout_init(H, I, n, ctypes.byref(lay)) == INVALID
    assert L.ft_fp8_slot_layout_init(256, 512, 1, None) == INVALID
    with pytest.raises(_lib.FtError):
        _lib.slot_layout(256, 512, 1, _lib.FT_SCALE_FP8, tiled=True)


def quant(L, x=A, t=0, M=4, K=100, ld=100, codes=A, ldc=112, s=A, lds=1):
    return L.ft_fp8_quant_rows(x, t, M, K, ld, codes, ldc, s, lds, None)


def test_quant_refusals(L):
    assert quant(L, M=0, x=None, codes=None, s=None) == _lib.FT_OK
    for kw in (dict(M=-1), dict(K=0), dict(t=3), dict(ld=99), dict(ldc=96), dict(ldc=120), dict(K=129, ld=129, ldc=144),
               dict(x=None), dict(codes=None), dict(s=None), dict(codes=A + 8), dict(x=A + 2), dict(s=A + 2),
               dict(M=1 << 30, K=512, ld=512, ldc=512, lds=4)):
        assert quant(L, **kw) == INVALID, kw


def test_pack_refusals(L):
    ok = dict(w=A, N=100, K=100, c=A, ldc=112, s=A, lds=1)
    for kw in (dict(N=0), dict(K=0), dict(ldc=96), dict(ldc=104), dict(lds=0), dict(w=None), dict(c=None), dict(s=None),
               dict(c=A + 8)):
        a = {**ok, **kw}
        assert L.ft_fp8_pack(a["w"], a["N"], a["K"], a["c"], a["ldc"], a["s"], a["lds"], None) == INVALID, kw
    lay = _lib.slot_layout(256, 512, 2, _lib.FT_SCALE_FP8)
    assert L.ft_pack_slot(None, 0, ctypes.byref(lay), A, A, None) == INVALID
    lay.tiled = 1
    assert L.ft_pack_slot(A, 0, ctypes.byref(lay), A, A, None) == INVALID


def gemm(L, a=A, lda=128, sa=A, lsa=1, b=A, ldb=128, sb=A, lsb=1, M=4, N=32, K=128, out=A, t=1, ldo=32):
    return L.ft_fp8_gemm(a, lda, sa, lsa, b, ldb, sb, lsb, M, N, K, out, t, ldo, None)


def test_gemm_refusals(L):
    assert gemm(L, M=0, a=None, sa=None, out=None) == _lib.FT_OK
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(lda=112), dict(lda=136), dict(ldb=120), dict(K=129, lda=144, ldb=144),
               dict(ldo=31), dict(t=2), dict(t=7), dict(a=None), dict(sa=None), dict(b=None), dict(sb=None),
               dict(out=None), dict(a=A + 8), dict(b=A + 4), dict(sa=A + 2), dict(out=A + 1),
               dict(K=1 << 24, lda=1 << 24, ldb=1 << 24, lsa=1 << 20, lsb=1 << 20)):
        assert gemm(L, **kw) == INVALID, kw


def ffn(L, layout, x=A, T=4, H=256, I=512, E=8, k=2, ps=A, off=A, st=A, pool=A, out=A, t=0, ws=A, n=1 << 30):
    return L.ft_moe_ffn_fp8(x, T, H, I, E, k, ps, off, st, pool, ctypes.byref(layout) if layout else None, out, t, ws, n,
                            None)


def test_ffn_refusals(L):
    lay = _lib.slot_layout(256, 512, 8, _lib.FT_SCALE_FP8)
    assert ffn(L, lay, T=0, x=None, ws=None) == _lib.FT_OK
    for kw in (dict(H=192), dict(I=500), dict(k=9), dict(E=2000, k=2), dict(T=-1), dict(T=1 << 24, k=2)):
        assert ffn(L, lay, **kw) == _lib.FT_ERR_UNSUPPORTED, kw
    for kw in (dict(x=None), dict(ps=None), dict(off=None), dict(st=None), dict(pool=None), dict(out=None), dict(ws=None),
               dict(t=2), dict(H=320), dict(x=A + 2), dict(pool=A + 128), dict(ws=A + 64), dict(out=A + 8), dict(n=16)):
        assert ffn(L, lay, **kw) == INVALID, kw
    assert ffn(L, None) == INVALID
    for other in (_lib.slot_layout(256, 512, 8), _lib.slot_layout(256, 512, 8, _lib.FT_SCALE_MXFP4)):
        assert ffn(L, other) == INVALID
    # and the other formats' calls refuse an FP8 layout
    assert L.ft_moe_ffn_nvfp4(A, 4, 256, 512, 8, 2, A, A, A, A, ctypes.byref(lay), A, A, 1 << 30, None) == INVALID
    assert L.ft_moe_layer_nvfp4(A, A, 4, 256, 512, 8, 2, 0, A, A, ctypes.byref(lay), A, A, A, A, A, A, A, A, 1 << 30,
                                None) == INVALID
    assert _lib.ffn_fp8_workspace_size(0, 256, 512, 8, 2) == 0


def test_combine_bf16_refusals(L):
    assert L.ft_moe_combine_bf16(None, None, None, 0, 2, 256, None, None) == _lib.FT_OK
    for a in ((A, A, A, 4, 2, 252, A), (A, A, A, 4, 0, 256, A), (None, A, A, 4, 2, 256, A), (A + 8, A, A, 4, 2, 256, A),
              (A, A, A, -1, 2, 256, A)):
        assert L.ft_moe_combine_bf16(*a, None) == INVALID, a


def balance(L, l=A, ld=8, ids=A, v=None, T=4, E=8, k=2, c=A, n=A, loss=A, ws=A, nb=1 << 30):
    return L.ft_moe_balance(l, ld, ids, v, T, E, k, 0.01, c, n, loss, ws, nb, None)


def test_balance_refusals(L):
    for kw in (dict(T=-1), dict(E=1025, ld=1025), dict(E=0), dict(k=0), dict(k=9), dict(E=64, ld=64, k=33), dict(ld=7),
               dict(l=None), dict(ids=None), dict(c=None), dict(n=None), dict(loss=None), dict(ws=None), dict(nb=8),
               dict(ws=A + 4), dict(T=1 << 30, k=2)):
        assert balance(L, **kw) == INVALID, kw
    assert _lib.balance_workspace_size(0, 8) == 0


def back(L, l=A, ld=8, ids=A, w=A, dw=A, T=4, E=8, k=2, c=A, n=A, d=A, ldd=8):
    return L.ft_moe_route_backward(l, ld, ids, w, dw, None, T, E, k, 0.01, c, n, None, d, ldd, None)


def test_route_backward_refusals(L):
    assert back(L, T=0) == _lib.FT_OK
    for kw in (dict(c=None, dw=None), dict(l=None), dict(n=None), dict(w=None), dict(ids=None), dict(d=None),
               dict(ld=7), dict(ldd=7), dict(k=9), dict(E=1025, ld=1025, ldd=1025), dict(T=-1)):
        assert back(L, **kw) == INVALID, kw


def test_python_refusals():
    x = torch.zeros(4, 128)
    codes = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    for call in (lambda: fp8.quantize_rows(x), lambda: fp8.quantize_rows(x.double()), lambda: fp8.pack_weight(x.T),
                 lambda: fp8.Fp8Linear(codes, torch.zeros(1, 1)), lambda: fp8.Fp8Linear(codes, torch.zeros(2, 1)),
                 lambda: fp8.Fp8Linear(x, torch.zeros(1, 1))):
        with pytest.raises(ValueError):
            call()


def test_ffn_refuses_more_blocks_than_32_bits_count(L):
    H = 65536      # 512 blocks a row
    lay = _lib.slot_layout(H, 256, 8, _lib.FT_SCALE_FP8)
    for T in (1 << 22, 1 << 23):
        assert ffn(L, lay, T=T, H=H, I=256, k=1) == _lib.FT_ERR_UNSUPPORTED
        assert _lib.ffn_fp8_workspace_size(T, H, 256, 8, 1) == 0
        assert _lib.ffn_fp8_workspace_size(T, 256, H, 8, 1) == 0
    assert _lib.ffn_fp8_workspace_size((1 << 22) - 1, H, 256, 8, 1) > 0


def test_sizes_at_the_end_of_int(L):
    big = (1 << 31) - 1
    assert quant(L, K=big, ld=big, ldc=1 << 31, lds=1 << 23) == INVALID      # fewer scales than blocks
    assert quant(L, M=128, K=big, ld=big, ldc=1 << 31, lds=1 << 24) == INVALID   # 2^31 blocks
    assert L.ft_fp8_pack(A, big, 128, A, 128, A, 1, None) == INVALID
    assert L.ft_fp8_pack(A, 128, big, A, 1 << 31, A, 1 << 23, None) == INVALID
