"""FP8 weights whose rows, or rows of scales, end just below 2^31."""
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib

pytestmark = pytest.mark.gpu


def _pack(w, K, codes, ldc, scales, lds):
    _lib.fp8_pack(w.data_ptr(), 1, K, codes.data_ptr(), ldc, scales.data_ptr(), lds,
                  torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()


@pytest.mark.parametrize("short", [100, 67, 1])
def test_pack_writes_no_code_past_a_row_that_ends_below_2_31(cuda_device, short):
    K = 2 ** 31 - short
    ldc, nb = (K + 15) // 16 * 16, (K + 127) // 128
    w = torch.zeros(K, device="cuda")
    w[0], w[K - 1], w[K - 29] = 7.0, -3.5, 1.75
    codes = torch.full((ldc + 256,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((nb + 64,), -3.0, device="cuda")
    _pack(w, K, codes, ldc, scales, nb)
    v = codes.view(torch.float8_e4m3fn)
    own_block = (K - 29) // 128 != (K - 1) // 128      # the largest value of a block has the code 448
    assert float(v[0]) == 448.0 and float(v[K - 1]) == -448.0 and float(v[K - 29]) == (448.0 if own_block else 224.0)
    assert float(scales[0]) * 448 == 7.0 and float(scales[nb - 1]) * 448 == 3.5
    assert int(codes.count_nonzero()) == 3 + ldc + 256 - K and (codes[K:] == 0x55).all() and (scales[nb:] == -3.0).all()


def test_pack_zeroes_the_columns_of_scale_rows_up_to_2_31(cuda_device):
    lds = 2 ** 31 - 1
    scales = torch.full((lds + 64,), -3.0, device="cuda")
    codes = torch.zeros(16, dtype=torch.uint8, device="cuda")
    _pack(torch.ones(1, device="cuda"), 1, codes, 16, scales, lds)
    assert abs(float(scales[0]) * 448 - 1.0) <= 2.0 ** -24 and (scales[lds:] == -3.0).all()
    assert int(scales.count_nonzero()) == 65
