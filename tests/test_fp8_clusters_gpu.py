"""FP8 products whose tiles are shared by clusters of CTAs, and kernels that share SMs."""
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib

from .test_fp8_gpu import Ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    _lib.device_status(clear=True)
    yield
    assert _lib.device_status(clear=True) == _lib.FT_DEV_OK


@pytest.mark.parametrize("rows,H,I,k", [([1, 1], 2880, 2880, 1), ([1], 2048, 768, 1), ([1] * 8, 2048, 768, 8)])
def test_kernels_that_share_sms_on_three_streams(rows, H, I, k):
    """Few tiles: gate/up and down of every stream fit a SM beside each other, their tiles split over clusters."""
    fs = [Ffn(rows, H, I, k, seed=50 + i) for i in range(3)]
    want = [f.run().clone() for f in fs]
    tables = [torch.from_numpy(f.table).cuda() for f in fs]
    streams = [torch.cuda.Stream() for _ in fs]
    fs[0].check(want[0])
    for f in fs:
        f.layer.out_perm.fill_(-5.0)
    torch.cuda.synchronize()
    for _ in range(60):
        for f, t, s in zip(fs, tables, streams):
            f.layer.ffn(f.x, t, f.pool, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(f.layer.out_perm, w) for f, w in zip(fs, want))
