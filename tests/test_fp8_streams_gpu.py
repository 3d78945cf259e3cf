"""FP8 layers on a stream that is given: their memory is not what the current stream still writes."""
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib
from moe_expert_layer_renorm_b200.layer import ExpertPool, MoELayer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4, 600])
def test_first_ffn_on_a_given_stream(cuda_device, T):
    E, H, I = 4, 256, 512
    gen = torch.Generator(device="cuda").manual_seed(T)
    pool = ExpertPool(H, I, E, fmt=_lib.FT_SCALE_FP8)
    for e in range(E):
        for mat in range(3):
            pool.pack_into(e, mat, torch.randn(*pool.shape(mat), generator=gen, device="cuda") * 0.02)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=gen, device="cuda")
    table = torch.arange(E, dtype=torch.int32, device="cuda")
    want = MoELayer(T, E, 2, H, I).forward(x, logits, table, pool).clone()
    lay = MoELayer(T, E, 2, H, I)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.empty(max(n, 256), dtype=torch.uint8, device="cuda") for n in (lay.perm_ws_bytes, lay.fp8_ws_bytes)]
    at = [h.data_ptr() for h in held]
    torch.cuda._sleep(20_000_000)      # some 10 ms, then the current stream writes what it has given back
    for h in held:
        h.fill_(0x2A)
    del held, h
    got = lay.forward(x, logits, table, pool, stream=side)
    assert not {lay.perm_ws.data_ptr(), lay.fp8_ws.data_ptr()} & set(at)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and _lib.device_status(clear=True) == _lib.FT_DEV_OK
