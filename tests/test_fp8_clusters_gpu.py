"""FP8 products whose tiles are shared by clusters of CTAs, kernels that share SMs, layers of hundreds of experts, and
rows beside other rows."""
import math

import numpy as np
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib, fp8

from oracle import fp8 as F

from .test_fp8_gpu import BF16_STEP, DTYPES, Ffn, _check_product, _f64, _operands

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


def _split(tiles, nk, sms, clusters):
    """(CTAs that share a tile, tiles of the busiest cluster) by the stream kernel's rule: K blocks of the busiest
    cluster, three more a split tile; clusters[S] of S CTAs fit the device."""
    best, split, most = math.ceil(tiles / sms) * nk, 1, math.ceil(tiles / sms)
    for S in (2, 4, 8):
        per = -(-nk // S)
        if S > nk or (S - 1) * per >= nk:
            continue
        cost = math.ceil(tiles / clusters[S]) * (per + 3)
        if cost < best:
            best, split, most = cost, S, math.ceil(tiles / clusters[S])
    return split, most


# tiles and K blocks -> the split, with several tiles a cluster
SHARED = [(100, 64, 4), (48, 64, 8), (184, 23, 2)]


def test_the_shapes_below_make_a_cluster_finish_several_split_tiles():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    full = {S: sms // S for S in (2, 4, 8)}
    for few in (0, 1, 2):       # a device holds no more clusters than its SMs allow, and may hold some fewer
        for tiles, nk, split in SHARED:
            got, most = _split(tiles, nk, sms, {S: n - few for S, n in full.items()})
            assert got == split and most >= 2, (tiles, nk, few, got, most)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,tiles,nk", [(4, 100, 64), (16, 48, 64), (27, 100, 64), (32, 48, 64), (1, 184, 23)])
def test_gemm_of_several_split_tiles_a_cluster(M, tiles, nk, out):
    assert (tiles, nk) in [t[:2] for t in SHARED]
    a, b = _operands(M, tiles * 128 - 5, nk * 128 - 17, M + tiles)
    lin = fp8.Fp8Linear(*b)
    y = lin.matmul(*a, out_dtype=DTYPES[out])
    _check_product(y, a, b)
    for _ in range(20):
        assert torch.equal(y, lin.matmul(*a, out_dtype=DTYPES[out]))


@pytest.mark.parametrize("rows,k", [([1] * 8 + [0] * 24, 4), ([20] * 8, 4), ([39, 41, 40, 40, 38, 42, 40, 40], 4)])
def test_ffn_of_several_split_tiles_a_cluster(rows, k):
    """8 groups of one tile each, 23 feature tiles of 23 K blocks: 184 tiles, two CTAs a tile (down; gate/up too while a
    tile has up to 32 rows)."""
    f = Ffn(np.random.default_rng(0).permutation(rows).tolist(), 2880, 2880, k, seed=70 + len(rows))
    out = f.run().clone()
    f.check(out)
    for _ in range(20):
        assert torch.equal(out, f.run())


def _check_elements(f, out):
    """Every element against its bound, which counts the codes of h that sit near a tie.  (A norm over a group says
    nothing here: a group may be one row of 256 h, of which one code that goes the other way at a tie, a sixteenth to
    an eighth of one h, is a percent.)"""
    x, got = _f64(f.x), _f64(out)
    for e in range(f.E):
        r0, r1 = f.off[e], f.off[e + 1]
        if r0 == r1:
            continue
        ref, bound = F.ffn_rows(x[f.perm[r0:r1] // f.k],
                                *[f.pool.tensor_bytes(int(f.table[e]), m)[:2] for m in range(3)])
        assert np.all(np.abs(got[r0:r1] - ref) <= bound + BF16_STEP * (np.abs(ref) + bound)), e
    assert (got[f.off[-1]:] == -5.0).all()


# groups per thread, work lists of up to 32 CTAs, tiles of 16, 32, 128 and 256 rows
@pytest.mark.parametrize("E,mean", [(512, 1), (512, 3), (1024, 2), (512, 18), (512, 60), (512, 200), (1024, 70)])
def test_ffn_of_hundreds_of_experts(E, mean):
    g = np.random.default_rng(E + mean)
    share = g.dirichlet(np.full(E, 1.5))
    rows = g.multinomial(E * mean, share)
    rows[g.integers(0, E, 5)] = 0
    rows[-1] += -rows.sum() % 2
    f = Ffn(rows.tolist(), 256, 256, 2, seed=E + mean, out=torch.bfloat16)
    _check_elements(f, f.run())


@pytest.mark.parametrize("M,N,K", [(5, 700, 1000), (40, 700, 1000), (300, 700, 1000), (1300, 2500, 300)])
def test_rows_do_not_depend_on_the_rows_beside_them(M, N, K):
    a, b = _operands(M, N, K, 11)
    other, _ = _operands(M, N, K, 12, spread=3.0)
    lin = fp8.Fp8Linear(*b)
    y = lin.matmul(*a, out_dtype=torch.float32)
    keep = torch.rand(M, generator=torch.Generator().manual_seed(M)) < 0.4
    keep[0], keep[M - 1] = True, False
    keep = keep.cuda()
    codes = torch.where(keep[:, None], a[0].view(torch.uint8), other[0].view(torch.uint8))
    pad = fp8.empty_codes(M, K, "cuda")
    pad.view(torch.uint8).copy_(codes)
    z = lin.matmul(pad, torch.where(keep[:, None], a[1], other[1]), out_dtype=torch.float32)
    assert torch.equal(y[keep], z[keep]) and not torch.equal(y[~keep], z[~keep])


@pytest.mark.parametrize("rows", [[1, 3, 2], [9, 14], [25, 30], [200, 130, 190]])
def test_ffn_rows_do_not_depend_on_the_rows_beside_them(rows):
    f = Ffn(rows, 512, 512, 1, seed=8)
    y = f.run().clone()
    keep = np.random.default_rng(1).random(sum(rows)) < 0.4
    keep[0], keep[-1] = True, False
    gone = torch.from_numpy(f.perm[~keep].astype(np.int64)).cuda()
    f.x[gone] = (f.x[gone].float() * -3.0 + 1.0).bfloat16()
    z = f.run()
    keep = torch.from_numpy(keep).cuda()
    assert torch.equal(y[keep], z[keep]) and not torch.equal(y[~keep], z[~keep])
