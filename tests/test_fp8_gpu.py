"""FP8 rows, weights, product and expert FFN on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from moe_expert_layer_renorm_b200 import _lib, fp8, inputs
from moe_expert_layer_renorm_b200.layer import ExpertPool, MoELayer
from oracle import fp8 as F
from oracle import moe_layer as M

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BF16_STEP, F32_STEP = 2.0 ** -8, 2.0 ** -24


def _u8(t):
    return t.view(torch.uint8).cpu().numpy()


def _f64(t):
    return t.double().cpu().numpy()


def _status():
    return _lib.device_status(clear=True)


@pytest.fixture(autouse=True)
def _clean_status(cuda_device):
    _status()
    yield
    assert _status() == _lib.FT_DEV_OK


# ------------------------------------------------------------- rows ---

@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("M,K,ld", [(1, 1, 1), (1, 128, 128), (3, 130, 130), (17, 200, 203), (64, 2048, 2048),
                                    (5, 2880, 2888), (257, 7, 9), (33, 127, 128)])
def test_quant_rows_bit_exact(dtype, M, K, ld):
    g = torch.Generator().manual_seed(M * 1000 + K)
    x = (torch.randn(M, ld, generator=g) * torch.exp(4 * torch.randn(M, 1, generator=g))).to(DTYPES[dtype])
    if M > 2:
        x[1] = 0
        x[2, :K // 2] *= 2.0 ** -12
    d = x.cuda()[:, :K]
    guard = torch.full((M, (K + 15) // 16 * 16 + 16), 0x55, dtype=torch.uint8, device="cuda")
    codes = guard.view(torch.float8_e4m3fn)[:, :K]
    scales = torch.full((M, (K + 127) // 128 + 2), -3.0, device="cuda")
    fp8.quantize_rows(d, codes, scales[:, :(K + 127) // 128])
    ref_c, ref_s, q = F.quant_rows(x[:, :K].double().numpy())
    got = _u8(codes)
    if dtype == "fp32":
        # 448 x is rounded once and the quotient once: off by at most 2^-23 of it, a step at a tie that near
        lo, hi = F.encode(q * (1 - 2.0 ** -23 * np.sign(q))), F.encode(q * (1 + 2.0 ** -23 * np.sign(q)))
        assert np.all((got == ref_c) | (got == lo) | (got == hi))
        assert np.mean(got != ref_c) < 1e-3
    else:
        assert np.array_equal(got, ref_c)
    got_s = _f64(scales)[:, :ref_s.shape[1]]
    fine = np.isfinite(ref_s)            # some fp16 rows overflow to infinity: their scale is infinite too
    assert np.all(np.abs(got_s - ref_s)[fine] <= F32_STEP * ref_s[fine]) and np.array_equal(got_s[~fine], ref_s[~fine])
    assert (scales[:, (K + 127) // 128:] == -3.0).all() and (guard[:, K:] == 0x55).all()


def test_quant_rows_ties_extremes_and_non_finite():
    x = torch.zeros(8, 128)
    x[0, :4] = torch.tensor([448.0, 17.0, 19.0, -21.0])      # 17 and 19 lie between 16, 18 and 20: ties to even
    x[1, :2] = torch.tensor([3.0e38, -1.0e38])               # 448 x would leave fp32
    x[2, :2] = torch.tensor([2.0 ** -120, 2.0 ** -101])      # below the floor of 2^-100
    x[3, :3] = torch.tensor([float("nan"), 7.0, -3.5])
    x[4, :3] = torch.tensor([float("inf"), 7.0, -3.5])
    x[5, :2] = torch.tensor([2.0 ** 100, 2.0 ** 90])
    x[6, :] = 2.0 ** -149
    codes, scales = fp8.quantize_rows(x.cuda())
    v = _f64(codes.float())
    assert v[0, :4].tolist() == [448.0, 16.0, 20.0, -20.0]
    assert v[1, 0] == 448.0 and v[1, 1] == -144.0            # -149.33: between 144 and 160
    assert v[2, :2].tolist() == [0.0, 224.0]                 # 448 2^-20 rounds to 0
    assert np.isnan(v[3, 0]) and v[3, 1:3].tolist() == [448.0, -224.0] and float(scales[3, 0]) == np.float32(7 / 448)
    assert np.isinf(float(scales[4, 0])) and np.isnan(v[4, 0]) and v[4, 1] == 0.0
    assert v[5, :2].tolist() == [448.0, 0.4375]
    assert not v[6].any() and not v[7].any() and torch.isfinite(scales[[6, 7]]).all()


@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (130, 257), (64, 2880), (300, 100), (2880, 64)])
def test_pack_weight(N, K):
    g = torch.Generator().manual_seed(N + K)
    w = torch.randn(N, K, generator=g) * 0.02
    codes, scales = fp8.pack_weight(w.cuda())
    ref_c, ref_s = F.pack(w.double().numpy())
    got = _u8(codes)
    assert np.all(np.abs(_f64(scales) - ref_s) <= F32_STEP * ref_s)
    s = np.repeat(np.repeat(ref_s, 128, 0)[:N], 128, 1)[:, :K]
    q = w.double().numpy() / s
    lo, hi = F.encode(q * (1 - 2.0 ** -23)), F.encode(q * (1 + 2.0 ** -23))
    assert np.all((got == ref_c) | (got == lo) | (got == hi)) and np.mean(got != ref_c) < 1e-3


# ---------------------------------------------------------- product ---

def _operands(M, N, K, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda") * torch.exp(spread * torch.randn(M, 1, generator=g, device="cuda"))
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    return fp8.quantize_rows(x), fp8.pack_weight(w)


def _check_product(out, a, b):
    av, bv = F.rows_value(_u8(a[0]), _f64(a[1])), F.weight_value(_u8(b[0]), _f64(b[1]))
    ref, bound = av @ bv.T, F.gemm_bound(av, bv)
    step = BF16_STEP if out.dtype == torch.bfloat16 else F32_STEP
    err = np.abs(_f64(out) - ref)
    assert np.all(err <= bound + step * (np.abs(ref) + bound)), float((err / (bound + step * np.abs(ref) + 1e-300)).max())
    if out.dtype == torch.float32 and ref.size > 1000:
        # in norm, additions that lose a half to a whole step each: far below the bound on every element
        assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(ref)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 2048, 2048), (2, 100, 130), (7, 257, 64), (8, 128, 128), (16, 130, 1100), (17, 384, 2880),
    (33, 1000, 15), (64, 2880, 2880), (65, 129, 257), (128, 256, 512), (129, 300, 700), (200, 1234, 1100),
    (300, 512, 127), (1, 7, 4096), (1037, 1234, 1100), (260, 5000, 96), (2, 20000, 64),
    (300, 6500, 200), (1100, 2500, 300), (600, 4104, 130), (513, 7001, 1030)])
def test_gemm(M, N, K, out):
    a, b = _operands(M, N, K, M * 7 + N * 3 + K)
    y = fp8.Fp8Linear(*b).matmul(*a, out_dtype=DTYPES[out])
    _check_product(y, a, b)


@pytest.mark.parametrize("M", [3, 300])
def test_gemm_pitches_and_guards(M):
    N, K = 333, 200
    a, b = _operands(M, N, K, 5)
    wide_a = torch.full((M, 224), 0x7F, dtype=torch.uint8, device="cuda")       # NaN codes behind every row
    wide_a[:, :K] = a[0].view(torch.uint8)
    wide_b = torch.full((N, 240), 0x7F, dtype=torch.uint8, device="cuda")
    wide_b[:, :K] = b[0].view(torch.uint8)
    sa = torch.full((M, 5), float("nan"), device="cuda")
    sa[:, :2] = a[1]
    sb = torch.full((3, 4), float("nan"), device="cuda")
    sb[:, :2] = b[1]
    out = torch.full((M + 1, 400), -7.0, device="cuda")
    lin = fp8.Fp8Linear(wide_b.view(torch.float8_e4m3fn)[:, :K], sb[:, :2])
    y = lin.matmul(wide_a.view(torch.float8_e4m3fn)[:, :K], sa[:, :2], out=out[:M, :N])
    _check_product(y, a, b)
    assert (out[M] == -7.0).all() and (out[:, N:] == -7.0).all()


@pytest.mark.parametrize("M", [1, 5, 200])
def test_gemm_is_repeatable_and_row_independent(M):
    a, b = _operands(M, 700, 1000, 11)
    lin = fp8.Fp8Linear(*b)
    y = lin.matmul(*a, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(y, lin.matmul(*a, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [4, 160])
def test_gemm_non_finite_rows_stay_in_their_rows(M):
    N, K = 200, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, K, generator=g, device="cuda")
    x[1, 5] = float("nan")
    x[2, 290] = float("inf")
    lin = fp8.Fp8Linear.from_weight(torch.randn(N, K, generator=g, device="cuda"))
    y = lin.forward(x, out_dtype=torch.float32)
    assert torch.isnan(y[1:3]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[3:]).all()


def test_gemm_no_rows_and_forward_types():
    lin = fp8.Fp8Linear.from_weight(torch.randn(48, 96, device="cuda"))
    assert lin.forward(torch.zeros(0, 96, device="cuda")).shape == (0, 48)
    x = torch.randn(6, 96, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    assert torch.equal(lin.forward(x), lin.forward(x.float()))


def test_gemm_on_two_streams_at_once_and_in_two_graphs():
    a, b = _operands(4, 4096, 2048, 21)
    a2, _ = _operands(4, 4096, 2048, 22)
    lin = fp8.Fp8Linear(*b)
    want, want2 = lin.matmul(*a), lin.matmul(*a2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got, got2 = [], []
    for _ in range(20):
        got.append(lin.matmul(*a, stream=s1))
        got2.append(lin.matmul(*a2, stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(want, y) for y in got) and all(torch.equal(want2, y) for y in got2)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        y1 = lin.matmul(*a)
    with torch.cuda.graph(g2):
        y2 = lin.matmul(*a2)
    for _ in range(10):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(y1, want) and torch.equal(y2, want2)


# ------------------------------------------------------- expert FFN ---

class Ffn:
    """An FFN call over given groups: rows[e] pairs for expert e, of T tokens with k pairs each."""

    def __init__(self, rows, H, I, k=1, out=torch.float32, seed=0, slots=None, tail=0, x_scale=1.0):
        g = np.random.default_rng(seed)
        self.E, self.H, self.I, self.k = len(rows), H, I, k
        P = sum(rows) + tail
        assert P % k == 0
        self.T = P // k
        self.off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.perm = g.permutation(P).astype(np.int32)
        S = slots or self.E + 1
        self.table = g.permutation(S)[:self.E].astype(np.int32)
        self.pool = ExpertPool(H, I, S, fmt=_lib.FT_SCALE_FP8)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for e in range(self.E):
            for mat in range(3):
                w = torch.randn(*self.pool.shape(mat), generator=gen, device="cuda") * 0.02
                self.pool.pack_into(int(self.table[e]), mat, w)
        self.x = (torch.randn(self.T, H, generator=gen, device="cuda") * x_scale).bfloat16()
        self.layer = MoELayer(self.T, self.E, k, H, I, out_dtype=out)

    def run(self):
        L = self.layer
        L.perm_src.copy_(torch.from_numpy(self.perm))
        L.offsets.copy_(torch.from_numpy(self.off))
        L.out_perm.fill_(-5.0)
        L.fp8_ws.fill_(0xFF)
        L.ffn(self.x, torch.from_numpy(self.table).cuda(), self.pool)
        return L.out_perm

    def check(self, out, skip=()):
        x = _f64(self.x)
        step = BF16_STEP if out.dtype == torch.bfloat16 else F32_STEP
        got = _f64(out)
        for e in range(self.E):
            r0, r1 = self.off[e], self.off[e + 1]
            if r0 == r1:
                continue
            if e in skip:
                assert (got[r0:r1] == -5.0).all()
                continue
            mats = [self.pool.tensor_bytes(int(self.table[e]), m)[:2] for m in range(3)]
            ref, bound = F.ffn_rows(x[self.perm[r0:r1] // self.k], *mats)
            err = np.abs(got[r0:r1] - ref)
            tol = bound + step * (np.abs(ref) + bound)
            assert np.all(err <= tol), (e, float((err / tol).max()))
            # most elements are far inside: codes near a tie are few
            assert np.linalg.norm(err) <= (3e-3 + step) * np.linalg.norm(ref)
        assert (got[self.off[-1]:] == -5.0).all()


FFN_SHAPES = [
    ([1], 256, 256, 1), ([0, 1, 0], 256, 512, 1), ([2, 0, 5, 1], 320, 448, 2), ([16, 17, 1, 30], 256, 512, 2),
    ([64, 65, 3], 512, 320, 3), ([128], 256, 256, 1), ([129, 0, 127], 320, 256, 2), ([300, 1, 210], 256, 576, 1),
    ([700, 0], 512, 256, 2), ([257, 255, 100, 513], 320, 448, 3), ([140, 90, 130], 256, 512, 1), ([1, 1, 1, 1, 1, 1, 1, 1], 2048, 768, 8), ([3, 2], 2880, 2880, 1), ([90, 160], 576, 2880, 2)]


def test_results_on_a_given_stream_are_not_memory_the_current_one_still_writes():
    M, N, K = 512, 1024, 4096
    x = torch.randn(M, K, device="cuda")
    lin = fp8.Fp8Linear.from_weight(torch.randn(N, K, device="cuda"))
    codes, scales = fp8.quantize_rows(x)
    want = lin.matmul(codes, scales)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def after_a_late_fill(call, *shapes):
        held = [torch.empty(s, dtype=t, device="cuda") for s, t in shapes]
        torch.cuda._sleep(20_000_000)      # some 10 ms, then the current stream writes what it has given back
        for h in held:
            h.view(torch.uint8).fill_(0x2A)
        del held, h
        got = call()
        torch.cuda.synchronize()
        return got

    got = after_a_late_fill(lambda: fp8.quantize_rows(x, stream=side), ((M, K), fp8.FP8), ((M, K // 128), torch.float32))
    assert np.array_equal(_u8(got[0]), _u8(codes)) and torch.equal(got[1], scales)
    got = after_a_late_fill(lambda: lin.matmul(codes, scales, stream=side), ((M, N), torch.bfloat16))
    assert torch.equal(got, want)
    got = after_a_late_fill(lambda: lin.forward(x, stream=side), ((M, K), fp8.FP8), ((M, N), torch.bfloat16))
    assert torch.equal(got, want)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,H,I,k", FFN_SHAPES)
def test_ffn(rows, H, I, k, out):
    f = Ffn(rows, H, I, k, out=DTYPES[out], seed=sum(rows) + H)
    f.check(f.run())


def test_ffn_large_rows_and_rows_of_zeros():
    f = Ffn([20, 140], 256, 512, 1, seed=9)
    f.x[:5] = 0
    f.x[5:9] *= 300.0
    f.x[9:12] *= 2.0 ** -30
    f.check(f.run())


@pytest.mark.parametrize("rows", [[3, 4, 2], [200, 130, 190]])
def test_ffn_rows_behind_the_groups_are_left(rows):
    f = Ffn(rows, 256, 512, 1, seed=4, tail=7)
    f.check(f.run())


@pytest.mark.parametrize("rows", [[3, 4, 2], [200, 130, 190]])
def test_ffn_missing_and_bad_slots(rows):
    f = Ffn(rows, 256, 512, 1, seed=4)
    keep = f.table.copy()
    for bad, code in ((-1, _lib.FT_DEV_NOT_RESIDENT), (f.pool.num_slots, _lib.FT_DEV_BAD_INDEX)):
        f.table[1] = bad
        out = f.run()
        assert _status() == code
        f.table[:] = keep
        f.check(out, skip=(1,))


@pytest.mark.parametrize("rows", [[3, 4, 2], [200, 130, 190]])
def test_ffn_bad_token_reads_as_zeros(rows):
    f = Ffn(rows, 256, 512, 1, seed=4)
    good = f.perm.copy()
    f.perm[1], f.perm[2] = f.T, -1
    out = f.run()
    assert _status() == _lib.FT_DEV_BAD_INDEX
    assert (out[1:3] == 0).all()
    f.x[torch.from_numpy(good[1:3]).long().cuda()] = 0
    f.perm[:] = good
    f.check(out)


def test_ffn_bad_token_of_rows_copied_from_their_tokens():
    f = Ffn([200, 130, 190], 320, 512, 2, seed=4)      # many rows, two a token
    good = f.perm.copy()
    f.perm[1], f.perm[2] = 2 * f.T, -1
    out = f.run()
    assert _status() == _lib.FT_DEV_BAD_INDEX
    assert (out[1:3] == 0).all()
    f.perm[:] = good
    kept = torch.ones(len(good), dtype=torch.bool)
    kept[1:3] = False
    again = f.run()
    assert torch.equal(out[kept], again[kept])
    f.check(again)


@pytest.mark.parametrize("rows,H,I,k", [([1] * 8, 2048, 768, 8), ([3, 0, 2, 4], 512, 320, 3), ([140, 90, 130], 256, 512, 2)])
def test_ffn_calls_at_once_on_three_streams_and_in_graphs(rows, H, I, k):
    fs = [Ffn(rows, H, I, k, seed=30 + i) for i in range(3)]
    want = [f.run().clone() for f in fs]
    tables = [torch.from_numpy(f.table).cuda() for f in fs]
    streams = [torch.cuda.Stream() for _ in fs]
    torch.cuda.synchronize()
    for f in fs:
        f.layer.out_perm.fill_(-5.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for f, t, s in zip(fs, tables, streams):
            f.layer.ffn(f.x, t, f.pool, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(f.layer.out_perm, w) for f, w in zip(fs, want))
    graphs = []
    for f, t in zip(fs, tables):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(4):
                f.layer.ffn(f.x, t, f.pool)
        f.layer.out_perm.fill_(-5.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(f.layer.out_perm, w) for f, w in zip(fs, want))


@pytest.mark.parametrize("rows", [[5, 4], [200, 130]])
def test_ffn_non_finite_tokens_stay_in_their_rows(rows):
    f = Ffn(rows, 256, 512, 1, seed=4)
    f.x[f.perm[2], 17] = float("nan")
    f.x[f.perm[4], 100] = float("-inf")
    out = f.run()
    assert torch.isnan(out[2]).all() and torch.isnan(out[4]).all()
    rest = [i for i in range(sum(rows)) if i not in (2, 4)]
    assert torch.isfinite(out[rest]).all()


@pytest.mark.parametrize("T", [1, 9, 64, 700])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_layer_over_fp8_experts(T, out):
    """route, permute, FP8 FFN and combine as one forward(), against the oracle."""
    w = inputs.WORKLOADS["tiny"]
    li = inputs.make_layer_inputs(w, T=T)
    pool = ExpertPool(w.H, w.I, w.slots, fmt=_lib.FT_SCALE_FP8)
    s = inputs.layer_seed(w.seed, 0)
    for e in range(w.E):
        for mat in range(3):
            pool.pack_into(int(li.slot_table[e]), mat,
                           inputs.make_weight_fp32_torch(*pool.shape(mat), s, e, mat, "cuda"))
    lay = MoELayer(T, w.E, w.k, w.H, w.I, out_dtype=out, whole=True)
    x = torch.from_numpy(li.x_bits.view(np.int16)).view(torch.bfloat16).cuda()
    args = (x, torch.from_numpy(li.logits).cuda(), torch.from_numpy(li.slot_table).cuda(), pool)
    y = lay.forward(*args)
    ids, wt = M.route(li.logits, w.k)
    xv = inputs.bf16_bits_to_fp32(li.x_bits).astype(np.float64)
    ref, tol = np.zeros((T, w.H)), np.zeros((T, w.H))
    step = BF16_STEP if out == torch.bfloat16 else F32_STEP
    for e in range(w.E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        o, b = F.ffn_rows(xv[t], *[pool.tensor_bytes(int(li.slot_table[e]), m)[:2] for m in range(3)])
        ref[t] += wt[t, j][:, None] * o
        # the weights are good to 2e-6 (the router's own test), the sum to k fp32 steps
        tol[t] += wt[t, j][:, None] * (b + (step + 2e-6 + (w.k + 1) * F32_STEP) * (np.abs(o) + b))
    assert np.all(np.abs(_f64(y) - ref) <= tol)
    y = y.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.forward(*args)
    for _ in range(3):
        lay.y.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lay.y, y)


def test_combine_bf16_equals_the_fp32_combine():
    g = torch.Generator(device="cuda").manual_seed(2)
    for T, k, H in ((1, 1, 8), (5, 3, 264), (200, 10, 2048)):
        o = torch.randn(T * k, H, generator=g, device="cuda").bfloat16()
        p2r = torch.randperm(T * k, generator=g, device="cuda").int()
        w = torch.rand(T, k, generator=g, device="cuda")
        y, z = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        of = o.float()
        _lib.combine(of.data_ptr(), p2r.data_ptr(), w.data_ptr(), T, k, H, y.data_ptr(), s)
        _lib.combine_bf16(o.data_ptr(), p2r.data_ptr(), w.data_ptr(), T, k, H, z.data_ptr(), s)
        assert torch.equal(y, z)


def test_slot_manager_streams_fp8_experts():
    """FP8 slots through the expert cache: filled from host banks, read by the FFN."""
    from moe_expert_layer_renorm_b200.layer import SlotManager
    f = Ffn([3, 0, 6, 2], 256, 512, 1, seed=12)
    want = f.run().clone()
    small = ExpertPool(256, 512, 3, fmt=_lib.FT_SCALE_FP8)
    banks = [torch.from_numpy(f.pool.export_slot(int(f.table[e]))).pin_memory() for e in range(4)]
    mgr = SlotManager(3, small.layout, small.ptr)
    for e, b in enumerate(banks):
        mgr.register_host(0, e, b.data_ptr())
    table = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    comp, copy = torch.cuda.current_stream(), torch.cuda.Stream()
    mgr.acquire(0, [0, 2, 3], table.data_ptr(), 4, comp.cuda_stream, copy.cuda_stream)
    f.layer.out_perm.fill_(0)
    f.layer.ffn(f.x, table, small)
    torch.cuda.synchronize()
    assert torch.equal(f.layer.out_perm, want)
    mgr.close()
