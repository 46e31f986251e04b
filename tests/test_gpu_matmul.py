"""FP8 block-scaled matrix product on the GPU against float64.

Tolerance per element, with A = sum over k of |a b| times the scales: half a
step of the output's type, eps/2 |out|; the fp32 sums, counted with a full
step (2^-23, as the matrix unit may truncate) for each of the 128 products and
some 32 partial sums of a block, and for each of the k / 128 blocks: (160 +
k / 128) 2^-23 A; the product of the two scales, 2^-23 A."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def codes(rng, rows, k):
    """Finite E4M3 codes over the whole range."""
    c = rng.integers(0, 256, (rows, k), dtype=np.uint8)
    return np.where((c & 127) == 127, 0x30, c).astype(np.uint8)


def values(c):
    return torch.from_numpy(c).view(torch.float8_e4m3fn).double()


def make(m, n, k, mode, seed=0):
    rng = np.random.default_rng(seed)
    a, b = codes(rng, m, k), codes(rng, n, k)
    # the products span 2^-18 .. 2^17; keep the sums inside fp16
    sa, sb = np.exp2(rng.uniform(-9, -5, (m, k // 128))), np.exp2(rng.uniform(-9, -6, (-(-n // 128), k // 128)))
    sa, sb = sa.astype(np.float32), sb.astype(np.float32)
    if "ue8m0" in mode or "e8m0" in mode:
        sa = np.exp2(np.floor(np.log2(sa))).astype(np.float32)
    given = sa
    if "ue8m0" in mode:
        given = ((sa.view(np.uint32) >> 23) & 255).astype(np.uint8)
    if "_col" in mode:
        per16 = 16 // given.itemsize
        cols = -(-m // per16) * per16 if "tma" in mode else m
        # what lies in the padding must not matter
        t = np.full((k // 128, cols), np.nan if given.dtype == np.float32 else 255, given.dtype)
        t[:, :m] = given.T
        given = t
    return a, sa, np.ascontiguousarray(given), b, sb


def reference(a, sa, b, sb):
    n = b.shape[0]
    x = values(a) * torch.from_numpy(sa).double().repeat_interleave(128, 1)
    w = values(b) * torch.from_numpy(sb).double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    return x @ w.t(), x.abs() @ w.abs().t()


def check(rq, m, n, k, mode, dtype, seed=0):
    a, sa, given, b, sb = make(m, n, k, mode, seed)
    buf = torch.full((m * n + 512,), 7.0, dtype=DT[dtype], device="cuda")
    out = buf[: m * n].view(m, n)
    dev = [torch.from_numpy(t).cuda() for t in (a, given, b, sb)]
    got = rq.fp8_block_matmul(dev[0], dev[1], mode, dev[2], dev[3], DT[dtype], out=out)
    torch.cuda.synchronize()
    assert rq.take_fault_flags() == 0
    assert got is out and (buf[m * n:] == 7).all()
    want, A = reference(a, sa, b, sb)
    tol = torch.finfo(DT[dtype]).eps / 2 * want.abs() + A * 2.0 ** -23 * (161 + k // 128)
    err = (out.double().cpu() - want).abs()
    assert (err <= tol).all(), f"{(err > tol).sum().item()} of {m * n} beyond; largest {(err / tol).max().item():.2f} of the bound"
    return dev, out


MODES = ["fp8_group128_row", "fp8_group128_col", "fp8_group128_col+tma", "fp8_group128_row+ue8m0",
         "fp8_group128_col+ue8m0+tma", "fp8_group128_row+e8m0"]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("m, n, k", [(1, 8, 128), (3, 136, 256), (130, 264, 384)])
def test_scale_layouts(rmsq_gpu, m, n, k, mode):
    check(rmsq_gpu, m, n, k, mode, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [1, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("n, k", [(128, 128), (1000, 640), (120, 2048)])
def test_few_rows(rmsq_gpu, m, n, k, dtype):
    check(rmsq_gpu, m, n, k, "fp8_group128_row", dtype, seed=m)


@pytest.mark.parametrize("m, n, k", [(100, 520, 7168), (128, 136, 4096), (200, 264, 7168), (65, 72, 7168)])
def test_some_rows_long_k(rmsq_gpu, m, n, k):
    """Few tiles and a long K, which a cluster divides: 128 tokens per CTA, one
    and two token tiles."""
    check(rmsq_gpu, m, n, k, "fp8_group128_col", "bf16", seed=m)


@pytest.mark.parametrize("m, n, k", [
    (520, 2680, 256),      # 128-column tiles, ragged both ways
    (1100, 4360, 384),     # 256-column tiles, more than one per CTA
    (2049, 2568, 128),     # one block of K, one row in the last tile
    (129, 20000, 128),     # two row tiles
    (300, 8, 256),         # fewer columns than a tile has
])
@pytest.mark.parametrize("mode", ["fp8_group128_col+tma", "fp8_group128_row+ue8m0"])
def test_many_rows(rmsq_gpu, m, n, k, mode):
    check(rmsq_gpu, m, n, k, mode, "bf16", seed=k)


@pytest.mark.parametrize("m, n", [(1, 64), (100, 136), (128, 2440)])
def test_longest_k(rmsq_gpu, m, n):
    check(rmsq_gpu, m, n, 32768, "fp8_group128_row", "bf16")


def test_zero_rows_and_nan_codes(rmsq_gpu):
    rq = rmsq_gpu
    dev, out = check(rq, 40, 256, 256, "fp8_group128_row", "bf16")
    assert rq.fp8_block_matmul(dev[0][:0], dev[1][:0], "fp8_group128_row", dev[2], dev[3]).shape == (0, 256)
    a = dev[0].clone()
    a[7, 200] = 0x7f
    got = rq.fp8_block_matmul(a, dev[1], "fp8_group128_row", dev[2], dev[3])
    assert torch.isnan(got[7]).all()
    keep = torch.arange(40, device="cuda") != 7
    assert torch.equal(got[keep], out[keep])


@pytest.mark.parametrize("m", [3, 300])
def test_extreme_scales(rmsq_gpu, m):
    """Zero and smallest scales, exact powers of two: a row's result is its
    integer sum times them."""
    rq = rmsq_gpu
    a = torch.full((m, 256), 0x38, dtype=torch.uint8, device="cuda")          # 1.0
    b = torch.full((136, 256), 0x38, dtype=torch.uint8, device="cuda")
    sb = torch.full((2, 2), 2.0 ** 40, device="cuda")
    sa = torch.full((m, 2), 127 - 40, dtype=torch.uint8, device="cuda")      # 2^-40
    sa[0], sa[1, 0] = 0, 0                                                   # 2^-127: lost beside the other block
    got = rq.fp8_block_matmul(a, sa, "fp8_group128_row+ue8m0", b, sb).float()
    assert (got[2:] == 256).all() and (got[1] == 128).all()
    assert (got[0] == 256 * 2.0 ** (40 - 127)).all()
    got = rq.fp8_block_matmul(a, torch.zeros(m, 2, device="cuda"), "fp8_group128_row", b, sb)
    assert (got == 0).all()


def test_fp16_overflows_to_infinity(rmsq_gpu):
    a = torch.full((2, 128), 0x7e, dtype=torch.uint8, device="cuda")
    one = torch.ones(2, 1, device="cuda")
    got = rmsq_gpu.fp8_block_matmul(a, one, "fp8_group128_row", a.repeat(4, 1), one[:1], torch.float16)
    assert torch.isinf(got).all()


@pytest.mark.parametrize("m, n, k", [(8, 512, 1024), (600, 2600, 512)])
def test_repeats_streams_and_graphs_agree(rmsq_gpu, m, n, k):
    """The same bits again, from several streams at once and from a replayed
    graph whose inputs have changed."""
    rq = rmsq_gpu
    dev, out = check(rq, m, n, k, "fp8_group128_row", "bf16")
    first = out.clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(first) for _ in range(12)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        rq.fp8_block_matmul(dev[0], dev[1], "fp8_group128_row", dev[2], dev[3], out=o, stream=streams[i % 3])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    g = torch.cuda.CUDAGraph()
    res = torch.empty_like(first)
    with torch.cuda.graph(g):
        for _ in range(2):
            rq.fp8_block_matmul(dev[0], dev[1], "fp8_group128_row", dev[2], dev[3], out=res)
    dev[1].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, first * 2) and rq.take_fault_flags() == 0


def test_float8_tensors_and_outputs_of_the_fused_ops(rmsq_gpu):
    """An MLP as a user writes it: norm + quant, up projection, SiLU+Mul +
    quant, down projection, against float64 products of the quantised values."""
    rq = rmsq_gpu
    torch.manual_seed(1)
    n, H, d = 37, 512, 640
    x, r = torch.randn(n, H, device="cuda").bfloat16(), torch.randn(n, H, device="cuda").bfloat16()
    w = torch.ones(H, device="cuda").bfloat16()

    def weight(rows, cols):
        c = torch.from_numpy(codes(np.random.default_rng(rows), rows, cols)).cuda()
        return c.view(torch.float8_e4m3fn), torch.rand(-(-rows // 128), cols // 128, device="cuda") * 0.002

    def want(q, s, wt):
        a = q.cpu().view(torch.float8_e4m3fn).double() * s.cpu().double().repeat_interleave(128, 1)
        b = wt[0].cpu().double() * wt[1].cpu().double().repeat_interleave(128, 0)[: len(wt[0])].repeat_interleave(128, 1)
        return a @ b.t(), a.abs() @ b.abs().t()

    up, down = weight(2 * d, H), weight(H, d)
    q, s, _ = rq.fused_add_rmsnorm_quant(x, r, w, 1e-6, "fp8_group128_col+tma")
    h = rq.fp8_block_matmul(q, s, "fp8_group128_col+tma", *up)
    y, A = want(q, s[:, :n].t(), up)
    assert ((h.double().cpu() - y).abs() <= y.abs() * 2.0 ** -8 + A * 2.0 ** -23 * 200).all()
    q2, s2 = rq.silu_mul_quant(h, "fp8_group128_row")
    o = rq.fp8_block_matmul(q2, s2, "fp8_group128_row", *down)
    y, A = want(q2, s2, down)
    assert ((o.double().cpu() - y).abs() <= y.abs() * 2.0 ** -8 + A * 2.0 ** -23 * 200).all()


@pytest.mark.parametrize("mode, dtype", [("fp8_group128_col+tma", "bf16"), ("fp8_group128_row+ue8m0", "fp16")])
@pytest.mark.parametrize("m, n", [(257, 9800), (600, 6912)])
def test_full_rounds_and_the_columns_left_over(rmsq_gpu, m, n, mode, dtype):
    """A little more than a round of wide tiles with a long K: the columns
    behind the full round go to narrow tiles of a second launch."""
    check(rmsq_gpu, m, n, 5120, mode, dtype, seed=m)


def test_both_launches_in_a_graph_follow_their_inputs(rmsq_gpu):
    rq = rmsq_gpu
    a, _, given, b, sb = make(257, 9800, 5120, "fp8_group128_row")
    x, s, w, t = [torch.from_numpy(v).cuda() for v in (a, given, b, sb)]
    out = torch.empty(257, 9800, dtype=torch.bfloat16, device="cuda")
    rq.fp8_block_matmul(x, s, "fp8_group128_row", w, t, out=out)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rq.fp8_block_matmul(x, s, "fp8_group128_row", w, t, out=out)
        y = out.flip(0).contiguous()
        x.copy_(x.flip(0))
        s.copy_(s.flip(0))
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(y, want.flip(0))
        want = want.flip(0)
    assert rq.take_fault_flags() == 0
