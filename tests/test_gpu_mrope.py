"""QK-norm + RoPE with three positions per token on the GPU: bit for bit against
the one-axis oracle given each token's own mixed row of the table, and within
the derived bound of float64."""
import dataclasses

import numpy as np
import pytest
import torch

import _parity as P
import _serve8_ref as ref
import oracle
import residual_add_rmsnorm_rmsq_gb300 as rq
import rmsq_inputs as ri

pytestmark = pytest.mark.gpu
VARIANTS = ["direct", "pipelined"]
MAX_POS = 500


@pytest.fixture(scope="module", autouse=True)
def _lib(rmsq_gpu):
    return rmsq_gpu


def positions(n, seed, outside=()):
    pos = np.random.default_rng(seed).integers(0, MAX_POS, (3, n))
    for axis, token, value in outside:
        pos[axis, token] = value
    return pos


def make(name, n, nq, nkv, D, dtype="bf16", neox=True, seed=0, sigma=1.0):
    return ri.make_qk_workload(name, n, nq, nkv, D, dtype=dtype, neox=neox, max_pos=MAX_POS, seed=seed, sigma=sigma)


def want_bits(wl, pos, sections, interleaved):
    """The oracle with a table of one row per token, mixed from its three."""
    half = wl.head_dim // 2
    ax = ref.axes(half, sections, interleaved)
    live = ((pos >= 0) & (pos < len(wl.cos_sin))).all(0)
    row = np.where(live, pos, 0)[ax].T
    i = np.arange(half)
    table = np.concatenate([wl.cos_sin[row, i], wl.cos_sin[row, half + i]], 1).astype(np.float32)
    mixed = dataclasses.replace(wl, positions=np.where(live, np.arange(wl.n_tokens), -1), cos_sin=table)
    return oracle.run_qk_norm_rope(mixed)


def run(wl, pos, sections, interleaved, *, norm=True, variant="auto", out=None, stream=None):
    qkv = P.dev_act(wl.qkv, wl.dtype)
    w = [P.dev_act(x, wl.dtype) for x in (wl.q_weight, wl.k_weight)] if norm else [None, None]
    got = rq.qk_norm_mrope(qkv, torch.from_numpy(pos).cuda(), torch.from_numpy(wl.cos_sin).cuda(), *w, wl.eps, wl.nq, wl.nkv,
                           wl.head_dim, sections, wl.neox, interleaved=interleaved, out=out, stream=stream, variant=variant)
    torch.cuda.synchronize()
    assert rq.take_fault_flags() == 0
    return qkv, got


def check(wl, pos, sections, interleaved, variant="auto"):
    want = want_bits(wl, pos, sections, interleaved)
    qkv, got = run(wl, pos, sections, interleaved, variant=variant)
    assert got is qkv and np.array_equal(P.host_bits(qkv), want)
    # into a buffer of its own: the same heads, qkv as it was, rows of bad positions not written
    width = (wl.nq + wl.nkv) * wl.head_dim
    out = torch.full((wl.n_tokens, width), 7.0, dtype=P._TDT[wl.dtype], device="cuda")
    qkv, got = run(wl, pos, sections, interleaved, variant=variant, out=out)
    live = ((pos >= 0) & (pos < len(wl.cos_sin))).all(0)
    assert np.array_equal(P.host_bits(qkv), wl.qkv)
    assert np.array_equal(P.host_bits(out)[live], want[live, :width]) and (out[torch.from_numpy(~live).cuda()] == 7).all()


def splits(D):
    """Sections one after the other (multiples of four, and not), and alternating."""
    h = D // 2
    return [((h // 4, h // 2 - h // 8, h - h // 4 - h // 2 + h // 8), False), ((h - 13, 6, 7), False),
            ((h - 2 * (h // 3), h // 3, h // 3), True), ((h - 5, 0, 5), True), ((0, 0, h), False), ((h, 0, 0), True)]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("neox", [True, False], ids=["neox", "gptj"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_sections(D, neox, dtype, variant):
    wl = make(f"mrope_{D}", 61, 6, 2, D, dtype, neox, seed=D, sigma=3.0)
    for k, (sections, interleaved) in enumerate(splits(D)):
        check(wl, positions(61, k), sections, interleaved, variant)


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("sections, interleaved", [((16, 24, 24), False), ((24, 20, 20), True)])
def test_sizes_and_positions_outside(sections, interleaved, variant):
    """One token, head counts that leave a warp part empty, no q or no k heads,
    more tokens than CTAs; tokens with one of the three positions outside."""
    bad = [(0, 3, -1), (1, 17, MAX_POS), (2, 49, 1 << 40), (1, 200, -(1 << 40)), (2, 349, -1)]
    for n, nq, nkv in ((1, 8, 1), (33, 0, 3), (33, 5, 0), (211, 7, 2), (1300, 28, 4)):
        wl = make(f"mrope_n{n}", n, nq, nkv, 128, seed=n)
        check(wl, positions(n, n, [b for b in bad if b[1] < n]), sections, interleaved, variant)


def test_automatic_choice_of_a_prefill():
    wl = make("mrope_prefill", 2500, 12, 4, 128, seed=1)
    check(wl, positions(2500, 9), (24, 20, 20), True)


@pytest.mark.parametrize("variant", VARIANTS)
def test_equal_positions_are_the_one_axis_op(variant):
    wl = make("mrope_equal", 150, 8, 2, 128, seed=4)
    qkv, _ = run(wl, np.stack([wl.positions] * 3), (24, 20, 20), True, variant=variant)
    one = P.dev_act(wl.qkv, wl.dtype)
    rq.qk_norm_rope(one, torch.from_numpy(wl.positions).cuda(), torch.from_numpy(wl.cos_sin).cuda(),
                    P.dev_act(wl.q_weight, wl.dtype), P.dev_act(wl.k_weight, wl.dtype), wl.eps, 8, 2, 128, variant=variant)
    assert torch.equal(one.view(torch.int16), qkv.view(torch.int16))


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D, neox, interleaved", [(64, True, True), (128, False, False), (256, True, False)])
def test_against_float64(D, neox, interleaved, norm, dtype, variant):
    wl = make("mrope_f64", 90, 5, 3, D, dtype, neox, seed=D + 1, sigma=2.0)
    pos, sections = positions(90, 2, [(1, 7, -1)]), (D // 2 - 20, 11 if not interleaved else 10, 9 if not interleaved else 10)
    qkv, _ = run(wl, pos, sections, interleaved, norm=norm, variant=variant)
    x = P.dev_act(wl.qkv, wl.dtype).double().cpu().numpy().reshape(90, 11, D)
    w = [P.dev_act(v, wl.dtype).double().cpu().numpy() if norm else None for v in (wl.q_weight, wl.k_weight)]
    y, tol, live = ref.rotate(x[:, :8], pos, wl.cos_sin.astype(np.float64), *w, wl.eps, 5, sections, interleaved, neox)
    got = qkv.double().cpu().numpy().reshape(90, 11, D)
    eps = torch.finfo(P._TDT[dtype]).eps
    # (fp16: a step of its subnormals is 2^-24)
    bound = tol + eps / 2 * (np.abs(y) + tol) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert (np.abs(got[:, :8] - y) <= bound)[live].all()
    assert np.array_equal(got[:, 8:], x[:, 8:]) and np.array_equal(got[~live], x[~live])


def test_a_captured_call_on_another_stream():
    """Captured, replayed on new positions and heads."""
    wl = make("mrope_graph", 700, 8, 2, 128, seed=6)
    pos = positions(700, 1)
    qkv, d_pos, cs = P.dev_act(wl.qkv, wl.dtype), torch.from_numpy(pos).cuda(), torch.from_numpy(wl.cos_sin).cuda()
    w = [P.dev_act(x, wl.dtype) for x in (wl.q_weight, wl.k_weight)]
    out = torch.zeros(700, 10 * 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: rq.qk_norm_mrope(qkv, d_pos, cs, *w, wl.eps, 8, 2, 128, (24, 20, 20), interleaved=True, out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (3, 4):
        new = positions(700, seed)
        d_pos.copy_(torch.from_numpy(new))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(P.host_bits(out), want_bits(wl, new, (24, 20, 20), True)[:, : 10 * 128])
    assert rq.take_fault_flags() == 0
