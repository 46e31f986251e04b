"""Refusals of the serving operators (no GPU needed, no kernel runs): every
bad argument is an error before anything is launched."""
import ctypes

import pytest
import torch

import residual_add_rmsnorm_rmsq_gb300 as rq

A = [0x10000000 * k for k in range(1, 16)]   # far-apart fake addresses
I32, F32 = torch.int32, torch.float32


@pytest.fixture(scope="module")
def L():
    from residual_add_rmsnorm_rmsq_gb300 import _build
    _build.build()
    return rq.load()


def vp(x):
    return ctypes.c_void_p(x) if x else None


def slots(L, ctx=A[0], ql=A[1], table=A[2], width=8, free=A[3], cap=100, nf=A[4], page=16, R=4, T=64, sm=A[5], pos=A[6],
          start=A[7], seq=A[8], out=A[9], st=A[10]):
    return L.rmsq_build_slot_map(vp(ctx), vp(ql), vp(table), width, vp(free), cap, vp(nf), page, R, T, vp(sm), vp(pos),
                                 vp(start), vp(seq), vp(out), vp(st), None)


NO_GPU = (rq.ERR_NO_DEVICE, rq.ERR_UNSUPPORTED_DEVICE)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")
def test_valid_calls_reach_the_device_check(L):
    assert slots(L) in NO_GPU
    assert slots(L, R=0, ctx=0, ql=0, seq=0, table=0) in NO_GPU
    assert store(L) in NO_GPU and load(L) in NO_GPU and attn(L) in NO_GPU
    # k and v as columns of one buffer
    assert store(L, k=A[0], v=A[0] + 1024, ks=2048, vs=2048) in NO_GPU
    assert load(L, k=A[0], v=A[0] + 1024, ks=1024, vs=1024) in NO_GPU
    assert attn(L, lse=0) in NO_GPU
    assert matmul(L) in NO_GPU and matmul(L, mode=3 | 0x40 | 0x20, sa=A[1] + 1) in NO_GPU


def test_slot_map_refusals(L):
    for kw in ("ctx", "ql", "table", "free", "nf", "sm", "pos", "start", "seq", "out", "st"):
        assert slots(L, **{kw: 0}) == rq.ERR_INVALID_ARG, kw
        assert slots(L, **{kw: A[12] + 2}) == rq.ERR_ALIGNMENT, kw
    assert slots(L, sm=A[12] + 4) == rq.ERR_ALIGNMENT
    for kw in ({"R": -1}, {"T": -1}, {"width": -1}, {"cap": -1}):
        assert slots(L, **kw) == rq.ERR_INVALID_ARG, kw
    for kw in ({"page": 0}, {"page": 8}, {"page": 24}, {"page": 512}, {"R": rq.MAX_REQUESTS + 1}, {"T": 1 << 30},
               {"cap": 1 << 31}, {"width": 1 << 28}):
        assert slots(L, **kw) == rq.ERR_UNSUPPORTED_SHAPE, kw
    assert slots(L, seq=A[0]) == rq.ERR_ALIAS             # seq_lens over context_lens
    assert slots(L, out=A[4]) == rq.ERR_ALIAS             # num_free in place
    assert slots(L, sm=A[5], pos=A[5] + 64) == rq.ERR_ALIAS
    assert slots(L, table=A[3]) == rq.ERR_ALIAS


def store(L, k=A[0], ks=256, v=A[1], vs=256, sm=A[2], kg=A[3], vg=A[4], cache=A[5], pages=10, page=16, n=4, h=2, d=128,
          dt=0):
    return L.rmsq_kv_cache_store_nvfp4(vp(k), ks, vp(v), vs, vp(sm), vp(kg), vp(vg), vp(cache), pages, page, n, h, d, dt,
                                       None)


def load(L, k=A[0], ks=256, v=A[1], vs=256, sm=A[2], kg=A[3], vg=A[4], cache=A[5], pages=10, page=16, n=4, h=2, d=128,
         dt=0):
    return L.rmsq_kv_cache_load_nvfp4(vp(cache), pages, page, vp(sm), vp(kg), vp(vg), vp(k), ks, vp(v), vs, n, h, d, dt,
                                      None)


@pytest.mark.parametrize("call", [store, load])
def test_cache_refusals(L, call):
    for kw in ("k", "v", "sm", "kg", "vg", "cache"):
        assert call(L, **{kw: 0}) == rq.ERR_INVALID_ARG, kw
        assert call(L, **{kw: A[12] + 2}) == rq.ERR_ALIGNMENT, kw
    for kw in ({"n": -1}, {"h": 0}, {"pages": 0}, {"dt": 2}, {"ks": 255}, {"vs": 128}, {"ks": 1 << 32}):
        assert call(L, **kw) == rq.ERR_INVALID_ARG, kw
    for kw in ({"d": 96}, {"d": 0}, {"d": 512}, {"page": 8}, {"page": 48}, {"h": 4097}, {"n": 1 << 31}):
        assert call(L, **(kw | {"ks": 1 << 30, "vs": 1 << 30})) == rq.ERR_UNSUPPORTED_SHAPE, kw
    assert call(L, ks=260) == rq.ERR_ALIGNMENT
    assert call(L, n=0) == rq.OK
    assert call(L, cache=A[0] + 512) == rq.ERR_ALIAS
    assert call is load or call(L, cache=A[2]) == rq.ERR_ALIAS   # (two inputs of the load)


def test_load_outputs_must_not_overlap(L):
    assert load(L, v=A[0]) == rq.ERR_ALIAS
    assert load(L, v=A[0] + 256, ks=512, vs=512) == rq.ERR_ALIAS      # columns that share elements
    assert load(L, v=A[0] + 512, ks=384, vs=384) == rq.ERR_ALIAS      # ... that wrap into the next row
    assert load(L, k=A[3]) == rq.ERR_ALIAS


def attn(L, q=A[0], qs=1024, cache=A[1], pages=10, page=16, table=A[2], width=8, start=A[3], seq=A[4], kg=A[5], vg=A[6],
         scale=0.1, window=0, out=A[7], lse=A[8], ws=A[9], wsb=1 << 27, T=4, R=3, h=8, kv=2, d=128, dt=0, var=0):
    return L.rmsq_paged_attention_nvfp4(vp(q), qs, vp(cache), pages, page, vp(table), width, vp(start), vp(seq), vp(kg),
                                        vp(vg), scale, window, vp(out), vp(lse), vp(ws), wsb, T, R, h, kv, d, dt, None, var)


def test_attention_refusals(L):
    for kw in ("q", "cache", "table", "start", "seq", "kg", "vg", "out", "ws"):
        assert attn(L, **{kw: 0}) == rq.ERR_INVALID_ARG, kw
        assert attn(L, **{kw: A[12] + 2}) == rq.ERR_ALIGNMENT, kw
    assert attn(L, lse=A[12] + 2) == rq.ERR_ALIGNMENT and attn(L, qs=1028) == rq.ERR_ALIGNMENT
    nan, inf = float("nan"), float("inf")
    for kw in ({"dt": 2}, {"T": -1}, {"R": -1}, {"h": 0}, {"kv": 0}, {"scale": 0.0}, {"scale": -1.0}, {"scale": nan},
               {"scale": inf}, {"window": -1}, {"qs": 1016}, {"pages": -1}, {"width": -1}, {"wsb": 100}, {"var": 3},
               {"var": -1}):
        assert attn(L, **kw) == rq.ERR_INVALID_ARG, kw
    for kw in ({"kv": 3}, {"d": 80}, {"d": 512}, {"page": 8}, {"R": rq.MAX_REQUESTS + 1}, {"T": 1 << 28},
               {"h": 8192, "kv": 8192}, {"width": 1 << 27}):
        assert attn(L, **kw) == rq.ERR_UNSUPPORTED_SHAPE, kw
    assert attn(L, T=0) == rq.OK and attn(L, R=0) == rq.OK
    for kw in ({"out": A[0]}, {"lse": A[7] + 64}, {"ws": A[1]}, {"out": A[4]}, {"lse": A[9] + 64}):
        assert attn(L, **kw) == rq.ERR_ALIAS, kw


def test_attention_workspace_size(L):
    small = rq.paged_attention_workspace_bytes(8, 8, 8, 1, 128)
    assert small > 0 and rq.paged_attention_workspace_bytes(8, 8, 16, 1, 128) >= small
    assert rq.paged_attention_workspace_bytes(8, 8, 8, 3, 128) == 0
    assert rq.paged_attention_workspace_bytes(8, 8, 8, 1, 100) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_workspace_of_the_largest_step_serves_the_smaller(L, D):
    most = rq.paged_attention_workspace_bytes(256, 256, 8, 4, D)
    for tokens, requests in ((256, 1), (256, 4), (200, 255), (1, 1)):
        assert rq.paged_attention_workspace_bytes(tokens, requests, 8, 4, D) <= most


def matmul(L, a=A[0], sa=A[1], mode=2, b=A[2], sb=A[3], out=A[4], m=4, n=256, k=512, dt=0):
    return L.rmsq_fp8_block_matmul(vp(a), vp(sa), mode, vp(b), vp(sb), vp(out), m, n, k, dt, None)


def test_matmul_refusals(L):
    for kw in ("a", "sa", "b", "sb", "out"):
        assert matmul(L, **{kw: 0}) == rq.ERR_INVALID_ARG, kw
        assert matmul(L, **{kw: A[12] + 2}) == rq.ERR_ALIGNMENT, kw
    # every mode without a scale per 128 columns, unknown bits, options that do not apply
    for mode in (0, 1, 4, 5, 6, 7, -1, 2 | 0x80, 2 | 0x20):
        assert matmul(L, mode=mode) == rq.ERR_INVALID_ARG, mode
    for kw in ({"dt": 2}, {"m": -1}, {"n": 0}, {"k": 0}):
        assert matmul(L, **kw) == rq.ERR_INVALID_ARG, kw
    for kw in ({"n": 257}, {"n": 252}, {"k": 64}, {"k": 500}, {"k": 32768 + 128}, {"m": 1 << 31}, {"n": 1 << 31}):
        assert matmul(L, **kw) == rq.ERR_UNSUPPORTED_SHAPE, kw
    assert matmul(L, m=0) == rq.OK
    for kw in ({"out": A[0]}, {"out": A[1]}, {"out": A[2] + 256}, {"out": A[3]}):
        assert matmul(L, **kw) == rq.ERR_ALIAS, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors")
def test_matmul_binding_refusals(L):
    u8 = torch.uint8
    a, b = torch.zeros(5, 256, dtype=u8), torch.zeros(200, 256, dtype=u8)
    sa, sb = torch.zeros(5, 2), torch.zeros(2, 2)
    with pytest.raises(rq.RmsqError) as e:
        rq.fp8_block_matmul(a, sa, "fp8_group128_row", b, sb, stream=0)
    assert e.value.status == rq.ERR_NO_DEVICE
    with pytest.raises(rq.RmsqError) as e:
        rq.fp8_block_matmul(a.view(torch.float8_e4m3fn), torch.zeros(2, 16, dtype=u8), "fp8_group128_col+ue8m0+tma", b, sb,
                            torch.float16, stream=0)
    assert e.value.status == rq.ERR_NO_DEVICE
    for args in ((a, sa, "fp8_per_token", b, sb), (a, sa, "fp8_group64_row", b, sb), (a, sa, "fp8_group128_col", b, sb),
                 (a, sa, "fp8_group128_row", b[:, :128], sb), (a, sa, "fp8_group128_row", b, sb[:1]),
                 (a[:, ::2], sa, "fp8_group128_row", b[:, ::2], sb), (a, sa[:, :1], "fp8_group128_row", b, sb)):
        with pytest.raises(ValueError):
            rq.fp8_block_matmul(*args, stream=0)
    for args in ((a.float(), sa, "fp8_group128_row", b, sb), (a, sa.double(), "fp8_group128_row", b, sb),
                 (a, sa, "fp8_group128_row+ue8m0", b, sb), (a, sa, "fp8_group128_row", b, sb.half()),
                 (a, sa, "fp8_group128_row", b, sb, torch.float32)):
        with pytest.raises(TypeError):
            rq.fp8_block_matmul(*args, stream=0)


def _attn_args(**kw):
    a = {"q": torch.zeros(4, 8, 128).bfloat16(), "cache": torch.zeros(rq.kv_cache_shape(10, 2, 128, 16), dtype=torch.uint8),
         "block_table": torch.zeros(3, 8, dtype=I32), "query_start": torch.zeros(4, dtype=I32),
         "seq_lens": torch.zeros(3, dtype=I32), "k_global_scale": torch.ones(1), "v_global_scale": torch.ones(1),
         "page_size": 16, "stream": 0}
    return a | kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors")
def test_binding_refusals(L):
    with pytest.raises(rq.RmsqError) as e:
        rq.paged_attention_nvfp4(**_attn_args())
    assert e.value.status == rq.ERR_NO_DEVICE
    z = torch.zeros
    for kw in ({"q": z(4, 8, 128)}, {"block_table": z(3, 8, dtype=torch.int64)}, {"seq_lens": z(3)},
               {"k_global_scale": torch.ones(1).double()}, {"cache": z(10, 2, 2, 1152)},
               {"lse": z(4, 8, dtype=torch.float64)}, {"out": z(4, 8, 128)}):
        with pytest.raises(TypeError):
            rq.paged_attention_nvfp4(**_attn_args(**kw))
    u8 = torch.uint8
    for kw in ({"q": z(4, 8, 256).bfloat16()[..., ::2]}, {"q": z(4, 128).bfloat16()}, {"page_size": 32},
               {"cache": z(10, 2, 2, 1151, dtype=u8)}, {"cache": z(10, 2, 2, 2304, dtype=u8)[..., ::2]},
               {"query_start": z(3, dtype=I32)}, {"seq_lens": z(4, dtype=I32)}, {"block_table": z(3, dtype=I32)},
               {"k_global_scale": torch.ones(2)}, {"out": z(5, 8, 128).bfloat16()}, {"lse": z(4, 9)}, {"variant": "fast"}):
        with pytest.raises(ValueError):
            rq.paged_attention_nvfp4(**_attn_args(**kw))
    k = z(4, 2, 128).bfloat16()
    sm, one, cache = torch.arange(4), torch.ones(1), z(rq.kv_cache_shape(10, 2, 128, 16), dtype=u8)
    for bad in ((k, k[:3], sm, one, one, cache, 16), (k, k, sm[:3], one, one, cache, 16), (k, k, sm, one, one, cache, 32),
                (k.transpose(0, 1), k.transpose(0, 1), sm[:2], one, one, cache, 16)):
        with pytest.raises(ValueError):
            rq.kv_cache_store_nvfp4(*bad, stream=0)
    with pytest.raises(TypeError):
        rq.kv_cache_store_nvfp4(k, k.half(), sm, one, one, cache, 16, stream=0)
    with pytest.raises(TypeError):
        rq.kv_cache_load_nvfp4(cache, sm, one, one, 128, 16, torch.float32, stream=0)
    with pytest.raises(ValueError):
        rq.kv_cache_load_nvfp4(cache, sm, one, one, 64, 16, stream=0)
    i = lambda *s: z(*s, dtype=I32)  # noqa: E731
    with pytest.raises(ValueError):
        rq.build_slot_map(i(3), i(2), i(3, 4), i(9), i(1), 16, 8, stream=0)
    with pytest.raises(ValueError):
        rq.build_slot_map(i(3), i(3), i(3, 4), i(9), i(1), 16, -1, stream=0)
    with pytest.raises(TypeError):
        rq.build_slot_map(i(3), i(3).long(), i(3, 4), i(9), i(1), 16, 8, stream=0)
    with pytest.raises(TypeError):
        rq.build_slot_map(i(3), i(3), i(3, 4), i(9), i(1), 16, 8, slot_map=i(8), stream=0)
    with pytest.raises(rq.RmsqError) as e:
        rq.build_slot_map(i(3), i(3), i(3, 4), i(9), i(1), 24, 8, stream=0)
    assert e.value.status == rq.ERR_UNSUPPORTED_SHAPE


class _FakeStream:
    device = None

    def __init__(self, handle):
        self.cuda_stream = handle


def _binding_calls():
    """Every binding that allocates, with none of its outputs given."""
    z, u8 = torch.zeros, torch.uint8
    i = lambda *s: z(*s, dtype=I32)  # noqa: E731
    x, w, gs = z(4, 128).bfloat16(), z(128).bfloat16(), torch.ones(1)
    cache = z(rq.kv_cache_shape(10, 2, 128, 16), dtype=u8)
    args = _attn_args()
    args.pop("stream")
    return {
        "fused_add_rmsnorm_quant": lambda s: rq.fused_add_rmsnorm_quant(x, x, w, 1e-6, "fp8_per_token", stream=s),
        "allreduce_add_rmsnorm_quant": lambda s: rq.allreduce_add_rmsnorm_quant([x, x], x, w, 1e-6, "fp8_per_token", stream=s),
        "fused_add_rmsnorm": lambda s: rq.fused_add_rmsnorm(x, x, w, 1e-6, stream=s),
        "quant": lambda s: rq.quant(x, "fp8_per_token", stream=s),
        "silu_mul_quant": lambda s: rq.silu_mul_quant(x, "fp8_group64_row", stream=s),
        "fused_add_rmsnorm_nvfp4_dynamic": lambda s: rq.fused_add_rmsnorm_nvfp4_dynamic(x, x, w, 1e-6, stream=s),
        "build_slot_map": lambda s: rq.build_slot_map(i(3), i(3), i(3, 4), i(9), i(1), 16, 8, stream=s),
        "kv_cache_load_nvfp4": lambda s: rq.kv_cache_load_nvfp4(cache, torch.arange(4), gs, gs, 128, 16, stream=s),
        "paged_attention_nvfp4": lambda s: rq.paged_attention_nvfp4(**args, return_lse=True, stream=s),
        "fp8_block_matmul": lambda s: rq.fp8_block_matmul(z(5, 256, dtype=u8), z(5, 2), "fp8_group128_row",
                                                          z(200, 256, dtype=u8), z(2, 2), stream=s),
        "debug_activation": lambda s: rq.debug_activation("silu_mul", z(4), z(4), s),
        "debug_convert": lambda s: rq.debug_convert("e4m3", z(4), s),
    }


@pytest.mark.skipif(torch.cuda.is_available(), reason="a fake of the streams")
@pytest.mark.parametrize("name", sorted(_binding_calls()))
def test_what_a_call_allocates_comes_from_the_launching_stream(monkeypatch, name):
    """With a stream that is not the current one, every output and workspace a
    binding allocates is taken while that stream is current; with the current
    one, nothing is switched."""
    import contextlib
    call = _binding_calls()[name]
    here, side = _FakeStream(0x100), _FakeStream(0x200)
    current, taken = [here], []

    @contextlib.contextmanager
    def switched(s):
        current.append(s)
        yield
        current.pop()

    class Lib:
        def __getattr__(self, fn):
            return lambda *a: 64 if fn.endswith("workspace_bytes") else taken.append((fn, a)) or 0

    monkeypatch.setattr(rq, "_lib", Lib())
    monkeypatch.setattr(rq, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", switched)
    for make in ("empty", "empty_like"):
        plain = getattr(torch, make)
        monkeypatch.setattr(torch, make, lambda *a, f=plain, **k: taken.append(("empty", current[-1])) or f(*a, **k))
    for given, owner in ((side, side), (here, here), (None, here)):
        taken.clear()
        call(given)
        made = [s for what, s in taken if what == "empty"]
        assert made and all(s is owner for s in made), name
        assert taken[-1][0].startswith("rmsq_") and current == [here]


def _function(source, name):
    at = source.index(f" {name}(")
    return source[at: source.index("\n}", at)]


def test_barriers_that_want_a_whole_warp_gather_it():
    """bar.sync and barrier.cluster...aligned are undefined for a warp that
    arrives in pieces, and their callers come from loops whose lanes leave at
    different turns (b's last block of columns, a few scales)."""
    import os
    csrc = os.path.join(os.path.dirname(rq.__file__), "csrc")
    tc = open(os.path.join(csrc, "rmsq_tc.cuh")).read()
    for name, barrier in (("named_sync", "bar.sync"), ("cluster_sync", "barrier.cluster.arrive")):
        body = _function(tc, name)
        assert body.index("__syncwarp();") < body.index(barrier), name
    sources = {f: open(os.path.join(csrc, f)).read() for f in os.listdir(csrc) if f.endswith((".cu", ".cuh"))}
    assert [f for f, s in sources.items() if "barrier.cluster" in s] == ["rmsq_tc.cuh"]
    assert sum(s.count('"bar.sync') for s in sources.values()) == 1


@pytest.mark.parametrize("T, h", [(1 << 60, 16), (1 << 61, 8), ((1 << 63) - 1, 2), (1 << 58, 64)])
def test_attention_sizes_whose_product_wraps_are_refused(L, T, h):
    assert attn(L, T=T, h=h, kv=1, qs=1 << 16) == rq.ERR_UNSUPPORTED_SHAPE
    assert rq.paged_attention_workspace_bytes(T, 3, h, 1, 128) == 0


def test_attention_with_a_bound_on_the_queries(L):
    def call(T=4, R=3, max_query=0, out=A[7]):
        return L.rmsq_paged_attention_nvfp4_ex(vp(A[0]), 1024, vp(A[1]), 10, 16, vp(A[2]), 8, vp(A[3]), vp(A[4]), vp(A[5]),
                                               vp(A[6]), 0.1, 0, vp(out), vp(A[8]), vp(A[9]), 1 << 27, T, R, 8, 2, 128, 0,
                                               None, 0, max_query)
    assert call(max_query=-1) == rq.ERR_INVALID_ARG
    assert call(out=A[0], max_query=3) == rq.ERR_ALIAS
    assert call(T=0, max_query=1) == rq.OK
    if not torch.cuda.is_available():       # fake addresses
        for q in (0, 1, 4, 1 << 40):
            assert call(max_query=q) in NO_GPU
        with pytest.raises(rq.RmsqError) as e:
            rq.paged_attention_nvfp4(**_attn_args(max_query=-3))
        assert e.value.status == rq.ERR_INVALID_ARG
