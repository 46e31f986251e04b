"""Refusals of the operators around the FP8 cache (no GPU needed, no kernel
runs): every bad argument is an error before anything is launched."""
import contextlib
import ctypes

import pytest
import torch

import residual_add_rmsnorm_rmsq_gb300 as rq

A = [0x10000000 * k for k in range(1, 16)]   # far-apart fake addresses
I32 = torch.int32
NO_GPU = (rq.ERR_NO_DEVICE, rq.ERR_UNSUPPORTED_DEVICE)


@pytest.fixture(scope="module")
def L():
    from residual_add_rmsnorm_rmsq_gb300 import _build
    _build.build()
    return rq.load()


def vp(x):
    return ctypes.c_void_p(x) if x else None


def mrope(L, qkv=A[0], out=A[1], pos=A[2], cs=A[3], max_pos=100, qw=A[4], kw=A[5], eps=1e-6, n=4, nq=8, nkv=2, d=128, t=24,
          h=20, w=20, il=1, neox=1, dt=0, var=0):
    return L.rmsq_qk_norm_mrope(vp(qkv), vp(out), vp(pos), vp(cs), max_pos, vp(qw), vp(kw), eps, n, nq, nkv, d, t, h, w, il, neox,
                                dt, None, var)


def store(L, k=A[0], ks=256, v=A[1], vs=256, sm=A[2], cache=A[3], scales=A[4], pages=10, page=16, n=4, h=2, d=128, dt=0):
    return L.rmsq_kv_cache_store_fp8(vp(k), ks, vp(v), vs, vp(sm), vp(cache), vp(scales), pages, page, n, h, d, dt, None)


def load(L, k=A[0], ks=256, v=A[1], vs=256, sm=A[2], cache=A[3], scales=A[4], pages=10, page=16, n=4, h=2, d=128, dt=0):
    return L.rmsq_kv_cache_load_fp8(vp(cache), vp(scales), pages, page, vp(sm), vp(k), ks, vp(v), vs, n, h, d, dt, None)


def attn(L, q=A[0], qs=1024, cache=A[1], scales=A[5], pages=10, page=16, table=A[2], width=8, start=A[3], seq=A[4], scale=0.1,
         window=0, out=A[7], lse=A[8], ws=A[9], wsb=1 << 27, T=4, R=3, h=8, kv=2, d=128, dt=0, var=0, most=0):
    return L.rmsq_paged_attention_fp8(vp(q), qs, vp(cache), vp(scales), pages, page, vp(table), width, vp(start), vp(seq), scale,
                                      window, vp(out), vp(lse), vp(ws), wsb, T, R, h, kv, d, dt, None, var, most)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")
def test_valid_calls_reach_the_device_check(L):
    assert mrope(L) in NO_GPU and mrope(L, out=0) in NO_GPU and mrope(L, qw=0, kw=0) in NO_GPU
    # sections at their ends: all of one axis, the last alternating angle, none
    for d, t, h, w, il in ((128, 64, 0, 0, 0), (128, 0, 0, 64, 0), (128, 1, 62, 1, 0), (64, 11, 11, 10, 1), (64, 12, 10, 10, 1),
                           (256, 44, 42, 42, 1), (128, 64, 0, 0, 1)):
        assert mrope(L, d=d, t=t, h=h, w=w, il=il) in NO_GPU, (d, t, h, w, il)
    assert store(L) in NO_GPU and load(L) in NO_GPU and attn(L) in NO_GPU
    assert store(L, scales=A[4] + 3) in NO_GPU and attn(L, scales=A[5] + 1, lse=0, most=3) in NO_GPU
    # k and v as columns of one buffer
    assert store(L, k=A[0], v=A[0] + 1024, ks=2048, vs=2048) in NO_GPU
    assert load(L, k=A[0], v=A[0] + 512, ks=1024, vs=1024) in NO_GPU


def test_mrope_refusals(L):
    for kw in ("qkv", "pos", "cs"):
        assert mrope(L, **{kw: 0}) == rq.ERR_INVALID_ARG, kw
    for kw in ("qkv", "out", "pos", "cs", "qw", "kw"):
        assert mrope(L, **{kw: A[12] + 4}) == rq.ERR_ALIGNMENT, kw
    nan, inf = float("nan"), float("inf")
    for kw in ({"dt": 2}, {"var": 3}, {"n": -1}, {"nq": -1}, {"nkv": -1}, {"nq": 0, "nkv": 0}, {"max_pos": 0}, {"neox": 2},
               {"il": 2}, {"il": -1}, {"eps": nan}, {"eps": inf}, {"eps": -1.0}, {"qw": 0}, {"kw": 0}, {"t": 25}, {"t": -1, "h": 45},
               {"h": -4, "t": 48}, {"w": -20, "h": 60, "il": 0}, {"t": 20, "h": 23, "w": 21}, {"t": 20, "h": 22, "w": 22},
               {"t": 2**31 - 1, "h": 2**31 - 1, "w": 66, "il": 0}):
        assert mrope(L, **kw) == rq.ERR_INVALID_ARG, kw
    for kw in ({"d": 96}, {"d": 512}, {"nq": 4097}, {"nkv": 4097}, {"n": 1 << 31}, {"n": (1 << 63) - 1}, {"max_pos": 1 << 60}):
        assert mrope(L, **kw) == rq.ERR_UNSUPPORTED_SHAPE, kw
    assert mrope(L, n=0, qkv=0) == rq.OK
    for kw in ({"out": A[0]}, {"out": A[0] + 64}, {"out": A[3]}, {"out": A[5]}, {"out": 0, "pos": A[0] + 128}, {"out": 0, "qw": A[0]}):
        assert mrope(L, **kw) == rq.ERR_ALIAS, kw


@pytest.mark.parametrize("call", [store, load])
def test_cache_refusals(L, call):
    for kw in ("k", "v", "sm", "cache", "scales"):
        assert call(L, **{kw: 0}) == rq.ERR_INVALID_ARG, kw
    for kw in ("k", "v", "sm", "cache"):
        assert call(L, **{kw: A[12] + 4}) == rq.ERR_ALIGNMENT, kw
    for kw in ({"n": -1}, {"h": 0}, {"pages": 0}, {"dt": 2}, {"ks": 255}, {"vs": 128}, {"ks": 1 << 32}):
        assert call(L, **kw) == rq.ERR_INVALID_ARG, kw
    for kw in ({"d": 96}, {"d": 0}, {"d": 512}, {"page": 8}, {"page": 48}, {"h": 4097}, {"n": 1 << 31}, {"pages": 1 << 31}):
        assert call(L, **(kw | {"ks": 1 << 30, "vs": 1 << 30})) == rq.ERR_UNSUPPORTED_SHAPE, kw
    assert call(L, ks=260) == rq.ERR_ALIGNMENT
    assert call(L, n=0) == rq.OK
    for kw in ({"cache": A[0] + 512}, {"scales": A[0] + 9}, {"scales": A[1]}):
        assert call(L, **kw) == rq.ERR_ALIAS, kw
    if call is store:
        assert store(L, scales=A[3] + 100) == rq.ERR_ALIAS and store(L, scales=A[2]) == rq.ERR_ALIAS
        assert store(L, cache=A[2]) == rq.ERR_ALIAS
    else:
        assert load(L, v=A[0]) == rq.ERR_ALIAS and load(L, v=A[0] + 256, ks=512, vs=512) == rq.ERR_ALIAS
        assert load(L, k=A[2]) == rq.ERR_ALIAS


def test_attention_refusals(L):
    for kw in ("q", "cache", "scales", "table", "start", "seq", "out", "ws"):
        assert attn(L, **{kw: 0}) == rq.ERR_INVALID_ARG, kw
    for kw in ("q", "cache", "table", "start", "seq", "out", "ws", "lse"):
        assert attn(L, **{kw: A[12] + 2}) == rq.ERR_ALIGNMENT, kw
    assert attn(L, qs=1028) == rq.ERR_ALIGNMENT
    nan, inf = float("nan"), float("inf")
    for kw in ({"dt": 2}, {"T": -1}, {"R": -1}, {"h": 0}, {"kv": 0}, {"scale": 0.0}, {"scale": -1.0}, {"scale": nan},
               {"scale": inf}, {"window": -1}, {"qs": 1016}, {"pages": -1}, {"width": -1}, {"wsb": 100}, {"var": 3},
               {"var": -1}, {"most": -1}):
        assert attn(L, **kw) == rq.ERR_INVALID_ARG, kw
    for kw in ({"kv": 3}, {"d": 80}, {"d": 512}, {"page": 8}, {"R": rq.MAX_REQUESTS + 1}, {"T": 1 << 28}, {"T": 1 << 61},
               {"h": 8192, "kv": 8192}, {"width": 1 << 27}):
        assert attn(L, **kw) == rq.ERR_UNSUPPORTED_SHAPE, kw
    assert attn(L, T=0) == rq.OK and attn(L, R=0) == rq.OK
    for kw in ({"out": A[0]}, {"lse": A[7] + 64}, {"ws": A[1]}, {"out": A[4]}, {"lse": A[9] + 64}, {"out": A[5]}, {"ws": A[5] - 64}):
        assert attn(L, **kw) == rq.ERR_ALIAS, kw


z, U8 = torch.zeros, torch.uint8


def _cache(pages=10, h=2, d=128, page=16):
    return tuple(z(s, dtype=U8) for s in rq.kv_cache_shapes_fp8(pages, h, d, page))


def _attn_args(**kw):
    cache, scales = _cache()
    a = {"q": z(4, 8, 128).bfloat16(), "cache": cache, "scales": scales, "block_table": z(3, 8, dtype=I32),
         "query_start": z(4, dtype=I32), "seq_lens": z(3, dtype=I32), "stream": 0}
    return a | kw


def _mrope_args(**kw):
    a = {"qkv": z(5, 12 * 128).bfloat16(), "positions": z(3, 5, dtype=torch.int64), "cos_sin_cache": z(9, 128),
         "q_weight": z(128).bfloat16(), "k_weight": z(128).bfloat16(), "eps": 1e-6, "num_q_heads": 8, "num_kv_heads": 2,
         "head_dim": 128, "sections": (24, 20, 20), "interleaved": True, "stream": 0}
    return a | kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors")
def test_binding_refusals(L):
    k, sm, (cache, scales) = z(4, 2, 128).bfloat16(), torch.arange(4), _cache()
    good = [lambda: rq.paged_attention_fp8(**_attn_args()), lambda: rq.qk_norm_mrope(**_mrope_args()),
            lambda: rq.qk_norm_mrope(**_mrope_args(q_weight=None, k_weight=None, out=z(5, 10 * 128).bfloat16())),
            lambda: rq.kv_cache_store_fp8(k, k.clone(), sm, cache.view(torch.float8_e4m3fn), scales, stream=0),
            lambda: rq.kv_cache_load_fp8(cache, scales, sm, torch.float16, stream=0)]
    for call in good:
        with pytest.raises(rq.RmsqError) as e:
            call()
        assert e.value.status == rq.ERR_NO_DEVICE
    half = torch.float16
    for kw in ({"q": z(4, 8, 128)}, {"cache": cache.float()}, {"scales": scales.float()}, {"block_table": z(3, 8).long()},
               {"seq_lens": z(3)}, {"lse": z(4, 8, dtype=torch.float64)}, {"out": z(4, 8, 128)}):
        with pytest.raises(TypeError):
            rq.paged_attention_fp8(**_attn_args(**kw))
    for kw in ({"q": z(4, 8, 64).bfloat16()}, {"q": z(4, 8, 256).bfloat16()[..., ::2]}, {"q": z(4, 128).bfloat16()},
               {"cache": cache[:, :1]}, {"cache": cache[..., ::2]}, {"cache": cache[:, 0]}, {"scales": scales[:9]},
               {"scales": z(10, 2, 2, 2, dtype=U8)}, {"query_start": z(3, dtype=I32)}, {"seq_lens": z(4, dtype=I32)},
               {"block_table": z(3, dtype=I32)}, {"out": z(5, 8, 128).bfloat16()}, {"lse": z(4, 9)}, {"variant": "fast"}):
        with pytest.raises(ValueError):
            rq.paged_attention_fp8(**_attn_args(**kw))
    for kw in ({"qkv": z(5, 12 * 128)}, {"positions": z(3, 5, dtype=I32)}, {"cos_sin_cache": z(9, 128).half()},
               {"q_weight": z(128).half()}, {"out": z(5, 10 * 128, dtype=half)}):
        with pytest.raises(TypeError):
            rq.qk_norm_mrope(**_mrope_args(**kw))
    for kw in ({"qkv": z(5, 11 * 128).bfloat16()}, {"positions": z(5, 3, dtype=torch.int64)}, {"positions": z(5, dtype=torch.int64)},
               {"cos_sin_cache": z(9, 64)}, {"k_weight": z(64).bfloat16()}, {"out": z(5, 12 * 128).bfloat16()}, {"sections": (64,)},
               {"variant": "fast"}):
        with pytest.raises(ValueError):
            rq.qk_norm_mrope(**_mrope_args(**kw))
    with pytest.raises(rq.RmsqError) as e:
        rq.qk_norm_mrope(**_mrope_args(sections=(24, 20, 21)))
    assert e.value.status == rq.ERR_INVALID_ARG
    for bad in ((k, k[:3], sm, cache, scales), (k, k, sm[:3], cache, scales), (k, k, sm, *_cache(h=3)), (k, k, sm, *_cache(d=64)),
                (k, k, sm, cache, scales[..., :0]), (k.transpose(0, 1), k.transpose(0, 1), sm[:2], cache, scales)):
        with pytest.raises(ValueError):
            rq.kv_cache_store_fp8(*bad, stream=0)
    for bad in ((k, k.half(), sm, cache, scales), (k, k, sm.int(), cache, scales), (k, k, sm, cache.int(), scales)):
        with pytest.raises(TypeError):
            rq.kv_cache_store_fp8(*bad, stream=0)
    with pytest.raises(TypeError):
        rq.kv_cache_load_fp8(cache, scales, sm, torch.float32, stream=0)
    with pytest.raises(ValueError):
        rq.kv_cache_load_fp8(cache, scales, sm, k_out=z(3, 2, 128).bfloat16(), stream=0)


class _FakeStream:
    device = None

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.skipif(torch.cuda.is_available(), reason="a fake of the streams")
@pytest.mark.parametrize("name", ["load", "attention"])
def test_what_a_call_allocates_comes_from_the_launching_stream(monkeypatch, name):
    args = _attn_args()
    args.pop("stream")
    call = {"load": lambda s: rq.kv_cache_load_fp8(args["cache"], args["scales"], torch.arange(4), stream=s),
            "attention": lambda s: rq.paged_attention_fp8(**args, return_lse=True, stream=s)}[name]
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
    plain = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: taken.append(("empty", current[-1])) or plain(*a, **k))
    for given, owner in ((side, side), (here, here), (None, here)):
        taken.clear()
        call(given)
        made = [s for what, s in taken if what == "empty"]
        assert made and all(s is owner for s in made)
        assert taken[-1][0].startswith("rmsq_") and current == [here]
