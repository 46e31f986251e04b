"""The operators around the FP8 cache beside one another: several streams at
once, graphs that share a workspace, calls that allocate on another stream."""
import numpy as np
import pytest
import torch

import test_gpu_attention_fp8 as attn

pytestmark = pytest.mark.gpu
dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731


def _attention(c):
    start = dev(np.concatenate([[0], np.cumsum(c["q_lens"])]).astype(np.int32))
    return [c["q"].cuda(), dev(c["codes"]), dev(c["scales"]), dev(c["table"]), start, dev(np.array(c["seq"], np.int32))]


def _calls(rq):
    """Calls that each have their buffers, and give their outputs."""
    prompt = _attention(attn.make([300, 260], [500, 260], 8, 2, 128, 16, "bf16", seed=2))
    decode = _attention(attn.make([1] * 40, list(range(40, 4040, 100)), 8, 2, 128, 16, "bf16", seed=40))
    slots = torch.randperm(decode[1].shape[0] * 16, device="cuda")[:256].contiguous()
    torch.manual_seed(5)
    qkv = torch.randn(1500, 12 * 128, device="cuda").bfloat16()
    pos = torch.randint(0, 400, (3, 1500), device="cuda")
    cs = torch.rand(400, 128, device="cuda")
    w = torch.ones(128, device="cuda").bfloat16()
    k, v = (torch.randn(300, 2, 128, device="cuda").bfloat16() for _ in range(2))
    cache = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in rq.kv_cache_shapes_fp8(20, 2, 128, 16)]
    at = torch.arange(5, 305, device="cuda")

    def store(s):
        rq.kv_cache_store_fp8(k, v, at, *cache, stream=s)
        return tuple(cache)

    return [lambda s: rq.paged_attention_fp8(*prompt, return_lse=True, stream=s, variant="pipelined"),
            lambda s: rq.paged_attention_fp8(*decode, return_lse=True, stream=s),
            lambda s: rq.kv_cache_load_fp8(decode[1], decode[2], slots, stream=s),
            lambda s: (rq.qk_norm_mrope(qkv, pos, cs, w, w, 1e-6, 8, 2, 128, (24, 20, 20), interleaved=True,
                                        out=torch.zeros(1500, 1280, device="cuda").bfloat16(), stream=s),),
            store]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_streams_of_all_kernels_at_once(rmsq_gpu):
    rq = rmsq_gpu
    calls = _calls(rq)
    want = [[t.clone() for t in f(None)] for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for turn in range(12):
        for i, f in enumerate(calls):
            # (one writer of a cache at a time: always its own stream)
            with torch.cuda.stream(streams[i if f is calls[-1] else (i + turn) % len(streams)]):
                got[i].append(f(None))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(_same(w, g) for g in gs)
    assert rq.take_fault_flags() == 0


def test_calls_on_another_stream_than_the_current(rmsq_gpu):
    rq = rmsq_gpu
    calls = _calls(rq)[:3]
    want = [[t.clone() for t in f(None)] for f in calls]
    torch.cuda.synchronize()
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for turn in range(20):
        torch.cuda._sleep(100_000)
        for size in (1 << 16, 1 << 20, 21 << 20):
            torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")     # let go before it is filled
        for f, ts in zip(calls, want):
            got = f(side.cuda_stream if turn % 2 else side)
            here.wait_stream(side)
            for g, t in zip(got, ts):
                wrong += (g.view(torch.uint8) != t.view(torch.uint8)).any()
            del got, g
    torch.cuda.synchronize()
    assert wrong.item() == 0 and rq.take_fault_flags() == 0


def test_two_graphs_with_one_workspace(rmsq_gpu):
    """Captured separately, replayed in turn, each between the other's replays."""
    rq = rmsq_gpu
    cases = [_attention(attn.make([1] * 9, [2000 + 50 * i for i in range(9)], 16, 4, 128, 16, "bf16", seed=1)),
             _attention(attn.make([1, 120, 4], [900, 700, 3000], 16, 4, 128, 16, "bf16", seed=2))]
    size = max(rq.paged_attention_workspace_bytes(c[0].shape[0], c[4].numel() - 1, 16, 4, 128) for c in cases)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = [rq.paged_attention_fp8(*c, workspace=ws).clone() for c in cases]
    graphs, outs = [], []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(rq.paged_attention_fp8(*c, workspace=ws))
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want)) and rq.take_fault_flags() == 0


def test_store_and_attention_follow_each_other_in_one_graph(rmsq_gpu):
    """A captured decode step (store, then attention that reads what it stored),
    replayed with new keys and slots; what runs without programmatic launch gives
    the same."""
    rq = rmsq_gpu
    torch.manual_seed(2)
    h, D, page, R = 2, 64, 16, 6
    table = torch.arange(R * 8, device="cuda").int().view(R, 8)
    start = torch.arange(R + 1, device="cuda").int()

    keys = [tuple(torch.randn(R, c, D, device="cuda").bfloat16() * (1 + n) for c in (8, h, h)) for n in range(40)]
    bufs = [torch.empty_like(t) for t in keys[0]]
    seq, slots = torch.zeros(R, device="cuda").int(), torch.zeros(R, dtype=torch.int64, device="cuda")

    def place(n, q, k, v):
        for b, t in zip(bufs, (q, k, v)):
            b.copy_(t)
        seq.fill_(n + 1)
        slots.copy_(table[:, n // page].long() * page + n % page)

    results = []
    for graph in (False, True):
        cache = [torch.full(s, 255, dtype=torch.uint8, device="cuda") for s in rq.kv_cache_shapes_fp8(R * 8, h, D, page)]

        def step():
            rq.kv_cache_store_fp8(bufs[1], bufs[2], slots, *cache)
            return rq.paged_attention_fp8(bufs[0], *cache, table, start, seq)

        if graph:
            place(0, *keys[0])
            step()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = step()
            for c in cache:
                c.fill_(255)

            def run(n, *t):
                place(n, *t)
                g.replay()
                return out
        else:
            rq.set_programmatic_launch(False)

            def run(n, *t):
                place(n, *t)
                return step()
        results.append(torch.stack([run(n, *t).clone() for n, t in enumerate(keys)]))
        rq.set_programmatic_launch(True)
    assert torch.equal(results[0], results[1])
