"""The serving operators beside one another: several streams at once, each
with a kernel that wants a whole SM's tensor memory or a part of it."""
import numpy as np
import pytest
import torch

import test_gpu_attention as attn
import test_gpu_matmul as mm

pytestmark = pytest.mark.gpu


def test_streams_of_all_kernels_at_once(rmsq_gpu):
    rq = rmsq_gpu
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    calls = []
    for m, n, k in ((700, 2048, 1024), (9, 2048, 4096), (100, 1024, 2048)):     # pairs; clusters of 8; the rule's choice
        a, _, given, b, sb = mm.make(m, n, k, "fp8_group128_row", seed=m)
        args = [dev(x) for x in (a, given, b, sb)]
        calls.append(lambda a=args: rq.fp8_block_matmul(a[0], a[1], "fp8_group128_row", a[2], a[3]))
    for q_lens, seq, variant in (([300, 260], [500, 260], "pipelined"), ([1] * 40, list(range(40, 4040, 100)), "direct")):
        c = attn.make(q_lens, seq, 8, 2, 128, 16, "bf16", seed=len(q_lens))
        start = dev(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32))
        g1, g2 = torch.tensor([c["k_gs"]], device="cuda"), torch.tensor([c["v_gs"]], device="cuda")
        args = [c["q"].cuda(), dev(c["cache"]), dev(c["table"]), start, dev(np.array(seq, np.int32)), g1, g2, 16]
        calls.append(lambda a=args, v=variant: rq.paged_attention_nvfp4(*a, variant=v))
        slots = torch.randperm(c["cache"].shape[0] * 16, device="cuda")[:256].contiguous()
        calls.append(lambda a=args, s=slots: torch.stack(rq.kv_cache_load_nvfp4(a[1], s, a[5], a[6], 128, 16)))
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for turn in range(12):
        for i, f in enumerate(calls):
            with torch.cuda.stream(streams[(i + turn) % len(streams)]):
                got[i].append(f())
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(w, g)
    assert rq.take_fault_flags() == 0


def test_calls_on_the_current_and_on_another_stream_in_turn(rmsq_gpu):
    """Calls that allocate their own workspace and outputs, in turn on the
    current stream and on others, next to memory that the current stream has let
    go while its work is still to come: all give what one call alone gives, and
    results that are read on the current stream and let go at once stay whole
    until then."""
    rq = rmsq_gpu
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    c = attn.make([1] * 16, [3000] * 16, 32, 8, 128, 16, "bf16", seed=51)
    start = dev(np.arange(17, dtype=np.int32))
    g1, g2 = torch.tensor([c["k_gs"]], device="cuda"), torch.tensor([c["v_gs"]], device="cuda")
    args = [c["q"].cuda(), dev(c["cache"]), dev(c["table"]), start, dev(np.array(c["seq"], np.int32)), g1, g2, 16]
    slots = torch.arange(256, device="cuda")
    a, _, given, b, sb = mm.make(33, 2048, 1024, "fp8_group128_row", seed=3)
    ops = [dev(x) for x in (a, given, b, sb)]
    x, w = torch.randn(256, 2048, device="cuda").bfloat16(), torch.ones(2048, device="cuda").bfloat16()
    calls = [lambda s: rq.paged_attention_nvfp4(*args, return_lse=True, stream=s),
             lambda s: rq.kv_cache_load_nvfp4(args[1], slots, g1, g2, 128, 16, stream=s),
             lambda s: (rq.fp8_block_matmul(ops[0], ops[1], "fp8_group128_row", ops[2], ops[3], stream=s),),
             lambda s: rq.fused_add_rmsnorm_nvfp4_dynamic(x, x, w, 1e-6, stream=s)]
    want = [[t.clone() for t in f(None)] for f in calls]
    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    side, handle = torch.cuda.Stream(), torch.cuda.Stream()
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for turn in range(40):
        torch.cuda._sleep(100_000)          # what follows on the current stream is late
        for size in (1 << 16, 1 << 20, 21 << 20):
            torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")     # let go before it is filled
        for f, ts in zip(calls, want):
            for s in ((side, None), (handle.cuda_stream, None), (None, side))[turn % 3]:
                got = f(s)
                if s is not None:
                    here.wait_stream(side if s is side else handle)
                for g, t in zip(got, ts):
                    wrong += (g.view(torch.uint8) != t.view(torch.uint8)).any()
                del got, g
    torch.cuda.synchronize()
    assert wrong.item() == 0 and rq.take_fault_flags() == 0


def test_a_call_on_a_forked_stream_of_a_capture(rmsq_gpu):
    """Inside a capture a call on a second stream takes its workspace and
    outputs from the graph's memory, and replays give what the call gives."""
    rq = rmsq_gpu
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    c = attn.make([1] * 8, [900] * 8, 16, 4, 128, 16, "bf16", seed=52)
    start = dev(np.arange(9, dtype=np.int32))
    g1, g2 = torch.tensor([c["k_gs"]], device="cuda"), torch.tensor([c["v_gs"]], device="cuda")
    args = [c["q"].cuda(), dev(c["cache"]), dev(c["table"]), start, dev(np.array(c["seq"], np.int32)), g1, g2, 16]
    want = rq.paged_attention_nvfp4(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        first = rq.paged_attention_nvfp4(*args, stream=side)
        other = rq.paged_attention_nvfp4(*args)
        here.wait_stream(side)
        total = first.float() + other.float()
        del first, other
    junk = [torch.full((1 << 20,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        graph.replay()
        assert torch.equal(total, 2 * want.float())
    del junk
    assert rq.take_fault_flags() == 0


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_handle(rmsq_gpu, handle):
    """Given as a raw handle while another stream is current, the default stream
    is a launching stream like any other."""
    rq = rmsq_gpu
    x = torch.randn(300, 1024, device="cuda").bfloat16()
    want = [t.clone() for t in rq.quant(x, "fp8_group128_row")]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(10):
            torch.full((300, 1024), 0xff, dtype=torch.uint8, device="cuda")
            got = rq.quant(x, "fp8_group128_row", stream=handle)
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            assert all(torch.equal(a, b) for a, b in zip(got, want))
