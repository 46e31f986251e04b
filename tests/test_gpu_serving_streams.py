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
