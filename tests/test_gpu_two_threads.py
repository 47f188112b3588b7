"""GPU tests of the hybrid block's calls made from two host threads at once, each on a stream and with
buffers of its own, at sizes that give a kernel different amounts of shared memory."""
import sys
import threading

import pytest
import torch

import kv_shared_b200 as hs

pytestmark = pytest.mark.gpu


def _at_once(calls, times):
    errors, ready = [], threading.Barrier(len(calls))
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)

    def go(call, stream):
        try:
            torch.zeros(1, device="cuda")                      # the device's context is the thread's, too
            ready.wait()
            for _ in range(times):
                call(stream)
        except Exception as e:                                 # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    workers = [threading.Thread(target=go, args=(c, torch.cuda.Stream())) for c in calls]
    for w in workers:
        w.start()
    for w in workers:
        w.join()
    sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    return errors


def _check(cases, times):
    """cases: (call, outputs).  The bits of calls made alone, and no call fails."""
    main = torch.cuda.current_stream()
    want = []
    for call, outs in cases:
        call(main)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    assert _at_once([c for c, _ in cases], times) == []
    for (_, outs), ws in zip(cases, want):
        assert all(torch.equal(t, w) for t, w in zip(outs, ws))


def test_selections():
    def case(T):
        desc = hs.make_desc(1, 1, 16, 128, window=128, budget=256, max_ctx=T)
        s = torch.rand(1, T, generator=torch.Generator().manual_seed(T)).cuda()
        pos0 = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
        idx, cnt = (torch.empty(1, n, dtype=torch.int32, device="cuda") for n in (384, 1))
        ws = hs.alloc_workspace(desc)
        return lambda st: hs.hs2_topk_select(desc, s, T, pos0, 1, idx, cnt, ws, stream=st), (idx, cnt)

    _check([case(11000), case(160000)], 20000)


def test_sparse_layers_of_many_rows():
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, 4000, 128, generator=g).bfloat16().cuda() for _ in range(2))

    def case(stride, rows=400):
        desc = hs.make_desc(1, rows, 16, 128, window=8, budget=stride - 8, max_ctx=4000)
        q = torch.randn(1, rows, 16, 128, generator=g).bfloat16().cuda()
        idx = torch.stack([torch.randperm(4000, generator=g)[:stride].sort().values for _ in range(rows)])[None].int().cuda()
        cnt = torch.full((1, rows), stride, dtype=torch.int32, device="cuda")
        o, lse, ws = torch.empty_like(q), torch.empty(1, rows, 16, device="cuda"), hs.alloc_workspace(desc)
        return lambda st: hs.hs2_sparse_attn(desc, q, k, v, None, None, idx, cnt, o, lse, ws, stream=st), (o, lse)

    _check([case(64), case(1400)], 4000)


def test_prefills():
    g = torch.Generator().manual_seed(2)

    def case(ctx, n=32):
        desc = hs.make_desc(1, n, 16, 128, window=128, budget=256, max_ctx=ctx)
        q, k, v = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((1, n, 16, 128), (1, ctx, 128), (1, ctx, 128)))
        pos0 = torch.tensor([ctx - n], dtype=torch.int32, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(1, n, 16, device="cuda")
        idx, cnt = torch.empty(1, n, 384, dtype=torch.int32, device="cuda"), torch.empty(1, n, dtype=torch.int32, device="cuda")
        ws = hs.alloc_workspace(desc)
        return (lambda st: hs.hs2_full_attn_select(desc, q, k, v, None, None, pos0, o, lse, idx, cnt, None, ws, stream=st),
                (o, lse, idx, cnt))

    _check([case(1000), case(250000)], 1000)
