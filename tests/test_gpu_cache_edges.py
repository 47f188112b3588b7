"""GPU tests of the calls around the block where buffers, streams and values meet their limits: outputs
in an input's place, two calls at once, captured calls, NaN and infinities in rows that are in use.

The forms, the checks and their tolerances are those of test_gpu_cache_ops.py."""
import math

import pytest
import torch

import cache_ops_ref as ref
import kv_shared_b200 as hs
import test_gpu_cache_ops as base

pytestmark = pytest.mark.gpu


def _evict_set(acc, lens, sinks, window, budget, kv, d, seed=0):
    """(description, inputs and outputs of an eviction on the GPU in the call's order)."""
    b, cap = acc.shape
    k, v, ks, vs = base._cache(base._gen(seed), b, cap, d, kv)
    keep = sinks + window + budget
    ko, vo = torch.full((b, keep, d), 7, dtype=k.dtype), torch.full((b, keep, d), 7, dtype=k.dtype)
    sc = [torch.full((b, keep), 5.0) if ks is not None else None for _ in range(2)]
    out = [ko, vo, *sc, torch.full((b, keep), 5.0), torch.full((b, keep), 99, dtype=torch.int32),
           torch.full((b,), 99, dtype=torch.int32)]
    desc = hs.make_evict_desc(b, d, base.KIND[kv], sinks=sinks, window=window, budget=budget, kv_capacity=cap)
    return desc, base._cu(torch.tensor(lens, dtype=torch.int32), acc, k, v, ks, vs), base._cu(*out)


# ------------------------------------------------------------------ eviction: lengths in place
@pytest.mark.parametrize("lens, cap, sinks, window, budget, kv", [
    ([5000, 300, 4000], 5000, 4, 96, 400, "bf16"),                     # one CTA a sequence
    ([60000, 59000, 200, 45000], 60000, 2, 10, 9000, "e4m3"),          # clusters
    ([300000, 299999], 300000, 0, 64, 90000, "e4m3"),                  # teams of all SMs
    ([700000], 700000, 0, 2, 9, "e4m3"),                               # slices that are read again
])
def test_evict_lengths_in_place(lens, cap, sinks, window, budget, kv):
    """new_len in len's place: the rows and lengths of a call with new_len apart, and a second cut of the
    same lengths that finds nothing left to cut."""
    acc = torch.rand(len(lens), cap, generator=base._gen(cap))
    desc, ins, outs = _evict_set(acc, lens, sinks, window, budget, kv, 64)
    hs.hs2_kv_evict(desc, *ins, *outs)
    torch.cuda.synchronize()
    want = [None if t is None else t.clone() for t in outs]
    keep = sinks + window + budget
    assert want[-1].tolist() == [min(n, keep) for n in lens]
    for _ in range(20):
        for t in outs[:-1]:
            if t is not None:
                t.zero_()
        ins[0].copy_(torch.tensor(lens, dtype=torch.int32))
        hs.hs2_kv_evict(desc, *ins, *outs[:-1], ins[0])
        torch.cuda.synchronize()
        assert torch.equal(ins[0], want[-1]) and torch.equal(outs[-2], want[-2])
        for s, m in enumerate(want[-1].tolist()):
            for got, w in zip(outs[:-2], want[:-2]):
                assert got is None or torch.equal(got[s, :m], w[s, :m])
    hs.hs2_kv_evict(desc, *ins, *outs[:-1], ins[0])
    assert ins[0].tolist() == want[-1].tolist()
    for s, m in enumerate(want[-1].tolist()):
        assert outs[-2][s, :m].tolist() == list(range(m)) and (outs[-2][s, m:] == -1).all()
