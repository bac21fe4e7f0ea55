"""Lengths that one call writes and the next one reads, with nothing between the two: the
attention calls read them before their dependency wait."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_tree_accept as acc
import test_gpu_decode_weights as weights
from longctx_reference import DIM
from tree_reference import make_tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = DIM ** -0.5


@pytest.mark.parametrize("layers", [1, 65])
def test_accepted_paths_then_a_decode(layers):
    """Every second sequence is refused: its length is -1, and the decode leaves its row."""
    rng = np.random.default_rng(1)
    S = 40
    trees = [make_tree("random", int(n), rng) for n in rng.integers(1, 20, S)]
    c = acc._case(trees, [len(t) + int(e) for t, e in zip(trees, rng.integers(1, 90, S))], 2, layers, "bf16", seed=1)
    lens = c["lens"].clone()
    lens[1::2] = 0  # shorter than the tree
    q = torch.randn((S, 4, DIM), device=DEV).bfloat16()
    before = [(k.clone(), v.clone()) for k, v in c["pools"]]
    want = None
    for rep in range(20):
        for (k, v), (k0, v0) in zip(c["pools"], before):
            k.copy_(k0), v.copy_(v0)
        out = torch.full_like(q, 3.0)
        torch.cuda.synchronize()
        new = pa.tree_accept(c["draft"], c["target"], c["parents"], c["n"], lens, c["handle"], c["bt"])[3]
        if rep == 0:
            torch.cuda.synchronize()
        pa.paged_attn_decode(q, *c["pools"][-1], c["bt"], new, SCALE, out=out)
        if rep == 0:
            want = out.clone()
            assert bool((new[1::2] == -1).all()) and bool((new[::2] > 0).all())
            assert bool((want[1::2] == 3.0).all()) and bool((want[::2] != 3.0).any(2).all())
        assert torch.equal(out, want)
    st, _ = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE"


def test_evicted_caches_then_a_decode():
    rng = np.random.default_rng(2)
    S, budget = 24, 64
    c = weights._case(rng.integers(20, 300, S), 4, 2, "f16", seed=2)
    lens = c["lens"].clone()
    lens[1::2] = 0
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    want = None
    for rep in range(20):
        c["kc"].copy_(kc0), c["vc"].copy_(vc0)
        out = torch.full_like(c["q"], 3.0)
        torch.cuda.synchronize()
        _, new = pa.kv_evict(c["kc"], c["vc"], c["bt"], lens, c["w"].clone(), budget, 8, 4)
        if rep == 0:
            torch.cuda.synchronize()
        pa.paged_attn_decode(c["q"], c["kc"], c["vc"], c["bt"], new, SCALE, out=out)
        if rep == 0:
            want = out.clone()
            assert bool((new[1::2] == -1).all()) and bool((want[1::2] == 3.0).all())
        assert torch.equal(out, want)
    st, _ = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE"
