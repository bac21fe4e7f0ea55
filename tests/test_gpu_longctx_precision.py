"""GPU checks of how exactly the long-context decodes multiply probabilities and
values: every probability goes in as two terms of the pool dtype.

Tolerances: those of test_gpu_decode_shared.py, with two terms (M 2^-16, M = sum |p v|)
for every group.  A term of fp16 is off by up to 2^-25 below fp16's normal range, where
the row's largest probability is 2^15 (2^13 in a shared prefix): by 2^-38 of it at most,
so an output by 2^-38 sum |v_j|, where the keys far below the largest matter."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_decode_shared as shared
import test_gpu_decode_weights as weights
from longctx_reference import DIM, HALF_STEP, HALF_TINY, attention_torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,size", [(32, 8, 32), (32, 8, 33), (16, 2, 17), (16, 2, 70), (4, 2, 130), (3, 3, 129)])
@pytest.mark.parametrize("prefix", [16, 400])
def test_large_groups_are_as_exact_as_small_ones(dtype, hq, hkv, size, prefix):
    """Few keys, so that roundings of the probabilities would not average out: one to five query tiles."""
    rng = np.random.default_rng(size)
    c = shared._case([(prefix, rng.integers(1, 4, size).tolist())], hq, hkv, dtype, seed=size + prefix)
    c["one_term"] = False
    shared._check(c, shared._run(c))


def test_one_more_sequence_keeps_the_precision_of_the_others():
    """The same sequences in a group that fills one query tile and in one that is a sequence larger."""
    c = shared._case([(64, [1] * 33)], 32, 8, "bf16", seed=5)
    c["one_term"] = False
    shared._check(c, shared._run(c))
    first = {k: c[k][:32] for k in ("q", "bt", "lens", "bt_h", "lens_h")}
    c = dict(c, **first, sizes=torch.full_like(c["sizes"], 32))
    shared._check(c, shared._run(c))


def _one_key_above(c, at, nats, hkv):
    """Key `at` of the first sequence lies so far above the others, and its value is zero.  (Dim 0 of the other keys
    is zero, the queries hold 16 there.)"""
    c["q"][:, :, 0] = 16.0
    c["kc"][..., 0] = torch.where(c["kc"][..., 0].isnan(), c["kc"][..., 0], 0.0)
    c["vc"] *= 64.0
    blk = int(c["bt_h"][0, at // 16])
    c["kc"][blk, at % 16] = 0.0
    c["kc"][blk, at % 16, :, 0] = nats * DIM ** 0.5 / 16.0
    c["vc"][blk, at % 16] = 0.0


def _check_tails(c, out):
    ref, mag, worst = attention_torch(c["q"], c["kc"], c["vc"], c["bt_h"], c["lens_h"], DIM ** -0.5)
    u = HALF_STEP[c["dtype"]]
    far = torch.zeros_like(mag)
    if c["dtype"] == "f16":
        G = c["q"].shape[1] // c["kc"].shape[2]
        for s, n in enumerate(c["lens_h"]):
            rows = torch.as_tensor(c["bt_h"][s][:-(-int(n) // 16)], device=DEV).long()
            far[s] = c["vc"][rows].flatten(0, 1)[:int(n)].double().abs().sum(0).repeat_interleave(G, 0) * 2.0 ** -38
    tol = u * ref.abs() + (1 + u) * (mag * (worst * 2.0 ** -17 + 2.0 ** -15) + far) + HALF_TINY[c["dtype"]]
    d = (out.double() - ref).abs()
    assert bool((d <= tol).all()), f"worst {float((d / tol).nan_to_num(9e9).max()):.3f} of the tolerance"


TAILS = [(nats, at) for nats in (16, 18, 20) for at in (0, 11003, 29983)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nats,at", TAILS)
@pytest.mark.parametrize("hq,hkv", [(4, 2), (8, 1)])
def test_weights_far_below_the_largest(dtype, nats, at, hq, hkv):
    c = weights._case([30000, 40], hq, hkv, dtype, seed=nats)
    _one_key_above(c, at, nats, hkv)
    out, _ = weights._run(c, None, torch.zeros_like(c["w"]))
    _check_tails(c, out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nats,at", TAILS)
@pytest.mark.parametrize("size", [2, 70])
def test_shared_weights_far_below_the_largest(dtype, nats, at, size):
    c = shared._case([(29984, [1, 30] * (size // 2))], 4, 2, dtype, seed=nats + size)
    _one_key_above(c, at, nats, 2)
    _check_tails(c, shared._run(c))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("large", [40.0, 200.0, 900.0])
def test_very_large_scores(dtype, large):
    """One key in each sequence, at any place, whose score is so far above the others that its value is the output."""
    c = shared._case([(1040, [1, 50] * 20)], 8, 2, dtype, seed=9)
    flat_k, flat_v = c["kc"].flatten(0, 1), c["vc"].flatten(0, 1)
    c["q"][:] = large
    live = ~flat_k[:, 0, 0].isnan()
    flat_k[live] = large / 2
    for at in (0, 130, 700, 1039):
        blk = int(c["bt_h"][0, at // 16])
        k = c["kc"].clone()
        k[blk, at % 16] = large
        x = dict(c, kc=k)
        want = c["vc"][blk, at % 16].repeat_interleave(4, 0).expand(40, -1, -1)
        assert torch.equal(shared._run(x), want)
        w = torch.zeros((40, 2, 16 * c["bt"].shape[1]), device=DEV)
        out, _ = pa.paged_attn_decode_weights(x["q"], x["kc"], x["vc"], x["bt"], x["lens"], DIM ** -0.5, None, w)
        assert torch.equal(out, want)
        assert torch.equal(w.sum(-1), torch.full((40, 2), 4.0, device=DEV)) and bool((w[:, :, at] == 4.0).all())


@pytest.mark.parametrize("dtype,step", [("f16", 0.5), ("bf16", 4.0)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_scores_that_rise_by_about_the_type_s_range(dtype, step, sign):
    """Scores of 2^21 (log2 units), where fp32 has steps of 0.125 to 0.25, that rise by 14 to 22 (fp16) or 112
    to 178 from one key tile to the next: what enters the tensor cores must stay finite.  (A weight is only good to some tens of percent there, so
    the outputs are held to the range of the values that weigh.)"""
    groups = 132  # (so that a CTA takes several key tiles in a row)
    c = shared._case([(512, [1, 5])] * groups, 4, 2, dtype, seed=21)
    c["kc"][~c["kc"].isnan()] = sign * 512.0
    heads = torch.as_tensor(c["bt_h"][::2, :32], device=DEV).long()
    for tile in range(1, 4):
        c["kc"][heads[:, 8 * tile:8 * tile + 8].flatten(), :, :, :tile] = sign * 512.0 + step
    q = 220 + 2 * (torch.arange(2 * groups, device=DEV) // 4)  # 220 to 350, exact in both types
    c["q"][:] = q[:, None, None].to(c["q"].dtype)
    out = shared._run(c).float()
    top = c["vc"].float().nan_to_num().abs().max()
    assert bool(out.isfinite().all()) and bool((out.abs() <= 1.01 * top).all())
