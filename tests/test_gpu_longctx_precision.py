"""GPU checks of how exactly the long-context decodes multiply probabilities and
values: every probability goes in as two terms of the pool dtype.

Tolerances: those of test_gpu_decode_shared.py, with two terms (M 2^-16, M = sum |p v|)
for every group."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_decode_shared as shared

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
