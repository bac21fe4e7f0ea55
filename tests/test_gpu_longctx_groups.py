"""GPU checks of group sizes that pa_paged_attn_decode_shared cannot take, wherever
in the list they stand: the error names the group, and every sequence is computed
right.  Tolerances: those of test_gpu_decode_shared.py."""
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


@pytest.mark.parametrize("sizes,prefix,bad", [
    ([8, 3], [256, 128], 0),                    # one more than there are, then a group
    ([2 ** 31 - 1, 4, 3], [256, 128, 64], 0),
    ([2, 6, 4], [256, 128, 64], 1),             # past the sequences, though not more than there are
    ([2, 2 ** 31 - 1, 4], [256, 128, 64], 1),
    ([2, 2 ** 31 - 1, 2 ** 31 - 1, 5], [256, 128, 64, 64], 1),
    ([2, 3, 2, 1], [256, 128, 64, 16], 3),      # the sequences are used up exactly
    ([7, 7, 7], [0, 256, 64], 1),
    ([2, -2 ** 31, 3, 2], [256, 64, 128, 64], 1),
    ([9] * 255 + [7], [256] * 256, 0),
])
def test_mis_sized_groups_before_others(sizes, prefix, bad):
    """Seven sequences in groups of 2, 3 and 2.  What follows the bad size would join sequences of two groups,
    whose keys differ, if it began where the bad one does."""
    good = shared._case([(256, [1, 30]), (128, [140, 150, 130]), (64, [209, 208])], 16, 4, "f16", seed=13)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    c = dict(good, sizes=i32(sizes), prefix=i32(prefix))
    out = shared._run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == bad
    shared._check(c, out)


def test_empty_groups_at_the_end():
    c = shared._case([(256, [1, 30]), (128, [140, 150, 130])], 16, 4, "f16", seed=14)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    c = dict(c, sizes=i32([0, 2, 0, 3, 0, 0]), prefix=i32([64, 256, 16, 128, 0, 256]))
    shared._check(c, shared._run(c))
