"""Host checks of pa_kv_evict_ex's flags (no GPU): nothing is enqueued."""
import ctypes
import os
import re

import pytest

import paged_kv_gqa_cache_gb300 as pa

P = 1 << 20  # a fake, 16-byte aligned "device" address; never dereferenced by these calls


@pytest.mark.parametrize("flags,S,status", [
    (0, 0, "PA_OK"), (1, 0, "PA_OK"), (3, 0, "PA_OK"), (4, 0, "PA_ERR_UNSUPPORTED"), (2 ** 31, 4, "PA_ERR_UNSUPPORTED"),
    (3, -1, "PA_ERR_SHAPE"),
])
def test_flags(flags, S, status):
    from paged_kv_gqa_cache_gb300 import _build
    _build.build()
    lib = pa.load_library()
    pool = pa.KVPool(k_cache=4096, v_cache=8192, num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=0)
    st = lib.pa_kv_evict_ex(ctypes.byref(pool), P, 16, P, S, P, 256, 64, 8, 4, P + 64, 4, P + 64, 64, P, P + 128, flags,
                            None)
    assert pa.STATUS[st] == status


def test_flags_match_the_header():
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                               "pagedattn.h")).read()
    defines = dict(re.findall(r"#define (PA_EVICT_[A-Z_]+) (\d+)u\b", header))
    assert {k: int(v) for k, v in defines.items()} == {"PA_EVICT_MARK_KEPT": pa.EVICT_MARK_KEPT,
                                                       "PA_EVICT_MARK_LENGTHS": pa.EVICT_MARK_LENGTHS}
