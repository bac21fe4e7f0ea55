"""Host checks (no GPU) of buffers of the long-context calls that may not overlap:
refused before anything is enqueued."""
import ctypes

import pytest

import paged_kv_gqa_cache_gb300 as pa

P = 1 << 20  # a fake, 16-byte aligned "device" address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from paged_kv_gqa_cache_gb300 import _build
    _build.build()
    return pa.load_library()


def _pool():
    return pa.KVPool(k_cache=4096, v_cache=8192, num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=0)


def _rope(lib, q, k, v, out, T=4, hq=16):
    rope = pa.Rope(inv_freq=64, rotary_dim=128, layout=0, attention_factor=1.0)
    return pa.STATUS[lib.pa_rope_kv_write(q, k, v, ctypes.byref(rope), None, None, 1e-6, 64, 64, T, hq, out,
                                          ctypes.byref(_pool()), None)]


Q, KV = 4 * 16 * 256, 4 * 8 * 256  # bytes of the queries and of the keys or values


@pytest.mark.parametrize("out", [P + 16, P - 16, P + Q - 16, P - Q + 16,            # in part over the queries
                                 2 * P, 2 * P + KV - 16, 2 * P - Q + 16,            # over the keys
                                 3 * P, 3 * P + 16, 3 * P - Q + 16])                # over the values
def test_rotated_queries_over_inputs(lib, out):
    assert _rope(lib, P, 2 * P, 3 * P, out) == "PA_ERR_SHAPE"


@pytest.mark.parametrize("k,v", [(P, 3 * P), (2 * P, P + Q - 16)])
def test_rotated_in_place_over_keys_or_values(lib, k, v):
    assert _rope(lib, P, k, v, P) == "PA_ERR_SHAPE"
