"""Host checks (no GPU) of long-context decodes whose pages 32 bits do not count:
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


def _pool(hkv):
    return pa.KVPool(k_cache=4096, v_cache=8192, num_blocks=64, block_size=16, num_kv_heads=hkv, head_dim=128, dtype=0)


@pytest.mark.parametrize("S,mcl,status", [
    (32, 2 ** 30, "PA_ERR_UNSUPPORTED"), (33, 2 ** 30 - 16, "PA_ERR_UNSUPPORTED"),
    (16384, 2 ** 21, "PA_ERR_UNSUPPORTED"), (16384, 2 ** 21 - 15, "PA_ERR_UNSUPPORTED"),
    (16384, 2 ** 21 - 16, "PA_ERR_WORKSPACE"), (31, 2 ** 30, "PA_ERR_WORKSPACE"), (32, 2 ** 30 - 16, "PA_ERR_WORKSPACE"),
])
def test_pages_of_a_decode_with_weights(lib, S, mcl, status):
    st = lib.pa_paged_attn_decode_weights(P, ctypes.byref(_pool(1)), P, -(-mcl // 16), P, S, 1, mcl, 0.1, None, P, mcl,
                                          P, None, 0, None)
    assert pa.STATUS[st] == status


@pytest.mark.parametrize("S,mb,status", [
    (6000, 357914, "PA_ERR_UNSUPPORTED"), (6000, 357913, "PA_ERR_WORKSPACE"), (2, 2 ** 30, "PA_ERR_UNSUPPORTED"),
    (2, 2 ** 30 - 1, "PA_ERR_WORKSPACE"),
])
def test_block_tables_of_a_shared_decode(lib, S, mb, status):
    st = lib.pa_paged_attn_decode_shared(P, ctypes.byref(_pool(1)), P, mb, P, S, 1, 256, 0.1, None, None, 0, P, None, 0,
                                         None)
    assert pa.STATUS[st] == status
