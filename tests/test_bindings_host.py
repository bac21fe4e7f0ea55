"""What the bindings show of themselves (no GPU)."""
import inspect

import pytest

import paged_kv_gqa_cache_gb300 as pa


@pytest.mark.parametrize("name", ["rope_kv_write", "rope_kv_write_axes", "rope_axes", "paged_attn_tree", "tree_accept",
                                  "tree_move", "layer_pools"])
def test_no_private_arguments(name):
    assert not [a for a in inspect.signature(getattr(pa, name)).parameters if a.startswith("_")]
