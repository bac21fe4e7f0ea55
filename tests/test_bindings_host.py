"""What the bindings show of themselves (no GPU)."""
import inspect

import paged_kv_gqa_cache_gb300 as pa


def test_public_calls_take_no_private_arguments():
    calls = {n: f for n, f in vars(pa).items() if inspect.isfunction(f) and not n.startswith("_")}
    assert "rope_kv_write" in calls and "paged_attn_tree" in calls
    private = {n: [a for a in inspect.signature(f).parameters if a.startswith("_")] for n, f in calls.items()}
    assert not {n: a for n, a in private.items() if a}
