"""What the sources of the library may not hold (no GPU)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_gqa_cache_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_nothing_is_multicast_in_a_cluster(name):
    """Every CTA fetches its own tiles and signals its own barriers: a pool may lie in another
    device's memory, and nobody waits for an arrival in a CTA that may have left."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert not re.search(r"multicast\s*::\s*cluster", text)


@pytest.mark.parametrize("name", ["evict.cu", "tree_accept.cu"])
def test_new_lengths_are_visible_before_their_kernel_ends(name):
    """The attention calls read the lengths before their dependency wait: a kernel that writes
    them fences behind the store and lets nothing start early."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    stores = re.findall(r"p\.new_lens\[s\] = [^;]*;(\s*__threadfence\(\);)?", text)
    assert stores and all(stores)
    assert "griddep_launch_dependents" not in text
