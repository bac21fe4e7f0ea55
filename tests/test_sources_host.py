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
