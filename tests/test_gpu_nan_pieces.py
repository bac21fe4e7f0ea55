"""A key that is NaN makes the rows that see it NaN, however the keys are dealt: also
where a worker's piece holds no other scores, so that it has a sum but no maximum."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_decode_shared as shared
import test_gpu_decode_weights as weights
import test_gpu_tree as tree
from tree_reference import make_case, make_tree

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _spoil(c, s, lo, hi, head):
    """NaN in an element of the keys lo .. hi - 1 of sequence s, one KV head."""
    pos = np.arange(lo, hi)
    rows = torch.from_numpy(np.asarray(c["bt_h"])[s, pos // 16].astype(np.int64)).to(DEV)
    c["kc"][rows, torch.from_numpy(pos % 16).to(DEV), head, 5] = float("nan")


def _heads(out, head, group):
    """(the rows' query heads of this KV head, the others)."""
    mine = torch.zeros(out.shape[1], dtype=torch.bool, device=DEV)
    mine[head * group:(head + 1) * group] = True
    return out[:, mine], out[:, ~mine]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_drafted_key_alone_in_its_piece(dtype):
    """256 drafts under the first, nothing committed: the later ones see of the first key tile only that token."""
    rng = np.random.default_rng(1)
    c = make_case([make_tree("star", 256, rng)], [256], 8, 1, dtype, seed=1)
    _spoil(c, 0, 0, 1, 0)
    out = tree._run(c)
    assert bool(out.isnan().all())
    tree._check(c, out)


@pytest.mark.parametrize("n", [5, 60])
def test_committed_keys_of_a_tree(n):
    """A front of NaN keys that grows by a key tile a time: somewhere it ends where a piece does."""
    rng = np.random.default_rng(2)
    c = make_case([make_tree("random", n, rng), make_tree("full", n, rng)], [20000 + n, 700], 32, 8, "bf16", seed=n)
    for lo in range(0, 5120, 128):
        _spoil(c, 0, lo, lo + 128, 2)
        out = tree._run(c)
        mine, rest = _heads(out[:n], 2, 4)
        assert bool(mine.isnan().all()) and not bool(rest.isnan().any()) and not bool(out[n:].isnan().any()), lo
    tree._check(c, out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_keys_of_a_shared_prefix(dtype):
    c = shared._case([(8192, [3000, 90, 1])], 16, 8, dtype, seed=3)
    for lo in range(0, 4096, 128):
        _spoil(c, 0, lo, lo + 128, 6)
        mine, rest = _heads(shared._run(c), 6, 2)
        assert bool(mine.isnan().all()) and not bool(rest.isnan().any()), lo


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_keys_of_a_suffix(dtype):
    """Without a prefix: the suffix's pieces alone."""
    c = shared._case([], 16, 8, dtype, seed=3, alone=[9000, 40])
    for lo in range(0, 2048, 16):
        _spoil(c, 0, lo, lo + 16, 6)
        mine, rest = _heads(shared._run(c), 6, 2)
        assert bool(mine[0].isnan().all()) and not bool(rest.isnan().any()) and not bool(mine[1].isnan().any()), lo


def test_outputs_of_the_decode_with_weights():
    c = weights._case([9000, 40], 16, 8, "bf16", seed=4)
    for lo in range(0, 2048, 16):
        _spoil(c, 0, lo, lo + 16, 1)
        mine, rest = _heads(weights._run(c, None, torch.zeros_like(c["w"]))[0], 1, 2)
        assert bool(mine[0].isnan().all()) and not bool(rest.isnan().any()) and not bool(mine[1].isnan().any()), lo


def test_weights_of_the_decode_with_weights():
    """The head's row sum is NaN, and so is the weight of every token."""
    c = weights._case([9000, 40], 16, 8, "bf16", seed=4)
    rest = [h for h in range(8) if h != 1]
    for lo in range(0, 2048, 16):
        _spoil(c, 0, lo, lo + 16, 1)
        _, w = weights._run(c, None, torch.zeros_like(c["w"]))
        assert bool(w[0, 1, :9000].isnan().all()) and not bool(w[0, 1, 9000:].isnan().any()), lo
        assert not bool(w[0, rest].isnan().any()) and not bool(w[1].isnan().any()), lo
