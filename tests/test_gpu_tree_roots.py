"""Accepted paths of trees whose tokens without parent are drafts like the others: the
model's choice after the committed context decides between them."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import bits
from test_gpu_tree_accept import _bits, _case, _moved, _run
from tree_reference import SHAPES, make_tree

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _judge(parents, draft, target, choice):
    """(path, next token): what greedy decoding produces as far as the tree has it drafted; of several such
    paths (the same token drafted twice) the deepest, of these the one that ends at the lowest index."""
    best = []
    ends = [[]]
    while ends:
        longer = []
        for path in ends:
            at = path[-1] if path else -1
            want = target[at] if path else choice
            longer += [path + [i] for i in range(len(parents)) if parents[i] == at and draft[i] == want]
        if longer:
            best = min(longer, key=lambda p: p[-1])
        ends = longer
    return best, int(target[best[-1]] if best else choice)


def _expect(c, choice, stride, skip=()):
    S = len(c["trees"])
    path, num, nxt, lens = np.full((S, stride), -1), np.zeros(S, int), np.full(S, -1), np.full(S, -1)
    at = 0
    for s, t in enumerate(c["trees"]):
        rows = slice(at, at + len(t))
        if s not in skip:
            way, nxt[s] = _judge(t, c["draft_h"][rows], c["target_h"][rows], choice[s])
            path[s, :len(way)], num[s] = way, len(way)
            lens[s] = c["lens_h"][s] - len(t) + len(way)
        at += len(t)
    return path, num, nxt, lens


def _choices(c, rng, right):
    """A choice per sequence: of one of its first tokens, or one that nobody drafted."""
    out, at = [], 0
    for t in c["trees"]:
        roots = [i for i, p in enumerate(t) if p < 0]
        out.append(c["draft_h"][at + int(rng.choice(roots))] if roots and rng.random() < right else 7)
        at += len(t)
    return np.array(out, np.int64)


@pytest.mark.parametrize("right", [0.0, 0.6, 1.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_shape(shape, right):
    rng = np.random.default_rng(3)
    trees = [make_tree(shape, int(n), rng) for n in [256, 0, 40, 3, 129, 17, 1, 64, 80]]
    c = _case(trees, [len(t) + 5 * i for i, t in enumerate(trees)], 2, 2, "bf16", seed=4)
    choice = _choices(c, rng, right)
    before = _bits(c)
    want = _expect(c, choice, 256)
    got = _run(c, context_targets=torch.from_numpy(choice).to(DEV))
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    for (k, v), (wk, wv) in zip(c["pools"], _moved(c, before, want[0], want[1])):
        assert np.array_equal(bits(k), wk) and np.array_equal(bits(v), wv)


def test_a_deeper_path_under_another_token_is_not_taken():
    """Two first tokens: greedy decoding would produce the second, and the first has the longer path."""
    c = _case([np.array([-1, 0, 1, -1, 3], np.int32)], [30], 2, 3, "f16", seed=5)
    draft, target = np.array([11, 12, 13, 21, 22]), np.array([12, 13, 14, 22, 23])
    c["draft"].copy_(torch.from_numpy(draft)), c["target"].copy_(torch.from_numpy(target))
    before = _bits(c)
    path, num, nxt, lens = _run(c, max_tree_len=5, context_targets=torch.tensor([21], device=DEV))
    assert path.tolist() == [[3, 4, -1, -1, -1]] and num.tolist() == [2] and nxt.tolist() == [23] and lens.tolist() == [27]
    for (k, v), (wk, wv) in zip(c["pools"], _moved(c, before, path.cpu().numpy(), [2])):
        assert np.array_equal(bits(k), wk) and np.array_equal(bits(v), wv)


def test_refused_and_many_layers():
    """A refused sequence gets -1 and not its choice; more layers than one launch takes."""
    rng = np.random.default_rng(6)
    trees = [make_tree("roots", 9, rng), make_tree("forest", 12, rng), make_tree("random", 7, rng)]
    c = _case(trees, [9, 30, 20], 2, 65, "f16", seed=6)
    choice = _choices(c, rng, 1.0)
    c["lens"][1] = 11  # shorter than its tree
    before = _bits(c)
    want = _expect(c, choice, 12, skip=(1,))
    got = _run(c, max_tree_len=12, context_targets=torch.from_numpy(choice).to(DEV))
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    for (k, v), (wk, wv) in zip(c["pools"], _moved(c, before, want[0], want[1])):
        assert np.array_equal(bits(k), wk) and np.array_equal(bits(v), wv)


def test_bindings_refuse():
    rng = np.random.default_rng(7)
    c = _case([make_tree("forest", 5, rng)] * 2, [20, 9], 2, 1, "f16", seed=7)
    with pytest.raises(TypeError):
        _run(c, context_targets=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        _run(c, context_targets=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        _run(c, context_targets=torch.zeros((2, 1), dtype=torch.int64, device=DEV))
