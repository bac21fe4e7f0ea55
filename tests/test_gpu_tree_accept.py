"""GPU checks of pa_tree_accept and pa_tree_move: paths, next tokens and lengths
equal to the definition's, rows moved bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import TORCH, bits, place, random_pool
from tree_reference import SHAPES, accept, make_tree, move

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _case(trees, ctx, hkv, layers, dtype, seed, right=0.7):
    """Drafts and choices over few token values (so that chance and repeats occur), a share of them made right."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = np.array([len(t) for t in trees])
    lens = np.asarray(ctx, np.int64)
    bt, nb = place(rng, np.maximum(lens, 1))
    total = int(n.sum())
    draft, target = rng.integers(0, 50, total) + (1 << 40), rng.integers(0, 50, total) + (1 << 40)
    at = 0
    for t in trees:
        for i, p in enumerate(t):
            if p >= 0 and rng.random() < right:
                draft[at + i] = target[at + p]
        at += len(t)
    cu = lambda x, d: torch.from_numpy(np.asarray(x).astype(d)).to(DEV)
    pools = [(random_pool(g, nb, hkv, dtype), random_pool(g, nb, hkv, dtype)) for _ in range(layers)]
    return dict(trees=trees, n=cu(n, np.int32), lens=cu(lens, np.int32), bt=cu(bt, np.int32), bt_h=bt, lens_h=lens,
                parents=cu(np.concatenate(trees) if total else np.zeros(0), np.int32), draft=cu(draft, np.int64),
                target=cu(target, np.int64), draft_h=draft, target_h=target, pools=pools,
                handle=pa.layer_pools(pools))


def _run(c, **kw):
    return pa.tree_accept(c["draft"], c["target"], c["parents"], c["n"], c["lens"], c["handle"], c["bt"], **kw)


def _expect(c, stride, skip=()):
    S = len(c["trees"])
    path, num, nxt, lens = np.full((S, stride), -1), np.zeros(S, int), np.full(S, -1), np.full(S, -1)
    at = 0
    for s, t in enumerate(c["trees"]):
        if s not in skip:
            way, nxt[s] = accept(t, c["draft_h"][at:at + len(t)], c["target_h"][at:at + len(t)])
            path[s, :len(way)], num[s] = way, len(way)
            lens[s] = c["lens_h"][s] - len(t) + len(way)
        at += len(t)
    return path, num, nxt, lens


def _moved(c, before, path, num):
    """The pools' bits after the moves."""
    out = []
    for pair in before:
        row = []
        for x in pair:
            x = x.copy()
            for s, t in enumerate(c["trees"]):
                move(x, c["bt_h"][s], int(c["lens_h"][s]) - len(t), [int(a) for a in path[s, :num[s]]])
            row.append(x)
        out.append(row)
    return out


def _check(c, got, before, stride, skip=(), pools=True):
    want = _expect(c, stride, skip)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    if pools:
        for (k, v), (wk, wv) in zip(c["pools"], _moved(c, before, want[0], want[1])):
            assert np.array_equal(bits(k), wk) and np.array_equal(bits(v), wv)


def _bits(c):
    return [(bits(k), bits(v)) for k, v in c["pools"]]


@pytest.mark.parametrize("dtype,hkv,layers", [("f16", 8, 3), ("bf16", 1, 5), ("bf16", 3, 1), ("f16", 4, 65)])
def test_ragged_trees(dtype, hkv, layers):
    rng = np.random.default_rng(hkv)
    sizes = [1, 5, 64, 0, 7, 33, 2, 16, 12, 100]
    trees = [make_tree(SHAPES[i % len(SHAPES)], n, rng) for i, n in enumerate(sizes)]
    ctx = [n + e for n, e in zip(sizes, [0, 11, 1, 30, 16, 100, 15, 47, 3, 9])]
    c = _case(trees, ctx, hkv, layers, dtype, seed=hkv)
    before = _bits(c)
    _check(c, _run(c, max_tree_len=100), before, 100)


@pytest.mark.parametrize("right", [0.0, 0.5, 0.95, 1.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_shape(shape, right):
    rng = np.random.default_rng(7)
    trees = [make_tree(shape, int(n), rng) for n in [256, 255, 40, 3, 129, 17, 1, 64, 80]]
    c = _case(trees, [len(t) + 5 * i for i, t in enumerate(trees)], 2, 2, "bf16", seed=11, right=right)
    before = _bits(c)
    _check(c, _run(c), before, 256)


def test_many_sequences():
    rng = np.random.default_rng(5)
    sizes = rng.integers(0, 12, 3000)
    trees = [make_tree("random", int(n), rng) for n in sizes]
    c = _case(trees, (sizes + rng.integers(0, 20, 3000)).tolist(), 1, 2, "f16", seed=5)
    before = _bits(c)
    _check(c, _run(c, max_tree_len=11), before, 11)


def test_without_pools():
    rng = np.random.default_rng(6)
    trees = [make_tree("random", 20, rng), make_tree("chain", 4, rng)]
    c = _case(trees, [40, 4], 8, 1, "f16", seed=6)
    before = _bits(c)
    got = pa.tree_accept(c["draft"], c["target"], c["parents"], c["n"], c["lens"], max_tree_len=20)
    _check(c, got, before, 20, pools=False)
    assert all(np.array_equal(bits(k), b[0]) for (k, v), b in zip(c["pools"], before))


def test_nothing_drafted():
    c = _case([np.zeros(0, np.int32)] * 3, [5, 0, 17], 8, 2, "f16", seed=1)
    before = _bits(c)
    _check(c, _run(c, max_tree_len=4), before, 4)


def test_refused_sequences():
    rng = np.random.default_rng(8)
    trees = [make_tree("random", n, rng) for n in (10, 6, 8, 12, 5)]
    c = _case(trees, [30, 40, 50, 60, 70], 8, 2, "bf16", seed=8, right=1.0)
    before = _bits(c)
    c["lens"][1] = 5                            # shorter than the tree
    c["lens"][2] = c["bt"].shape[1] * 16 + 1    # beyond the table
    c["parents"][10 + 6 + 8 + 4] = 4            # its own parent
    got = _run(c, max_tree_len=11)              # (the tree of 12 does not fit either)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail in (1, 2, 3)
    _check(c, got, before, 11, skip=(1, 2, 3))


@pytest.mark.parametrize("value", [-1, 257, 2 ** 31 - 1, -2 ** 31])
def test_bad_tree_lengths(value):
    rng = np.random.default_rng(9)
    trees = [make_tree("random", n, rng) for n in (10, 6)]
    c = _case(trees, [30, 40], 8, 1, "bf16", seed=9, right=1.0)
    c["n"][1] = value
    before = _bits(c)
    got = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    _check(c, got, before, 256, skip=(1,))


def test_a_tree_past_the_tokens_is_refused():
    rng = np.random.default_rng(10)
    trees = [make_tree("random", n, rng) for n in (10, 6, 4)]
    c = _case(trees, [30, 40, 20], 8, 1, "f16", seed=10)
    short = dict(c, draft=c["draft"][:18], target=c["target"][:18], parents=c["parents"][:18])
    before = _bits(c)
    got = _run(short)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 2
    _check(c, got, before, 256, skip=(2,))


def test_a_bad_block_moves_the_rest():
    trees = [np.array([-1, 0, 0, 2, 3], np.int32)]
    c = _case(trees, [36], 8, 2, "f16", seed=12, right=0.0)
    c["draft"][2:] = torch.tensor([7, 8, 9], device=DEV)
    c["target"][0], c["target"][2], c["target"][3] = 7, 8, 9   # path 0 2 3 4: positions 31 33 34 35 to 31 .. 34
    c["draft_h"], c["target_h"] = c["draft"].cpu().numpy(), c["target"].cpu().numpy()
    c["bt"][0, 1] = -1                                         # (block of position 31: its token stays anyway)
    before = _bits(c)
    got = _run(c)
    assert got[0][0, :4].tolist() == [0, 2, 3, 4] and pa.get_device_error()[0] == 0
    _check(c, got, before, 256)
    c["bt"][0, 2] = c["pools"][0][0].shape[0]                  # the others' block
    before = _bits(c)
    got = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 0
    assert got[0][0, :4].tolist() == [0, 2, 3, 4] and all(np.array_equal(bits(k), b[0])
                                                          for (k, _), b in zip(c["pools"], before))


def test_given_paths():
    rng = np.random.default_rng(13)
    trees = [make_tree("random", n, rng) for n in (10, 6, 8, 12, 5, 3)]
    c = _case(trees, [30, 40, 50, 60, 70, 3], 3, 66, "bf16", seed=13)
    paths = [[0, 3, 9], [], [1, 2, 7], [0, 1, 2, 3], [4], [2]]
    path = np.full((6, 7), 99)
    for s, w in enumerate(paths):
        path[s, :len(w)] = w
    num = np.array([len(w) for w in paths])
    before = _bits(c)
    cu = lambda x: torch.from_numpy(x.astype(np.int32)).to(DEV)
    given, nums = cu(path), cu(num)
    lens = pa.tree_move(given, nums, c["n"], c["lens"], c["handle"], c["bt"])
    assert lens.tolist() == [int(L) - len(t) + m for L, t, m in zip(c["lens_h"], trees, num)]
    assert np.array_equal(given.cpu().numpy(), path) and np.array_equal(nums.cpu().numpy(), num)
    for (k, v), (wk, wv) in zip(c["pools"], _moved(c, before, path, num)):
        assert np.array_equal(bits(k), wk) and np.array_equal(bits(v), wv)


@pytest.mark.parametrize("bad", [[3, 2], [1, 1], [0, 10], [-1, 2], [0, 2 ** 31 - 1]])
def test_bad_given_paths(bad):
    rng = np.random.default_rng(14)
    trees = [make_tree("random", n, rng) for n in (10, 6)]
    c = _case(trees, [30, 40], 8, 2, "bf16", seed=14)
    before = _bits(c)
    path = torch.tensor([bad + [0], [0, 2, 5]], dtype=torch.int32, device=DEV)
    lens = pa.tree_move(path, torch.tensor([2, 3], dtype=torch.int32, device=DEV), c["n"], c["lens"], c["handle"], c["bt"])
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 0 and lens.tolist() == [-1, 37]
    want = _moved(c, before, np.array([[0, 0, 0], [0, 2, 5]]), np.array([0, 3]))
    assert all(np.array_equal(bits(k), w[0]) and np.array_equal(bits(v), w[1]) for (k, v), w in zip(c["pools"], want))
    for num in (-1, 4, 11):
        lens = pa.tree_move(path, torch.tensor([num, 0], dtype=torch.int32, device=DEV), c["n"], c["lens"], c["handle"],
                            c["bt"])
        assert pa.STATUS[pa.get_device_error()[0]] == "PA_ERR_RANGE" and lens.tolist() == [-1, 34]


def test_stream_and_graph():
    rng = np.random.default_rng(15)
    trees = [make_tree("random", n, rng) for n in (10, 60, 8)]
    c = _case(trees, [30, 90, 50], 8, 4, "f16", seed=15)
    before = _bits(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(c, got, before, 256)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(c, max_tree_len=60)
    for _ in range(2):  # (each replay moves once more, from where the last one left the rows)
        before = _bits(c)
        graph.replay()
        torch.cuda.synchronize()
        _check(c, got, before, 60)


def test_bindings_refuse():
    rng = np.random.default_rng(16)
    c = _case([make_tree("random", 5, rng)], [30], 8, 1, "f16", seed=16)
    with pytest.raises(TypeError):
        pa.tree_accept(c["draft"].int(), c["target"], c["parents"], c["n"], c["lens"])
    with pytest.raises(ValueError):
        pa.tree_accept(c["draft"], c["target"][:-1], c["parents"], c["n"], c["lens"])
    with pytest.raises(TypeError):
        pa.tree_accept(c["draft"], c["target"], c["parents"], c["n"], c["lens"], c["pools"], c["bt"])
    with pytest.raises((TypeError, ValueError)):
        pa.tree_accept(c["draft"], c["target"], c["parents"], c["n"], c["lens"], c["handle"])
    with pytest.raises(ValueError):
        _run(c, max_tree_len=0)
    with pytest.raises(ValueError):
        pa.tree_move(c["parents"].view(1, 5), c["n"].repeat(2), c["n"], c["lens"], c["handle"], c["bt"])
    k, v = c["pools"][0]
    for pools in ([(k, v), (k, v)], [(k, k)], [(k[:2], v[:2]), (k[1:3], v[2:4])]):  # a row of them would move twice
        with pytest.raises(ValueError):
            pa.layer_pools(pools)
    pa.layer_pools([(k[:2], v[:2]), (k[2:4], v[2:4])])
    assert TORCH["f16"] is c["pools"][0][0].dtype
