"""Attention of drafted trees with more than 128 query rows per KV head (two query tiles to a
pair of CTAs): what test_gpu_tree.py looks at with one, and tables past 2^31 entries."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import DIM, bits
from test_gpu_tree import SCALE, _check, _run
from test_gpu_tree_steps import Model, _depths
from tree_reference import SHAPES, accept, ancestors, make_case, make_tree

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _case(sizes, ctx, hq, hkv, dtype, seed, shapes=SHAPES, **kw):
    """Trees that fill more than a query tile on average (by which the call takes two)."""
    rng = np.random.default_rng(seed)
    assert sum(sizes) * (hq // hkv) > 128 * len(sizes)
    trees = [make_tree(shapes[i % len(shapes)], n, rng) for i, n in enumerate(sizes)]
    return make_case(trees, ctx, hq, hkv, dtype, seed, **kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,sizes", [(32, 8, [64, 33, 1, 60, 0, 97, 32, 128]), (8, 8, [256, 129, 5, 128, 255]),
                                          (16, 2, [17, 1, 200, 16, 33]), (8, 1, [256, 240]), (6, 3, [100, 65, 64, 70])])
def test_tiles_of_every_fill(dtype, hq, hkv, sizes):
    """Second tiles that are full, hold one token or none; a third tile; short contexts and long ones."""
    ctx = [n + (0, 5000, 130, 1, 900, 12000, 64, 2047)[i % 8] for i, n in enumerate(sizes)]
    c = _case(sizes, ctx, hq, hkv, dtype, seed=hq)
    _check(c, _run(c))
    _check(c, _run(c, max_context_len=max(ctx)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,sizes,ctx", [(32, 8, [60, 64, 50], [1500, 700, 9000]), (16, 2, [31, 40], [30000, 200]),
                                              (8, 8, [256], [20000])])
def test_sharp_softmax(dtype, hq, hkv, sizes, ctx):
    """Scores tens of units apart: the running maximum moves from tile to tile."""
    c = _case(sizes, ctx, hq, hkv, dtype, seed=5, peak=8.0)
    _check(c, _run(c))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rising_maxima(dtype):
    """Every key tile's largest score lies above the one before: O is rescaled at each."""
    c = _case([64, 40], [6000, 700], 32, 8, dtype, seed=6, peak=2.0)
    for s in range(2):
        L = int(c["lens_h"][s])
        pos = np.arange(L)
        rows, cols = (torch.from_numpy(x.astype(np.int64)).to(DEV) for x in (c["bt_h"][s][pos // 16], pos % 16))
        grow = torch.from_numpy(1.0 + 3.0 * pos / 6000).to(DEV)
        c["kc"][rows, cols] = (c["kc"][rows, cols].double() * grow[:, None, None]).to(c["kc"].dtype)
    _check(c, _run(c))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("what", ["vc", "kc"])
@pytest.mark.parametrize("hq,hkv,n,ctx,bad", [(32, 8, 64, 174, 7), (32, 8, 60, 20060, 40), (16, 2, 200, 9000, 5),
                                             (8, 8, 256, 256, 130)])
def test_what_a_branch_does_not_see_has_no_effect(dtype, value, what, hq, hkv, n, ctx, bad):
    """Infinities and NaN in one drafted token's key or value: the rows that do not see it are as without it."""
    c = _case([n, n], [ctx, n + 700], hq, hkv, dtype, seed=8, shapes=("full", "random"))
    clean = _run(c).clone()
    _check(c, clean)
    pos, head, group = ctx - n + bad, hkv - 1, hq // hkv
    c[what][int(c["bt_h"][0, pos // 16]), pos % 16, head, 17:19] = value
    out = _run(c)
    hit = np.zeros((2 * n, hq), bool)
    hit[:n, head * group:(head + 1) * group] = ancestors(c["trees"][0])[:, bad][:, None]
    hit = torch.from_numpy(hit).to(DEV)
    assert torch.equal(out[~hit], clean[~hit])
    if what == "vc" or value != value:
        assert bool(out[hit].isnan().all())
    else:  # (an infinite key is a weight of 0, 1 or NaN: not finite scores end as NaN or as the rest)
        assert not bool((out[hit] == clean[hit]).all())


def test_rows_behind_and_refused_sequences_are_left():
    sizes = [64, 60, 50, 40, 70, 33]
    c = _case(sizes, [100, 60, 90, 300, 5000, 700], 32, 8, "bf16", seed=9)
    good = _run(c).clone()
    total = sum(sizes)
    q = torch.cat([c["q"], torch.full_like(c["q"][:5], float("nan"))])
    parents = torch.cat([c["parents"], torch.full_like(c["parents"][:5], 77)])
    lens = c["lens"].clone()
    lens[1] = 5                              # shorter than its tree
    lens[3] = c["bt"].shape[1] * 16 + 1      # beyond the table
    out = torch.full_like(q, 3.0)
    pa.paged_attn_tree(q, c["kc"], c["vc"], c["bt"], lens, c["n"], parents, SCALE, out=out)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail in (1, 3)
    first = np.concatenate([[0], np.cumsum(sizes)])
    rows = torch.ones(total + 5, dtype=torch.bool, device=DEV)
    rows[total:] = False
    for s in (1, 3):
        rows[first[s]:first[s + 1]] = False
    assert bool((out[~rows] == 3.0).all())
    # (the others' keys are dealt differently without the refused ones: equal within the tolerance)
    _check(c, torch.where(rows[:total, None, None], out[:total], good), skip=(1, 3))


@pytest.mark.parametrize("bad", [40, 63, 2 ** 31 - 1, -2, -2 ** 31])
def test_a_bad_parent_is_reported_and_taken_as_none(bad):
    c = _case([64, 64], [500, 9000], 32, 8, "bf16", seed=11, shapes=("chain",))
    c["parents"][64 + 40] = bad
    out = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    trees = [t.copy() for t in c["trees"]]
    trees[1][40] = -1
    _check(dict(c, trees=trees), out)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_bad_block_is_reported(dtype):
    """Committed pages, and the one with the last drafted token."""
    c = _case([60, 64, 90], [500, 4000, 3000], 32, 8, dtype, seed=12)
    good = _run(c).clone()
    c["bt"][1, 3] = c["kc"].shape[0]
    c["bt"][1, 77] = -4
    c["bt"][1, 249] = 2 ** 31 - 1
    out = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    assert torch.equal(out[:60], good[:60]) and torch.equal(out[124:], good[124:])


def test_repeats_streams_and_graphs_agree():
    """The same bits again and again, on another stream, and from captured calls that share a workspace."""
    c = _case([60, 64, 90], [3000, 700, 15000], 32, 8, "bf16", seed=15)
    d = _case([200], [9000], 16, 8, "f16", seed=16)
    ref_c, ref_d = _run(c).clone(), _run(d).clone()
    _check(c, ref_c)
    _check(d, ref_d)
    for _ in range(20):
        assert torch.equal(_run(c), ref_c) and torch.equal(_run(d), ref_d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = _run(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref_c)
    ws = pa.alloc_tree_workspace(3, 32, 8)
    oc, od = torch.zeros_like(ref_c), torch.zeros_like(ref_d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(c, out=oc, workspace=ws)
        _run(d, out=od, workspace=ws)
        _run(c, out=oc, workspace=ws)
    for _ in range(3):
        oc.zero_(), od.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oc, ref_c) and torch.equal(od, ref_d)


def test_a_drafted_step():
    """Wide trees rotated and written, attended, judged and compacted in two layers: the cache is that of the
    accepted tokens written in a line, and the attention the plain form's over what was written."""
    layers, vocab, hq, hkv, dtype = 2, 23, 32, 8, torch.bfloat16
    model = Model(layers, hq, hkv, dtype, vocab, seed=1)
    rng = np.random.default_rng(2)
    inv, _ = pa.rope_inv_freq(DIM, 1e4)
    starts, sizes = [37, 500], [64, 50]
    tokens = [rng.integers(0, vocab, n) for n in starts]
    trees = [make_tree(s, n, rng) for s, n in zip(("random", "full"), sizes)]
    alloc, other = pa.BlockAllocator(200), pa.BlockAllocator(200)
    fresh = lambda: [tuple(torch.zeros((200, 16, hkv, DIM), dtype=dtype, device=DEV) for _ in range(2))
                     for _ in range(layers)]
    pools, pools2 = fresh(), fresh()
    seqs, seqs2 = [alloc.sequence() for _ in starts], [other.sequence() for _ in starts]
    cu = lambda x, d=np.int32: torch.from_numpy(np.asarray(x).astype(d)).to(DEV)

    def write(to, slots, ids, pos):
        ids = torch.from_numpy(np.asarray(ids)).to(DEV)
        return [pa.rope_kv_write(model.q[la][ids], model.k[la][ids], model.v[la][ids], inv, cu(pos), cu(slots, np.int64),
                                 *to[la]) for la in range(layers)]

    for s, t in zip(seqs, tokens):
        write(pools, s.reserve(len(t)), t, np.arange(len(t)))
        s.commit(len(t))
    drafts = [rng.integers(0, 2, n) for n in sizes]
    slots = [s.reserve(n) for s, n in zip(seqs, sizes)]
    bt, _, tree_lens, lens = pa.build_step_tables(seqs, 40)
    pos = np.concatenate([n + _depths(t) for n, t in zip(starts, trees)])
    queries = write(pools, np.concatenate(slots), np.concatenate(drafts), pos)
    parents = cu(np.concatenate(trees))
    for la in range(layers):
        out = pa.paged_attn_tree(queries[la], *pools[la], cu(bt), cu(lens), cu(tree_lens), parents, SCALE)
        _check(dict(q=queries[la], kc=pools[la][0], vc=pools[la][1], trees=trees, bt_h=np.asarray(bt),
                    lens_h=np.asarray(lens), dtype="bf16"), out)
    target = rng.integers(0, 2, sum(sizes))
    path, num, nxt, new = pa.tree_accept(cu(np.concatenate(drafts), np.int64), cu(target, np.int64), parents,
                                         cu(tree_lens), cu(lens), pa.layer_pools(pools), cu(bt))
    at = 0
    for i, (s, s2, t) in enumerate(zip(seqs, seqs2, tokens)):
        n = sizes[i]
        way, after = accept(trees[i], drafts[i], target[at:at + n])
        assert path[i, :int(num[i])].tolist() == way and int(nxt[i]) == after and int(new[i]) == starts[i] + len(way)
        s.commit(n)
        s.truncate(int(new[i]))
        line = np.concatenate([t, drafts[i][way]]).astype(np.int64)
        write(pools2, s2.reserve(len(line)), line, np.arange(len(line)))
        s2.commit(len(line))
        rows = lambda pair, q: [x[torch.tensor(q.blocks, device=DEV).long()].flatten(0, 1)[:len(line)] for x in pair]
        for la in range(layers):
            for a, b in zip(rows(pools[la], s), rows(pools2[la], s2)):
                assert np.array_equal(bits(a), bits(b))
        at += n


@pytest.mark.parametrize("sizes,hq", [([5, 7, 9], 16), ([70, 64, 80], 16)])
def test_tables_past_two_to_the_31_entries(sizes, hq):
    """The third sequence's row of the table begins 2^31 entries behind the first one's."""
    rng = np.random.default_rng(19)
    trees = [make_tree("random", n, rng) for n in sizes]
    c = make_case(trees, [n + e for n, e in zip(sizes, (300, 20, 1000))], hq, 8, "f16", seed=19)
    width = 1 << 30
    wide = torch.empty((3, width), dtype=torch.int32, device=DEV)
    wide[:, :4096] = -1
    wide[:, :c["bt"].shape[1]] = c["bt"]
    c["bt"] = wide
    _check(c, _run(c, max_context_len=4096))
    draft = torch.from_numpy(rng.integers(0, 2, sum(sizes))).to(DEV)
    target = torch.from_numpy(rng.integers(0, 2, sum(sizes))).to(DEV)
    kc, vc = c["kc"].clone(), c["vc"].clone()
    narrow = wide[:, :128].contiguous()
    got = pa.tree_accept(draft, target, c["parents"], c["n"], c["lens"], pa.layer_pools([(c["kc"], c["vc"])]), wide)
    want = pa.tree_accept(draft, target, c["parents"], c["n"], c["lens"], pa.layer_pools([(kc, vc)]), narrow)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert np.array_equal(bits(c["kc"]), bits(kc)) and np.array_equal(bits(c["vc"]), bits(vc))
