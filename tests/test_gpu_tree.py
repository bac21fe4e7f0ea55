"""GPU checks of pa_paged_attn_tree against a plain form in 64 bits.

Tolerance of an output element, with u the type's half step and M = sum |p v|:
u |ref| for its rounding; (1 + u) M (a 2^-17 + 2^-16) for fp32 scores, exponentials
and sums, a = scale sum |q_i k_i| (each score is summed at most 40 roundings deep and a
weight moves by at most twice its score's error); and (1 + u) M 2^-16 for probabilities
in two terms of the type."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import DIM, HALF_STEP, HALF_TINY, bits
from tree_reference import SHAPES, attention, make_case, make_tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = DIM ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _run(c, **kw):
    return pa.paged_attn_tree(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["n"], c["parents"], SCALE, **kw)


def _check(c, out, skip=()):
    ref, mag, worst = attention(c, SCALE, skip)
    u = HALF_STEP[c["dtype"]]
    d = (out.double() - ref).abs()
    tol = u * ref.abs() + (1 + u) * mag * (worst * 2.0 ** -17 + 2.0 ** -15) + HALF_TINY[c["dtype"]]
    rows = np.concatenate([np.full(len(t), s not in skip) for s, t in enumerate(c["trees"])])
    rows = torch.from_numpy(rows).to(out.device)
    ok = torch.where(ref.isnan(), out.isnan(), d <= tol)[rows]
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} outside, worst {float((d / tol)[rows].nan_to_num(9e9).max()):.3f}"


HEADS = [(3, 3), (4, 2), (16, 8), (32, 8), (16, 2)]


def _trees(rng, sizes):
    return [make_tree(SHAPES[i % len(SHAPES)], n, rng) for i, n in enumerate(sizes)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_ragged_trees_and_contexts(dtype, hq, hkv):
    """Trees of one token up, contexts that end inside, at and just past pages and key tiles; no committed context."""
    rng = np.random.default_rng(hq)
    sizes = [1, 5, 16, 3, 31, 64, 1, 7, 2, 40, 12, 9]
    extra = [776, 0, 112, 124, 1, 63, 0, 1024, 127, 88, 130, 2039]
    _check_case = make_case(_trees(rng, sizes), [n + e for n, e in zip(sizes, extra)], hq, hkv, dtype, seed=hq + hkv)
    _check(_check_case, _run(_check_case))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("hq,hkv,n", [(8, 8, 256), (16, 8, 128), (32, 8, 100), (16, 2, 255), (8, 1, 200)])
def test_large_trees_of_every_shape(shape, hq, hkv, n):
    """Several query tiles; trees that reach over up to four key tiles."""
    rng = np.random.default_rng(n)
    trees = [make_tree(shape, n, rng), make_tree(shape, 17, rng), make_tree(shape, n - 3, rng)]
    c = make_case(trees, [n + 100, 17 + 300, n - 3], hq, hkv, "bf16", seed=n)
    _check(c, _run(c))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,ctx,n", [(16, 8, 40011, 9), (8, 1, 30000, 13), (32, 8, 20021, 64), (16, 2, 9999, 200),
                                          (1, 1, 50001, 1), (8, 1, 25000, 100)])
def test_one_long_context(dtype, hq, hkv, ctx, n):
    """One sequence over the whole GPU: pieces of every CTA, key blocks with several query tiles."""
    rng = np.random.default_rng(ctx)
    c = make_case([make_tree("random", n, rng)], [ctx], hq, hkv, dtype, seed=ctx)
    _check(c, _run(c))


def test_many_sequences_of_all_sizes():
    rng = np.random.default_rng(3)
    sizes = rng.integers(0, 9, 300)
    ctx = sizes + (np.exp(rng.uniform(0, 7, 300)).astype(int) - 1)
    c = make_case(_trees(rng, sizes.tolist()), ctx.tolist(), 16, 8, "bf16", seed=3)
    _check(c, _run(c, max_context_len=int(ctx.max())))


def test_the_most_sequences():
    rng = np.random.default_rng(4)
    sizes = rng.integers(1, 3, pa.MAX_TREE_SEQS)
    c = make_case(_trees(rng, sizes.tolist()), (sizes + rng.integers(0, 40, len(sizes))).tolist(), 4, 2, "f16", seed=4)
    _check(c, _run(c))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sharp_softmax(dtype):
    """Scores tens of units apart: the running maximum moves from tile to tile."""
    rng = np.random.default_rng(5)
    c = make_case(_trees(rng, [20, 33, 6]), [1500, 700, 3000], 16, 8, dtype, seed=5, peak=8.0)
    _check(c, _run(c))


def test_one_token_is_the_plain_decode():
    rng = np.random.default_rng(6)
    c = make_case([make_tree("chain", 1, rng) for _ in range(6)], [1, 16, 17, 500, 2000, 129], 16, 8, "bf16", seed=6)
    out = _run(c)
    _check(c, out)
    plain = pa.paged_attn_decode(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], SCALE)
    assert float((out.float() - plain.float()).abs().max()) <= 2 * 2.0 ** -8 * float(plain.float().abs().max())


def test_a_chain_is_the_causal_chunk():
    rng = np.random.default_rng(7)
    sizes, ctx = [100, 33], [1100, 33]
    c = make_case([make_tree("chain", n, rng) for n in sizes], ctx, 32, 8, "f16", seed=7)
    out = _run(c)
    _check(c, out)
    starts = torch.tensor([b - a for a, b in zip(sizes, ctx)], dtype=torch.int32, device=DEV)
    chunk = pa.paged_attn_prefill_chunk(c["q"], starts, c["n"], c["kc"], c["vc"], c["bt"], c["lens"], SCALE)
    assert float((out.float() - chunk.float()).abs().max()) <= 2e-3 + 1e-2 * float(chunk.float().abs().max())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("what", ["vc", "kc"])
def test_what_a_branch_does_not_see_has_no_effect(dtype, value, what):
    """Infinities and NaN in one drafted token's key or value: the rows that do not see it are as without it."""
    rng = np.random.default_rng(8)
    trees = [make_tree("full", 30, rng), make_tree("random", 9, rng)]
    c = make_case(trees, [30 + 110, 9 + 700], 16, 8, dtype, seed=8)
    clean = _run(c).clone()
    _check(c, clean)
    bad = 7
    pos = 110 + bad
    c[what][int(c["bt_h"][0, pos // 16]), pos % 16, 3, 17:19] = value
    out = _run(c)
    sees = np.zeros(39, bool)
    from tree_reference import ancestors
    sees[:30] = ancestors(trees[0])[:, bad]
    hit = np.zeros((39, 16), bool)
    hit[:, 6:8] = sees[:, None]  # the query heads of KV head 3
    hit = torch.from_numpy(hit).to(DEV)
    assert torch.equal(out[~hit], clean[~hit])
    if what == "vc":
        assert bool(out[hit].isnan().all())
    else:  # (an infinite key is a weight of 0, 1 or NaN: not finite scores end as NaN or as the rest)
        assert not bool((out[hit] == clean[hit]).all())


def test_rows_behind_and_refused_sequences_are_left():
    rng = np.random.default_rng(9)
    sizes = [4, 6, 5, 3, 8, 2]
    c = make_case(_trees(rng, sizes), [100, 60, 90, 300, 50, 700], 16, 8, "bf16", seed=9)
    good = _run(c).clone()
    q = torch.cat([c["q"], torch.full_like(c["q"][:5], float("nan"))])
    parents = torch.cat([c["parents"], torch.full_like(c["parents"][:5], 77)])
    lens, n = c["lens"].clone(), c["n"].clone()
    lens[1] = 5                              # shorter than its tree
    lens[3] = c["bt"].shape[1] * 16 + 1      # beyond the table
    out = torch.full_like(q, 3.0)
    pa.paged_attn_tree(q, c["kc"], c["vc"], c["bt"], lens, n, parents, SCALE, out=out)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail in (1, 3)
    first = np.concatenate([[0], np.cumsum(sizes)])
    for s in range(6):
        rows = slice(first[s], first[s + 1])
        assert torch.equal(out[rows], torch.full_like(out[rows], 3.0) if s in (1, 3) else good[rows])
    assert bool((out[28:] == 3.0).all())


def test_bad_tree_lengths():
    rng = np.random.default_rng(10)
    c = make_case(_trees(rng, [4, 6, 5]), [100, 60, 90], 4, 2, "f16", seed=10)
    good = _run(c).clone()
    for s, value, left in [(1, -1, None), (2, 6, [2]), (1, 257, [1, 2]), (0, 2 ** 31 - 1, [0, 1, 2])]:
        n = c["n"].clone()
        n[s] = value
        out = torch.full_like(good, 3.0)
        pa.paged_attn_tree(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], n, c["parents"], SCALE, out=out)
        st, detail = pa.get_device_error()
        assert pa.STATUS[st] == "PA_ERR_RANGE" and 0 <= detail < 3
        if left is not None:  # (a negative length moves the trees behind it: their rows are others')
            for i, rows in enumerate([slice(0, 4), slice(4, 10), slice(10, 15)]):
                assert torch.equal(out[rows], torch.full_like(out[rows], 3.0) if i in left else good[rows])


@pytest.mark.parametrize("bad", [3, 4, 2 ** 31 - 1, -2, -2 ** 31])
def test_a_bad_parent_is_reported_and_taken_as_none(bad):
    rng = np.random.default_rng(11)
    trees = [make_tree("chain", 6, rng), make_tree("chain", 5, rng)]
    c = make_case(trees, [500, 40], 16, 8, "bf16", seed=11)
    c["parents"][6 + 3] = bad
    out = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    trees[1][3] = -1
    _check(dict(c, trees=trees), out)


def test_a_bad_block_is_reported():
    rng = np.random.default_rng(12)
    c = make_case(_trees(rng, [6, 5, 9]), [500, 400, 300], 16, 8, "bf16", seed=12)
    good = _run(c).clone()
    c["bt"][1, 3] = c["kc"].shape[0]
    c["bt"][1, 7] = -4
    out = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    assert torch.equal(out[:6], good[:6]) and torch.equal(out[11:], good[11:])


def test_a_longer_sequence_than_the_bound_is_refused():
    rng = np.random.default_rng(13)
    c = make_case(_trees(rng, [6, 5]), [500, 400], 16, 8, "bf16", seed=13)
    good = _run(c).clone()
    out = torch.full_like(good, 3.0)
    _run(c, out=out, max_context_len=450)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 0
    assert bool((out[:6] == 3.0).all()) and torch.equal(out[6:], good[6:])


def test_no_rows():
    rng = np.random.default_rng(14)
    c = make_case(_trees(rng, [0, 0]), [50, 0], 16, 8, "bf16", seed=14)
    assert _run(c).shape == (0, 16, DIM)


def test_repeats_streams_and_graphs_agree():
    """The same bits again, on another stream, and from two captured calls that share a workspace in one graph."""
    rng = np.random.default_rng(15)
    c = make_case(_trees(rng, [9, 30, 4]), [3000, 700, 5000], 32, 8, "bf16", seed=15)
    d = make_case(_trees(rng, [64]), [9000], 32, 8, "f16", seed=16)
    ref_c, ref_d = _run(c).clone(), _run(d).clone()
    _check(c, ref_c)
    for _ in range(5):
        assert torch.equal(_run(c), ref_c)
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
    c["q"].mul_(0.5)  # a replay reads what is there then
    graph.replay()
    _check(c, oc)


def test_two_calls_on_two_streams():
    rng = np.random.default_rng(17)
    a = make_case(_trees(rng, [9, 30]), [30000, 700], 16, 8, "bf16", seed=17)
    b = make_case(_trees(rng, [5, 16, 2]), [8000, 70, 20000], 16, 8, "f16", seed=18)
    ref_a, ref_b = _run(a).clone(), _run(b).clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        x, y = _run(a, stream=s1), _run(b, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(x, ref_a) and torch.equal(y, ref_b)


def test_a_wide_block_table():
    """A table far wider than any context (offsets past 2^31 entries' bytes stay apart)."""
    rng = np.random.default_rng(19)
    c = make_case(_trees(rng, [5, 7]), [300, 100], 16, 8, "f16", seed=19, width=100000)
    _check(c, _run(c, max_context_len=1024))


@pytest.mark.parametrize("hq,hkv", [(8, 8), (16, 2)])
def test_bindings_refuse(hq, hkv):
    rng = np.random.default_rng(20)
    c = make_case(_trees(rng, [5, 7]), [300, 100], hq, hkv, "f16", seed=20)
    with pytest.raises(TypeError):
        pa.paged_attn_tree(c["q"].bfloat16(), c["kc"], c["vc"], c["bt"], c["lens"], c["n"], c["parents"], SCALE)
    with pytest.raises(TypeError):
        pa.paged_attn_tree(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["n"], c["parents"].long(), SCALE)
    with pytest.raises(ValueError):
        pa.paged_attn_tree(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["n"], c["parents"][:-1], SCALE)
    with pytest.raises(ValueError):
        pa.paged_attn_tree(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["n"][:1], c["parents"], SCALE)
    with pytest.raises(ValueError):
        pa.paged_attn_tree(c["q"][:, :, :64], c["kc"], c["vc"], c["bt"], c["lens"], c["n"], c["parents"], SCALE)
    with pytest.raises(ValueError):
        _run(c, out=c["q"][:3].clone())
    with pytest.raises(pa.PagedAttnError):
        _run(c, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert np.array_equal(bits(_run(c)), bits(_run(c)))
