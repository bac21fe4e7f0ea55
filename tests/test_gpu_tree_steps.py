"""Steps of speculative decoding over one cache as a user runs them: drafts rotated and
written, attended as trees, judged, the cache compacted, the next step on what is left;
against the same tokens one by one (plain decode over a cache of its own)."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import DIM, bits
from tree_reference import accept, make_tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = DIM ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return np.array(d)


class Model:
    """Queries, keys and values of a token from its number alone, per layer (what is tested is the cache)."""

    def __init__(self, layers, hq, hkv, dtype, vocab, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda n: torch.randn((layers, vocab, n, DIM), generator=g, device=DEV).to(dtype)
        self.q, self.k, self.v = r(hq), r(hkv), r(hkv)


@pytest.mark.parametrize("dtype,hq,hkv", [(torch.bfloat16, 32, 8), (torch.float16, 16, 8)])
def test_drafted_steps_leave_the_cache_of_single_steps(dtype, hq, hkv):
    layers, vocab, steps = 3, 23, 6
    model = Model(layers, hq, hkv, dtype, vocab, seed=1)
    rng = np.random.default_rng(2)
    inv, factor = pa.rope_inv_freq(DIM, 1e4)
    axes = pa.rope_axes([16, 24, 24])
    starts = [37, 16, 120, 5]
    S = len(starts)
    alloc = pa.BlockAllocator(200)
    pools = [tuple(torch.zeros((200, 16, hkv, DIM), dtype=dtype, device=DEV) for _ in range(2)) for _ in range(layers)]
    handle = pa.layer_pools(pools)
    seqs = [alloc.sequence() for _ in range(S)]
    tokens = [[int(x) for x in rng.integers(0, vocab, n)] for n in starts]
    cu = lambda x, d=np.int32: torch.from_numpy(np.asarray(x).astype(d)).to(DEV)

    def write(slots, ids, pos):
        """Every layer's rows of these tokens; the queries of each."""
        p3 = cu(np.stack([pos, pos + 1, pos + 2]))  # three axes, apart
        return [pa.rope_kv_write_axes(model.q[la][ids], model.k[la][ids], model.v[la][ids], inv, p3, axes,
                                      cu(slots, np.int64), *pools[la], attention_factor=factor) for la in range(layers)]

    for s, t in zip(seqs, tokens):
        write(s.reserve(len(t)), torch.tensor(t, device=DEV), np.arange(len(t)))
        s.commit(len(t))
    accepted = 0
    for step in range(steps):
        shapes = [("random", "full", "chain", "forest")[(i + step) % 4] for i in range(S)]
        trees = [make_tree(shape, int(rng.integers(1, 14)), rng) for shape in shapes]
        drafts = [rng.integers(0, 3, len(t)) for t in trees]
        slots = [s.reserve(len(t)) for s, t in zip(seqs, trees)]
        bt, _, tree_lens, lens = pa.build_step_tables(seqs, 24)
        bt, tree_lens, lens = cu(bt), cu(tree_lens), cu(lens)
        ids = torch.from_numpy(np.concatenate(drafts)).to(DEV)
        pos = np.concatenate([s.length + _depths(t) for s, t in zip(seqs, trees)])
        queries = write(np.concatenate(slots), ids, pos)
        parents = cu(np.concatenate(trees))
        outs = [pa.paged_attn_tree(queries[la], *pools[la], bt, lens, tree_lens, parents, SCALE)
                for la in range(layers)]
        # what the "model" chooses after each token: any function of the outputs that is the same below
        target = (outs[-1].float().sum((1, 2)).abs() * 64).long() % 3
        path, num, nxt, new_lens = pa.tree_accept(ids, target, parents, tree_lens, lens, handle, bt, max_tree_len=16)
        at = 0
        for i, s in enumerate(seqs):
            n = len(trees[i])
            way, after = accept(trees[i], drafts[i], target[at:at + n].cpu().numpy())
            assert path[i, :int(num[i])].tolist() == way and int(nxt[i]) == after
            s.commit(n)
            s.truncate(int(new_lens[i]))
            tokens[i] += [int(drafts[i][a]) for a in way]
            assert s.length == len(tokens[i]) == int(new_lens[i])
            accepted += len(way)
            at += n
    assert accepted > 2 * steps * S // 2
    # the same tokens written in one go into another cache: the same rows, and a decode over either gives the same
    other = pa.BlockAllocator(200)
    pools2 = [tuple(torch.zeros_like(x) for x in pair) for pair in pools]
    seqs2 = [other.sequence() for _ in range(S)]
    pools, mine = pools2, pools
    for s, t in zip(seqs2, tokens):
        write(s.reserve(len(t)), torch.tensor(t, device=DEV), np.arange(len(t)))
        s.commit(len(t))
    for s, s2, t in zip(seqs, seqs2, tokens):
        n = len(t)
        rows = lambda pair, q: [x[torch.tensor(q.blocks, device=DEV).long()].flatten(0, 1)[:n] for x in pair]
        for la in range(layers):
            for a, b in zip(rows(mine[la], s), rows(pools[la], s2)):
                assert np.array_equal(bits(a), bits(b))
    q = model.q[0][torch.tensor([t[-1] for t in tokens], device=DEV)].contiguous()
    got = []
    for pair, group in ((mine[0], seqs), (pools[0], seqs2)):
        for s in group:
            s.reserve(1)
        bt, _, _, lens = pa.build_step_tables(group, 24)
        got.append(pa.paged_attn_decode(q, *pair, cu(bt), cu(lens - 1), SCALE))
    assert torch.equal(got[0], got[1])


def test_a_captured_step():
    """Write, attention over two layers' pools, judgement and compaction in one graph, replayed on new drafts."""
    rng = np.random.default_rng(5)
    g = torch.Generator(device=DEV).manual_seed(5)
    S, n, hq, hkv = 3, 9, 16, 8
    trees = [make_tree("random", n, rng) for _ in range(S)]
    ctx = np.array([100, 48, 700])
    pages = [-(-int(c) // 16) for c in ctx]
    bt = np.full((S, max(pages)), -1, np.int32)
    at = 0
    for s in range(S):
        bt[s, :pages[s]] = np.arange(at, at + pages[s])
        at += pages[s]
    start = torch.randn((2, 2, at, 16, hkv, DIM), generator=g, device=DEV).half()
    pool = start.clone()
    cu = lambda x, d=np.int32: torch.from_numpy(np.asarray(x).astype(d)).to(DEV)
    slots = np.concatenate([bt[s, np.arange(c - n, c) // 16].astype(np.int64) * 16 + np.arange(c - n, c) % 16
                            for s, c in enumerate(ctx)])
    pos = np.concatenate([c - n + _depths(t) for c, t in zip(ctx, trees)])
    r = lambda h: torch.randn((S * n, h, DIM), generator=g, device=DEV).half()
    q, k, v = r(hq), r(hkv), r(hkv)
    draft, target = cu(rng.integers(0, 2, S * n), np.int64), cu(rng.integers(0, 2, S * n), np.int64)
    a = dict(bt=cu(bt), lens=cu(ctx), n=cu([n] * S), parents=cu(np.concatenate(trees)), pos=cu(np.stack([pos] * 3)),
             slots=cu(slots, np.int64))
    inv, _ = pa.rope_inv_freq(DIM, 1e4)
    handle = pa.layer_pools([(pool[0, 0], pool[0, 1]), (pool[1, 0], pool[1, 1])])
    ws = pa.alloc_tree_workspace(S, hq, hkv)

    def step():
        outs = []
        for la in range(2):
            kc, vc = pool[la]
            rq = pa.rope_kv_write_axes(q, k, v, inv, a["pos"], pa.rope_axes([64, 0, 0]), a["slots"], kc, vc)
            outs.append(pa.paged_attn_tree(rq, kc, vc, a["bt"], a["lens"], a["n"], a["parents"], SCALE, workspace=ws))
        return outs + list(pa.tree_accept(draft, target, a["parents"], a["n"], a["lens"], handle, a["bt"],
                                          max_tree_len=n))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(3):
        new = np.random.default_rng(seed)
        draft.copy_(cu(new.integers(0, 2, S * n), np.int64))
        target.copy_(cu(new.integers(0, 2, S * n), np.int64))
        k.normal_(generator=g)
        pool.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        got, after = [x.clone() for x in captured], pool.clone()
        pool.copy_(start)
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(after, pool)
