"""GPU checks of pa_kv_evict against a plain form in 64 bits.  Everything it
returns is a selection or a copy, so every comparison is exact."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import bits, evict_keep, place, random_pool

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _weights(rng, shape, kind):
    w = rng.random(shape, np.float32)
    if kind == "ties":
        w = np.floor(w * 3).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":
        w = np.where(w < 0.9, 0.0, w).astype(np.float32)
        w[w == 0] *= rng.choice([1.0, -1.0], int((w == 0).sum())).astype(np.float32)  # both zeros, equal
    elif kind == "odd":  # any sign, infinities, NaN, subnormals
        w = (w - 0.5).astype(np.float32)
        pick = rng.random(shape)
        w[pick < 0.10] = np.nan
        w[(pick >= 0.10) & (pick < 0.15)] = np.inf
        w[(pick >= 0.15) & (pick < 0.25)] = -np.inf
        w[(pick >= 0.25) & (pick < 0.35)] = 1e-42
    elif kind == "near":  # neighbours in the last bits: every radix pass decides
        w = (np.float32(1.0).view(np.int32) + rng.integers(0, 300, shape)).astype(np.int32).view(np.float32)
    return w


def _case(lens, hkv, dtype, seed, budget, kind="random", in_place=False, stride=None):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    left = np.minimum(lens, budget)
    bt, nb = place(rng, lens, extra=0)
    if in_place:
        dst, total = bt, nb + 2
    else:
        dst, total = place(rng, left, extra=2, first=nb)
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = _weights(rng, (len(lens), hkv, stride or int(lens.max())), kind)
    c = dict(lens=lens, hkv=hkv, budget=budget, bt=bt, dst=dst, w=w, kc=random_pool(g, total, hkv, dtype),
             vc=random_pool(g, total, hkv, dtype))
    c["dev"] = {n: torch.from_numpy(np.array(c[n])).to(DEV) for n in ("lens", "bt", "dst", "w")}
    return c


def _expect(c, recent, sinks, w_out, skip=()):
    S, hkv, budget = len(c["lens"]), c["hkv"], c["budget"]
    kept = np.full((S, hkv, budget), -1, np.int32)
    k, v = bits(c["kc"]), bits(c["vc"])
    k0, v0 = k.copy(), v.copy()
    w_out = w_out.copy()
    for s in range(S):
        if s in skip:
            continue
        n = int(c["lens"][s])
        for h in range(hkv):
            at = evict_keep(c["w"][s, h], n, budget, recent, sinks)
            m = len(at)
            kept[s, h, :m] = at
            to = c["dst"][s][np.arange(m) // 16], np.arange(m) % 16, h
            src = c["bt"][s][at // 16], at % 16, h
            k[to], v[to] = k0[src], v0[src]
            w_out[s, h, :m] = c["w"][s, h, at]
            w_out[s, h, m:min(n, w_out.shape[2])] = 0
    return kept, k, v, w_out


def _run(c, recent, sinks, in_place=False, out_stride=None, **kw):
    d = c["dev"]
    w_out = None if in_place else torch.full((len(c["lens"]), c["hkv"], out_stride or c["budget"]), 7.0, device=DEV)
    before = (c["w"] if in_place else w_out.cpu().numpy()).copy()
    kept, new = pa.kv_evict(c["kc"], c["vc"], d["bt"], d["lens"], d["w"], c["budget"], recent=recent, sinks=sinks,
                            dst_block_tables=None if in_place else d["dst"], weights_out=w_out, **kw)
    return kept, new, (d["w"] if in_place else w_out), before


def _check(c, recent, sinks, in_place=False, out_stride=None):
    d = c["dev"]
    before = c["w"] if in_place else np.full((len(c["lens"]), c["hkv"], out_stride or c["budget"]), 7.0, np.float32)
    kept, k, v, w_out = _expect(c, recent, sinks, before)
    got_kept, new, got_w, _ = _run(c, recent, sinks, in_place, out_stride)
    assert np.array_equal(new.cpu().numpy(), np.minimum(c["lens"], c["budget"]))
    assert np.array_equal(got_kept.cpu().numpy(), kept)
    assert np.array_equal(bits(c["kc"]), k) and np.array_equal(bits(c["vc"]), v)
    assert np.array_equal(got_w.cpu().numpy().view(np.int32), w_out.view(np.int32))
    if not in_place:
        assert np.array_equal(d["w"].cpu().numpy().view(np.int32), c["w"].view(np.int32))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "zeros", "odd", "near"])
def test_weights_of_every_kind(in_place, kind):
    c = _case([700, 33, 5, 257, 1, 64], 3, "bf16", 11, 64, kind, in_place)
    _check(c, recent=9, sinks=3, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (17, 17, 0), (16, 0, 16),
                                                 (40, 20, 20), (333, 5, 0), (2048, 100, 4), (5000, 0, 0)])
def test_budgets(in_place, budget, recent, sinks):
    c = _case([2600, 16, 17, 2049], 2, "f16", budget, budget, "random", in_place)
    _check(c, recent, sinks, in_place=in_place)


@pytest.mark.parametrize("S,hkv,ctx", [(1, 1, 40000), (1, 8, 30001), (20, 3, 900), (60, 2, 1500), (160, 1, 301),
                                       (40, 8, 200), (1, 1, 200000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_every_cluster_size_and_long_slices(S, hkv, ctx, in_place):
    rng = np.random.default_rng(S)
    lens = rng.integers(1, ctx + 1, S)
    lens[-1] = ctx
    c = _case(lens, hkv, "bf16", S, max(1, ctx // 3), "random", in_place)
    _check(c, recent=ctx // 50, sinks=min(4, ctx // 10), in_place=in_place)


def test_slices_past_shared_memory_in_place():
    """160 sequences take one CTA each, so a long one overflows the keys kept in shared memory."""
    lens = np.full(160, 20)
    lens[3], lens[90] = 50000, 16385
    c = _case(lens, 1, "bf16", 77, 9000, "ties", in_place=True)
    _check(c, recent=100, sinks=7, in_place=True)


@pytest.mark.parametrize("ctx", [700, 5000, 140000])
@pytest.mark.parametrize("more", [0, 1, 20, 300])
def test_infinite_weights_beside_tokens_that_stay_anyway(ctx, more):
    """The leading bits of +inf and of the largest numbers are those of no other weight, and are held apart from the
    first and last tokens' whatever those weigh: as many heavy tokens as may stay, a few more, many more."""
    rng = np.random.default_rng(ctx + more)
    budget, recent, sinks = 100, 30, 10
    c = _case([ctx], 2, "bf16", 31, budget)
    mid = np.arange(sinks, ctx - recent)
    for h in range(2):
        heavy = rng.choice(mid, budget - recent - sinks + more, replace=False)
        c["w"][0, h, heavy] = np.inf if h else np.float32(3.4e38)
    c["dev"]["w"].copy_(torch.from_numpy(c["w"]))
    _check(c, recent, sinks)


@pytest.mark.parametrize("ctx", [3000, 20000, 150000])
@pytest.mark.parametrize("ties", [2, 31, 32, 33, 200])
def test_ties_at_the_border_among_distinct_weights(ctx, ties):
    rng = np.random.default_rng(ctx + ties)
    budget = 257
    c = _case([ctx], 2, "f16", 41, budget, stride=ctx + 3)  # (rows that do not start on 16 bytes)
    c["w"][0, :, :ctx] = np.float32(1) + rng.permutation(ctx).astype(np.float32) / ctx
    order = np.argsort(-c["w"][0, 0, :ctx])
    c["w"][0, :, order[budget - 5 - 1:budget - 5 - 1 + ties]] = c["w"][0, 0, order[budget - 6]]
    c["dev"]["w"].copy_(torch.from_numpy(c["w"]))
    _check(c, 0, 5)


def test_wider_and_narrower_weights():
    c = _case([300, 20], 2, "f16", 5, 64, stride=513)
    _check(c, 8, 2, out_stride=200)
    c = _case([300, 20], 2, "f16", 6, 64, in_place=True, stride=513)
    _check(c, 8, 2, in_place=True)


def test_bad_sequences_are_reported_and_left():
    c = _case([100, 90, 80, 70], 2, "bf16", 9, 32)
    for what, value in (("zero", 0), ("beyond its table", 16 * c["bt"].shape[1] + 1), ("beyond the weights", 101)):
        lens = c["lens"].copy()
        lens[1] = value
        x = dict(c, kc=c["kc"].clone(), vc=c["vc"].clone(), lens=lens)
        x["dev"] = dict(c["dev"], lens=torch.from_numpy(lens).to(DEV))
        kept0 = torch.full((4, 2, 32), 5, dtype=torch.int32, device=DEV)
        new0 = torch.full((4,), 6, dtype=torch.int32, device=DEV)
        exp_kept, k, v, _ = _expect(x, 4, 2, np.zeros((4, 2, 32), np.float32), skip=(1,))
        kept, new, _, _ = _run(x, 4, 2, kept=kept0, new_context_lens=new0)
        st, detail = pa.get_device_error()
        assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1, what
        exp_kept[1] = 5
        assert np.array_equal(kept.cpu().numpy(), exp_kept), what
        assert new.cpu().tolist() == [32, 6, 32, 32]
        assert np.array_equal(bits(x["kc"]), k) and np.array_equal(bits(x["vc"]), v)


def test_bad_block_ids_are_reported_and_their_rows_left():
    c = _case([100, 90], 1, "bf16", 10, 90)
    c["dev"]["bt"][0, 2] = 10 ** 6
    c["dev"]["dst"][1, 1] = -1
    k0 = bits(c["kc"])
    kept, k, v, _ = _expect(c, 4, 2, np.zeros((2, 1, 90), np.float32))
    got, new, _, _ = _run(c, 4, 2)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail in (0, 1)
    assert np.array_equal(got.cpu().numpy(), kept)
    k[c["dst"][1, 1]] = k0[c["dst"][1, 1]]
    for i, j in enumerate(kept[0, 0]):  # rows whose source page is bad stay what they were
        if j // 16 == 2:
            k[c["dst"][0, i // 16], i % 16] = k0[c["dst"][0, i // 16], i % 16]
    assert np.array_equal(bits(c["kc"]), k)


def test_stream_graph_and_repeat():
    c = _case([700, 33, 5, 257], 4, "bf16", 12, 64)
    kept, k, v, w_out = _expect(c, 9, 3, np.full((4, 4, 64), 7.0, np.float32))
    d = c["dev"]
    w = torch.full((4, 4, 64), 7.0, device=DEV)
    out = [torch.empty((4, 4, 64), dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int32, device=DEV)]
    call = lambda stream=None: pa.kv_evict(c["kc"], c["vc"], d["bt"], d["lens"], d["w"], 64, 9, 3, d["dst"], w, *out,
                                           stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        c["kc"].view(torch.int16)[c["dst"].ravel()[0]] = 0
        out[0].zero_(), out[1].zero_()
        g.replay()
        assert np.array_equal(out[0].cpu().numpy(), kept)
        assert np.array_equal(bits(c["kc"]), k) and np.array_equal(bits(c["vc"]), v)


def test_evict_with_the_allocator():
    """Two sequences on shared blocks; one is shortened in place after it got blocks of its own."""
    hkv, n, budget = 2, 100, 40
    alloc = pa.BlockAllocator(32)
    a, b = alloc.sequence(), alloc.sequence()
    a.reserve(n)
    a.commit(n)
    b.fork_from(a)
    g = torch.Generator(device=DEV).manual_seed(3)
    kc, vc = random_pool(g, 32, hkv, "bf16"), random_pool(g, 32, hkv, "bf16")
    k0, v0 = bits(kc), bits(vc)
    w = torch.rand((1, hkv, n), generator=g, device=DEV)
    w_h = w.cpu().numpy().copy()
    old = list(b.blocks)
    b.unshare(-(-budget // 16))
    pairs = alloc.take_copies()
    assert [p[0] for p in pairs] == old[:3] and b.blocks[3:] == old[3:]
    pa.kv_block_copy([(kc, vc)], torch.tensor(pairs, dtype=torch.int32, device=DEV))
    table = torch.tensor([b.blocks], dtype=torch.int32, device=DEV)
    kept, new = pa.kv_evict(kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), w, budget, 8, 2)
    b.truncate(int(new[0]))
    assert b.length == budget and len(b.blocks) == 3 and a.length == n
    assert alloc.stats()["shared"] == 0 and alloc.stats()["used"] == 7 + 3
    k1, v1 = bits(kc), bits(vc)
    for blk in a.blocks:
        assert np.array_equal(k1[blk], k0[blk]) and np.array_equal(v1[blk], v0[blk])
    for h in range(hkv):
        at = evict_keep(w_h[0, h], n, budget, 8, 2)
        assert np.array_equal(kept[0, h].cpu().numpy(), at)
        for i, j in enumerate(at):
            assert np.array_equal(k1[b.blocks[i // 16], i % 16, h], k0[old[j // 16], j % 16, h])
            assert np.array_equal(v1[b.blocks[i // 16], i % 16, h], v0[old[j // 16], j % 16, h])
