"""GPU checks of pa_paged_attn_decode_shared against a plain form in 64 bits and
against the plain decode over the same tables.

Tolerance of an output element, with u the type's half step and M = sum |p v|:
u |ref| for its rounding; (1 + u) M (a 2^-17 + 2^-16) for fp32 scores, exponentials
and sums, a = scale sum |q_i k_i| (each score is summed at most 40 roundings deep and a
weight moves by at most twice its score's error); and (1 + u) M u where the
probabilities are rounded once to the type (groups of more than 128 query rows per KV
head; elsewhere two terms leave M 2^-16, of the same order as the second)."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import DIM, HALF_STEP, HALF_TINY, TORCH, attention_torch, random_pool

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = DIM ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _case(groups, hq, hkv, dtype, seed, alone=(), peak=1.0, width=0):
    """groups: [(prefix length, [suffix lengths])]; alone: lengths of sequences behind the last group."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    lens = [p + n for p, suf in groups for n in suf] + list(alone)
    pages = [-(-n // 16) for n in lens]
    need = sum(p // 16 for p, _ in groups) + sum(-(-n // 16) for _, suf in groups for n in suf) + \
        sum(-(-n // 16) for n in alone)
    nb = need + 3
    perm = rng.permutation(nb)
    bt = np.full((len(lens), max(max(pages + [1]), width)), -1, np.int32)
    at = s = 0
    for p, suf in groups:
        head = perm[at:at + p // 16]
        at += p // 16
        for n in suf:
            own = -(-n // 16)
            bt[s, :p // 16] = head
            bt[s, p // 16:p // 16 + own] = perm[at:at + own]
            at += own
            s += 1
    for n in alone:
        own = -(-n // 16)
        bt[s, :own] = perm[at:at + own]
        at += own
        s += 1
    kc, vc = random_pool(g, nb, hkv, dtype), random_pool(g, nb, hkv, dtype)
    live = torch.zeros((nb, 16), dtype=torch.bool)
    for i, n in enumerate(lens):
        pos = np.arange(n)
        live[bt[i, pos // 16], pos % 16] = True
    kc[~live.to(DEV)] = float("nan")  # slots that hold no token
    vc[~live.to(DEV)] = float("nan")
    q = (torch.randn((len(lens), hq, DIM), generator=g, device=DEV) * peak).to(TORCH[dtype])
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device=DEV)
    return dict(q=q, kc=kc, vc=vc, bt=i32(bt), lens=i32(lens), sizes=i32([len(s) for _, s in groups]),
                prefix=i32([p for p, _ in groups]), bt_h=bt, lens_h=lens, dtype=dtype,
                one_term=any(len(s) * (hq // hkv) > 128 for _, s in groups))


def _run(c, **kw):
    return pa.paged_attn_decode_shared(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["sizes"], c["prefix"], SCALE,
                                       **kw)


def _check(c, out, rows=None):
    ref, mag, worst = attention_torch(c["q"], c["kc"], c["vc"], c["bt_h"], c["lens_h"], SCALE)
    u = HALF_STEP[c["dtype"]]
    rel = worst * 2.0 ** -17 + 2.0 ** -16 + (u if c["one_term"] else 2.0 ** -16)
    d = (out.double() - ref).abs()
    tol = u * ref.abs() + (1 + u) * mag * rel + HALF_TINY[c["dtype"]]
    ok = d <= tol
    if rows is not None:
        ok = ok[rows]
    assert bool(ok.all()), f"worst {float((d / tol).nan_to_num(9e9).max()):.3f} of the tolerance"


HEADS = [(3, 3), (4, 2), (16, 8), (32, 8), (16, 2)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_prefix_ends_and_ragged_suffixes(dtype, hq, hkv):
    """Prefixes that end inside, at and just past a key tile; suffixes of one token to several pages."""
    c = _case([(16, [1, 2, 17]), (128, [5, 1]), (144, [16, 33, 1, 400]), (112, [3, 3]), (1024, [1, 90]),
               (2064, [7, 250, 16])], hq, hkv, dtype, seed=hq + hkv)
    _check(c, _run(c))


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("size", [2, 31, 33, 64, 65, 130])
def test_one_group_of_every_tile_count(hq, hkv, size):
    rng = np.random.default_rng(size)
    c = _case([(848, rng.integers(1, 40, size).tolist())], hq, hkv, "bf16", seed=size)
    _check(c, _run(c))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_prefix_few_sequences(dtype):
    c = _case([(40000, [1, 700, 16])], 16, 8, dtype, seed=1)
    _check(c, _run(c))


@pytest.mark.parametrize("sizes", [[100, 60], [40, 2, 90, 33]])
def test_long_prefixes_several_query_tiles(sizes):
    rng = np.random.default_rng(len(sizes))
    c = _case([(int(rng.integers(20, 500)) * 16, rng.integers(1, 90, n).tolist()) for n in sizes], 32, 8, "bf16",
              seed=len(sizes))
    _check(c, _run(c))


def test_many_groups():
    rng = np.random.default_rng(5)
    groups = [(int(rng.integers(0, 12)) * 16, rng.integers(1, 50, int(rng.integers(1, 6))).tolist())
              for _ in range(pa.MAX_PREFIX_GROUPS)]
    c = _case(groups, 8, 2, "bf16", seed=6)
    _check(c, _run(c))


def test_sequences_behind_the_groups_and_groups_that_share_nothing():
    c = _case([(256, [1, 30]), (0, [40, 500, 3]), (512, [9]), (160, [4, 4, 4])], 16, 4, "f16", seed=7,
              alone=[1, 16, 900, 2500])
    _check(c, _run(c))
    none = dict(c, sizes=c["sizes"][:0], prefix=c["prefix"][:0])
    plain = pa.paged_attn_decode(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], SCALE)
    out = _run(none)
    _check(none, out)
    _check(c, plain)


def test_context_equal_to_the_prefix():
    """No suffix at all for some members, then for every one (no split work)."""
    c = _case([(128, [0, 3, 0]), (32, [1, 0])], 16, 8, "bf16", seed=8)
    _check(c, _run(c))
    c = _case([(400, [0, 0, 0, 0])], 16, 8, "bf16", seed=9)
    _check(c, _run(c))


def test_only_the_first_table_is_read_for_the_prefix():
    c = _case([(320, [20, 30, 40])], 8, 4, "bf16", seed=10)
    want = _run(c)
    c["bt"][1:, :20] = -1
    assert torch.equal(_run(c), want)


def test_peaked_rows():
    """Large queries: maxima that move from key tile to key tile (the accumulators are rescaled)."""
    for size in (6, 80):
        c = _case([(3000 // 16 * 16, [10] * size)], 32, 8, "bf16", seed=11, peak=16.0)
        _check(c, _run(c))


def test_rising_maxima():
    """Keys aligned with the query more and more from tile to tile: every key tile raises the maximum."""
    c = _case([(1280, [5] * 40)], 4, 1, "f16", seed=12)
    d = torch.randn(DIM, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    d = d / d.norm() * 4
    c["q"] = (c["q"].float() * 0.2 + d * 4).half()
    rows = c["bt"][0, :80].long()
    ramp = torch.linspace(0, 3, 1280, device=DEV).view(80, 16, 1, 1)
    c["kc"][rows] = (c["kc"][rows].float() * 0.2 + ramp * d).half()
    _check(c, _run(c))


def test_bad_groups_share_nothing():
    good = _case([(256, [1, 30]), (128, [40, 50, 3]), (64, [9, 8])], 16, 4, "f16", seed=13)
    for what, (sizes, prefix, bad) in dict(
            negative_length=([2, 3, 2], [256, -16, 64], 1), odd_length=([2, 3, 2], [256, 100, 64], 1),
            beyond_the_table=([2, 3, 2], [256, 16 * good["bt"].shape[1] + 16, 64], 1),
            negative_size=([2, 3, -2], [256, 128, 64], 2), too_many=([2, 3, 3], [256, 128, 64], 2),
            huge=([2, 3, 2 ** 31 - 1], [256, 128, 64], 2)).items():
        c = dict(good, sizes=torch.tensor(sizes, dtype=torch.int32, device=DEV),
                 prefix=torch.tensor(prefix, dtype=torch.int32, device=DEV))
        out = _run(c)
        st, detail = pa.get_device_error()
        assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == bad, what
        _check(c, out)


def test_bad_sequences_are_left():
    c = _case([(256, [1, 30, 5]), (128, [40, 50, 3])], 16, 4, "f16", seed=14, alone=[50])
    for value, which in ((240, 1), (0, 4), (16 * c["bt"].shape[1] + 1, 6), (-5, 2)):
        lens = c["lens"].clone()
        lens[which] = value
        out = torch.full_like(c["q"], 7.0)
        _run(dict(c, lens=lens), out=out)
        st, detail = pa.get_device_error()
        assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == which
        assert (out[which] == 7.0).all()
        _check(c, out, rows=[i for i in range(7) if i != which])


def test_bad_blocks_are_reported():
    c = _case([(256, [1, 30, 5])], 16, 4, "bf16", seed=15, alone=[50])
    c["bt"][0, 3] = 10 ** 6     # a page of the prefix
    out = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 0
    _check(c, out, rows=[3])
    c["bt"][0, 3] = int(c["bt_h"][0, 3])
    c["bt"][1, 17] = -7         # a page of one suffix
    out = _run(c)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    _check(c, out, rows=[0, 2, 3])


def test_workspace_needs_no_clearing_and_calls_repeat():
    a = _case([(2000, [1, 30, 5] * 20), (512, [9] * 3)], 32, 8, "bf16", seed=16)
    b = _case([(64, [3, 4])], 32, 8, "bf16", seed=17)
    ws = pa.alloc_decode_shared_workspace(63, 2, 32, 8)
    ws.fill_(0xff)
    first = _run(a, workspace=ws)
    small = _run(b, workspace=ws)
    again = _run(a, workspace=ws)
    assert torch.equal(first, again)
    _check(a, again)
    _check(b, small)


def test_stream_graph_and_writes_right_before():
    """Captured behind the KV write of the step's tokens and replayed with other queries and tokens."""
    c = _case([(512, [17, 30, 5] * 4)], 16, 8, "f16", seed=18)
    S = 12
    ws = pa.alloc_decode_shared_workspace(S, 1, 16, 8)
    out = torch.zeros_like(c["q"])
    k, v = (torch.randn((S, 8, DIM), device=DEV).half() for _ in range(2))
    pos = torch.tensor(c["lens_h"], device=DEV) - 1
    slots = torch.gather(c["bt"].long(), 1, (pos // 16)[:, None])[:, 0] * 16 + pos % 16

    def step():
        pa.kv_cache_write(k, v, slots, c["kc"], c["vc"])
        _run(c, out=out, workspace=ws, max_context_len=544)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    _check(c, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            step()
    for i in range(4):
        gen = torch.Generator(device=DEV).manual_seed(i)
        c["q"].copy_(torch.randn(c["q"].shape, generator=gen, device=DEV))
        k.copy_(torch.randn(k.shape, generator=gen, device=DEV))
        v.copy_(torch.randn(k.shape, generator=gen, device=DEV))
        out.zero_()
        g.replay()
        _check(c, out)


def test_many_layers_back_to_back():
    """Thirty calls in a row on one workspace, each reading the one before's output as its query."""
    c = _case([(1024, [20] * 36), (300 // 16 * 16, [5, 6])], 32, 8, "bf16", seed=19)
    ws = pa.alloc_decode_shared_workspace(38, 2, 32, 8)
    q = c["q"]
    for _ in range(30):
        q = (_run(dict(c, q=q), workspace=ws).float() * 8).bfloat16()
    before = q
    out = _run(dict(c, q=before), workspace=ws)
    _check(dict(c, q=before), out)


def test_empty_batch():
    c = _case([(64, [3, 4])], 16, 8, "bf16", seed=20)
    e = dict(c, q=c["q"][:0], bt=c["bt"][:0], lens=c["lens"][:0])
    assert _run(e).shape[0] == 0


def test_with_the_allocator():
    """A prefix adopted by reference, one token per sequence and step."""
    hq, hkv, S = 16, 8, 5
    alloc = pa.BlockAllocator(128)
    donor = alloc.sequence()
    g = torch.Generator(device=DEV).manual_seed(22)
    kc, vc = (torch.full((128, 16, hkv, DIM), float("nan"), device=DEV).half() for _ in range(2))
    slots = donor.reserve(320)
    donor.commit(320)
    new = lambda n: (torch.randn((n, hkv, DIM), generator=g, device=DEV).half() for _ in range(2))
    pa.kv_cache_write(*new(320), torch.tensor(slots, device=DEV), kc, vc)
    seqs = [alloc.sequence() for _ in range(S)]
    for s in seqs:
        s.adopt_prefix(donor.blocks)
    one = lambda x: torch.tensor([x], dtype=torch.int32, device=DEV)
    for step in range(20):
        slots = [s.reserve(1)[0] for s in seqs]
        bt, _, _, ctx = pa.build_step_tables(seqs, 24)
        pa.kv_cache_write(*new(S), torch.tensor(slots, device=DEV), kc, vc)
        q = torch.randn((S, hq, DIM), generator=g, device=DEV).half()
        c = dict(q=q, kc=kc, vc=vc, bt=torch.from_numpy(bt).to(DEV), lens=torch.from_numpy(ctx).to(DEV), bt_h=bt,
                 lens_h=ctx, sizes=one(S), prefix=one(320), dtype="f16", one_term=False)
        _check(c, _run(c))
        for s in seqs:
            s.commit(1)
