"""GPU checks of pa_paged_attn_decode_weights against a plain form in 64 bits,
alone and in the loop it is made for: rotated keys written, a decode that
accumulates, an eviction by what it accumulated, and on.

Tolerances.  A score's fp32 error: its 128 products are summed at most 40 roundings
deep, so it is off by at most a 2^-18.6 where a = scale sum |q_i k_i| (its
products' magnitudes); a softmax weight moves by at most twice that relatively (its own
score and its row's sum), and the exponential, the sums of l over at most 2^12 keys of
one lane, the merges and the division add less than 2^-16 together.  So a weight is
off by at most (a 2^-17 + 2^-16) relatively, an output by as much of sum |p v|, plus
one rounding to its type."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import (DIM, HALF_STEP, HALF_TINY, TORCH, attention, bits, evict_keep, f64, gather, place,
                               random_pool, rotate)

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = DIM ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _case(lens, hq, hkv, dtype, seed, peak=1.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    lens = np.asarray(lens, np.int32)
    bt, nb = place(rng, lens)
    kc, vc = random_pool(g, nb, hkv, dtype), random_pool(g, nb, hkv, dtype)
    live = torch.zeros((nb, 16), dtype=torch.bool)
    for s, n in enumerate(lens):
        pos = np.arange(n)
        live[bt[s, pos // 16], pos % 16] = True
    kc[~live.to(DEV)] = float("nan")  # slots that hold no token
    vc[~live.to(DEV)] = float("nan")
    q = (torch.randn((len(lens), hq, DIM), generator=g, device=DEV) * peak).to(TORCH[dtype])
    w = torch.rand((len(lens), hkv, int(lens.max()) + 3), generator=g, device=DEV) * 3
    return dict(q=q, kc=kc, vc=vc, bt=torch.from_numpy(bt).to(DEV), lens=torch.from_numpy(lens).to(DEV), w=w,
                lens_h=lens, bt_h=bt, dtype=dtype)


def _magnitude(c):
    """Largest scale * sum |q_i k_i| of the case's (query, key) pairs."""
    q, worst = np.abs(f64(c["q"])), 0.0
    G = q.shape[1] // c["kc"].shape[2]
    kc = np.abs(f64(c["kc"]))
    for s, n in enumerate(c["lens_h"]):
        for h in range(kc.shape[2]):
            worst = max(worst, float((q[s, h * G:(h + 1) * G] @ gather(kc, c["bt_h"][s], int(n), h).T).max()) * SCALE)
    return worst


def _check(c, out, w_out, w_in, before=None):
    ref, got_w, mag = attention(f64(c["q"]), f64(c["kc"]), f64(c["vc"]), c["bt_h"], c["lens_h"], SCALE)
    rel = _magnitude(c) * 2.0 ** -17 + 2.0 ** -16
    u = HALF_STEP[c["dtype"]]
    assert (np.abs(f64(out) - ref) <= u * np.abs(ref) + (1 + u) * mag * rel + HALF_TINY[c["dtype"]]).all()
    w_out = w_out.cpu().numpy()
    for s, n in enumerate(c["lens_h"]):
        base = np.zeros(got_w[s, :, :n].shape) if w_in is None else w_in[s, :, :n].cpu().numpy().astype(np.float64)
        want = base + got_w[s, :, :n]
        tol = got_w[s, :, :n] * rel + 2.0 ** -24 * want + 1e-37
        assert (np.abs(w_out[s, :, :n] - want) <= tol).all(), s
        if before is not None:
            assert np.array_equal(w_out[s, :, n:], before[s, :, n:].cpu().numpy())


def _run(c, w_in, w_out, **kw):
    return pa.paged_attn_decode_weights(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], SCALE, w_in, w_out, **kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(3, 3), (4, 2), (16, 8), (32, 8), (16, 2)])
def test_lengths_and_head_ratios(dtype, hq, hkv):
    c = _case([1, 15, 16, 17, 33, 250, 1023, 4097, 4096, 5000], hq, hkv, dtype, seed=hq * 10 + hkv)
    before = torch.full_like(c["w"], -2.0)
    w_out = before.clone()
    out, got = _run(c, c["w"], w_out)
    assert got is w_out
    _check(c, out, w_out, c["w"], before)


@pytest.mark.parametrize("lens", [[1], [777], [30000], [9000, 1] * 3, [40] * 300])
def test_few_and_many_sequences(lens):
    c = _case(lens, 8, 2, "bf16", seed=len(lens))
    w_out = torch.zeros_like(c["w"])
    out, _ = _run(c, None, w_out)
    _check(c, out, w_out, None, torch.zeros_like(c["w"]))


def test_same_outputs_as_the_plain_decode():
    c = _case([300, 5, 1000], 16, 8, "f16", seed=4)
    out, _ = _run(c, None, torch.zeros_like(c["w"]))
    plain = pa.paged_attn_decode(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], SCALE)
    ref, _, mag = attention(f64(c["q"]), f64(c["kc"]), f64(c["vc"]), c["bt_h"], c["lens_h"], SCALE)
    tol = 2 * (HALF_STEP["f16"] * np.abs(ref) + 1.01 * mag * (_magnitude(c) * 2.0 ** -17 + 2.0 ** -16))
    assert (np.abs(f64(out) - f64(plain)) <= tol).all()


def test_peaked_rows():
    """Large queries: most weights vanish, some below the smallest fp32 number."""
    c = _case([700, 50], 8, 2, "bf16", seed=6, peak=24.0)
    w_out = torch.zeros_like(c["w"])
    out, _ = _run(c, None, w_out)
    _check(c, out, w_out, None)


def test_in_place_over_several_steps():
    c = _case([130, 2000, 7], 8, 2, "f16", seed=7)
    w = torch.zeros_like(c["w"])
    rel = total = 0.0
    for step in range(3):
        c["q"] = torch.randn(c["q"].shape, generator=torch.Generator(device=DEV).manual_seed(step), device=DEV).half()
        _run(c, w, w)
        total = total + attention(f64(c["q"]), f64(c["kc"]), f64(c["vc"]), c["bt_h"], c["lens_h"], SCALE)[1]
        rel = max(rel, _magnitude(c) * 2.0 ** -17 + 2.0 ** -16)
    got = w.cpu().numpy()[:, :, :total.shape[2]]
    assert (np.abs(got - total) <= total * (rel + 3 * 2.0 ** -24) + 1e-37).all()
    assert np.array_equal(got[:, 0, :7] > 0, np.ones((3, 7), bool))


def test_bad_lengths_and_blocks():
    c = _case([100, 90, 80], 4, 2, "bf16", seed=8)
    limit = int(c["lens_h"].max())
    c["lens"][1] = limit + 1  # beyond the bound, within the table
    w_out = torch.full_like(c["w"], -2.0)
    out = torch.full_like(c["q"], 9.0)
    _run(c, None, w_out, out=out, max_context_len=limit)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    assert (out[1] == 9.0).all() and (w_out[1] == -2.0).all()
    good = dict(c, q=c["q"][::2], bt_h=c["bt_h"][::2], lens_h=c["lens_h"][::2])
    _check(good, out[::2], w_out[::2], None)
    c["lens"][1] = 90
    c["bt"][2, 1] = 10 ** 6  # keys 16 .. 31 of sequence 2 cannot be read
    _run(c, None, w_out, out=out)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 2
    assert (w_out[2, :, 16:32] == 0).all()
    assert abs(float(w_out[2, :, :80].sum()) - 4.0) < 1e-4


def test_no_page_readable():
    c = _case([20], 4, 2, "bf16", seed=9)
    c["bt"][:] = -1
    w_out = torch.full_like(c["w"], -2.0)
    _run(c, c["w"], w_out)
    assert pa.STATUS[pa.get_device_error()[0]] == "PA_ERR_RANGE"
    assert torch.equal(w_out[:, :, :20], c["w"][:, :, :20])


def test_stream_graph_and_empty():
    c = _case([300, 5, 1000], 16, 8, "f16", seed=14)
    ws = pa.alloc_decode_weights_workspace(3, 16, 8, 1000)
    ref_w = torch.zeros_like(c["w"])
    ref, _ = _run(c, c["w"], ref_w, max_context_len=1000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w2 = torch.zeros_like(c["w"])
    out, _ = _run(c, c["w"], w2, max_context_len=1000, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref) and torch.equal(w2, ref_w)
    ws.fill_(0xff)  # NaN everywhere: nothing in it need be initialised
    out, w2 = torch.zeros_like(ref), torch.zeros_like(c["w"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(c, c["w"], w2, out=out, workspace=ws, max_context_len=1000)
    for _ in range(3):
        out.zero_(), w2.zero_()
        g.replay()
        assert torch.equal(out, ref) and torch.equal(w2, ref_w)
    e = dict(c, q=c["q"][:0], bt=c["bt"][:0], lens=c["lens"][:0])
    out, _ = _run(e, c["w"][:0], c["w"][:0].clone())
    assert out.shape[0] == 0


def test_offsets_beyond_32_bits():
    """More than 2^31 scores in the workspace: 2100 sequences that all read the same 131072 cached tokens."""
    S, hq, hkv, n = 2100, 8, 1, 131072
    assert S * n * hq > 1 << 31
    c = _case([n, 5], hq, hkv, "bf16", seed=15)
    bt = c["bt"][:1].expand(S, -1).contiguous()
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    q = torch.randn((S, hq, DIM), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    w_out = torch.zeros((S, hkv, n), device=DEV)
    out, _ = pa.paged_attn_decode_weights(q, c["kc"], c["vc"], bt, lens, SCALE, None, w_out)
    for s in (0, 1000, S - 1):
        one = dict(c, q=q[s:s + 1], bt_h=c["bt_h"][:1], lens_h=c["lens_h"][:1])
        _check(one, out[s:s + 1], w_out[s:s + 1], None)


def test_rotate_decode_evict_and_on():
    """Four sequences grow token by token under a budget: the loop a server runs."""
    S, hq, hkv, budget, recent, sinks, start, steps = 4, 8, 2, 48, 8, 2, 60, 6
    u = HALF_STEP["f16"]
    g = torch.Generator(device=DEV).manual_seed(31)
    alloc = pa.BlockAllocator(64)
    seqs = [alloc.sequence() for _ in range(S)]
    kc, vc = (torch.full((64, 16, hkv, DIM), float("nan"), device=DEV).half() for _ in range(2))
    inv, factor = pa.rope_inv_freq(96, 1e6, pa.ROPE_YARN, factor=4.0, trained_length=32768)
    w = torch.zeros((S, hkv, 80), device=DEV)
    position = start

    def write(tokens):
        slots = [s.reserve(tokens) for s in seqs]
        n = S * tokens
        q, k, v = (torch.randn((n, h, DIM), generator=g, device=DEV).half() for h in (hq, hkv, hkv))
        first = 0 if tokens > 1 else position
        pos = torch.arange(first, first + tokens, dtype=torch.int32, device=DEV).repeat(S)
        out = pa.rope_kv_write(q, k, v, inv, pos, torch.tensor(sum(slots, []), device=DEV), kc, vc, interleaved=True,
                               attention_factor=factor)
        ref, mag = rotate(f64(q), pos.cpu().numpy(), inv.cpu().numpy(), factor, True)
        assert (np.abs(f64(out) - ref) <= u * np.abs(ref) + mag * 2.0 ** -20).all()
        for s in seqs:
            s.commit(tokens)
        return out

    write(start)
    model = [[list(range(start)) for _ in range(hkv)] for _ in range(S)]  # which token each cache row holds
    evictions = 0
    for step in range(steps):
        q = write(1)
        position += 1
        for s in range(S):
            for h in range(hkv):
                model[s][h].append(position - 1)
        bt, _, _, _ = pa.build_step_tables(seqs, 8)
        lens = np.array([s.length for s in seqs], np.int32)
        c = dict(q=q, kc=kc, vc=vc, bt_h=bt, lens_h=lens, bt=torch.from_numpy(bt).to(DEV),
                 lens=torch.from_numpy(lens).to(DEV), dtype="f16")
        w_before = w.clone()
        out, _ = _run(c, w, w)
        _check(c, out, w, w_before, w_before)
        if lens[0] > budget + 2:
            w_h = w.cpu().numpy()
            kept, new = pa.kv_evict(kc, vc, c["bt"], c["lens"], w, budget, recent, sinks)
            for s in range(S):
                for h in range(hkv):
                    at = evict_keep(w_h[s, h], int(lens[s]), budget, recent, sinks)
                    assert np.array_equal(kept[s, h].cpu().numpy(), at)
                    model[s][h] = [model[s][h][j] for j in at]
                seqs[s].truncate(int(new[s]))
            evictions += 1
            assert (w[:, :, budget:int(lens.max())] == 0).all()
    assert evictions == 2
    assert len({tuple(m) for row in model for m in row}) > 1  # the heads kept tokens of their own
