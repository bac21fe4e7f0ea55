"""GPU checks of pa_rope_kv_write against a plain form in 64 bits: layouts,
rotary widths, norms, far positions, bad tokens, in place, captured, on another
stream, and a step that decodes over what it wrote.

Tolerance of a rotated element, with u the type's half step and m the sum of the
magnitudes that enter it (|a| + |b|) |factor|: u |ref| for the one rounding, plus
m (1 + u) times the fp32 error: 2^-23 for each of cos and sin (2 ulp at most below 1),
2^-23.3 of angle (pi 2^-25 from the conversion of the turn to fp32), two products and
a sum (3 2^-24), the factor (2^-24): below 2^-21 in all; with the norm its sum of 128
squares (at most 11 roundings deep, so 2^-21), rsqrt (2^-22) and two products more:
below 2^-19.  Far positions add 3 p f 2^-53 rad: the frequency in turns is off by two roundings,
the reference by one of its product; 2^-51 p f is taken."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
from longctx_reference import DIM, HALF_STEP, HALF_TINY, TORCH, attention, bits, f64, random_pool, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _case(T, hq, hkv, dtype, rotary, seed, pos_hi=4096, norm=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    nb = -(-T // 16) + 2
    r = lambda n: torch.randn((T, n, DIM), generator=g, device=DEV).to(TORCH[dtype])
    c = dict(q=r(hq), k=r(hkv), v=r(hkv), kc=random_pool(g, nb, hkv, dtype), vc=random_pool(g, nb, hkv, dtype),
             pos=torch.from_numpy(rng.integers(0, pos_hi, T).astype(np.int32)).to(DEV),
             slots=torch.from_numpy(rng.permutation(nb * 16)[:T].astype(np.int64)).to(DEV),
             inv=1e4 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=DEV) / rotary), dtype=dtype)
    c["qw"], c["kw"] = ((1 + 0.3 * torch.randn(DIM, generator=g, device=DEV)).to(TORCH[dtype]) if norm else None
                        for _ in range(2))
    return c


def _run(c, interleaved, factor=1.0, q_out=None, stream=None):
    return pa.rope_kv_write(c["q"], c["k"], c["v"], c["inv"], c["pos"], c["slots"], c["kc"], c["vc"],
                            interleaved=interleaved, attention_factor=factor, q_norm_weight=c["qw"],
                            k_norm_weight=c["kw"], eps=1e-6, q_out=q_out, stream=stream)


def _close(got, x, weight, c, interleaved, factor):
    inv, pos = c["inv"].cpu().numpy(), c["pos"].cpu().numpy()
    w = None if weight is None else f64(weight)
    ref, mag = rotate(f64(x), pos, inv, factor, interleaved, w, 1e-6)
    u = HALF_STEP[c["dtype"]]
    far = (pos.astype(np.float64) * (inv.max() if len(inv) else 0.0) * 2.0 ** -51)[:, None, None]
    tol = u * np.abs(ref) + (1 + u) * mag * ((2.0 ** -21 if w is None else 2.0 ** -19) + far) + HALF_TINY[c["dtype"]]
    d = np.abs(got - ref)
    assert (d <= tol).all(), f"worst {np.max(d / tol):.3f} of the tolerance at {np.unravel_index(np.argmax(d / tol), d.shape)}"


def _check(c, out, before_k, before_v, interleaved, factor=1.0, skip=()):
    keep = np.array([t for t in range(len(c["pos"])) if t not in skip], np.int64)
    sub = dict(c, pos=c["pos"][keep])
    _close(f64(out)[keep], c["q"][keep], c["qw"], sub, interleaved, factor)
    kc, vc = c["kc"].flatten(0, 1), c["vc"].flatten(0, 1)
    sl = c["slots"][keep]
    _close(f64(kc[sl]), c["k"][keep], c["kw"], sub, interleaved, factor)
    assert np.array_equal(bits(vc[sl]), bits(c["v"][keep]))
    rest = np.ones(kc.shape[0], bool)
    rest[sl.cpu().numpy()] = False
    assert np.array_equal(bits(kc)[rest], bits(before_k.flatten(0, 1))[rest])
    assert np.array_equal(bits(vc)[rest], bits(before_v.flatten(0, 1))[rest])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [2, 6, 16, 64, 90, 96, 128])
@pytest.mark.parametrize("dtype,norm", [("bf16", False), ("f16", True)])
def test_layouts_and_widths(interleaved, rotary, dtype, norm):
    c = _case(37, 8, 2, dtype, rotary, seed=rotary + interleaved, norm=norm)
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    out = _run(c, interleaved, factor=1.25)
    _check(c, out, k0, v0, interleaved, 1.25)


@pytest.mark.parametrize("T,hq,hkv", [(1, 16, 8), (3, 1, 1), (700, 32, 8), (129, 64, 3), (5, 13, 7)])
@pytest.mark.parametrize("norm", [False, True])
def test_sizes_and_heads(T, hq, hkv, norm):
    c = _case(T, hq, hkv, "bf16", 128, seed=T, norm=norm)
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    _check(c, _run(c, False), k0, v0, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_and_odd_frequencies(interleaved):
    c = _case(64, 4, 2, "f16", 128, seed=3)
    c["pos"][:8] = torch.tensor([0, 1, 2 ** 20 - 1, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, 65535, 131071])
    c["inv"][:4] = torch.tensor([0.0, -0.37, 3.0, 7.5], dtype=torch.float64)  # still, backwards, near and past half a turn
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    _check(c, _run(c, interleaved), k0, v0, interleaved)


def test_in_place_query():
    c = _case(50, 8, 4, "bf16", 96, seed=8)
    apart = _run(c, False)
    again = c["q"].clone()
    c2 = dict(c, q=again)
    out = _run(c2, False, q_out=again)
    assert out.data_ptr() == again.data_ptr() and torch.equal(out, apart)


def test_bad_tokens_are_skipped():
    c = _case(40, 8, 4, "bf16", 128, seed=9)
    c["pos"][7] = -1
    c["slots"][11] = c["kc"].shape[0] * 16
    c["slots"][12] = -5
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    q_out = torch.full_like(c["q"], 3.0)
    _run(c, False, q_out=q_out)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail in (7, 11, 12)
    assert (q_out[[7, 11, 12]] == 3.0).all()
    _check(c, q_out, k0, v0, False, skip=(7, 11, 12))


def test_empty_step():
    c = _case(1, 8, 4, "bf16", 128, seed=1)
    e = dict(c, q=c["q"][:0], k=c["k"][:0], v=c["v"][:0], pos=c["pos"][:0], slots=c["slots"][:0])
    assert _run(e, False).shape == (0, 8, DIM)


def test_other_stream_and_graph_replay():
    c = _case(33, 8, 4, "f16", 64, seed=5)
    ref_k, ref_v = c["kc"].clone(), c["vc"].clone()
    ref = _run(dict(c, kc=ref_k, vc=ref_v), True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = _run(c, True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref) and torch.equal(c["kc"], ref_k) and torch.equal(c["vc"], ref_v)
    g = torch.cuda.CUDAGraph()
    q_out = torch.zeros_like(ref)
    with torch.cuda.graph(g):
        _run(c, True, q_out=q_out)
    for shift in (0, 100):
        c["pos"] += shift
        c["kc"].zero_()
        g.replay()
        want_k = torch.zeros_like(c["kc"])
        want = _run(dict(c, kc=want_k, vc=ref_v), True)
        assert torch.equal(q_out, want) and torch.equal(c["kc"], want_k)


def test_write_then_decode():
    """The rotated keys of a whole sequence, then a decode over them."""
    T, hq, hkv = 75, 16, 8
    c = _case(T, hq, hkv, "f16", 64, seed=21)
    c["pos"] = torch.arange(1000, 1000 + T, dtype=torch.int32, device=DEV)
    bt = torch.randperm(c["kc"].shape[0], generator=torch.Generator().manual_seed(2))[:5].int()
    slots = bt[torch.arange(T) // 16].long() * 16 + torch.arange(T) % 16
    c["slots"] = slots.to(DEV)
    q = _run(c, True)
    out = pa.paged_attn_decode(q[-1:].contiguous(), c["kc"], c["vc"], bt[None].to(DEV),
                               torch.tensor([T], dtype=torch.int32, device=DEV), DIM ** -0.5)
    ref, _, mag = attention(f64(q[-1:]), f64(c["kc"]), f64(c["vc"]), bt[None].numpy(), np.array([T]), DIM ** -0.5)
    # fp32 scores of magnitude at most 2^4 over 128 products (2^-17 absolute), then one rounding
    assert (np.abs(f64(out) - ref) <= HALF_STEP["f16"] * np.abs(ref) + mag * 2.0 ** -15).all()
