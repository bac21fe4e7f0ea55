"""GPU checks of pa_rope_kv_write_axes: against the one-axis call, whose every pair
must turn as if its axis's position were the token's (the same bits), and against a
plain form in 64 bits with the tolerance of test_gpu_rope_kv.py."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_rope_kv as one
from longctx_reference import DIM, HALF_STEP, HALF_TINY, bits, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _case(T, hq, hkv, dtype, sections, seed, woven=False, norm=False, pos_hi=4096):
    c = one._case(T, hq, hkv, dtype, 2 * sum(sections), seed, pos_hi, norm)
    rng = np.random.default_rng(seed + 1)
    c["pos"] = torch.from_numpy(rng.integers(0, pos_hi, (len(sections), T)).astype(np.int32)).to(DEV)
    c["axes"] = pa.rope_axes(sections, woven)
    return c


def _run(c, interleaved, factor=1.0, q_out=None, stream=None):
    return pa.rope_kv_write_axes(c["q"], c["k"], c["v"], c["inv"], c["pos"], c["axes"], c["slots"], c["kc"], c["vc"],
                                 interleaved=interleaved, attention_factor=factor, q_norm_weight=c["qw"],
                                 k_norm_weight=c["kw"], eps=1e-6, q_out=q_out, stream=stream)


def _rotate(x, c, interleaved, factor, weight):
    y = f64(x)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6) * f64(weight)
    out, mag, far = y.copy(), np.abs(y), 0.0
    pos, inv = c["pos"].cpu().numpy().astype(np.float64), c["inv"].cpu().numpy()
    half = len(inv)
    for i, f in enumerate(inv):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = pos[c["axes"][i]] * f
        far = max(far, float(np.abs(angle).max()))
        co, si = (np.cos(angle) * factor)[:, None], (np.sin(angle) * factor)[:, None]
        out[..., a], out[..., b] = y[..., a] * co - y[..., b] * si, y[..., b] * co + y[..., a] * si
        mag[..., a] = mag[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * abs(factor)
    return out, mag, far


def _close(got, x, c, interleaved, factor, weight):
    ref, mag, far = _rotate(x, c, interleaved, factor, weight)
    u = HALF_STEP[c["dtype"]]
    rel = (2.0 ** -21 if weight is None else 2.0 ** -19) + far * 2.0 ** -51
    tol = u * np.abs(ref) + (1 + u) * mag * rel + HALF_TINY[c["dtype"]]
    d = np.abs(got - ref)
    assert (d <= tol).all(), f"worst {np.max(d / tol):.3f} of the tolerance"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections,woven", [([16, 24, 24], False), ([24, 20, 20], True), ([1, 31], False), ([64], False),
                                            ([3, 2, 9, 1], True), ([0, 5, 0, 8], False), ([1], True)])
@pytest.mark.parametrize("dtype,norm", [("bf16", False), ("f16", True)])
def test_sections(interleaved, sections, woven, dtype, norm):
    c = _case(41, 8, 2, dtype, sections, seed=sum(sections), woven=woven, norm=norm)
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    out = _run(c, interleaved, 1.25)
    _close(f64(out), c["q"], c, interleaved, 1.25, c["qw"])
    kc, vc, sl = c["kc"].flatten(0, 1), c["vc"].flatten(0, 1), c["slots"]
    _close(f64(kc[sl]), c["k"], c, interleaved, 1.25, c["kw"])
    assert np.array_equal(bits(vc[sl]), bits(c["v"]))
    rest = np.ones(kc.shape[0], bool)
    rest[sl.cpu().numpy()] = False
    assert np.array_equal(bits(kc)[rest], bits(k0.flatten(0, 1))[rest])
    assert np.array_equal(bits(vc)[rest], bits(v0.flatten(0, 1))[rest])


@pytest.mark.parametrize("T,hq,hkv", [(1, 16, 8), (3, 1, 1), (457, 32, 8), (2003, 8, 4), (129, 64, 3)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_every_axis_turns_as_the_one_axis_call(T, hq, hkv, interleaved, norm):
    """Pair by pair the bits of the one-axis call at that axis's positions."""
    sections = [10, 26, 28]
    c = _case(T, hq, hkv, "bf16", sections, seed=T, woven=T % 2 == 0, norm=norm, pos_hi=100000)
    out = _run(c, interleaved)
    kc = c["kc"].flatten(0, 1)[c["slots"]].clone()
    for a in range(3):
        pairs = [i for i in range(64) if c["axes"][i] == a]
        dims = torch.tensor([d for i in pairs for d in ((2 * i, 2 * i + 1) if interleaved else (i, i + 64))], device=DEV)
        alone = one._run(dict(c, pos=c["pos"][a].contiguous()), interleaved)
        assert torch.equal(out[..., dims], alone[..., dims])
        assert torch.equal(kc[..., dims], c["kc"].flatten(0, 1)[c["slots"]][..., dims])


def test_equal_axes_are_one_axis():
    c = _case(600, 16, 8, "f16", [16, 24, 24], seed=4)
    c["pos"][1:] = c["pos"][0]
    out = _run(c, False)
    assert torch.equal(out, one._run(dict(c, pos=c["pos"][0].contiguous()), False))


def test_far_positions():
    c = _case(64, 4, 2, "f16", [20, 22, 22], seed=3)
    c["pos"][1, :6] = torch.tensor([0, 2 ** 20 - 1, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, 65535])
    out = _run(c, False)
    _close(f64(out), c["q"], c, False, 1.0, None)


@pytest.mark.parametrize("T", [40, 1000])
def test_a_negative_position_on_any_axis_is_refused(T):
    c = _case(T, 8, 4, "bf16", [16, 24, 24], seed=9)
    c["pos"][0, 7], c["pos"][1, 11], c["pos"][2, 12] = -1, -2 ** 31, -7
    c["slots"][20] = -5
    bad = [7, 11, 12, 20]
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    q_out = torch.full_like(c["q"], 3.0)
    _run(c, False, q_out=q_out)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail in bad
    assert bool((q_out[bad] == 3.0).all())
    for now, was in ((c["kc"], k0), (c["vc"], v0)):
        assert torch.equal(now.flatten(0, 1)[c["slots"][bad[:3]]], was.flatten(0, 1)[c["slots"][bad[:3]]])
    keep = [t for t in range(T) if t not in bad]
    sub = dict(c, pos=c["pos"][:, keep])
    _close(f64(q_out)[keep], c["q"][keep], sub, False, 1.0, None)


def test_in_place_stream_and_graph():
    c = _case(50, 8, 4, "bf16", [12, 18, 18], seed=8)
    apart = _run(c, False)
    again = c["q"].clone()
    assert torch.equal(_run(dict(c, q=again), False, q_out=again), apart)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = _run(c, False, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, apart)
    out = torch.zeros_like(apart)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(c, False, q_out=out)
    c["pos"][1] += 5
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _run(c, False))


def test_bindings_refuse():
    c = _case(5, 8, 4, "bf16", [16, 24, 24], seed=2)
    for change, error in [(dict(axes=list(c["axes"])), TypeError), (dict(axes=c["axes"][:-1]), ValueError),
                          (dict(pos=c["pos"][0]), ValueError), (dict(pos=c["pos"][:, :4].contiguous()), ValueError),
                          (dict(pos=c["pos"].long()), TypeError), (dict(pos=c["pos"][:2].contiguous()), pa.PagedAttnError)]:
        with pytest.raises(error):
            _run(dict(c, **change), False)
    empty = dict(c, q=c["q"][:0], k=c["k"][:0], v=c["v"][:0], pos=c["pos"][:, :0].contiguous(), slots=c["slots"][:0])
    assert _run(empty, False).shape == (0, 8, DIM)
