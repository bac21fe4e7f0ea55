"""Host checks of the long-context calls (no GPU): refusals before anything is
enqueued, the scaled rotary frequencies, and the allocator's unshare / truncate."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_gqa_cache_gb300 as pa

P = 1 << 20  # a fake, 16-byte aligned "device" address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from paged_kv_gqa_cache_gb300 import _build
    _build.build()
    return pa.load_library()


def _pool(**kw):
    d = dict(k_cache=4096, v_cache=8192, num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=0)
    d.update(kw)
    return pa.KVPool(**d)


def _rope(**kw):
    d = dict(inv_freq=P, rotary_dim=128, layout=0, attention_factor=1.0)
    d.update(kw)
    return pa.Rope(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "PA_OK"), (dict(T=-1), "PA_ERR_SHAPE"), (dict(rope=None), "PA_ERR_NULL"),
    (dict(rope=_rope(inv_freq=0)), "PA_ERR_NULL"), (dict(rope=_rope(rotary_dim=0)), "PA_ERR_SHAPE"),
    (dict(rope=_rope(rotary_dim=7)), "PA_ERR_SHAPE"), (dict(rope=_rope(rotary_dim=130)), "PA_ERR_SHAPE"),
    (dict(rope=_rope(layout=2)), "PA_ERR_UNSUPPORTED"),
    (dict(rope=_rope(attention_factor=math.inf)), "PA_ERR_SHAPE"), (dict(rope=_rope(inv_freq=P + 4)), "PA_ERR_ALIGN"),
    (dict(q=0), "PA_ERR_NULL"), (dict(v=0), "PA_ERR_NULL"), (dict(pos=0), "PA_ERR_NULL"),
    (dict(qw=P), "PA_ERR_NULL"), (dict(qw=P, kw=P, eps=-1.0), "PA_ERR_SHAPE"),
    (dict(qw=P, kw=P, eps=math.nan), "PA_ERR_SHAPE"), (dict(qw=P + 2, kw=P), "PA_ERR_ALIGN"),
    (dict(hq=0), "PA_ERR_SHAPE"), (dict(hq=1025), "PA_ERR_SHAPE"), (dict(q=P + 8), "PA_ERR_ALIGN"),
    (dict(pos=P + 2), "PA_ERR_ALIGN"), (dict(slots=P + 4), "PA_ERR_ALIGN"),
    (dict(pool=_pool(dtype=5)), "PA_ERR_DTYPE"), (dict(pool=_pool(head_dim=64)), "PA_ERR_UNSUPPORTED"),
])
def test_rope_kv_write_refusals(lib, kw, status):
    rope = kw.get("rope", _rope())
    st = lib.pa_rope_kv_write(kw.get("q", P), kw.get("k", P), kw.get("v", P),
                              None if rope is None else ctypes.byref(rope), kw.get("qw"), kw.get("kw"),
                              kw.get("eps", 1e-6), kw.get("pos", P), kw.get("slots", P), kw.get("T", 4),
                              kw.get("hq", 16), kw.get("out", P), ctypes.byref(kw.get("pool", _pool())), None)
    assert pa.STATUS[st] == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), "PA_OK"), (dict(S=-1), "PA_ERR_SHAPE"), (dict(w=0), "PA_ERR_NULL"), (dict(kept=0), "PA_ERR_NULL"),
    (dict(dst=0), "PA_ERR_NULL"), (dict(new=0), "PA_ERR_NULL"), (dict(w_out=0), "PA_ERR_NULL"),
    (dict(budget=0), "PA_ERR_SHAPE"), (dict(recent=-1), "PA_ERR_SHAPE"), (dict(sinks=-1), "PA_ERR_SHAPE"),
    (dict(budget=8, recent=5, sinks=4), "PA_ERR_SHAPE"), (dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), "PA_ERR_SHAPE"),
    (dict(new=P), "PA_ERR_SHAPE"), (dict(w_out=P, out_stride=99), "PA_ERR_SHAPE"),
    (dict(dst=P, dst_blocks=3), "PA_ERR_SHAPE"), (dict(stride=0), "PA_ERR_SHAPE"), (dict(mb=0), "PA_ERR_SHAPE"),
    (dict(S=16385), "PA_ERR_UNSUPPORTED"), (dict(w=P + 2), "PA_ERR_ALIGN"), (dict(kept=P + 2), "PA_ERR_ALIGN"),
    (dict(budget=2 ** 30 + 1), "PA_ERR_UNSUPPORTED"), (dict(budget=2 ** 31 - 1), "PA_ERR_UNSUPPORTED"),
    (dict(w_out=P + 4), "PA_ERR_SHAPE"), (dict(w=P + (1 << 20), w_out=P + (1 << 20) - 4), "PA_ERR_SHAPE"),
    (dict(w_out=P + 4 * 8 * 256 * 4 - 4), "PA_ERR_SHAPE"), (dict(new=P + 12), "PA_ERR_SHAPE"),
    (dict(new=P - 12), "PA_ERR_SHAPE"),
    (dict(pool=_pool(num_blocks=0)), "PA_ERR_SHAPE"), (dict(pool=_pool(k_cache=0)), "PA_ERR_NULL"),
])
def test_kv_evict_refusals(lib, kw, status):
    st = lib.pa_kv_evict(ctypes.byref(kw.get("pool", _pool())), P, kw.get("mb", 16), P, kw.get("S", 4),
                         kw.get("w", P), kw.get("stride", 256), kw.get("budget", 64), kw.get("recent", 8),
                         kw.get("sinks", 4), kw.get("dst", P + 64), kw.get("dst_blocks", 4), kw.get("w_out", P + 64),
                         kw.get("out_stride", 64), kw.get("kept", P), kw.get("new", P + 128), None)
    assert pa.STATUS[st] == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), "PA_OK"), (dict(S=-1), "PA_ERR_SHAPE"), (dict(w_out=0), "PA_ERR_NULL"), (dict(q=0), "PA_ERR_NULL"),
    (dict(w_in=None, ws=0), "PA_ERR_WORKSPACE"), (dict(wsb=-1), "PA_ERR_WORKSPACE"), (dict(stride=255), "PA_ERR_SHAPE"),
    (dict(mcl=257), "PA_ERR_SHAPE"), (dict(mcl=0), "PA_ERR_SHAPE"), (dict(hq=24), "PA_ERR_UNSUPPORTED"),
    (dict(hq=12), "PA_ERR_SHAPE"), (dict(scale=0.0), "PA_ERR_SHAPE"), (dict(w_in=P + 2), "PA_ERR_ALIGN"),
    (dict(w_out=P + 2), "PA_ERR_ALIGN"), (dict(ws=P + 8), "PA_ERR_ALIGN"), (dict(S=9000, wsb=1 << 40), "PA_ERR_UNSUPPORTED"),
    (dict(pool=_pool(dtype=5)), "PA_ERR_DTYPE"),
    (dict(w_out=P + 4), "PA_ERR_SHAPE"), (dict(w_out=P + 4 * 8 * 256 * 4 - 4), "PA_ERR_SHAPE"),
    (dict(w_in=P + 512), "PA_ERR_SHAPE"),
    (dict(mb=2 ** 27, mcl=2 ** 30 + 1, stride=2 ** 31 - 1, wsb=2 ** 62), "PA_ERR_UNSUPPORTED"),
    (dict(mb=2 ** 27, mcl=2 ** 31 - 1, stride=2 ** 31 - 1, wsb=2 ** 62), "PA_ERR_UNSUPPORTED"),
])
def test_decode_weights_refusals(lib, kw, status):
    S, mcl = kw.get("S", 4), kw.get("mcl", 256)
    need = lib.pa_decode_weights_workspace_bytes(max(S, 1), kw.get("hq", 16), 8, max(mcl, 1))
    wsb = kw.get("wsb", need)
    st = lib.pa_paged_attn_decode_weights(kw.get("q", P), ctypes.byref(kw.get("pool", _pool())), P, kw.get("mb", 16), P, S,
                                          kw.get("hq", 16), mcl, kw.get("scale", 0.1), kw.get("w_in", P),
                                          kw.get("w_out", P), kw.get("stride", 256), P, kw.get("ws", P),
                                          need - 1 if wsb == -1 else wsb, None)
    assert pa.STATUS[st] == status


def test_decode_weights_workspace_size(lib):
    f = lib.pa_decode_weights_workspace_bytes
    assert f(4, 16, 8, 256) >= lib.pa_decode_workspace_bytes(4, 16, 8, 256) + 4 * 256 * 16 * 4
    assert f(4, 16, 8, 257) > f(4, 16, 8, 256)
    assert f(70, 32, 4, 1 << 19) > 1 << 32  # 64-bit arithmetic
    assert f(-1, 16, 8, 256) == 0 and f(4, 12, 8, 256) == 0 and f(4, 16, 8, 0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), "PA_OK"), (dict(S=-1), "PA_ERR_SHAPE"), (dict(q=0), "PA_ERR_NULL"), (dict(groups=-1), "PA_ERR_SHAPE"),
    (dict(sizes=0), "PA_ERR_NULL"), (dict(prefix=0), "PA_ERR_NULL"), (dict(groups=257), "PA_ERR_UNSUPPORTED"),
    (dict(S=6001), "PA_ERR_UNSUPPORTED"), (dict(ws=0), "PA_ERR_WORKSPACE"), (dict(ws=P + 8), "PA_ERR_ALIGN"),
    (dict(sizes=P + 2), "PA_ERR_ALIGN"), (dict(prefix=P + 1), "PA_ERR_ALIGN"), (dict(mcl=257), "PA_ERR_SHAPE"),
    (dict(hq=24), "PA_ERR_UNSUPPORTED"), (dict(scale=-1.0), "PA_ERR_SHAPE"), (dict(pool=_pool(dtype=9)), "PA_ERR_DTYPE"),
    (dict(mb=1 << 30), "PA_ERR_UNSUPPORTED"),
])
def test_decode_shared_refusals(lib, kw, status):
    st = lib.pa_paged_attn_decode_shared(kw.get("q", P), ctypes.byref(kw.get("pool", _pool())), P, kw.get("mb", 16), P,
                                         kw.get("S", 4), kw.get("hq", 16), kw.get("mcl", 256), kw.get("scale", 0.1),
                                         kw.get("sizes", P), kw.get("prefix", P), kw.get("groups", 2), P,
                                         kw.get("ws", P), kw.get("wsb", 1 << 40), None)
    assert pa.STATUS[st] == status


def test_shared_prefix_limits_match_the_header(lib):
    import os
    import re
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                               "pagedattn.h")).read()
    defines = dict(re.findall(r"#define (PA_[A-Z0-9_]+) (\d+)\b", header))
    assert int(defines["PA_MAX_PREFIX_GROUPS"]) == pa.MAX_PREFIX_GROUPS
    for name in ("HALF", "INTERLEAVED", "PLAIN", "LINEAR", "NTK", "BANDS", "YARN"):
        assert int(defines["PA_ROPE_" + name]) == getattr(pa, "ROPE_" + name)
    f = lib.pa_decode_shared_workspace_bytes
    assert f(4, 257, 16, 8) == 0 and f(6001, 1, 16, 8) == 0 and f(4, 1, 12, 8) == 0 and f(-1, 1, 16, 8) == 0


# ---- rotary frequencies ----------------------------------------------------------------

def _freqs(*a, **kw):
    f, att = pa.rope_inv_freq(*a, device="cpu", **kw)
    return f.numpy(), att


@pytest.mark.parametrize("d", [2, 6, 96, 128])
def test_plain_linear_and_ntk_frequencies(d):
    base = 1e6 ** (-np.arange(0, d, 2) / d)
    f, att = _freqs(d, 1e6)
    assert att == 1.0 and np.allclose(f, base, rtol=1e-14, atol=0)
    f, att = _freqs(d, 1e6, pa.ROPE_LINEAR, factor=3.0)
    assert att == 1.0 and np.allclose(f, base / 3, rtol=1e-14, atol=0)
    f, att = _freqs(d, 1e6, pa.ROPE_NTK, factor=3.0)
    assert f[0] == 1.0
    if d > 2:  # the slowest pair turns exactly `factor` times slower
        assert abs(f[-1] / (base[-1] / 3) - 1) < 1e-12
    assert all(f[i] <= base[i] * (1 + 1e-12) for i in range(d // 2))


def test_bands_keep_fast_pairs_and_stretch_slow_ones():
    d, L, slow, fast, factor = 128, 8192, 1.0, 4.0, 8.0
    base = 5e5 ** (-np.arange(0, d, 2) / d)
    f, att = _freqs(d, 5e5, pa.ROPE_BANDS, factor=factor, trained_length=L, slow=slow, fast=fast)
    turns = L * base / (2 * math.pi)
    assert att == 1.0 and (turns > fast).any() and (turns < slow).any()
    for i in range(d // 2):
        if turns[i] >= fast:
            want = base[i]
        elif turns[i] <= slow:
            want = base[i] / factor
        else:
            mix = (turns[i] - slow) / (fast - slow)
            want = (1 - mix) * base[i] / factor + mix * base[i]
        assert abs(f[i] / want - 1) < 1e-12


def test_yarn_ramp_and_attention_factor():
    d, theta, L, factor = 128, 1e6, 32768, 4.0
    base = theta ** (-np.arange(0, d, 2) / d)
    f, att = _freqs(d, theta, pa.ROPE_YARN, factor=factor, trained_length=L, slow=1.0, fast=32.0)
    assert abs(att - (0.1 * math.log(4.0) + 1.0)) < 1e-7
    ratio = f / base
    turns = L * base / (2 * math.pi)
    # the pair nearest the border may sit on either side of it: borders are rounded outwards
    assert np.allclose(ratio[turns > 32.0 * (theta ** (2 / d))], 1.0)
    assert np.allclose(ratio[turns < 1.0 / (theta ** (2 / d))], 1 / factor)
    assert (np.diff(ratio) <= 1e-12).all()
    f, att = _freqs(d, theta, pa.ROPE_YARN, factor=1.0, trained_length=L, slow=1.0, fast=32.0)
    assert att == 1.0 and np.allclose(f, base, rtol=1e-14)


@pytest.mark.parametrize("kw,status", [
    (dict(d=0), "PA_ERR_SHAPE"), (dict(d=3), "PA_ERR_SHAPE"), (dict(d=130), "PA_ERR_SHAPE"),
    (dict(theta=1.0), "PA_ERR_SHAPE"), (dict(theta=math.nan), "PA_ERR_SHAPE"), (dict(scaling=5), "PA_ERR_UNSUPPORTED"),
    (dict(scaling=-1), "PA_ERR_UNSUPPORTED"), (dict(scaling=1, factor=0.5), "PA_ERR_SHAPE"),
    (dict(scaling=3, factor=2.0, length=0.0), "PA_ERR_SHAPE"), (dict(scaling=4, factor=2.0, slow=32.0), "PA_ERR_SHAPE"),
    (dict(scaling=4, factor=2.0, slow=0.0), "PA_ERR_SHAPE"), (dict(scaling=2, factor=math.inf), "PA_ERR_SHAPE"),
    (dict(), "PA_OK"), (dict(factor=0.0), "PA_OK"),
])
def test_inv_freq_refusals(lib, kw, status):
    buf, att = (ctypes.c_double * 64)(), ctypes.c_float()
    st = lib.pa_rope_inv_freq(kw.get("scaling", 0), kw.get("d", 128), kw.get("theta", 1e4), kw.get("factor", 1.0),
                              kw.get("length", 4096.0), kw.get("slow", 1.0), kw.get("fast", 32.0), buf,
                              ctypes.byref(att))
    assert pa.STATUS[st] == status
    assert pa.STATUS[lib.pa_rope_inv_freq(0, 128, 1e4, 1, 1, 1, 2, None, ctypes.byref(att))] == "PA_ERR_NULL"


# ---- unshare and truncate -----------------------------------------------------------------

def test_unshare_copies_only_shared_blocks():
    alloc = pa.BlockAllocator(12)
    a, b = alloc.sequence(), alloc.sequence()
    a.reserve(70)
    a.commit(70)
    b.fork_from(a)
    b.unshare(2)
    assert alloc.take_copies() == [(0, 5), (1, 6)]
    assert b.blocks == [5, 6, 2, 3, 4] and a.blocks == [0, 1, 2, 3, 4]
    b.unshare(2)  # nothing left to do
    assert alloc.take_copies() == [] and alloc.stats()["n_cow"] == 2
    st = alloc.stats()
    assert st["used"] == 7 and st["shared"] == 3


def test_unshare_is_all_or_nothing():
    alloc = pa.BlockAllocator(6)
    a, b = alloc.sequence(), alloc.sequence()
    a.reserve(80)
    a.commit(80)
    b.fork_from(a)
    with pytest.raises(pa.PagedAttnError) as e:
        b.unshare(2)  # one block is free
    assert pa.STATUS[e.value.status] == "PA_ERR_NO_BLOCKS"
    assert b.blocks == a.blocks and alloc.take_copies() == [] and alloc.stats()["free"] == 1
    for n in (-1, 6):
        with pytest.raises(pa.PagedAttnError):
            b.unshare(n)


def test_truncate_releases_the_blocks_past_the_length():
    alloc = pa.BlockAllocator(8)
    a = alloc.sequence()
    a.reserve(100)
    with pytest.raises(pa.PagedAttnError) as e:
        a.truncate(0)  # tokens are reserved
    assert pa.STATUS[e.value.status] == "PA_ERR_STATE"
    a.commit(100)
    for n in (-1, 101):
        with pytest.raises(pa.PagedAttnError):
            a.truncate(n)
    a.truncate(33)
    assert a.length == 33 and a.blocks == [0, 1, 2] and alloc.stats()["free"] == 5
    assert a.reserve(16)[:2] == [2 * 16 + 1, 2 * 16 + 2]
    a.commit(16)
    a.truncate(0)
    assert a.length == 0 and a.blocks == [] and alloc.stats()["free"] == 8


def test_truncated_fork_still_copies_on_write():
    alloc = pa.BlockAllocator(8)
    a, b = alloc.sequence(), alloc.sequence()
    a.reserve(40)
    a.commit(40)
    b.fork_from(a)
    b.truncate(20)
    assert b.blocks == a.blocks[:2]
    b.reserve(1)
    assert alloc.take_copies() == [(1, 3)] and b.blocks == [0, 3]
