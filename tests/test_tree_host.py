"""Host checks of the calls on trees of drafted tokens and of the rotary write with
several axes (no GPU): refusals before anything is enqueued, and the axes' order."""
import ctypes

import pytest
import torch

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


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), "PA_OK"), (dict(T=0), "PA_OK"), (dict(S=-1), "PA_ERR_SHAPE"), (dict(T=-1), "PA_ERR_SHAPE"),
    (dict(S=-1, T=0), "PA_ERR_SHAPE"), (dict(q=0), "PA_ERR_NULL"), (dict(out=0), "PA_ERR_NULL"),
    (dict(n=0), "PA_ERR_NULL"), (dict(parents=0), "PA_ERR_NULL"), (dict(lens=0), "PA_ERR_NULL"),
    (dict(S=2049), "PA_ERR_UNSUPPORTED"), (dict(T=2 ** 20 - 1), "PA_ERR_UNSUPPORTED"), (dict(ws=0), "PA_ERR_WORKSPACE"),
    (dict(ws=P + 8), "PA_ERR_ALIGN"), (dict(n=P + 2), "PA_ERR_ALIGN"), (dict(parents=P + 1), "PA_ERR_ALIGN"),
    (dict(q=P + 8), "PA_ERR_ALIGN"), (dict(mcl=257), "PA_ERR_SHAPE"), (dict(mcl=0), "PA_ERR_SHAPE"),
    (dict(hq=24), "PA_ERR_UNSUPPORTED"), (dict(hq=12), "PA_ERR_SHAPE"), (dict(scale=-1.0), "PA_ERR_SHAPE"),
    (dict(scale=float("nan")), "PA_ERR_SHAPE"), (dict(pool=_pool(dtype=9)), "PA_ERR_DTYPE"),
    (dict(pool=_pool(block_size=32)), "PA_ERR_UNSUPPORTED"), (dict(pool=None), "PA_ERR_NULL"),
    (dict(mb=1 << 26, mcl=1 << 30, S=40, T=100), "PA_ERR_UNSUPPORTED"),
    (dict(mb=(1 << 26) + 1, mcl=(1 << 30) + 1, S=1, T=1), "PA_ERR_UNSUPPORTED"),
])
def test_attn_tree_refusals(lib, kw, status):
    pool = kw.get("pool", _pool())
    st = lib.pa_paged_attn_tree(kw.get("q", P), None if pool is None else ctypes.byref(pool), P, kw.get("mb", 16),
                                kw.get("lens", P), kw.get("S", 4), kw.get("hq", 16), kw.get("mcl", 256),
                                kw.get("scale", 0.1), kw.get("n", P), kw.get("parents", P), kw.get("T", 20),
                                kw.get("out", P), kw.get("ws", P), 1 << 40, None)
    assert pa.STATUS[st] == status


def test_tree_workspace_size(lib):
    f = lib.pa_tree_workspace_bytes
    assert f(1, 16, 8) == f(2048, 32, 4) > 0  # a piece or two per CTA, whatever the batch
    assert f(-1, 16, 8) == f(2049, 16, 8) == f(4, 12, 8) == f(4, 0, 8) == 0


def _accept(lib, kw, move):
    pools = kw.get("pools", (pa.KVPool * 2)(_pool(), _pool(k_cache=1 << 14, v_cache=1 << 15)))
    S, layers = kw.get("S", 4), kw.get("layers", 2)
    if move:
        return lib.pa_tree_move(kw.get("path", P), kw.get("stride", 8), kw.get("plens", P), kw.get("n", P),
                                kw.get("lens", P), S, pools, layers, kw.get("bt", P), kw.get("mb", 16),
                                kw.get("new", P + 64), None)
    return lib.pa_tree_accept(kw.get("draft", P), kw.get("target", P), kw.get("parents", P), kw.get("T", 20),
                              kw.get("n", P), kw.get("lens", P), S, pools, layers, kw.get("bt", P), kw.get("mb", 16),
                              kw.get("path", P), kw.get("stride", 8), kw.get("plens", P), kw.get("next", P),
                              kw.get("new", P + 64), None)


BOTH = [
    (dict(S=0), "PA_OK"), (dict(S=-1), "PA_ERR_SHAPE"), (dict(layers=-1), "PA_ERR_SHAPE"),
    (dict(stride=0), "PA_ERR_SHAPE"), (dict(path=0), "PA_ERR_NULL"), (dict(plens=0), "PA_ERR_NULL"),
    (dict(n=0), "PA_ERR_NULL"), (dict(lens=0), "PA_ERR_NULL"), (dict(new=0), "PA_ERR_NULL"), (dict(bt=0), "PA_ERR_NULL"),
    (dict(pools=None), "PA_ERR_NULL"), (dict(mb=0), "PA_ERR_SHAPE"), (dict(S=65537, new=P << 4), "PA_ERR_UNSUPPORTED"),
    (dict(path=P + 2), "PA_ERR_ALIGN"), (dict(plens=P + 1), "PA_ERR_ALIGN"), (dict(n=P + 2), "PA_ERR_ALIGN"),
    (dict(bt=P + 2), "PA_ERR_ALIGN"), (dict(new=P), "PA_ERR_SHAPE"), (dict(new=P + 12), "PA_ERR_SHAPE"),
    (dict(new=P - 12), "PA_ERR_SHAPE"),
    (dict(pools=(pa.KVPool * 2)(_pool(), _pool(num_blocks=63))), "PA_ERR_SHAPE"),
    (dict(pools=(pa.KVPool * 2)(_pool(), _pool(dtype=1))), "PA_ERR_SHAPE"),
    (dict(pools=(pa.KVPool * 2)(_pool(), _pool(v_cache=0))), "PA_ERR_NULL"),
]


@pytest.mark.parametrize("kw,status", BOTH)
@pytest.mark.parametrize("move", [False, True])
def test_accept_and_move_refusals(lib, kw, status, move):
    assert pa.STATUS[_accept(lib, kw, move)] == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "PA_ERR_SHAPE"), (dict(draft=0), "PA_ERR_NULL"), (dict(target=0), "PA_ERR_NULL"),
    (dict(parents=0), "PA_ERR_NULL"), (dict(next=0), "PA_ERR_NULL"), (dict(draft=P + 4), "PA_ERR_ALIGN"),
    (dict(target=P + 4), "PA_ERR_ALIGN"), (dict(next=P + 4), "PA_ERR_ALIGN"), (dict(parents=P + 2), "PA_ERR_ALIGN"),
])
def test_accept_refusals(lib, kw, status):
    assert pa.STATUS[_accept(lib, kw, False)] == status


def _apart(**kw):
    """Addresses that no two arrays of a call share, but for those given."""
    names = ["draft", "target", "parents", "n", "lens", "bt", "path", "plens", "next", "new"]
    d = {name: P + (i << 16) for i, name in enumerate(names)}
    d.update({a: d[b] + off for a, (b, off) in kw.items()})
    return d


@pytest.mark.parametrize("out,of,off", [  # 4 sequences, 20 tokens, paths of 8, tables of 16 blocks
    *[(out, of, 0) for out in ("path", "plens", "next", "new")
      for of in ("draft", "target", "parents", "n", "lens", "bt", "path", "plens", "next", "new") if of != out],
    ("new", "n", 12), ("new", "path", 124), ("path", "parents", 76), ("next", "target", 152), ("plens", "bt", 252),
])
def test_accept_outputs_apart(lib, out, of, off):
    assert pa.STATUS[_accept(lib, _apart(**{out: (of, off)}), False)] == "PA_ERR_SHAPE"


@pytest.mark.parametrize("of,off", [("n", 0), ("lens", 12), ("bt", 252), ("path", 124), ("plens", 12)])
def test_move_output_apart(lib, of, off):
    assert pa.STATUS[_accept(lib, _apart(new=(of, off)), True)] == "PA_ERR_SHAPE"


def _rope(**kw):
    d = dict(inv_freq=P, rotary_dim=128, layout=0, attention_factor=1.0)
    d.update(kw)
    return pa.Rope(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "PA_OK"), (dict(axes=0), "PA_ERR_SHAPE"), (dict(axes=5), "PA_ERR_SHAPE"),
    (dict(pairs=None), "PA_ERR_NULL"), (dict(pairs=b"\0" * 63 + b"\3"), "PA_ERR_SHAPE"),
    (dict(pairs=b"\xff" * 64), "PA_ERR_SHAPE"), (dict(pairs=b"\0" * 31 + b"\3" * 33, rope=_rope(rotary_dim=62), T=0), "PA_OK"),
    (dict(rope=None), "PA_ERR_NULL"), (dict(rope=_rope(rotary_dim=7)), "PA_ERR_SHAPE"), (dict(q=0), "PA_ERR_NULL"),
    (dict(pos=P + 2), "PA_ERR_ALIGN"), (dict(T=-1), "PA_ERR_SHAPE"), (dict(out=P + 4096), "PA_ERR_SHAPE"),
])
def test_rope_axes_refusals(lib, kw, status):
    rope = kw.get("rope", _rope())
    st = lib.pa_rope_kv_write_axes(kw.get("q", P), P << 4, P << 5, None if rope is None else ctypes.byref(rope),
                                   kw.get("pairs", b"\0" * 20 + b"\1" * 20 + b"\2" * 24), kw.get("axes", 3), None, None,
                                   1e-6, kw.get("pos", P), P, kw.get("T", 4), 16, kw.get("out", P),
                                   ctypes.byref(_pool()), None)
    assert pa.STATUS[st] == status


def test_rope_axes_order():
    assert pa.rope_axes([2, 1, 3]) == bytes([0, 0, 1, 2, 2, 2])
    assert pa.rope_axes([2, 1, 3], woven=True) == bytes([0, 1, 2, 0, 2, 2])
    assert pa.rope_axes([0, 4], woven=True) == bytes([1] * 4)
    assert len(pa.rope_axes((16, 24, 24))) == 64
    for bad in ([], [1] * 5, [-1, 3], [0, 0], [40, 40]):
        with pytest.raises(ValueError):
            pa.rope_axes(bad)


def test_bindings_want_cuda_tensors():
    q = torch.zeros(3, 16, 128, dtype=torch.float16)
    kc = torch.zeros(4, 16, 8, 128, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises((TypeError, AssertionError, RuntimeError)):
        pa.paged_attn_tree(q, kc, kc, i.view(1, 3), i[:1], i[:1], i, 0.1)
    with pytest.raises((TypeError, AssertionError, RuntimeError)):
        pa.tree_accept(i.long(), i.long(), i, i[:1], i[:1])
    with pytest.raises(TypeError):
        pa.layer_pools([(kc, kc)])
