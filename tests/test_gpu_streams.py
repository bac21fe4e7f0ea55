"""GPU checks of calls on another stream than the current one that allocate their
own outputs and workspaces: that memory belongs to the stream of the call, so work
still queued on the current stream over a block it has freed cannot meet it, and an
output stays the caller's until the current stream is done with it."""
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_decode_shared as shared
import test_gpu_decode_weights as weights
import test_gpu_evict as evict
import test_gpu_rope_kv as rope
from longctx_reference import DIM

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = DIM ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def _calls():
    """name -> a call taking stream=, whose results do not depend on how often it ran."""
    hq, hkv = 16, 8
    c = weights._case([300, 5, 1000], hq, hkv, "f16", seed=1)
    s = shared._case([(512, [40, 3, 90])], hq, hkv, "f16", seed=2)
    e = evict._case([700, 33, 257], 4, "bf16", 3, 64)
    r = rope._case(40, hq, hkv, "f16", 96, seed=4)
    g = torch.Generator(device=DEV).manual_seed(5)
    randn = lambda *n: torch.randn(n, generator=g, device=DEV).half()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    qc = randn(70, hq, DIM)
    pages = c["bt"][:1, :19].contiguous()  # one chunk of 70 tokens at the end of 300
    one = dict(starts=i32(230), lens=i32(70), ctx=i32(300))
    kq, vq, ks, vs = pa.alloc_pool_q8(c["kc"].shape[0], hkv)
    kf, vf, fs, gs = pa.alloc_pool_f8(c["kc"].shape[0], hkv)
    everywhere = torch.arange(c["kc"].shape[0] * 16, device=DEV)
    rows_k, rows_v = (x.flatten(0, 1).nan_to_num().contiguous() for x in (c["kc"], c["vc"]))
    pa.kv_cache_write_q8(rows_k, rows_v, everywhere, kq, vq, ks, vs)
    pa.kv_cache_write_f8(rows_k, rows_v, everywhere, kf, vf, fs, gs)
    kn, vn = randn(3, hkv, DIM), randn(3, hkv, DIM)
    kt, vt, qt = randn(40, hkv, DIM), randn(40, hkv, DIM), randn(40, hq, DIM)
    table = torch.rand((64, DIM), generator=g, device=DEV).half()
    norm, pos = torch.ones(DIM, device=DEV).half(), r["pos"] % 64
    base = (c["q"], c["kc"], c["vc"], c["bt"], c["lens"], SCALE)
    w_out = torch.zeros_like(c["w"])
    mixed_ws = pa.alloc_mixed_step_workspace(3, hq, hkv)
    d = e["dev"]
    e_out = torch.full((3, 4, 64), 7.0, device=DEV)
    chunk_args = (qc, one["starts"], one["lens"])
    return dict(
        decode=lambda **kw: pa.paged_attn_decode(*base, **kw),
        decode_window=lambda **kw: pa.paged_attn_decode_window(*base, 100, **kw),
        decode_append=lambda **kw: pa.paged_attn_decode_append(c["q"], kn, vn, *base[1:], **kw),
        decode_noalloc=lambda **kw: pa.paged_attn_decode_noalloc(*base, **kw),
        decode_q8=lambda **kw: pa.paged_attn_decode_q8(c["q"], kq, vq, ks, vs, c["bt"], c["lens"], SCALE, **kw),
        decode_f8=lambda **kw: pa.paged_attn_decode_f8(c["q"], kf, vf, fs, gs, c["bt"], c["lens"], SCALE, **kw),
        prefill=lambda **kw: pa.paged_attn_prefill_chunk(*chunk_args, c["kc"], c["vc"], pages, one["ctx"], SCALE, **kw),
        prefill_q8=lambda **kw: pa.paged_attn_prefill_chunk_q8(*chunk_args, kq, vq, ks, vs, pages, one["ctx"], SCALE,
                                                               **kw),
        mixed_step=lambda **kw: pa.mixed_step(c["kc"], c["vc"], SCALE, mixed_ws, q=c["q"], block_tables=c["bt"],
                                              context_lens=c["lens"], **kw)[1],
        qk_norm_rope=lambda **kw: pa.qk_norm_rope_kv_write(qt, kt, vt, norm, norm, 1e-6, table, table, pos,
                                                           r["slots"], r["kc"], r["vc"], **kw),
        rope=lambda **kw: rope._run(r, True, **kw),
        shared=lambda **kw: shared._run(s, **kw),
        weights=lambda **kw: pa.paged_attn_decode_weights(*base, c["w"], w_out, **kw),
        evict=lambda **kw: pa.kv_evict(e["kc"], e["vc"], d["bt"], d["lens"], d["w"], 64, 9, 3, d["dst"], e_out, **kw),
    )


NAMES = ["decode", "decode_window", "decode_append", "decode_noalloc", "decode_q8", "decode_f8", "prefill", "prefill_q8",
         "mixed_step", "qk_norm_rope", "rope", "shared", "weights", "evict"]


def _results(x):
    return [t for t in (x if isinstance(x, tuple) else (x,))]


def _stream_of_block(t):
    """The stream whose part of the allocator a tensor's memory belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_call_belongs_to_its_stream(name, monkeypatch):
    call = _calls()[name]
    want = [t.clone() for t in _results(call())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    spaces = []
    for fn in [n for n in dir(pa) if n.startswith("alloc_") and n.endswith("_workspace")]:
        def make(*a, _f=getattr(pa, fn), **kw):
            spaces.append(torch.cuda.current_stream().cuda_stream)
            return _f(*a, **kw)
        monkeypatch.setattr(pa, fn, make)
    got = _results(call(stream=side))
    torch.cuda.synchronize()
    given = [t for t in got if name != "weights" or t is not got[1]]  # (weights_out is the caller's)
    assert all(_stream_of_block(t) == side.cuda_stream for t in given)
    assert all(s == side.cuda_stream for s in spaces)
    assert len(spaces) == (name in ("decode", "decode_window", "decode_append", "decode_q8", "decode_f8", "shared", "weights"))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_behind_queued_work_over_freed_memory(name):
    """The current stream still has fills of freed blocks of every likely size to come when the call runs."""
    call = _calls()[name]
    want = [t.clone() for t in _results(call())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(60_000_000)
    for shift in range(9, 26):
        junk = [torch.empty(3 << (shift - 1), dtype=torch.uint8, device=DEV) for _ in range(2)]
        for j in junk:
            j.fill_(0x55)
        del junk, j
    got = _results(call(stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_results_last_until_the_current_stream_is_done(name):
    call = _calls()[name]
    want = [t.clone() for t in _results(call())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _results(call(stream=side))
    sizes = [t.numel() * t.element_size() for t in got]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(60_000_000)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        for n in sizes * 2:
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x55)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
