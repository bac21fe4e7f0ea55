"""GPU checks of the long-context calls at the ends of their ranges and in use
beside each other: as many sequences as a call takes, two streams at once, graphs
that take turns on one workspace, many steps of the rotary kernel's loop.
Tolerances: those of each operator's own tests."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_decode_shared as shared
import test_gpu_decode_weights as weights
import test_gpu_evict as evict
import test_gpu_rope_kv as rope
from longctx_reference import DIM, HALF_STEP

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = DIM ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    pa.get_device_error()
    yield
    st, detail = pa.get_device_error()
    assert st == 0, f"unexpected device error {pa.STATUS.get(st, st)} at index {detail}"


def test_shared_as_many_sequences_and_groups_as_a_call_takes():
    rng = np.random.default_rng(1)
    sizes = rng.integers(2, 20, pa.MAX_PREFIX_GROUPS - 1).tolist() + [1000]
    groups = [(16 * int(rng.integers(0, 4)), rng.integers(1, 20, n).tolist()) for n in sizes]
    c = shared._case(groups, 8, 4, "bf16", seed=2, alone=rng.integers(1, 40, 6000 - sum(sizes)).tolist())
    assert len(c["lens_h"]) == 6000
    out = shared._run(c)
    shared._check(c, out)
    # a small call behind it, and the plain decode of the same tables beside it
    small = shared._case([(64, [3, 5])], 8, 4, "bf16", seed=3)
    shared._check(small, shared._run(small))


def test_weights_as_many_sequences_as_a_call_takes():
    """16383 sequences of at most one page, over pages that they share (they are only read)."""
    g = torch.Generator(device=DEV).manual_seed(4)
    S, hkv, G, nb = 16383, 4, 2, 50
    kc, vc = (torch.randn((nb, 16, hkv, DIM), generator=g, device=DEV).half() for _ in range(2))
    q = torch.randn((S, hkv * G, DIM), generator=g, device=DEV).half()
    bt = torch.randint(0, nb, (S, 1), generator=g, device=DEV, dtype=torch.int32)
    lens = torch.randint(1, 17, (S,), generator=g, device=DEV, dtype=torch.int32)
    w_out = torch.full((S, hkv, 16), -1.0, device=DEV)
    out, _ = pa.paged_attn_decode_weights(q, kc, vc, bt, lens, SCALE, None, w_out)
    k, v = (x[bt[:, 0].long()].double().transpose(1, 2) for x in (kc, vc))  # [S, Hkv, 16, 128]
    qd = q.double().view(S, hkv, G, DIM)
    x = SCALE * qd @ k.transpose(2, 3)
    seen = (torch.arange(16, device=DEV) < lens[:, None])[:, None, None]
    p = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
    rel = float((SCALE * qd.abs() @ k.abs().transpose(2, 3)).max()) * 2.0 ** -17 + 2.0 ** -16
    ref, mag = p @ v, p @ v.abs()
    u = HALF_STEP["f16"]
    assert bool(((out.double().view(ref.shape) - ref).abs() <= u * ref.abs() + (1 + u) * mag * rel + 2.0 ** -25).all())
    want = torch.where(seen[:, :, 0], p.sum(2), -1.0)
    assert bool(((w_out.double() - want).abs() <= want.abs() * (rel + 2.0 ** -23)).all())


def test_evict_thousands_of_sequences():
    rng = np.random.default_rng(5)
    c = evict._case(rng.integers(1, 60, 3000), 2, "bf16", 6, 24, "ties")
    evict._check(c, recent=5, sinks=2)


@pytest.mark.parametrize("interleaved,rotary", [(True, 96), (False, 128), (False, 64), (False, 90)])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_many_steps_of_four_tokens(interleaved, rotary, norm):
    c = rope._case(4003, 5, 3, "f16", rotary, seed=rotary, norm=norm)
    bad = {7: (-1, None), 2000: (None, -5), 4002: (None, 10 ** 12)}
    for t, (pos, slot) in bad.items():
        if pos is not None:
            c["pos"][t] = pos
        if slot is not None:
            c["slots"][t] = slot
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    out = torch.full_like(c["q"], 3.0)
    rope._run(c, interleaved, factor=0.75, q_out=out)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail in bad
    assert all(bool((out[t] == 3.0).all()) for t in bad)
    rope._check(c, out, k0, v0, interleaved, 0.75, skip=tuple(bad))


def test_rope_in_place_over_many_steps():
    c = rope._case(2500, 8, 2, "bf16", 128, seed=9, norm=True)
    apart = rope._run(c, False)
    again = c["q"].clone()
    rope._run(dict(c, q=again), False, q_out=again)
    assert torch.equal(again, apart)


def test_two_streams_at_once():
    """Two decodes and two evictions on two streams, each with buffers of its own, many times over."""
    a = [shared._case([(2048, [30, 200, 7] * 10), (512, [50] * 5)], 32, 8, "bf16", seed=11 + i) for i in range(2)]
    b = [weights._case([3000, 17, 900, 2500], 16, 8, "f16", seed=21 + i) for i in range(2)]
    e = [evict._case([700, 5000, 33], 4, "bf16", 31 + i, 64) for i in range(2)]
    want = []
    for i in range(2):
        w = torch.zeros_like(b[i]["w"])
        out, _ = weights._run(b[i], b[i]["w"], w)
        want.append((shared._run(a[i]), out, w, evict._expect(e[i], 9, 3, np.full((3, 4, 64), 7.0, np.float32))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                w = torch.zeros_like(b[i]["w"])
                out, _ = weights._run(b[i], b[i]["w"], w)
                got[i].append((shared._run(a[i]), out, w))
    kept = []
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            kept.append(evict._run(e[i], 9, 3))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, want[i][:3]))
        k, kc, vc, w_out = want[i][3]
        assert np.array_equal(kept[i][0].cpu().numpy(), k)
        assert np.array_equal(evict.bits(e[i]["kc"]), kc) and np.array_equal(evict.bits(e[i]["vc"]), vc)
        assert np.array_equal(kept[i][2].cpu().numpy(), w_out)


def test_graphs_that_take_turns_on_one_workspace():
    """A shared decode and a decode with weights captured twice each; all four graphs use one workspace."""
    a = [shared._case([(1024, [30, 200, 7] * 4)], 16, 8, "f16", seed=41), shared._case([(160, [9, 500])], 16, 8, "f16",
                                                                                     seed=42)]
    b = [weights._case([3000, 17, 900], 16, 8, "f16", seed=43), weights._case([5, 1200], 16, 8, "f16", seed=44)]
    want = [shared._run(c).clone() for c in a]
    ww = []
    for c in b:
        w = torch.zeros_like(c["w"])
        want.append(weights._run(c, None, w)[0].clone())
        ww.append(w)
    need = max([pa.alloc_decode_shared_workspace(c["q"].shape[0], 1, 16, 8).numel() for c in a] +
               [pa.alloc_decode_weights_workspace(c["q"].shape[0], 16, 8, 16 * c["bt"].shape[1]).numel() for c in b])
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(x) for x in want]
    w_outs = [torch.zeros_like(w) for w in ww]
    calls = [lambda i=i: shared._run(a[i], out=outs[i], workspace=ws) for i in range(2)] + \
        [lambda i=i: weights._run(b[i], None, w_outs[i], out=outs[2 + i], workspace=ws) for i in range(2)]
    graphs = []
    for f in calls:
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for order in ([0, 1, 2, 3], [3, 0, 2, 1], [2, 2, 0, 0, 3, 1]):
        for x in outs + w_outs:
            x.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
        assert all(torch.equal(x, y) for x, y in zip(w_outs, ww))
