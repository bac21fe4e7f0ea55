"""GPU checks of what pa.kv_evict returns for a sequence that the device refuses,
through outputs that the binding allocates over memory with plausible contents."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_evict as evict

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _recycle(shape, value):
    """Blocks of this size that the allocator hands out next hold the value."""
    for t in [torch.full(shape, value, dtype=torch.int32, device=DEV) for _ in range(6)]:
        del t


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("heads,ctx", [(3, 100), (2, 60000)])
@pytest.mark.parametrize("what", ["zero", "negative", "beyond its table", "beyond the weights"])
def test_refused_sequences_through_outputs_of_the_binding(in_place, heads, ctx, what):
    c = evict._case([ctx - 5, ctx, 7, 70], heads, "bf16", 9, 32, in_place=in_place)
    lens = c["lens"].copy()
    lens[1] = dict(zero=0, negative=-3).get(what, 16 * c["bt"].shape[1] + 1)
    if what == "beyond the weights":
        c["w"] = c["w"][:, :, :ctx - 2].copy()
        c["dev"]["w"] = torch.from_numpy(c["w"]).to(DEV)
        lens[1] = ctx - 1
    x = dict(c, lens=lens, dev=dict(c["dev"], lens=torch.from_numpy(lens).to(DEV)))
    want, k, v, _ = evict._expect(x, 4, 2, np.zeros((4, heads, max(32, c["w"].shape[2])), np.float32), skip=(1,))
    pa.get_device_error()
    _recycle((4, heads, 32), 20)
    _recycle((4,), 20)
    kept, new, _, _ = evict._run(x, 4, 2, in_place=in_place)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1
    assert new.cpu().tolist() == [32, -1, 7, 32]
    assert np.array_equal(kept.cpu().numpy(), want)  # (-1 throughout for sequence 1)
    assert np.array_equal(evict.bits(c["kc"]), k) and np.array_equal(evict.bits(c["vc"]), v)


def test_a_given_output_keeps_what_it_held():
    c = evict._case([100, 90], 2, "f16", 10, 32)
    c["dev"]["lens"][1] = 0
    pa.get_device_error()
    mine = torch.full((2, 2, 32), 5, dtype=torch.int32, device=DEV)
    kept, new, _, _ = evict._run(c, 4, 2, kept=mine)
    assert kept is mine and bool((mine[1] == 5).all()) and new.cpu().tolist() == [32, -1]
    mine = torch.full((2,), 6, dtype=torch.int32, device=DEV)
    kept, new, _, _ = evict._run(c, 4, 2, new_context_lens=mine)
    assert mine.cpu().tolist() == [32, 6] and bool((kept[1] == -1).all())
    assert pa.STATUS[pa.get_device_error()[0]] == "PA_ERR_RANGE"


def test_the_length_of_a_refused_sequence_is_refused_by_what_follows():
    c = evict._case([100, 90], 2, "f16", 11, 32)
    c["dev"]["lens"][1] = 0
    _recycle((2,), 20)
    _, new, _, _ = evict._run(c, 4, 2)
    pa.get_device_error()
    out = torch.full((2, 4, 128), 7.0, device=DEV).half()
    q = torch.randn((2, 4, 128), device=DEV).half()
    pa.paged_attn_decode(q, c["kc"], c["vc"], c["dev"]["dst"], new, 0.1, out=out)
    st, detail = pa.get_device_error()
    assert pa.STATUS[st] == "PA_ERR_RANGE" and detail == 1 and bool((out[1] == 7.0).all())
