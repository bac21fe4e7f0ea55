"""GPU checks of pa.rope_kv_write on buffers that lie next to each other, and of its
refusals of those that overlap and of shapes that are none."""
import pytest
import torch

import paged_kv_gqa_cache_gb300 as pa
import test_gpu_rope_kv as rope
from longctx_reference import DIM

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [5, 700])
def test_neighbours_in_one_buffer(T):
    """k, the output, q, v one behind the other."""
    hq, hkv = 8, 2
    c = rope._case(T, hq, hkv, "bf16", 96, seed=T)
    buf = torch.zeros((T * (2 * hq + 2 * hkv), DIM), device=DEV).bfloat16()
    parts = [x.view(T, -1, DIM) for x in buf.split([T * hkv, T * hq, T * hq, T * hkv])]
    for at, name in ((0, "k"), (2, "q"), (3, "v")):
        parts[at].copy_(c[name])
    x = dict(c, k=parts[0], q=parts[2], v=parts[3])
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    out = rope._run(x, True, q_out=parts[1])
    rope._check(x, out, k0, v0, True)
    assert torch.equal(parts[2], c["q"]) and torch.equal(parts[0], c["k"])


def test_overlaps_are_refused():
    T, hq, hkv = 6, 4, 2
    c = rope._case(T, hq, hkv, "f16", 128, seed=1)
    buf = torch.zeros((T + 1, hq, DIM), device=DEV).half()
    buf[:T].copy_(c["q"])
    over_k = torch.zeros((T, hq, DIM), device=DEV).half()
    for q, k, out in ((buf[:T], c["k"], buf[1:]), (buf[1:], c["k"], buf[:T]),
                      (c["q"], over_k.view(-1)[:T * hkv * DIM].view(T, hkv, DIM), over_k)):
        before = [t.clone() for t in (q, k, out, c["kc"])]
        with pytest.raises(pa.PagedAttnError) as e:
            rope._run(dict(c, q=q, k=k), False, q_out=out)
        assert pa.STATUS[e.value.status] == "PA_ERR_SHAPE"
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16))
                   for a, b in zip((q, k, out, c["kc"]), before))


@pytest.mark.parametrize("shape", [(), (DIM,), (6, 4 * DIM), (6, 4, 1, DIM)])
def test_queries_that_are_no_rows_of_heads(shape):
    c = rope._case(6, 4, 2, "f16", 128, seed=2)
    with pytest.raises(ValueError):
        rope._run(dict(c, q=torch.zeros(shape, device=DEV).half()), False)
