"""Host checks of pa_tree_accept_ex's choices after the committed context (no GPU): nothing is enqueued."""
import pytest

import paged_kv_gqa_cache_gb300 as pa
from test_tree_host import P, _apart, _pool, lib  # noqa: F401 (lib: a fixture)


def _accept_ex(lib, a, choice, S=4):
    pools = (pa.KVPool * 2)(_pool(), _pool(k_cache=1 << 14, v_cache=1 << 15))
    return lib.pa_tree_accept_ex(a["draft"], a["target"], choice, a["parents"], 20, a["n"], a["lens"], S, pools, 2,
                                 a["bt"], 16, a["path"], 8, a["plens"], a["next"], a["new"], None)


def test_a_misaligned_choice(lib):  # noqa: F811
    assert pa.STATUS[_accept_ex(lib, _apart(), P + (20 << 16) + 4)] == "PA_ERR_ALIGN"


@pytest.mark.parametrize("out,off", [("next", 0), ("next", 24), ("path", 120), ("plens", 8), ("new", 8)])
def test_a_choice_that_overlaps_an_output(lib, out, off):  # noqa: F811
    a = _apart()
    assert pa.STATUS[_accept_ex(lib, a, a[out] + off)] == "PA_ERR_SHAPE"


def test_no_sequences(lib):  # noqa: F811
    assert pa.STATUS[_accept_ex(lib, _apart(), None, S=0)] == "PA_OK"
