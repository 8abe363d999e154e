"""What the calls of the 8-bit paged cache promise, without a GPU: overlaps that are refused, the number of rows from which
the caches are expanded."""
import ctypes

import pytest

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib
from tests.test_q8_host import _append, _append8, _cache, _cache8, _rope, _shape

P = ctypes.c_void_p
BASE = 1 << 32  # aligned, never dereferenced: every call below fails validation first


# ----------------------------------------------------------------------------- overlaps
@pytest.mark.parametrize("heads", [2, 16])
def test_rotated_queries_may_not_overwrite_inputs(heads):
    """Other blocks still read the new keys and values, the frequencies and the positions when a query is written."""
    s = _shape(h=heads)
    tokens = 2 * 8
    qb, kb = tokens * heads * 128 * 2, tokens * 2 * 128 * 2
    far = BASE << 1
    for at in (BASE, BASE + kb - 16, BASE - qb + 16):
        for k, v in ((BASE, far), (far, BASE)):
            r = _rope(q=far << 1, q_out=at)
            for call, c in ((_append, _cache()), (_append8, _cache8())):
                assert call(s, c, r, k=P(k), v=P(v)) == 1
                assert b"overlap" in nsa.load().nsa_last_error()
    for name, size in (("inv_freq", 64 * 4), ("positions", tokens * 4)):
        for at in (BASE, BASE + size - 16, BASE - qb + 16):
            r = _rope(q=far << 1, q_out=at, **{name: BASE})
            for call, c in ((_append, _cache()), (_append8, _cache8())):
                assert call(s, c, r, k=P(far), v=P(far)) == 1
                assert b"overlap" in nsa.load().nsa_last_error()


# ----------------------------------------------------------------------------- forms
@pytest.mark.parametrize("h,h_kv", [(1, 1), (16, 2), (6, 2), (128, 1)])
def test_the_number_of_rows_that_expands(h, h_kv):
    """256 rows read the codes as they are (no bound of the lengths sizes the workspace), 257 do not."""
    lib = nsa.load()

    def sized_by_the_bound(q_len):
        s = _shape(seqlen=q_len, h=h, h_kv=h_kv)
        c = _cache8(max_pages=1 << 12, page_stride=64 * h_kv * 128)
        size = [lib.nsa_paged_q8_attn_fwd_workspace_size(ctypes.byref(s), ctypes.byref(c), b, 0, 0) for b in (64, 1 << 18)]
        return size[0] != size[1]

    group = h // h_kv
    assert not sized_by_the_bound(1) and not sized_by_the_bound(256 // group)
    assert sized_by_the_bound(256 // group + 1) and sized_by_the_bound(4096)
