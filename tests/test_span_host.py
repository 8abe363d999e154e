"""Paged-cache and sink-window operators without a GPU: the 64-bit reference against library
attention, hand counts and differences, and every refusal of the C and Python entry points."""
import ctypes
import math

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib
from tests import span_reference as ref

P = ctypes.c_void_p
FAKE = P(0x10000)  # aligned, never dereferenced: every call below fails validation first
MIS = P(0x10002)


# ----------------------------------------------------------------------------- the reference
def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (5, 0), (5, 3), (64, 4), (3, 100)])
def test_reference_attention_matches_library_attention(window, n_sink):
    Q, n, H, hk, d = 9, 21, 6, 2, 16
    q, k, v = _rand(Q, H, d, seed=1), _rand(n, hk, d, seed=2), _rand(n, hk, d, seed=3)
    see = ref.visible(range(n - Q, n), n, window, n_sink)
    for i in range(Q):  # the mask, counted by hand
        p = n - Q + i
        for j in range(n):
            want = j <= p and (window == 0 or j > p - window or j < n_sink)
            assert bool(see[i, j]) == want
    o, lse, _, _ = ref.attend(q, k, v, see, 0.25)
    kk, vv = (x.repeat_interleave(H // hk, 1).transpose(0, 1) for x in (k, v))
    lib = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=see, scale=0.25)
    assert torch.allclose(o, lib.transpose(0, 1), atol=1e-12)
    w, _ = ref.key_weights(q, k, see, lse, 0.25)
    assert math.isclose(float(w.sum()), Q * H, rel_tol=1e-12)  # every row's probabilities add up to one


def test_reference_rows_without_keys():
    q, k, v = _rand(3, 2, 8), _rand(2, 1, 8, seed=1), _rand(2, 1, 8, seed=2)
    o, lse, _, _ = ref.attend(q, k, v, ref.visible([-1, 0, 1], 2, 0, 0), 1.0)
    assert torch.equal(o[0], torch.zeros(2, 8, dtype=torch.float64)) and torch.isinf(lse[0]).all()
    assert torch.allclose(o[1, 0], v[0, 0])


@pytest.mark.parametrize("window,n_sink", [(4, 0), (4, 3), (100, 2)])
def test_reference_gradients_match_differences(window, n_sink):
    T, H, hk, d = 11, 4, 2, 8
    q, k, v, do = (_rand(T, h, d, seed=s) for s, h in enumerate((H, hk, hk, H)))
    see = ref.visible(range(T), T, window, n_sink)
    o, lse, _, _ = ref.attend(q, k, v, see, 0.3)
    grads, _ = ref.gradients(q, k, v, do, o, lse, see, 0.3)

    def loss(a, b, c):
        return float((ref.attend(a, b, c, see, 0.3)[0] * do).sum())

    for at in range(3):
        step = _rand(*(q, k, v)[at].shape, seed=10 + at)
        up, down = [list((q, k, v)) for _ in range(2)]
        up[at], down[at] = up[at] + 1e-5 * step, down[at] - 1e-5 * step
        diff = (loss(*up) - loss(*down)) / 2e-5
        assert math.isclose(diff, float((grads[at] * step).sum()), rel_tol=1e-6, abs_tol=1e-7)


def test_reference_choice():
    inf, nan = math.inf, math.nan
    w = [0.0, 5.0, 1.0, 1.0, -inf, nan, 1.0, inf, -0.0, 2.0]
    assert ref.choose(w, 10, 10, 0, 0) == list(range(10))
    assert ref.choose(w, 10, 3, 0, 0) == [1, 7, 9]
    assert ref.choose(w, 10, 5, 0, 0) == [1, 2, 3, 7, 9]       # equal weights: the lower positions
    assert ref.choose(w, 10, 9, 0, 0) == [0, 1, 2, 3, 4, 6, 7, 8, 9]  # NaN goes first
    assert ref.choose(w, 10, 4, 1, 2) == [0, 7, 8, 9]
    assert ref.choose(w, 10, 3, 1, 2) == [0, 8, 9]


# ----------------------------------------------------------------------------- refusals, C
def _shape(**kw):
    s = _lib.NsaShape()
    s.batch, s.seqlen, s.h, s.h_kv, s.d, s.dtype = 2, 128, 16, 2, 128, _lib.NSA_BF16
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _cache(**kw):
    c = _lib.NsaPagedCache()
    for n in ("k_pages", "v_pages", "weights", "block_table", "cache_lens"):
        setattr(c, n, 0x10000)
    c.n_pages, c.page_size, c.max_pages, c.page_stride = 8, 64, 4, 64 * 2 * 128
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(s, c):
    return nsa.load().nsa_paged_append(ctypes.byref(s), FAKE, FAKE, ctypes.byref(c), None)


def _attn(s, c, window=0, n_sink=0, bound=0, q=FAKE, o=FAKE, lse=None, ws=FAKE, n=1 << 40):
    return nsa.load().nsa_paged_attn_fwd(ctypes.byref(s), q, ctypes.byref(c), bound, window, n_sink, 0.0, o, lse, ws, n,
                                         None)


def _weights(s, c, window=0, n_sink=0, lse=FAKE, out=FAKE):
    return nsa.load().nsa_paged_attn_weights(ctypes.byref(s), FAKE, ctypes.byref(c), lse, window, n_sink, 0.0, 1.0, out,
                                             None)


def _evict(c, n=2, hk=2, d=128, budget=64, sink=4, recent=16, table=FAKE, pages=1, keep=FAKE, lens=FAKE):
    return nsa.load().nsa_paged_evict(n, hk, d, ctypes.byref(c), budget, sink, recent, table, pages, keep, lens, None)


def _sink_fwd(s, window=64, n_sink=4, q=FAKE, ws=FAKE, n=1 << 40):
    return nsa.load().nsa_swa_sink_fwd(ctypes.byref(s), q, FAKE, FAKE, window, n_sink, 0.0, FAKE, None, ws, n, None)


def _sink_bwd(s, window=64, n_sink=4, lse=FAKE, ws=FAKE, n=1 << 40):
    return nsa.load().nsa_swa_sink_bwd(ctypes.byref(s), FAKE, FAKE, FAKE, window, n_sink, 0.0, FAKE, lse, FAKE, FAKE,
                                       FAKE, FAKE, ws, n, None)


@pytest.mark.parametrize("kw,expect", [
    ({"h": 0}, 1), ({"h": 15}, 1), ({"dtype": 7}, 1), ({"batch": -1}, 1), ({"dtype": _lib.NSA_F32}, 2), ({"d": 96}, 2),
    ({"h": 258, "h_kv": 2}, 2), ({"batch": 65536, "seqlen": 1}, 2), ({"batch": 1 << 20, "seqlen": 1 << 20}, 2),
])
def test_shapes_refused(kw, expect):
    s = _shape(**kw)
    for call in (lambda: _append(s, _cache()), lambda: _attn(s, _cache()), lambda: _weights(s, _cache()),
                 lambda: _sink_fwd(s), lambda: _sink_bwd(s)):
        assert call() == expect
        assert nsa.load().nsa_last_error()


@pytest.mark.parametrize("kw,expect", [
    ({"k_pages": None}, 1), ({"k_pages": 0x10008}, 1), ({"block_table": None}, 1), ({"cache_lens": None}, 1),
    ({"block_table": 0x10002}, 1), ({"n_pages": 0}, 1), ({"max_pages": 0}, 1), ({"page_size": 0}, 2),
    ({"page_size": 48}, 2), ({"page_size": 8}, 2), ({"page_size": 512}, 2), ({"page_stride": 64 * 2 * 128 - 8}, 1),
    ({"page_stride": 64 * 2 * 128 + 4}, 1), ({"page_stride": 1 << 38}, 2), ({"max_pages": 1 << 24}, 2),
    ({"weights": 0x10001}, 1),
])
def test_caches_refused(kw, expect):
    c = _cache(**kw)
    for call in (lambda: _append(_shape(), c), lambda: _attn(_shape(), c), lambda: _weights(_shape(), c),
                 lambda: _evict(c)):
        assert call() == expect
        assert nsa.load().nsa_last_error()


def test_calls_refused():
    s, c = _shape(), _cache()
    assert _append(s, _cache(v_pages=None)) == 1
    assert _attn(s, _cache(v_pages=None)) == 1
    assert _attn(s, c, window=-1) == 1 and _attn(s, c, n_sink=-1) == 1 and _attn(s, c, bound=-1) == 1
    assert _attn(s, c, window=(1 << 28) + 1) == 2
    assert _attn(s, c, q=None) == 1 and _attn(s, c, o=MIS) == 1 and _attn(s, c, lse=MIS) == 1
    one = _shape(seqlen=1)  # few rows: the keys are divided and the call needs a workspace
    need = nsa.load().nsa_paged_attn_fwd_workspace_size(ctypes.byref(one), 4096, 0, 0)
    assert need > 0
    assert _attn(one, c, bound=4096, ws=None) == 1 and _attn(one, c, bound=4096, ws=MIS) == 1
    assert _attn(one, c, bound=4096, n=need - 1) == 1
    assert _weights(s, c, lse=None) == 1 and _weights(s, c, out=None) == 1 and _weights(s, c, out=MIS) == 1
    assert _evict(_cache(weights=None)) == 1
    assert _evict(c, budget=0) == 1 and _evict(c, sink=-1) == 1 and _evict(c, sink=60, recent=5) == 1
    assert _evict(c, n=-1) == 1 and _evict(c, n=65536) == 2 and _evict(c, d=96) == 2
    assert _evict(_cache(max_pages=1), budget=(1 << 28) + 1) == 2
    assert _evict(c, budget=65) == 1  # one page of 64 does not hold it
    assert _evict(c, table=None) == 1 and _evict(c, keep=None) == 1 and _evict(c, lens=MIS) == 1
    assert _sink_fwd(s, window=0) == 1 and _sink_fwd(s, n_sink=-1) == 1 and _sink_fwd(s, q=None) == 1
    assert _sink_bwd(s, window=0) == 1 and _sink_bwd(s, n_sink=1025) == 2 and _sink_bwd(s, lse=None) == 1
    need = nsa.load().nsa_swa_sink_bwd_workspace_size(ctypes.byref(s), 64, 4)
    assert need > 0 and _sink_bwd(s, n=need - 1) == 1 and _sink_bwd(s, ws=None) == 1


def test_overlapping_outputs_refused():
    """Addresses are compared, never read."""
    lib, s, c = nsa.load(), ctypes.byref(_shape()), _cache()
    tokens, h, hk, d = _shape().batch * _shape().seqlen, _shape().h, _shape().h_kv, _shape().d
    qb, kb, at = tokens * h * d * 2, tokens * hk * d * 2, 1 << 32
    q, k, v, o, d_o, dq, dk, dv = (at + i * (qb + 256) for i in range(8))
    assert lib.nsa_paged_attn_fwd(s, q, ctypes.byref(c), 0, 0, 0, 0.0, q, None, FAKE, 1 << 40, None) == 1
    assert b"overlap" in lib.nsa_last_error()
    assert lib.nsa_paged_attn_fwd(s, q, ctypes.byref(c), 0, 0, 0, 0.0, q + qb - 16, None, FAKE, 1 << 40, None) == 1
    for bad in (q, q - qb + 16, k, k + kb - 16, v):
        assert lib.nsa_swa_sink_fwd(s, q, k, v, 64, 4, 0.0, bad, None, FAKE, 1 << 40, None) == 1
        assert b"overlap" in lib.nsa_last_error()
    for bad in ((q, dk, dv), (dq, k, dv), (dq, dk, o), (d_o, dk, dv), (dq, dq, dv), (dq, dk, dk), (dq, dk, dk + kb - 16)):
        assert lib.nsa_swa_sink_bwd(s, q, k, v, 64, 4, 0.0, o, FAKE, d_o, *bad, FAKE, 1 << 40, None) == 1
        assert b"overlap" in lib.nsa_last_error()


def test_nothing_to_do_is_no_error():
    empty = _shape(batch=0)
    assert _append(empty, _cache()) == 0 and _attn(empty, _cache()) == 0 and _weights(empty, _cache()) == 0
    assert _sink_fwd(empty) == 0 and _sink_bwd(empty) == 0 and _evict(_cache(), n=0) == 0


# ----------------------------------------------------------------------------- refusals, Python
def test_python_refuses_tensors_of_the_cpu():
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        nsa.nsa_paged_attn_fwd(z(1, 4, 64), z(2, 16, 2, 64), z(2, 16, 2, 64), z(1, 2), z(1))
    with pytest.raises(ValueError, match="GPU"):
        nsa.nsa_swa_sink_fwd(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64))


def test_python_checks():
    """The checks themselves, on CPU tensors."""
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(3, 16, 2, 64, dtype=bf)
    table, lens = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)
    c, page, hk, d = _lib._paged_cache("f", k, k, table, lens, 2)
    assert (c.n_pages, c.page_size, c.max_pages, c.page_stride, page, hk, d) == (3, 16, 4, 16 * 2 * 64, 16, 2, 64)
    pool = torch.zeros(3, 2, 16, 2, 64, dtype=bf)  # K and V of a page side by side
    assert _lib._paged_cache("f", pool[:, 0], pool[:, 1], table, lens, 2)[0].page_stride == 2 * 16 * 2 * 64
    for bad in (dict(v=torch.zeros(3, 16, 2, 128, dtype=bf)), dict(k=k.transpose(1, 2)), dict(k=k.float()),
                dict(k=k[..., :32]), dict(k=k[0]), dict(table=table.long()), dict(table=table.t()), dict(lens=lens[:1]),
                dict(v=pool[:, 0]), dict(table=torch.zeros(2, 8, dtype=i32)[:, ::2]),
                dict(w=torch.zeros(3, 16, 2)), dict(w=torch.zeros(3, 2, 16, dtype=torch.float64))):
        with pytest.raises((TypeError, ValueError)):
            _lib._paged_cache("f", bad.get("k", k), bad.get("v", bad.get("k", k)), bad.get("table", table),
                              bad.get("lens", lens), 2, bad.get("w"))
    q = torch.zeros(5, 4, 64, dtype=bf)
    cu = torch.zeros(3, dtype=i32)
    assert _lib._span_shape("f", q, 2, 64, q.device, cu, 3)[2] == 2
    with pytest.raises(ValueError):
        _lib._span_shape("f", q, 0, 64, q.device, cu, 3)
    for args in ((q.float(), cu), (q[:, :3], cu), (q[..., :32], cu), (q[:, ::2], cu), (q, cu.long()), (q, cu[:1]),
                 (q[None], cu)):
        with pytest.raises((TypeError, ValueError)):
            _lib._span_shape("f", args[0], 2, 64, q.device, args[1], 3)
