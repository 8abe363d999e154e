"""The rotating append and the 8-bit paged cache without a GPU: the 64-bit reference against independent forms, and
every refusal of the C and Python entry points."""
import ctypes
import os
import re

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib
from tests import q8_reference as ref8
from tests import span_reference as ref

P = ctypes.c_void_p
FAKE = P(0x10000)  # aligned, never dereferenced: every call below fails validation first
MIS = P(0x10002)
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_compress_gb300", "csrc")


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


# ----------------------------------------------------------------------------- the reference
def test_reference_code_is_the_cast():
    x = torch.cat([_rand(50000) * 10 ** (7 * torch.rand(50000, dtype=torch.float64) - 5),
                   torch.tensor([0.0, 2 ** -10, 3 * 2 ** -10, 2 ** -6, 17.0, 19.0, 248.0, 432.0, 448.0, -448.0]).double()])
    x = x.float().clamp(-448, 448)
    assert torch.equal(ref8.code(x), x.to(torch.float8_e4m3fn).double())
    assert ref8.code(torch.tensor([1e9, -500.0])).tolist() == [448.0, -448.0]


def test_reference_scales():
    for top, want in ((0.0, 2.0 ** -60), (448.0, 1.0), (448.0001, 2.0), (447.0, 1.0), (224.0, 0.5), (1e-30, 2.0 ** -60),
                      (1e30, 2.0 ** 60), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7)):
        assert ref8.scale_for(top) == want


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_is_a_complex_product(interleaved):
    x, n = _rand(7, 3, 16, seed=1), 5
    f, pos = torch.rand(n, generator=torch.Generator().manual_seed(2)), torch.tensor([0, 1, -3, 100, 4096, 7, 2])
    got, _ = ref8.rotate(x, f, pos, interleaved)
    j = torch.arange(n)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
    z = torch.complex(x[..., a], x[..., b]) * torch.exp(1j * pos[:, None, None].double() * f.double())
    assert torch.allclose(got[..., a], z.real, atol=1e-12) and torch.allclose(got[..., b], z.imag, atol=1e-12)
    assert torch.equal(got[..., 2 * n:], x[..., 2 * n:])
    # what attention sees depends on the distance alone
    k, _ = ref8.rotate(x, f, pos + 50, interleaved)
    q, _ = ref8.rotate(x.flip(0), f, pos + 50, interleaved)
    q0, _ = ref8.rotate(x.flip(0), f, pos, interleaved)
    assert torch.allclose((k * q).sum(-1), (got * q0).sum(-1), atol=1e-10)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (5, 3)])
def test_reference_attention_is_that_of_the_values(window, n_sink):
    Q, n, H, hk, d = 6, 21, 4, 2, 16
    q, kc, vc = _rand(Q, H, d, seed=3), _rand(n, hk, d, seed=4), _rand(n, hk, d, seed=5)
    ks, vs = torch.exp2(_rand(n, hk, seed=6).round()), torch.exp2(_rand(n, hk, seed=7).round())
    see = ref.visible(range(n - Q, n), n, window, n_sink)
    o, lse, _, _ = ref8.attend(q, kc, ks, vc, vs, see, 0.25)
    o2, lse2, _, _ = ref.attend(q, kc * ks[..., None], vc * vs[..., None], see, 0.25)
    assert torch.allclose(o, o2, atol=1e-12) and torch.allclose(lse, lse2, atol=1e-12)


def test_reference_store():
    old = ref8.code(torch.tensor([[400.0, -3.0], [0.0, 2.0 ** -9]]))
    codes = torch.cat([old, torch.full((2, 2), 7.0, dtype=torch.float64)])
    got, s = ref8.store(codes, 1.0, 2, torch.tensor([[100.0, 1.0]]).double())
    assert s == 1.0 and torch.equal(got[:2], old) and got[2].tolist() == [ref8.code(torch.tensor(100.0)), 1.0]
    assert (got[3] == 7).all()
    got, s = ref8.store(codes, 1.0, 2, torch.tensor([[1000.0, 1.0]]).double())
    assert s == 4.0 and got[0].tolist() == [ref8.code(torch.tensor(100.0)), -0.75] and got[1].tolist() == [0.0, 0.0]
    got, s = ref8.store(codes, 1.0, 0, torch.tensor([[1e-3, 0.0]]).double())
    assert s == 2.0 ** -18 and got[0, 0] * s == pytest.approx(1e-3, rel=2 ** -4)


# ----------------------------------------------------------------------------- refusals, C
def _shape(**kw):
    s = _lib.NsaShape()
    s.batch, s.seqlen, s.h, s.h_kv, s.d, s.dtype = 2, 8, 16, 2, 128, _lib.NSA_BF16
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _fill(c, kw):
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _cache(**kw):
    c = _lib.NsaPagedCache()
    for n in ("k_pages", "v_pages", "weights", "block_table", "cache_lens"):
        setattr(c, n, 0x10000)
    c.n_pages, c.page_size, c.max_pages, c.page_stride = 8, 64, 4, 64 * 2 * 128
    return _fill(c, kw)


def _cache8(**kw):
    c = _lib.NsaPagedCacheQ8()
    for n in ("k_pages", "v_pages", "k_scales", "v_scales", "block_table", "cache_lens"):
        setattr(c, n, 0x10000)
    c.n_pages, c.page_size, c.max_pages, c.block_size, c.page_stride = 8, 64, 4, 64, 64 * 2 * 128
    return _fill(c, kw)


def _rope(**kw):
    return _fill(_lib.NsaRope(0x10000, None, 128, 0, None, None), kw)


def _append(s, c, r=None, k=FAKE, v=FAKE):
    return nsa.load().nsa_paged_append_rope(ctypes.byref(s), k, v, ctypes.byref(_rope() if r is None else r),
                                            ctypes.byref(c), None)


def _append8(s, c, r=None, k=FAKE, v=FAKE):
    return nsa.load().nsa_paged_q8_append(ctypes.byref(s), k, v, None if r is None else ctypes.byref(r), ctypes.byref(c),
                                          None)


def _attn8(s, c, window=0, n_sink=0, bound=0, q=FAKE, o=FAKE, lse=None, ws=FAKE, n=1 << 50):
    return nsa.load().nsa_paged_q8_attn_fwd(ctypes.byref(s), q, ctypes.byref(c), bound, window, n_sink, 0.0, o, lse, ws, n,
                                            None)


@pytest.mark.parametrize("kw,expect", [
    ({"h": 0}, 1), ({"h": 15}, 1), ({"dtype": 7}, 1), ({"batch": -1}, 1), ({"dtype": _lib.NSA_F32}, 2), ({"d": 96}, 2),
    ({"h": 258, "h_kv": 2}, 2), ({"batch": 65536, "seqlen": 1}, 2), ({"batch": 1 << 20, "seqlen": 1 << 20}, 2),
])
def test_shapes_refused(kw, expect):
    s = _shape(**kw)
    for call in (lambda: _append(s, _cache()), lambda: _append8(s, _cache8()), lambda: _attn8(s, _cache8())):
        assert call() == expect
        assert nsa.load().nsa_last_error()


COMMON = [
    ({"k_pages": None}, 1), ({"v_pages": None}, 1), ({"k_pages": 0x10008}, 1), ({"block_table": None}, 1),
    ({"cache_lens": None}, 1), ({"block_table": 0x10002}, 1), ({"n_pages": 0}, 1), ({"max_pages": 0}, 1),
    ({"page_size": 0}, 2), ({"page_size": 48}, 2), ({"page_size": 512}, 2), ({"page_stride": 64 * 2 * 128 - 16}, 1),
    ({"page_stride": 64 * 2 * 128 + 4}, 1), ({"page_stride": 1 << 38}, 2), ({"max_pages": 1 << 24}, 2),
]


@pytest.mark.parametrize("kw,expect", COMMON)
def test_caches_refused(kw, expect):
    for call in (lambda: _append(_shape(), _cache(**kw)), lambda: _append8(_shape(), _cache8(**kw)),
                 lambda: _attn8(_shape(), _cache8(**kw))):
        assert call() == expect
        assert nsa.load().nsa_last_error()


@pytest.mark.parametrize("kw,expect", [
    ({"k_scales": None}, 1), ({"v_scales": None}, 1), ({"v_scales": 0x10002}, 1), ({"block_size": 0}, 2),
    ({"block_size": 8}, 2), ({"block_size": 48}, 2), ({"block_size": 128}, 2), ({"page_size": 256, "block_size": 256, "page_stride": 256 * 2 * 128}, 2),
    ({"page_stride": 64 * 2 * 128 + 8}, 1),  # fine for bf16 pages, no 16 bytes here
])
def test_8_bit_caches_refused(kw, expect):
    for call in (_append8, _attn8):
        assert call(_shape(), _cache8(**kw)) == expect
        assert nsa.load().nsa_last_error()
    need = nsa.load().nsa_paged_q8_attn_fwd_workspace_size(ctypes.byref(_shape()), ctypes.byref(_cache8(**kw)), 0, 0, 0)
    assert need == 0


@pytest.mark.parametrize("kw,expect", [
    ({"rot_dim": 0}, 2), ({"rot_dim": 8}, 2), ({"rot_dim": 24}, 2), ({"rot_dim": 144}, 2), ({"rot_dim": -16}, 2),
    ({"inv_freq": None}, 1), ({"inv_freq": 0x10002}, 1), ({"positions": 0x10001}, 1), ({"q": 0x10000}, 1),
    ({"q_out": 0x10000}, 1), ({"q": 0x10000, "q_out": 0x10008}, 1), ({"q": 0x10000, "q_out": 0x10010}, 1),
])
def test_rotations_refused(kw, expect):
    assert _append(_shape(), _cache(), _rope(**kw)) == expect
    assert _append8(_shape(), _cache8(), _rope(**kw)) == expect
    assert nsa.load().nsa_last_error()


def test_calls_refused():
    s, c = _shape(), _cache8()
    lib = nsa.load()
    assert lib.nsa_paged_append_rope(ctypes.byref(s), FAKE, FAKE, None, ctypes.byref(_cache()), None) == 1
    assert lib.nsa_paged_append_rope(ctypes.byref(s), FAKE, FAKE, ctypes.byref(_rope()), None, None) == 1
    assert lib.nsa_paged_q8_append(ctypes.byref(s), FAKE, FAKE, None, None, None) == 1
    for k, v in ((None, FAKE), (FAKE, None), (MIS, FAKE), (FAKE, MIS)):
        assert _append(s, _cache(), k=k, v=v) == 1 and _append8(s, c, k=k, v=v) == 1
    assert _attn8(s, c, window=-1) == 1 and _attn8(s, c, n_sink=-1) == 1 and _attn8(s, c, bound=-1) == 1
    assert _attn8(s, c, window=(1 << 28) + 1) == 2
    assert _attn8(s, c, q=None) == 1 and _attn8(s, c, o=MIS) == 1 and _attn8(s, c, lse=MIS) == 1
    for seqlen in (1, 100):  # codes as they are, and expanded
        x = _shape(seqlen=seqlen)
        need = lib.nsa_paged_q8_attn_fwd_workspace_size(ctypes.byref(x), ctypes.byref(c), 0, 0, 0)
        assert need > 0
        assert _attn8(x, c, ws=None) == 1 and _attn8(x, c, ws=MIS) == 1 and _attn8(x, c, n=need - 1) == 1
    assert lib.nsa_paged_q8_attn_fwd_workspace_size(ctypes.byref(s), ctypes.byref(c), 0, -1, 0) == 0
    qb = 2 * 8 * 16 * 128 * 2
    for o in (1 << 32, (1 << 32) + qb - 16, (1 << 32) - qb + 16):
        assert _attn8(s, c, q=P(1 << 32), o=P(o)) == 1
        assert b"overlap" in lib.nsa_last_error()


def test_nothing_to_do_is_no_error():
    empty = _shape(batch=0)
    assert _append(empty, _cache()) == 0 and _append8(empty, _cache8()) == 0 and _attn8(empty, _cache8()) == 0


def test_the_workspace_of_expanded_caches_is_bounded():
    """By the window, by the caller's bound of the lengths and by the room of a group."""
    lib, c = nsa.load(), _cache8(max_pages=1 << 14, n_pages=1 << 20)  # rows of 2^20 positions
    size = lambda s, bound, window: lib.nsa_paged_q8_attn_fwd_workspace_size(  # noqa: E731
        ctypes.byref(s), ctypes.byref(c), bound, window, 4 if window else 0)
    one = _shape(batch=1, seqlen=512)
    key = 2 * 128 * 4  # bytes of a key's K and V in bf16, 2 kv-heads
    assert (1 << 20) * key <= size(one, 0, 0) <= (1 << 20) * key * 1.1 + (1 << 26)
    assert 8192 * key <= size(one, 8192, 0) <= 8192 * key + (1 << 26)
    assert size(one, 0, 1024) <= (1024 + 512 + 3 * 64) * key + (1 << 26)
    many = _shape(batch=64, seqlen=512)
    assert size(many, 32768, 0) <= (512 << 20) + 32768 * key + (1 << 27)


# ----------------------------------------------------------------------------- refusals, Python
def test_python_refuses_tensors_of_the_cpu():
    z, f8 = torch.zeros, torch.float8_e4m3fn
    pages = z(2, 16, 2, 64).to(f8)
    with pytest.raises(ValueError, match="GPU"):
        nsa.nsa_paged_append_rope(z(4, 2, 64), z(4, 2, 64), z(2, 16, 2, 64), z(2, 16, 2, 64), z(1, 2), z(1), z(32))
    with pytest.raises(ValueError, match="GPU"):
        nsa.nsa_paged_q8_append(z(4, 2, 64), z(4, 2, 64), pages, pages, z(2, 2, 1), z(2, 2, 1), z(1, 2), z(1))
    with pytest.raises(ValueError, match="GPU"):
        nsa.nsa_paged_q8_attn_fwd(z(1, 4, 64), pages, pages, z(2, 2, 1), z(2, 2, 1), z(1, 2), z(1))


@pytest.mark.parametrize("value", [(1 << 32) + 5, 1 << 31, -(1 << 31) - 1])
@pytest.mark.parametrize("name", ["window", "n_sink"])
def test_numbers_past_32_bits_are_refused(name, value):
    z = torch.zeros
    pages = z(2, 16, 2, 64).to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match=f"{name} = {value}"):
        nsa.nsa_paged_q8_attn_fwd(z(1, 4, 64), pages, pages, z(2, 2, 1), z(2, 2, 1), z(1, 2), z(1), **{name: value})
    with pytest.raises(ValueError, match=f"{name} = {value}"):
        nsa.nsa_paged_q8_attn_fwd_workspace_size(nsa.make_shape(1, 4, 2, 64, _lib.NSA_BF16), _cache8(), 64, **{name: value})


def test_python_checks_of_the_cache():
    """The checks themselves, on CPU tensors."""
    f8, i32, z = torch.float8_e4m3fn, torch.int32, torch.zeros
    k, sc = z(3, 32, 2, 64).to(f8), z(3, 2, 2)
    table, lens = z(2, 4, dtype=i32), z(2, dtype=i32)
    c, page = _lib._paged_cache_q8("f", k, k, sc, sc, table, lens, 2)
    assert (c.n_pages, c.page_size, c.max_pages, c.block_size, c.page_stride, page) == (3, 32, 4, 16, 32 * 2 * 64, 32)
    pool = z(3, 2, 32, 2, 64).to(f8)  # K and V of a page side by side
    assert _lib._paged_cache_q8("f", pool[:, 0], pool[:, 1], sc, sc, table, lens, 2)[0].page_stride == 2 * 32 * 2 * 64
    for bad in (dict(v=z(3, 32, 2, 128).to(f8)), dict(k=k.transpose(1, 2)), dict(k=k.float()), dict(k=k.view(torch.uint8)),
                dict(k=k[..., :32]), dict(k=k[0]), dict(table=table.long()), dict(table=table.t()), dict(lens=lens[:1]),
                dict(v=pool[:, 0]), dict(v=None), dict(ks=z(3, 2, 3)), dict(ks=z(3, 2, 0)), dict(ks=z(3, 2)), dict(ks=None),
                dict(vs=None), dict(vs=z(3, 2, 1)), dict(vs=z(3, 2, 2, dtype=torch.float64)), dict(table=None),
                dict(lens=None)):
        with pytest.raises((TypeError, ValueError)):
            _lib._paged_cache_q8("f", bad.get("k", k), bad.get("v", bad.get("k", k)), bad.get("ks", sc), bad.get("vs", sc),
                                 bad.get("table", table), bad.get("lens", lens), 2)


def test_python_checks_of_the_rotation():
    bf, i32, z = torch.bfloat16, torch.int32, torch.zeros
    cpu = torch.device("cpu")

    class Dev:  # (a device whose tensors answer -1, as the CPU's do)
        type, index = "cpu", -1

        def __eq__(self, other):
            return other == cpu

        def __str__(self):
            return "cpu"

    k, q, f = (5, 2, 64), z(5, 6, 64, dtype=bf), z(16)
    call = lambda **kw: _lib._rope("f", Dev(), 5, k, 2, 64, **(dict(  # noqa: E731
        q=q, inv_freq=f, positions=None, interleaved=False, q_out=q, share=None) | kw))
    r, out = call(positions=z(5, dtype=i32), interleaved=True)
    assert (r.rot_dim, r.interleaved, out) == (32, 1, q)
    assert call(q=None, q_out=None)[1] is None
    for bad in (dict(inv_freq=None), dict(inv_freq=z(4, 4)), dict(inv_freq=f.double()), dict(inv_freq=z(32)[::2]),
                dict(positions=z(4, dtype=i32)), dict(positions=z(5)), dict(q=None), dict(q=q[:4]), dict(q=q[:, :5]),
                dict(q=q.float()), dict(q=q[None]), dict(q_out=q.float()), dict(q_out=q[:, :4])):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)


# ----------------------------------------------------------------------------- sources
def test_the_join_reads_parts_coherently():
    """q8_combine_kernel starts before the kernel whose parts it joins has ended: no read-only loads of them, none before
    wait_primary()."""
    with open(os.path.join(CSRC, "span_q8.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    body = code[code.index("q8_combine_kernel(const Q8Params p)"):]
    body = body[:body.index("\n}\n")]
    before, after = body.split("wait_primary();")
    for name in ("info", "part_ml", "part_o"):
        assert f"p.{name}" not in before and f"p.{name}" in after
        assert not re.search(rf"__ldg\([^;]*\b{name}\b", code)
    assert "__restrict__ part" not in code
