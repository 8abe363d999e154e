"""The forms of the 8-bit cache's attention at the sizes that choose them: up to 32 rows (queries x heads of a group) a
sequence and kv-head, up to 256, and more, where the caches are expanded.  Every test asks the library which form a call
takes, so that a boundary that moves cannot empty one."""
import math
import random

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib
from tests import q8_reference as ref8
from tests import span_reference as ref
from tests.test_q8_gpu import BF, F8, I32, NAN, Cache8, _bf, _cached8, _check, _gen, _inv_freq, _queries, _reference

pytestmark = pytest.mark.gpu


def expands(c, n_seqs, q_len, H):
    """Whether calls of q_len tokens expand the cache: only then a bound of the lengths sizes the workspace."""
    s = nsa.make_shape(n_seqs * q_len, H, c.hk, c.d, _lib.NSA_BF16, batch=n_seqs, seqlen=q_len)
    cc, page = _lib._paged_cache_q8("f", *c.args, n_seqs)
    cc.max_pages = 1 << 12
    size = lambda bound: nsa.nsa_paged_q8_attn_fwd_workspace_size(s, cc, bound)  # noqa: E731
    return size(page) != size(page << 12)


# ----------------------------------------------------------------------------- more than 256 rows
def _many_rows(seed):
    r = random.Random(3000 + seed)
    d, hk = r.choice([64, 128]), r.choice([1, 2, 3])
    page = (16, 32, 64, 128, 256)[seed % 5]
    blocks = [b for b in (16, 32, 64, 128) if b <= page]
    block = blocks[seed // 5 % len(blocks)]
    group, n = r.choice([1, 2, 3, 5, 8, 16, 40, 128]), r.choice([1, 2, 3, 5])
    top = -(-r.choice([257, 258, 300, r.randint(257, 1000), r.randint(600, 1500)]) // group)
    q_lens = [r.choice([0, 1, r.randint(0, top)]) for _ in range(n)]
    q_lens[r.randrange(n)] = top
    # (shorter caches than chunks among them)
    lens = [r.choice([q, q + r.randint(0, 900), r.randint(0, 300), 128 * r.randint(1, 5)]) for q in q_lens]
    window = r.choice([0, 0, 1, r.randint(1, 50), r.randint(50, 600), 2000])
    return lens, q_lens, group * hk, hk, d, page, block, window, r.choice([0, r.randint(1, 40), r.randint(1, 300)]) if window else 0


@pytest.mark.parametrize("seed", range(60))
def test_expanded_calls_at_random_sizes(seed):
    """Ragged chunks of more than 256 rows under windows and sinks; bounds that are none, exact, larger, and below some of
    the lengths, whose queries then see no key."""
    lens, q_lens, H, hk, d, page, block, window, n_sink = _many_rows(seed)
    c = Cache8(lens, hk, d, page, block, seed, interleave=seed % 2 == 1, odd_scales=seed % 3 == 1, spread=seed % 4)
    assert expands(c, len(lens), max(q_lens), H)
    longest = max(1, max(lens))
    bound = [None, longest, longest + seed, max(1, sorted(lens)[len(lens) // 2])][seed % 4]
    q, cu = _queries(q_lens, H, d, 4000 + seed, scale=(0.3, 1.0, 3.0)[seed % 3])
    pad = torch.full((3, H, d), NAN, dtype=BF)  # rows of no sequence
    dq = torch.cat([q, pad]).cuda()
    lse, out = torch.full((dq.shape[0], H), 7.0, device="cuda"), torch.full_like(dq, 7.0)
    kw = dict(window=window, n_sink=n_sink, cu_seqlens=cu.cuda(), max_seqlen=max(q_lens), max_cache_len=bound)
    nsa.nsa_paged_q8_attn_fwd(dq, *c.args, lse=lse, out=out, **kw)
    assert nsa.nsa_device_status() == 0
    for b, L in enumerate(lens):
        a, e = int(cu[b]), int(cu[b + 1])
        if bound is not None and L > -(-bound // page) * page:
            assert (out[a:e] == 0).all() and (lse[a:e] == -math.inf).all(), b
            continue
        _, _, (ro, rl, eo, el) = _reference(c, q, cu, b, window, n_sink, 1.0 / math.sqrt(d))
        ref.within(lse[a:e], rl, el, f"lse of sequence {b}")
        ref.within(out[a:e], ro, eo, f"o of sequence {b}")
    assert (out[q.shape[0]:] == 7).all() and (lse[q.shape[0]:] == 7).all()
    assert torch.equal(out[:q.shape[0]], nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw)[:q.shape[0]])


@pytest.mark.parametrize("window", [0, 100])
def test_expanded_chunks_beside_single_tokens(window):
    """A call that mixes a chunk with single tokens of longer caches, missing pages among them."""
    c = Cache8([700, 2900, 1, 1300], 2, 128, 64, 32, 5, odd_scales=True)
    q, cu = _queries([40, 1, 1, 3], 16, 128, 6)
    assert expands(c, 4, 40, 16)
    hide = [(64, 128), (640, 700)]
    for lo, hi in hide:
        c.dev_table[0, lo // 64:-(-hi // 64)] = -1
    lse = torch.empty(45, 16, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, window=window, n_sink=5 if window else 0, cu_seqlens=cu.cuda(),
                                  max_seqlen=40, lse=lse)
    assert nsa.nsa_device_status() == 0
    for b in range(4):
        a, e, (ro, rl, eo, el) = _reference(c, q, cu, b, window, 5 if window else 0, 1 / math.sqrt(128), hide if b == 0 else ())
        ref.within(lse[a:e], rl, el, f"lse of {b}")
        ref.within(o[a:e], ro, eo, f"o of {b}")


def test_expanded_pools_past_32_bits():
    """Pages and scales' cells that lie past 2^32 bytes, expanded."""
    hk, d, page, block, n_pages, L = 4, 128, 256, 64, 20000, 1000  # K and V side by side: 5.2 GB
    pool = torch.empty(n_pages, 2, page, hk, d, dtype=torch.uint8, device="cuda")
    c = Cache8([0], hk, d, page, block, 140)
    c.k_pages, c.v_pages = pool[:, 0].view(F8), pool[:, 1].view(F8)
    c.k_scales, c.v_scales = (torch.zeros(n_pages, hk, page // block, device="cuda") for _ in range(2))
    c.table, c.lens = torch.tensor([[n_pages - 1, 3, n_pages - 7, 12345]], dtype=I32), [L]
    c.dev_table, c.dev_lens = c.table.cuda(), torch.tensor([L], dtype=I32, device="cuda")
    k, v = _bf((1, L, hk, d), _gen(141)), _bf((1, L, hk, d), _gen(142))
    nsa.nsa_paged_q8_append(k.cuda(), v.cuda(), *c.args)
    c.codes[0], c.scales[0] = (torch.stack(x) for x in zip(*_cached8(c, 0)))
    q, cu = _queries([70], 16, d, 143)
    assert expands(c, 1, 70, 16)
    lse = torch.empty(70, 16, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, cu_seqlens=cu.cuda(), max_seqlen=70, lse=lse)
    _check(c, q, cu, o, lse, 0, 0, 1 / math.sqrt(d))


# ----------------------------------------------------------------------------- weights in f16
@pytest.mark.parametrize("seed", range(20))
def test_weights_of_33_to_256_rows_count_to_f16(seed, monkeypatch):
    """P is rounded once, to f16, there: 2^-11 of a weight, and half of f16's least step, 2^-25, where the row's largest is
    at least 2^9.  (Fewer rows have three 8-bit terms, 2^-9 and 2^-26, which the bounds count otherwise.)"""
    monkeypatch.setattr(ref8, "P_REL", 2.0 ** -11)
    monkeypatch.setattr(ref8, "P_ABS", 2.0 ** -34)
    r = random.Random(5000 + seed)
    d, hk, page = r.choice([64, 128]), r.choice([1, 2]), r.choice([16, 64, 256])
    group = r.choice([1, 3, 8, 16])
    q_len = r.randint(-(-33 // group), 256 // group)
    lens = [q_len + r.randint(0, 900), q_len + 128 * r.randint(0, 20)]
    window = r.choice([0, 0, r.randint(1, 600)])
    c = Cache8(lens, hk, d, page, 16, seed, odd_scales=seed % 2 == 1, spread=r.choice([0, 3]))
    assert not expands(c, 2, q_len, group * hk)
    q, cu = _queries([q_len, q_len], group * hk, d, seed, r.choice([0.3, 1.0, 3.0]))
    lse = torch.full((q.shape[0], group * hk), NAN, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, window=window, n_sink=3 if window else 0, cu_seqlens=cu.cuda(),
                                  max_seqlen=q_len, lse=lse)
    assert nsa.nsa_device_status() == 0
    _check(c, q, cu, o, lse, window, 3 if window else 0, 1.0 / math.sqrt(d))


# ----------------------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 8, 10, 20, 40, 64, 70])  # 4, 12, 32, 40, 80, 160, 256 and 280 rows
def test_rows_that_are_not_finite(n, d):
    """NaN and infinities spoil their own rows: NaN in o and lse where the codes are read as they are, zeros and -inf (the
    bf16 cache's answer) where they are expanded.  Whole units and joined ones, the first and the last row tile."""
    lens = [700, 9000, 129]
    c = Cache8(lens, 2, d, 64, 32, 160)
    q, cu = _queries([n] * 3, 8, d, 161)
    bad = q.clone()
    bad[0, 1, 5] = NAN
    bad[n, 6, d - 1] = NAN
    bad[2 * n - 1, 2, 0] = -math.inf
    bad[3 * n - 1, 0, 0] = math.inf
    bad[3 * n - 1, 7, :] = NAN
    rows = ~torch.isfinite(bad.float()).all(-1)
    lse = torch.full((q.shape[0], 8), 7.0, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(bad.cuda(), *c.args, lse=lse, cu_seqlens=cu.cuda(), max_seqlen=n).cpu()
    assert nsa.nsa_device_status() == 0
    lse = lse.cpu()
    if expands(c, 3, n, 8):
        assert n == 70 and (o[rows] == 0).all() and (lse[rows] == -math.inf).all()
    else:
        assert torch.isnan(o[rows]).all() and torch.isnan(lse[rows]).all()
    for b in range(3):
        a, e, (ro, rl, eo, el) = _reference(c, q, cu, b, 0, 0, 1.0 / math.sqrt(d))
        k = ~rows[a:e]
        ref.within(lse[a:e][k], rl[k], el[k], f"lse of sequence {b}")
        ref.within(o[a:e][k], ro[k], eo[k], f"o of sequence {b}")


# ----------------------------------------------------------------------------- graphs, waits
@pytest.mark.parametrize("n", [9, 40])  # 72 and 320 rows
def test_captured_chunks_share_nothing(n):
    """Two captured chunk steps (append and attention, workspaces of their own), replayed in turn and on new contents."""
    def make(seed):
        c = Cache8([700, 300], 2, 128, 64, 64, seed)
        k, v, q = (_bf((2, n, h, 128), _gen(seed + i)).cuda() for i, h in enumerate((2, 2, 16)))
        return c, k, v, q, _inv_freq(128).cuda(), torch.empty_like(q), torch.empty(2 * n, 16, device="cuda")

    def step(c, k, v, q, inv, out, lse):
        nsa.nsa_paged_q8_append(k, v, *c.args, q=q, q_out=out, inv_freq=inv)
        return nsa.nsa_paged_q8_attn_fwd(out, *c.args, lse=lse, window=500, n_sink=4)

    states = [make(70), make(80)]
    assert expands(states[0][0], 2, n, 16) == (n == 40)
    want = []
    for st in states:
        o = step(*st)
        want.append((o.clone(), st[-1].clone(), st[0].k_pages.view(torch.uint8).clone()))
    graphs, outs = [], []
    for st in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*st))
        graphs.append(g)
    for st in states:
        st[-1].fill_(7.0)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for st, o, (wo, wl, wk) in zip(states, outs, want):
        assert torch.equal(o, wo) and torch.equal(st[-1], wl) and torch.equal(st[0].k_pages.view(torch.uint8), wk)
    states[0][3].copy_(_bf((2, n, 16, 128), _gen(90)).cuda())
    graphs[0].replay()
    torch.cuda.synchronize()
    again = step(*states[0])
    assert torch.equal(outs[0], again) and not torch.equal(outs[0], want[0][0])
    assert nsa.nsa_device_status() == 0


@pytest.fixture
def clean_status():
    assert nsa.nsa_device_status(reset=True) == 0
    yield
    nsa.nsa_set_wait_limit_ns(0)
    nsa.nsa_device_status(reset=True)


@pytest.mark.parametrize("n", [30, 40])  # 240 rows (two row tiles) and 320
@pytest.mark.parametrize("limit", [1, 2000])
def test_waits_of_many_rows_run_out_and_recover(clean_status, n, limit):
    """Limits below and about a copy's time: the call returns, and with limit and word reset it gives what it gave."""
    c = Cache8([5000, 1200, 1], 2, 128, 64, 64, 150)
    q, cu = _queries([n, n, 1], 16, 128, 151)
    assert expands(c, 3, n, 16) == (n == 40)
    dq, kw = q.cuda(), dict(cu_seqlens=cu.cuda(), max_seqlen=n)
    want = nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw)
    for _ in range(2):
        torch.empty(96 << 20, device="cuda").fill_(1.0)  # (nothing of it in L2)
        torch.cuda.synchronize()
        nsa.nsa_set_wait_limit_ns(limit)
        nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw)
        torch.cuda.synchronize()  # it returned
        if limit == 1:
            assert nsa.nsa_device_status() == 4
            nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw)
            torch.cuda.synchronize()  # (a call that finds the word set returns, too)
        nsa.nsa_set_wait_limit_ns(0)
        nsa.nsa_device_status(reset=True)
        assert torch.equal(nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw), want)
        assert nsa.nsa_device_status() == 0
