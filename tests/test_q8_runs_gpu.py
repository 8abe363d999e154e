"""The rotating append and the 8-bit paged cache as programs use them: a serving run, captured steps, several streams and
host threads, many sequences, pools past 32 bits, waits that run out."""
import ctypes
import math
import random
import threading

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib
from tests import q8_reference as ref8
from tests import span_reference as ref
from tests.test_q8_gpu import BF, F8, I32, NAN, Cache8, _bf, _cached8, _check, _gen, _inv_freq, _queries, _reference

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- sizes
def _random_case(seed):
    r = random.Random(seed)
    d, hk = r.choice([64, 128]), r.choice([1, 2, 3])
    page = r.choice([16, 32, 64, 128, 256])
    block = r.choice([b for b in (16, 32, 64, 128) if b <= page])
    group, n = r.choice([1, 2, 3, 5, 8, 13, 16, 40]), r.choice([1, 2, 3, 5])
    top = max(1, (159 if d == 128 else 127) // group) if r.random() < 0.8 else 200 // group + 1
    q_lens = [r.randint(0, min(top, 40)) for _ in range(n)]
    q_lens[r.randrange(n)] = min(top, 40)
    lens = [max(0, r.choice([q, q + r.randint(0, 900), r.randint(0, 300), 128 * r.randint(1, 5)])) for q in q_lens]
    window = r.choice([0, 0, 1, r.randint(1, 50), r.randint(50, 600)])
    return lens, q_lens, group * hk, hk, d, page, block, window, r.choice([0, r.randint(1, 200)]) if window else 0


@pytest.mark.parametrize("seed", range(60))
def test_attention_at_random_sizes(seed):
    lens, q_lens, H, hk, d, page, block, window, n_sink = _random_case(seed)
    c = Cache8(lens, hk, d, page, block, seed, interleave=seed % 2 == 1, spread=seed % 5)
    q, cu = _queries(q_lens, H, d, 1000 + seed, scale=(0.3, 1.0, 3.0)[seed % 3])
    lse = torch.full((q.shape[0], H), NAN, device="cuda")
    bound = max(lens) + seed % 7 if seed % 3 == 0 else None
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, window=window, n_sink=n_sink, cu_seqlens=cu.cuda(), lse=lse,
                                  max_seqlen=max(q_lens), max_cache_len=bound)
    assert nsa.nsa_device_status() == 0
    _check(c, q, cu, o, lse, window, n_sink, 1.0 / math.sqrt(d))


@pytest.mark.parametrize("seed", range(24))
def test_attention_of_33_to_256_rows(seed):
    r = random.Random(1000 + seed)
    d, hk, page = r.choice([64, 128]), r.choice([1, 2, 3]), r.choice([16, 32, 64, 128, 256])
    block = r.choice([b for b in (16, 32, 64, 128) if b <= page])
    group, n = r.choice([1, 3, 5, 8, 16, 40, 128]), r.choice([1, 2, 5, 9])
    top = max(1, r.randint(33, 256) // group)
    q_lens = [r.randint(0, top) for _ in range(n)]
    q_lens[r.randrange(n)] = top
    lens = [r.choice([q, q + r.randint(0, 900), r.randint(0, 300), 128 * r.randint(1, 9), q + r.randint(2000, 5000)])
            for q in q_lens]
    window = r.choice([0, 0, 1, r.randint(1, 50), r.randint(50, 600)])
    n_sink = r.choice([0, r.randint(1, 200)]) if window else 0
    c = Cache8(lens, hk, d, page, block, seed, odd_scales=seed % 2 == 1, spread=r.choice([0, 3, 20]))
    q, cu = _queries(q_lens, group * hk, d, seed, r.choice([0.3, 1.0, 6.0]))
    lse = torch.full((q.shape[0], group * hk), NAN, device="cuda")
    kw = dict(window=window, n_sink=n_sink, cu_seqlens=cu.cuda(), max_seqlen=top)
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, lse=lse, **kw)
    assert nsa.nsa_device_status() == 0
    _check(c, q, cu, o, lse, window, n_sink, 1.0 / math.sqrt(d))
    assert torch.equal(o, nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, **kw))


@pytest.mark.parametrize("n,hk,H,q_len", [(1300, 1, 4, 1), (700, 2, 2, 1), (350, 2, 22, 5), (200, 7, 14, 20), (350, 2, 14, 7), (200, 2, 32, 12)])
def test_more_units_than_runs_take(n, hk, H, q_len):
    """Calls of so many units that each takes a CTA (and no join), ragged, some without queries or keys."""
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 300, (n,), generator=g).tolist()
    q_lens = [0 if i % 11 == 5 else q_len for i in range(n)]
    c = Cache8(lens, hk, 64, 64, 32, 8)
    q, cu = _queries(q_lens, H, 64, 9)
    lse = torch.full((q.shape[0], H), NAN, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, cu_seqlens=cu.cuda(), max_seqlen=q_len, lse=lse).cpu()
    assert nsa.nsa_device_status() == 0
    lse = lse.cpu()
    for b in list(range(0, n, 37)) + [n - 1]:
        a, e = int(cu[b]), int(cu[b + 1])
        see = ref.visible(range(lens[b] - (e - a), lens[b]), lens[b], 0, 0)
        ro, rl, eo, el = c.reference(q[a:e].double(), b, see, 1 / 8)
        ref.within(o[a:e], ro, eo, f"o of {b}")
        ref.within(lse[a:e], rl, el, f"lse of {b}")


def test_a_long_cache():
    """One token and a few over 100000 keys: many parts of a row."""
    c = Cache8([100003], 1, 64, 256, 128, 10)
    for n in (1, 5):
        q, cu = _queries([n], 8, 64, 11)
        lse = torch.empty(n, 8, device="cuda")
        o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, cu_seqlens=cu.cuda(), max_seqlen=n, lse=lse)
        _check(c, q, cu, o, lse, 0, 0, 1 / 8)


def test_one_key_that_outweighs_the_rest():
    """Late and early keys that make up the row: the output is their value."""
    for at in (3, 250, 299):
        c = Cache8([300], 1, 128, 64, 64, 12)
        q = torch.ones(1, 1, 4, 128, dtype=BF)
        c.k_pages.view(torch.uint8)[:] = 0
        c.k_scales[:] = 1.0
        pid = c.table[0, at // 64].item()
        c.k_pages[pid, at % 64, 0] = torch.full((128,), 8.0, device="cuda").to(F8)
        lse = torch.empty(1, 4, device="cuda")
        o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, scale=0.1, lse=lse)
        want = c.codes[0][1][at, 0] * c.scales[0][1][at, 0]  # the others weigh e^-102 together with 299
        err = (o[0, 0, 0].cpu().double() - want).abs()
        # a weight of 2^9 is exactly its three terms: what is left is the output's rounding
        assert (err <= 2.0 ** -8 * want.abs()).all()


# ----------------------------------------------------------------------------- a serving run
def test_serving_run():
    """Prompts in chunks, then tokens, over an 8-bit cache with rotation on the way; each step's attention against the
    64-bit form of what the cache holds, and the cache against the rotated keys."""
    hk, H, d, page, block = 2, 8, 64, 32, 16
    inv = _inv_freq(d).cuda()
    n_pages, g = 64, _gen(50)
    k_pages = torch.full((n_pages, page, hk, d), 0x7f, dtype=torch.uint8, device="cuda").view(F8)
    v_pages = k_pages.clone()
    k_scales = torch.full((n_pages, hk, page // block), NAN, device="cuda")
    v_scales = k_scales.clone()
    table = torch.randperm(n_pages, generator=g)[:48].view(2, 24).to(I32)
    c = Cache8([0, 0], hk, d, page, block, 51)
    c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.table = k_pages, v_pages, k_scales, v_scales, table
    dev_table, lens = table.cuda(), [0, 0]
    values = [[], []]
    for step, q_lens in enumerate([[37, 5], [64, 1], [3, 130], [1, 1], [1, 1], [0, 1], [1, 1], [300, 40], [1, 1]]):
        lens = [a + b for a, b in zip(lens, q_lens)]
        k, cu = _queries(q_lens, hk, d, 52 + step, scale=1.0 + step)
        v, _ = _queries(q_lens, hk, d, 72 + step)
        q, _ = _queries(q_lens, H, d, 92 + step)
        dl, packed = torch.tensor(lens, dtype=I32, device="cuda"), dict(cu_seqlens=cu.cuda(), max_seqlen=max(q_lens))
        rotated = nsa.nsa_paged_q8_append(k.cuda(), v.cuda(), k_pages, v_pages, k_scales, v_scales, dev_table, dl,
                                          q=q.cuda(), inv_freq=inv, **packed)
        lse = torch.empty(q.shape[0], H, device="cuda")
        o = nsa.nsa_paged_q8_attn_fwd(rotated, k_pages, v_pages, k_scales, v_scales, dev_table, dl, lse=lse, **packed)
        c.lens = lens
        for b in range(2):
            a, e = int(cu[b]), int(cu[b + 1])
            pos = torch.arange(lens[b] - (e - a), lens[b])
            values[b].append((ref8.rotate(k[a:e].double(), inv.cpu(), pos, False)[0], v[a:e].double()))
            held = _cached8(c, b)
            c.codes[b], c.scales[b] = (torch.stack(x) for x in zip(*held))
            for (codes, scales), x in zip(held, (torch.cat(y) for y in zip(*values[b]))):
                err = (codes * scales[..., None] - x).abs()
                assert (err <= 2.0 ** -4 * x.abs() + 2.0 ** -9 * scales[..., None] + 1e-6).all(), step
        _check(c, rotated.cpu(), cu, o, lse, 0, 0, 1 / 8)
    assert nsa.nsa_device_status() == 0


def test_bf16_and_8_bit_caches_agree():
    """The same prompt through nsa_paged_append_rope and through nsa_paged_append of keys rotated before give the same
    cache; the 8-bit cache's attention is near the bf16 one's."""
    T, hk, H, d, page = 500, 2, 8, 128, 64
    k, v, q = (_bf((1, T, x, d), _gen(60 + i)).cuda() for i, x in enumerate((hk, hk, H)))
    table = torch.arange(8, dtype=I32, device="cuda")[None].contiguous()
    lens = torch.tensor([T], dtype=I32, device="cuda")
    inv = _inv_freq(d).cuda()
    pages = [torch.zeros(8, page, hk, d, dtype=BF, device="cuda") for _ in range(4)]
    rq = nsa.nsa_paged_append_rope(k, v, pages[0], pages[1], table, lens, inv, q=q)
    rk, _ = ref8.rotate(k[0].cpu().double(), inv.cpu(), torch.arange(T), False)
    nsa.nsa_paged_append(rk.to(BF).cuda()[None].contiguous(), v, pages[2], pages[3], table, lens)
    off = (pages[0].float() - pages[2].float()).abs()  # (a value next to a border may round to either side)
    assert torch.equal(pages[1], pages[3]) and (off <= 2.0 ** -7 * pages[2].float().abs()).all() and (off > 0).sum() < 100
    o = nsa.nsa_paged_attn_fwd(rq, pages[0], pages[1], table, lens)
    k8, v8 = (torch.zeros(8, page, hk, d, device="cuda").to(F8) for _ in range(2))
    sc = [torch.zeros(8, hk, 2, device="cuda") for _ in range(2)]
    rq8 = nsa.nsa_paged_q8_append(k, v, k8, v8, *sc, table, lens, q=q, inv_freq=inv)
    assert torch.equal(rq, rq8)
    o8 = nsa.nsa_paged_q8_attn_fwd(rq, k8, v8, *sc, table, lens)
    # rounding K and V to 4 significant bits is of the order of 3% of a value, less what a row's keys average out
    assert float((o8.float() - o.float()).norm() / o.float().norm()) < 0.04


# ----------------------------------------------------------------------------- graphs, streams, threads
def test_captured_steps_share_nothing():
    """Two captured decode steps (append and attention, workspaces of their own) replayed in turn and on new contents give
    what eager calls give."""
    def make(seed):
        c = Cache8([700, 300], 2, 128, 64, 64, seed)
        k, v, q = (_bf((2, 1, h, 128), _gen(seed + i)).cuda() for i, h in enumerate((2, 2, 16)))
        return c, k, v, q, _inv_freq(128).cuda(), torch.empty_like(q), torch.empty(2, 16, device="cuda")

    def step(c, k, v, q, inv, out, lse):
        nsa.nsa_paged_q8_append(k, v, *c.args, q=q, q_out=out, inv_freq=inv)
        return nsa.nsa_paged_q8_attn_fwd(out, *c.args, lse=lse)

    states = [make(70), make(80)]
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
    # new contents in the captured tensors
    states[0][3].copy_(_bf((2, 1, 16, 128), _gen(90)).cuda())
    graphs[0].replay()
    torch.cuda.synchronize()
    again = step(*states[0])
    assert torch.equal(outs[0], again) and not torch.equal(outs[0], want[0][0])
    assert nsa.nsa_device_status() == 0


@pytest.mark.parametrize("n", [1, 3, 40])
def test_calls_on_other_streams_at_once(n):
    work = []
    for i in range(4):
        c = Cache8([3000, 900], 2, 128, 64, 32, 100 + i)
        q, cu = _queries([n, n], 16, 128, 110 + i)
        kw = dict(cu_seqlens=cu.cuda(), max_seqlen=n)
        work.append((c, q.cuda(), kw, torch.cuda.Stream(), nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, **kw)))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [nsa.nsa_paged_q8_attn_fwd(q, *c.args, stream=st, **kw) for c, q, kw, st, _ in work]
        torch.cuda.synchronize()
        for o, (*_, want) in zip(outs, work):
            assert torch.equal(o, want)


def test_calls_of_other_row_counts_from_several_threads():
    """The launches' settings belong to the kernels: threads with other row counts do not refuse one another's."""
    work, errors = [], []
    for i, (h, hk, t, d) in enumerate([(16, 2, 1, 128), (16, 1, 1, 128), (16, 1, 2, 128), (8, 1, 16, 128), (8, 1, 1, 64)]):
        c = Cache8([500], hk, d, 64, 64, 120 + i)
        q = _bf((1, t, h, d), _gen(130 + i)).cuda()
        o, lse, stream = torch.empty_like(q), torch.empty(t, h, device="cuda"), torch.cuda.Stream()
        s = nsa.make_shape(t, h, hk, d, _lib.NSA_BF16)
        cc, _ = _lib._paged_cache_q8("f", *c.args, 1)
        size = nsa.nsa_paged_q8_attn_fwd_workspace_size(s, cc, 512)
        ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
        args = (ctypes.byref(s), q.data_ptr(), ctypes.byref(cc), 512, 0, 0, 0.0, o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                size, stream.cuda_stream)
        torch.cuda.synchronize()
        assert nsa.load().nsa_paged_q8_attn_fwd(*args) == 0
        torch.cuda.synchronize()
        work.append((args, o, o.clone(), (s, cc, c, q, lse, ws, stream)))
    start = threading.Barrier(len(work))

    def run(args):
        try:
            start.wait()
            for _ in range(1000):
                rc = nsa.load().nsa_paged_q8_attn_fwd(*args)
                if rc:
                    raise RuntimeError(nsa.load().nsa_last_error().decode())
        except BaseException as e:  # noqa: BLE001  (reported below, in the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(w[0],)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for _, o, want, _ in work:
        assert torch.equal(o, want)


# ----------------------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 40])  # 8 rows, more, many
def test_queries_that_are_not_finite_spoil_their_own_rows(n, d):
    """Where codes are read as they are, rows with NaN or an infinity give NaN, not zeros (calls of many rows have
    the bf16 cache's answer, zeros).  Every other row is as without them."""
    c = Cache8([700, 3000, 129], 2, d, 64, 32, 160)
    q, cu = _queries([n] * 3, 8, d, 161)
    bad = q.clone()
    bad[0, 1, 5] = NAN
    bad[n, 6, d - 1] = NAN
    bad[3 * n - 1, 0, 0] = math.inf
    bad[3 * n - 1, 7, :] = NAN
    lse = torch.full((q.shape[0], 8), 7.0, device="cuda")
    kw = dict(cu_seqlens=cu.cuda(), max_seqlen=n)
    o = nsa.nsa_paged_q8_attn_fwd(bad.cuda(), *c.args, lse=lse, **kw)
    assert nsa.nsa_device_status() == 0
    rows = torch.zeros(q.shape[0], 8, dtype=torch.bool)
    for t, h in ((0, 1), (n, 6), (3 * n - 1, 0), (3 * n - 1, 7)):
        rows[t, h] = True
        assert n == 40 or torch.isnan(o[t, h]).all(), (t, h)
    keep = ~rows
    scale = 1.0 / math.sqrt(d)
    for b in range(3):
        a, e, (ro, rl, eo, el) = _reference(c, q, cu, b, 0, 0, scale)
        k = keep[a:e]
        ref.within(lse[a:e].cpu()[k], rl[k], el[k], f"lse of sequence {b}")
        ref.within(o[a:e].cpu()[k], ro[k], eo[k], f"o of sequence {b}")


# ----------------------------------------------------------------------------- 32 bits
def test_pools_past_32_bits():
    """Pages, scales' cells and table entries that lie past 2^32 bytes."""
    hk, d, page, block, n_pages = 4, 128, 256, 64, 20000  # K and V side by side: 5.2 GB
    pool = torch.empty(n_pages, 2, page, hk, d, dtype=torch.uint8, device="cuda")
    k_pages, v_pages = pool[:, 0].view(F8), pool[:, 1].view(F8)
    k_scales, v_scales = (torch.zeros(n_pages, hk, page // block, device="cuda") for _ in range(2))
    ids = torch.tensor([[n_pages - 1, 3, n_pages - 7, 12345]], dtype=I32)
    L = 1000
    c = Cache8([0], hk, d, page, block, 140)
    c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.table, c.lens = k_pages, v_pages, k_scales, v_scales, ids, [L]
    c.dev_table, c.dev_lens = ids.cuda(), torch.tensor([L], dtype=I32, device="cuda")
    k, v = _bf((1, L, hk, d), _gen(141)), _bf((1, L, hk, d), _gen(142))
    nsa.nsa_paged_q8_append(k.cuda(), v.cuda(), *c.args)
    held = _cached8(c, 0)
    for (codes, scales), x in zip(held, (k, v)):
        err = (codes * scales[..., None] - x[0].double()).abs()
        assert (err <= 2.0 ** -4 * x[0].double().abs() + 2.0 ** -10 * scales[..., None]).all()
    c.codes[0], c.scales[0] = (torch.stack(x) for x in zip(*held))
    for n in (1, 5, 40):
        q, cu = _queries([n], 16, d, 143)
        lse = torch.empty(n, 16, device="cuda")
        o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, cu_seqlens=cu.cuda(), max_seqlen=n, lse=lse)
        _check(c, q, cu, o, lse, 0, 0, 1 / math.sqrt(d))
    del pool, k_pages, v_pages
    c.k_pages = c.v_pages = None
    bf = torch.empty(9000, page, hk, d, dtype=BF, device="cuda")  # 2.4 GB each of K and V
    ids = torch.tensor([[8999, 8998]], dtype=I32, device="cuda")
    vf = torch.empty_like(bf)
    inv = _inv_freq(d).cuda()
    nsa.nsa_paged_append_rope(k[:, :400].cuda().contiguous(), v[:, :400].cuda().contiguous(), bf, vf, ids,
                              torch.tensor([400], dtype=I32, device="cuda"), inv)
    rk, ek = ref8.rotate(k[0, :400].double(), inv.cpu(), torch.arange(400), False)
    got = torch.cat([bf[8999], bf[8998]])[:400]
    ref.within(got, rk, ek + ref.B * (rk.abs() + ek), "k")
    assert torch.equal(torch.cat([vf[8999], vf[8998]])[:400].cpu(), v[0, :400])


# ----------------------------------------------------------------------------- waits that run out
@pytest.fixture
def clean_status():
    assert nsa.nsa_device_status(reset=True) == 0
    yield
    nsa.nsa_set_wait_limit_ns(0)
    nsa.nsa_device_status(reset=True)


def _flush_l2():
    torch.empty(96 << 20, device="cuda").fill_(1.0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [1, 2, 4, 14])
@pytest.mark.parametrize("limit", [1, 1000, 2000, 4000])
def test_waits_run_out_and_recover(clean_status, n, limit):
    """Limits below and about a copy's time: the kernel gives up wherever it is and returns, later calls skip their work,
    and with limit and word reset the call gives what it gave."""
    c = Cache8([5000, 1200, 1], 2, 128, 64, 64, 150)
    q, cu = _queries([n, n, 1], 16, 128, 151)
    dq, kw = q.cuda(), dict(cu_seqlens=cu.cuda(), max_seqlen=n)
    want = nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw)
    for _ in range(3):
        _flush_l2()
        nsa.nsa_set_wait_limit_ns(limit)
        nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw)
        torch.cuda.synchronize()  # it returned
        if limit == 1:
            assert nsa.nsa_device_status() == 4
            out = torch.full_like(want, 7.0)
            nsa.nsa_paged_q8_attn_fwd(dq, *c.args, out=out, **kw)
            torch.cuda.synchronize()
            assert (out == 7.0).all()  # skipped while the word is set
        nsa.nsa_set_wait_limit_ns(0)
        nsa.nsa_device_status(reset=True)
        assert torch.equal(nsa.nsa_paged_q8_attn_fwd(dq, *c.args, **kw), want)
        assert nsa.nsa_device_status() == 0
