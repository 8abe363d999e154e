"""The rotating append and the 8-bit paged cache on the GPU against the 64-bit reference, elementwise
within the bounds of the kernels' own roundings (tests/q8_reference.py)."""
import math

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from tests import q8_reference as ref8
from tests import span_reference as ref

pytestmark = pytest.mark.gpu

BF, F8, I32, NAN = torch.bfloat16, torch.float8_e4m3fn, torch.int32, float("nan")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(BF)


def _f8(bits):
    return bits.view(F8)


class Cache8:
    """Codes, scales and a table.  Slots that hold no position have NaN codes, blocks without any
    NaN scales."""

    def __init__(self, lens, hk, d, page, block, seed, spare=2, interleave=False, odd_scales=False, spread=3):
        g = _gen(seed)
        self.lens, self.hk, self.d, self.page, self.block = lens, hk, d, page, block
        need = [-(-n // page) for n in lens]
        n_pages, nb = sum(need) + spare, page // block
        order = torch.randperm(n_pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(1, max(need)) + 1), -1, dtype=I32)
        pool = torch.full((n_pages, 2, page, hk, d), 0x7f, dtype=torch.uint8)
        sc = torch.full((2, n_pages, hk, nb), NAN)
        self.codes, self.scales = [], []  # per sequence: [2][n, hk, d] and [2][n, hk], 64 bits
        for b, n in enumerate(lens):
            x = (torch.randn((2, n, hk, d), generator=g) * 60).clamp(-448, 448).to(F8)
            nblk = -(-n // block)
            s = torch.exp2(torch.randint(-spread, spread + 1, (2, nblk, hk), generator=g).float() - 6)
            if odd_scales:
                s *= 1.0 + torch.rand((2, nblk, hk), generator=g)
            at = torch.arange(n)
            self.codes.append(x.double())
            self.scales.append(s[:, at // block].double())
            for i in range(need[b]):
                pid = order.pop()
                self.table[b, i] = pid
                m = min(page, n - i * page)
                pool[pid, :, :m] = x[:, i * page:i * page + m].view(torch.uint8)
                part = s[:, i * nb:min((i + 1) * nb, nblk)]
                sc[:, pid, :, :part.shape[1]] = part.transpose(1, 2)
        self.free = order
        dev = pool.cuda()
        if interleave:
            self.k_pages, self.v_pages = dev[:, 0].view(F8), dev[:, 1].view(F8)
        else:
            self.k_pages, self.v_pages = dev[:, 0].contiguous().view(F8), dev[:, 1].contiguous().view(F8)
        self.k_scales, self.v_scales = sc[0].cuda(), sc[1].cuda()
        self.dev_table, self.dev_lens = self.table.cuda(), torch.tensor(lens, dtype=I32, device="cuda")

    @property
    def args(self):
        return self.k_pages, self.v_pages, self.k_scales, self.v_scales, self.dev_table, self.dev_lens

    def reference(self, q, b, see, scale, many=False):
        """`many`: a call of more than 256 rows, whose keys and values are rounded to bf16 and whose weights are bf16."""
        (kc, vc), (ks, vs) = self.codes[b], self.scales[b]
        if many:
            k, v = ((c * s[..., None]).to(BF).double() for c, s in ((kc, ks), (vc, vs)))
            return ref.attend(q, k, v, see, scale)
        return ref8.attend(q, kc, ks, vc, vs, see, scale)


def _queries(q_lens, H, d, seed, scale=1.0):
    cu = torch.tensor([0] + q_lens).cumsum(0).to(I32)
    return _bf((int(cu[-1]), H, d), _gen(seed), scale), cu


def _reference(c, q, cu, b, window, n_sink, scale, hide=()):
    a, e = int(cu[b]), int(cu[b + 1])
    see = ref.visible(range(c.lens[b] - (e - a), c.lens[b]), c.lens[b], window, n_sink)
    for lo, hi in hide:
        see[:, lo:hi] = False
    many = int((cu[1:] - cu[:-1]).max()) * q.shape[1] // c.hk > 256
    return a, e, c.reference(q[a:e].double(), b, see, scale, many)


def _check(c, q, cu, o, lse, window, n_sink, scale, hide=()):
    for b in range(len(c.lens)):
        a, e, (ro, rl, eo, el) = _reference(c, q, cu, b, window, n_sink, scale, hide)
        ref.within(lse[a:e], rl, el, f"lse of sequence {b}")
        ref.within(o[a:e], ro, eo, f"o of sequence {b}")


# ----------------------------------------------------------------------------- attention
# lengths (cached), lengths (new), heads, kv-heads, d, page, block, window, sinks
CASES = [
    ([1], [1], 1, 1, 128, 16, 16, 0, 0),
    ([40], [1], 8, 1, 128, 64, 64, 0, 0),
    ([1, 130, 0, 77], [1, 1, 1, 1], 16, 2, 128, 64, 32, 0, 0),           # a sequence with an empty cache
    ([300, 17, 128, 129], [1, 1, 1, 1], 6, 2, 64, 16, 16, 0, 0),         # group 3, pages of 16
    ([5, 260], [9, 12], 4, 4, 128, 32, 16, 0, 0),                        # more queries than cached tokens
    ([127, 128, 129, 400], [127, 1, 0, 130], 8, 1, 128, 128, 128, 0, 0),  # a sequence without queries
    ([513, 255], [200, 33], 16, 1, 64, 256, 64, 0, 0),
    ([700, 40], [300, 40], 10, 2, 128, 64, 64, 100, 0),                  # group 5
    ([700, 1000, 3], [300, 1, 3], 8, 2, 128, 16, 16, 37, 5),
    ([900, 640], [1, 1], 32, 2, 64, 32, 32, 64, 130),                    # sinks over more than a tile
    ([450], [450], 12, 4, 64, 16, 16, 1, 1),
    ([333], [90], 128, 1, 128, 64, 32, 50, 16),                          # group 128: two row tiles a token
    ([2000, 1500], [1, 3], 16, 2, 128, 64, 64, 1000, 4),
    ([200, 650], [2, 2], 16, 1, 128, 32, 32, 0, 0),                      # 32 rows
    ([700, 650], [19, 1], 8, 1, 128, 32, 32, 0, 0),                      # 152 rows: two row tiles
    ([700, 650], [20, 1], 8, 1, 128, 32, 32, 0, 0),                      # 160 rows
    ([700, 650], [127, 1], 1, 1, 64, 16, 16, 0, 0),                      # 127 rows
    ([700, 650], [128, 1], 1, 1, 64, 16, 16, 0, 0),                      # 128 rows: a whole row tile
    ([700, 650], [32, 1], 8, 1, 128, 32, 32, 0, 0),                      # 256 rows: codes
    ([700, 650], [257, 1], 1, 1, 128, 32, 32, 0, 0),                     # 257 rows: expanded
    ([700, 650], [64, 3], 4, 1, 64, 16, 16, 200, 7),                     # 256 rows: codes
    ([700, 650], [86, 1], 3, 1, 64, 16, 16, 0, 0),                       # 258 rows: expanded
    ([9, 33], [1, 1], 9, 1, 64, 32, 32, 0, 0),                           # 9 rows
    ([200, 650], [3, 1], 11, 1, 64, 64, 16, 90, 2),                      # 33 rows
]


@pytest.mark.parametrize("lens,q_lens,H,hk,d,page,block,window,n_sink", CASES)
@pytest.mark.parametrize("interleave", [False, True])
def test_attention(lens, q_lens, H, hk, d, page, block, window, n_sink, interleave):
    c = Cache8(lens, hk, d, page, block, 1, interleave=interleave, odd_scales=interleave)
    q, cu = _queries(q_lens, H, d, 2)
    lse = torch.full((q.shape[0], H), NAN, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, window=window, n_sink=n_sink, cu_seqlens=cu.cuda(),
                                  max_seqlen=max(q_lens), lse=lse)
    assert nsa.nsa_device_status() == 0
    _check(c, q, cu, o, lse, window, n_sink, 1.0 / math.sqrt(d))


def test_attention_is_the_same_on_every_run_and_for_every_division():
    """Any bound of the cached lengths divides the keys differently and gives the same rows."""
    c = Cache8([5000, 1200], 2, 128, 64, 64, 5)
    for q_lens in ([1, 1], [3, 2], [40, 3]):
        q, cu = _queries(q_lens, 16, 128, 6)
        kw = dict(cu_seqlens=cu.cuda(), max_seqlen=max(q_lens))
        for bound in (None, 5000, 1 << 20):
            lse = torch.empty(q.shape[0], 16, device="cuda")
            o = [nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, max_cache_len=bound, lse=lse, **kw) for _ in range(2)]
            assert torch.equal(*o)
            _check(c, q, cu, o[0], lse, 0, 0, 1.0 / math.sqrt(128))


def test_a_bound_that_is_too_small():
    """Codes read as they are need no bound; a call of many rows shows by -inf which caches exceeded it."""
    c = Cache8([500, 120], 2, 64, 64, 64, 40)
    q, cu = _queries([3, 1], 8, 64, 41)
    lse = torch.empty(4, 8, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, max_cache_len=128, lse=lse, cu_seqlens=cu.cuda(), max_seqlen=3)
    _check(c, q, cu, o, lse, 0, 0, 1 / 8)
    q, cu = _queries([90, 70], 8, 64, 42)
    lse = torch.empty(160, 8, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, max_cache_len=128, lse=lse, cu_seqlens=cu.cuda(), max_seqlen=90)
    assert (o[:90] == 0).all() and (lse[:90] == -math.inf).all()
    a, e, (ro, rl, eo, el) = _reference(c, q, cu, 1, 0, 0, 1 / 8)
    ref.within(lse[a:e], rl, el, "lse")
    ref.within(o[a:e], ro, eo, "o")


def test_expanded_groups_of_sequences():
    """More caches than the room for expanded pages holds at a time (dense and packed): 10 of 4096 tokens x 32 heads."""
    hk, d, n = 32, 128, 10
    c = Cache8([260] * n, hk, d, 128, 64, 43, spread=1)
    table = torch.cat([c.table[:, :3], torch.full((n, 29), -1, dtype=I32)], 1)  # rows of 4096 positions
    c.dev_table = table.cuda()
    q, cu = _queries([320] * n, hk, d, 44)
    keep = slice(250, 320)  # (positions from 190 on)
    for dense in (False, True):
        lse = torch.empty(n * 320, hk, device="cuda")
        kw = {} if dense else dict(cu_seqlens=cu.cuda(), max_seqlen=320)
        x = q.view(n, 320, hk, d) if dense else q
        o = nsa.nsa_paged_q8_attn_fwd(x.cuda(), *c.args, lse=lse, **kw).view(n, 320, hk, d)
        for b in (0, 3, n - 1):
            see = ref.visible(range(190, 260), 260, 0, 0)
            for h in (0, 31):
                (kc, vc), (ks, vs) = c.codes[b], c.scales[b]
                k, v = ((y[:, h:h + 1] * s[:, h:h + 1, None]).to(BF).double() for y, s in ((kc, ks), (vc, vs)))
                qq = q[b * 320:(b + 1) * 320][keep, h:h + 1].double()
                ro, rl, eo, el = ref.attend(qq, k, v, see, 1 / math.sqrt(d))
                ref.within(o[b, keep, h:h + 1], ro, eo, f"o of {b}, {h}")
                ref.within(lse.view(n, 320, hk)[b, keep, h:h + 1], rl, el, f"lse of {b}, {h}")


@pytest.mark.parametrize("scale", [0.3, 4.0])
@pytest.mark.parametrize("n", [1, 4, 100])
def test_large_scores_and_a_rising_maximum(scale, n):
    """Key scales that grow along the cache move the running maximum in every tile."""
    c = Cache8([900], 1, 64, 64, 16, 7)
    for g in range(900 // 16 + 1):
        c.scales[0][0, g * 16:(g + 1) * 16] = 2.0 ** (g // 12 - 8)
        c.k_scales[c.table[0, g // 4].item(), :, g % 4] = 2.0 ** (g // 12 - 8)
    q, cu = _queries([n], 4, 64, 8)
    lse = torch.empty(n, 4, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, scale=scale, cu_seqlens=cu.cuda(), max_seqlen=n, lse=lse)
    _check(c, q, cu, o, lse, 0, 0, scale)


@pytest.mark.parametrize("n", [1, 3, 50])
def test_value_scales_far_apart(n):
    """The weight that counts is p times the value scale: blocks whose scales are up to 2^80 apart, the
    large ones late and early."""
    for order in (1, -1):
        c = Cache8([700], 2, 128, 32, 32, 9)
        blocks = 700 // 32 + 1
        for i in range(blocks):
            s = 2.0 ** (order * (i - blocks // 2) * 4)
            c.scales[0][1, i * 32:(i + 1) * 32] = s
            c.v_scales[c.table[0, i].item()] = s
        q, cu = _queries([n], 8, 128, 10)
        lse = torch.empty(n, 8, device="cuda")
        o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, cu_seqlens=cu.cuda(), max_seqlen=n, lse=lse)
        _check(c, q, cu, o, lse, 0, 0, 1.0 / math.sqrt(128))


def test_queries_with_an_outlier_dimension():
    """A dimension 1000 times the others: the rest of the row still counts to 2^-24 of it."""
    c = Cache8([300], 1, 128, 64, 64, 11)
    c.k_pages.view(torch.uint8)[..., 5] &= 0x80  # the keys have nothing there
    c.codes[0][0][..., 5] = 0.0
    for n in (1, 20):
        q, cu = _queries([n], 8, 128, 12)
        q[..., 5] = 1000.0
        lse = torch.empty(n, 8, device="cuda")
        o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, scale=0.05, cu_seqlens=cu.cuda(), max_seqlen=n, lse=lse)
        _check(c, q, cu, o, lse, 0, 0, 0.05)


@pytest.mark.parametrize("size", [0.0, 1e-38, 1e-30, 1e30])
def test_queries_of_any_size(size):
    c = Cache8([200], 1, 64, 64, 64, 13)
    q, cu = _queries([2], 4, 64, 14)
    q = (q.double().clamp(-2, 2) * size).to(BF)
    lse = torch.empty(2, 4, device="cuda")
    scale = 0.1 / max(size, 1e-30)
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, scale=scale, cu_seqlens=cu.cuda(), max_seqlen=2, lse=lse)
    _check(c, q, cu, o, lse, 0, 0, scale)


@pytest.mark.parametrize("bad", [-1, 1 << 20])
@pytest.mark.parametrize("n", [1, 4, 70])
def test_missing_pages_are_masked(bad, n):
    c = Cache8([600], 2, 128, 32, 16, 15)
    hide = [(64, 96), (224, 288), (576, 600)]
    for lo, hi in hide:
        c.dev_table[0, lo // 32:-(-hi // 32)] = bad
    q, cu = _queries([n], 8, 128, 16)
    lse = torch.empty(n, 8, device="cuda")
    kw = dict(cu_seqlens=cu.cuda(), max_seqlen=n)
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, lse=lse, **kw)
    _check(c, q, cu, o, lse, 0, 0, 1.0 / math.sqrt(128), hide)
    c.dev_table.fill_(bad)  # nothing left: no key
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, lse=lse, **kw)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("n", [2, 20, 100])
def test_pages_behind_a_window_may_leave_the_table(n):
    c = Cache8([800], 1, 64, 16, 16, 17)
    q, cu = _queries([n], 4, 64, 18)
    kw = dict(window=100, n_sink=4, cu_seqlens=cu.cuda(), max_seqlen=n)
    whole = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, **kw)
    c.dev_table[0, 1:(800 - n - 100) // 16] = -1
    assert torch.equal(whole, nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, **kw))


def test_rows_past_the_last_sequence_stay():
    c = Cache8([100, 50], 2, 64, 16, 16, 19)
    for q_lens in ([1, 1], [3, 5], [60, 20]):
        q, cu = _queries(q_lens, 4, 64, 20)
        n = int(cu[-1])
        q = torch.cat([q, torch.full((9, 4, 64), NAN, dtype=BF)]).cuda()
        out, lse = torch.full_like(q, 7.0), torch.full((n + 9, 4), 7.0, device="cuda")
        nsa.nsa_paged_q8_attn_fwd(q, *c.args, cu_seqlens=cu.cuda(), max_seqlen=max(q_lens), out=out, lse=lse)
        assert (out[n:] == 7).all() and (lse[n:] == 7).all() and torch.isfinite(out[:n]).all()


def test_dense_batches_and_lengths_past_the_table():
    """[B, T, H, d] queries; lengths outside the table row are clamped to it."""
    c = Cache8([96, 64, 80], 1, 64, 16, 16, 21)
    c.dev_lens[0] = 1 << 30
    c.dev_lens[1] = -5
    c.dev_table[0, 6] = -1
    q = _bf((3, 3, 4, 64), _gen(22))
    lse = torch.empty(9, 4, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, lse=lse)
    assert o.shape == q.shape
    # sequence 0 ends at the table's end (its last page missing), sequence 1 has no keys
    cap = c.table.shape[1] * 16
    see = (torch.arange(96)[None] <= torch.arange(cap - 3, cap)[:, None])
    ro, rl, eo, el = c.reference(q[0].double(), 0, see, 1 / 8)
    ref.within(o[0], ro, eo, "o of sequence 0")
    assert (o[1] == 0).all() and (lse[3:6] == -math.inf).all()
    see = ref.visible(range(77, 80), 80, 0, 0)
    ro, rl, eo, el = c.reference(q[2].double(), 2, see, 1 / 8)
    ref.within(o[2], ro, eo, "o of sequence 2")
    ref.within(lse[6:], rl, el, "lse of sequence 2")


# ----------------------------------------------------------------------------- rotating append
def _inv_freq(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2).double() / rot)).float()


# lengths (cached), lengths (new), heads, kv-heads, d, page, rot
APPENDS = [
    ([1], [1], 2, 1, 64, 16, 64), ([17, 200, 64, 5], [17, 1, 0, 9], 6, 3, 128, 32, 128),
    ([70, 300], [33, 255], 2, 2, 64, 256, 16), ([400] * 40, [1] * 40, 16, 2, 128, 64, 128),
    ([900, 700], [900, 333], 4, 1, 128, 128, 96),
]


@pytest.mark.parametrize("lens,q_lens,H,hk,d,page,rot", APPENDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("where", ["cache", "given"])
def test_append_rope(lens, q_lens, H, hk, d, page, rot, interleaved, where):
    g = _gen(23)
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=I32)
    order = torch.randperm(sum(need) + 2, generator=g).tolist()
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
    pool = torch.full((sum(need) + 2, 2, page, hk, d), 5.0, dtype=BF, device="cuda")
    k_pages, v_pages = pool[:, 0], pool[:, 1]
    weights = torch.full((pool.shape[0], hk, page), 3.0, device="cuda")
    k, cu = _queries(q_lens, hk, d, 24, scale=3.0)
    v, _ = _queries(q_lens, hk, d, 25)
    q, _ = _queries(q_lens, H, d, 26)
    n = int(cu[-1])
    place = torch.cat([torch.arange(lens[b] - q_lens[b], lens[b]) for b in range(len(lens))])
    pos = place if where == "cache" else torch.randint(-(1 << 31), (1 << 31) - 1, (n,), generator=g)
    inv = _inv_freq(rot)
    out = nsa.nsa_paged_append_rope(k.cuda(), v.cuda(), k_pages, v_pages, table.cuda(),
                                    torch.tensor(lens, dtype=I32, device="cuda"), inv.cuda(), q=q.cuda(),
                                    positions=None if where == "cache" else pos.to(I32).cuda(),
                                    interleaved=interleaved, weights=weights, cu_seqlens=cu.cuda(),
                                    max_seqlen=max(q_lens))
    rk, ek = ref8.rotate(k.double(), inv, pos, interleaved)
    rq, eq = ref8.rotate(q.double(), inv, pos, interleaved)
    ref.within(out, rq, eq + ref.B * (rq.abs() + eq), "q")
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(q_lens)])
    has = place >= 0  # (more new tokens than cached ones: the first are dropped)
    pid, slot = table[seq[has], place[has] // page].long(), place[has] % page
    ref.within(k_pages.cpu()[pid, slot], rk[has], (ek + ref.B * (rk.abs() + ek))[has], "k")
    assert torch.equal(k_pages.cpu()[pid, slot][..., rot:], k[has][..., rot:])
    assert torch.equal(v_pages.cpu()[pid, slot], v[has])
    w = weights.cpu()
    assert (w[pid, :, slot] == 0).all()
    w[pid, :, slot] = 3.0
    assert (w == 3.0).all()
    rest = pool.cpu()
    rest[pid, :, slot] = 5.0
    assert (rest == 5.0).all()
    # the same in place, without the weights
    q2 = q.cuda()
    assert nsa.nsa_paged_append_rope(k.cuda(), v.cuda(), k_pages, v_pages, table.cuda(),
                                     torch.tensor(lens, dtype=I32, device="cuda"), inv.cuda(), q=q2, q_out=q2,
                                     positions=None if where == "cache" else pos.to(I32).cuda(),
                                     interleaved=interleaved, cu_seqlens=cu.cuda(), max_seqlen=max(q_lens)) is q2
    assert torch.equal(q2, out)


def test_rotation_of_unusual_frequencies():
    """Frequencies from denormal to 2 pi, negative ones and zero, at large positions."""
    inv = torch.tensor([0.0, 1e-40, -1e-40, 1e-30, 1e-9, -1e-3, 0.5, 1.0, -1.0, 1.5, 3.0, -3.14159, 6.28, 1e-5, 0.1, 2.0])
    pos = torch.tensor([0, 1, -1, 77, 1 << 20, -(1 << 31), (1 << 31) - 1, 123456789], dtype=I32)
    k = _bf((8, 1, 64), _gen(27))
    pages = torch.zeros(1, 16, 1, 64, dtype=BF, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=I32, device="cuda"), torch.tensor([8], dtype=I32, device="cuda")
    nsa.nsa_paged_append_rope(k.cuda(), k.cuda(), pages, torch.zeros_like(pages), table, lens, inv.cuda(),
                              positions=pos.cuda())
    rk, ek = ref8.rotate(k.double(), inv, pos, False)
    ref.within(pages[0, :8], rk, ek + ref.B * (rk.abs() + ek), "k")


def test_appends_drop_tokens_without_a_place():
    for eight in (False, True):
        table = torch.tensor([[0, 1, -1, 3], [4, 5, 6, 7], [8, 9, 10, 11]], dtype=I32, device="cuda")
        lens = torch.tensor([64, 200, 20], dtype=I32, device="cuda")  # one past its row, one longer chunk than cached
        k = torch.ones(3, 40, 1, 64, dtype=BF, device="cuda")
        q = torch.ones(3, 40, 2, 64, dtype=BF, device="cuda")
        inv = torch.zeros(32, device="cuda")
        pages = torch.zeros(12, 16, 1, 64, dtype=BF, device="cuda")
        if eight:
            pages = pages.to(F8)
            sc = torch.full((12, 1, 1), 1.0, device="cuda")
            out = nsa.nsa_paged_q8_append(k, k, pages, pages.clone(), sc, sc.clone(), table, lens, q=q, inv_freq=inv)
        else:
            out = nsa.nsa_paged_append_rope(k, k, pages, pages.clone(), table, lens, inv, q=q)
        assert torch.equal(out, q)  # (a turn by nothing)
        rows = (pages.float() != 0).all(-1).any(-1).sum(1).tolist()
        # sequence 0: positions 24 .. 63 but for the missing page; 1: none; 2: positions 0 .. 19
        assert rows == [0, 8, 0, 16, 0, 0, 0, 0, 16, 4, 0, 0]


# ----------------------------------------------------------------------------- 8-bit append
def _plain_store(c, b, q_len, k, v):
    """The blocks of sequence b after an append of its last q_len tokens (k, v in 64 bits)."""
    n, first = c.lens[b], c.lens[b] - q_len
    want = []
    for x, new in ((0, k), (1, v)):
        codes, scales = c.codes[b][x].clone(), c.scales[b][x].clone()
        for p0 in range(max(0, first) // c.block * c.block, n, c.block):
            lo, hi = max(p0, first), min(p0 + c.block, n)
            for g in range(c.hk):
                got, s = ref8.store(codes[p0:hi, g], float(scales[p0, g]), lo - p0, new[lo - first:hi - first, g])
                codes[p0:hi, g], scales[p0:hi, g] = got, s
        want.append((codes, scales))
    return want


def _cached8(c, b):
    """Codes and scales [2][n, hk(, d)] of sequence b as the device holds them."""
    at = torch.arange(c.lens[b])
    pid, slot = c.table[b].long()[at // c.page], at % c.page
    codes = [x.cpu().view(torch.uint8)[pid, slot].view(F8).double() for x in (c.k_pages, c.v_pages)]
    return list(zip(codes, (x.cpu()[pid, :, slot // c.block].double() for x in (c.k_scales, c.v_scales))))


Q8_APPENDS = [
    ([1], [1], 1, 64, 16, 16), ([17, 200, 64, 5], [17, 1, 0, 5], 3, 128, 32, 16), ([70, 300], [33, 255], 2, 64, 256, 128),
    ([130, 128, 129, 300], [1, 1, 1, 1], 2, 128, 64, 64), ([1000, 700], [600, 333], 2, 128, 128, 128),
    ([257, 65], [130, 2], 1, 128, 64, 32),
]


@pytest.mark.parametrize("lens,q_lens,hk,d,page,block", Q8_APPENDS)
@pytest.mark.parametrize("size", [1e-3, 1.0, 30.0])
@pytest.mark.parametrize("interleave", [False, True])
def test_q8_append(lens, q_lens, hk, d, page, block, size, interleave):
    """Exact: scales, new codes, earlier codes where the scale grew, and everything else as it was."""
    c = Cache8(lens, hk, d, page, block, 28, interleave=interleave)
    k, cu = _queries(q_lens, hk, d, 29, scale=size)
    v, _ = _queries(q_lens, hk, d, 30, scale=size)
    before = [x.cpu().clone() for x in (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scales, c.v_scales)]
    assert nsa.nsa_paged_q8_append(k.cuda(), v.cuda(), *c.args, cu_seqlens=cu.cuda(), max_seqlen=max(q_lens)) is None
    after = [x.cpu() for x in (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scales, c.v_scales)]
    for b in range(len(lens)):
        a, e = int(cu[b]), int(cu[b + 1])
        for (codes, scales), (rc, rs) in zip(_cached8(c, b), _plain_store(c, b, q_lens[b], k[a:e].double(), v[a:e].double())):
            assert torch.equal(scales, rs)
            assert torch.equal(codes, rc)
        # what lies outside the sequence's positions is as it was
        at = torch.arange(lens[b])
        pid, slot = c.table[b].long()[at // page], at % page
        for x, y in zip(before[:2], after[:2]):
            y[pid, slot] = x[pid, slot]
        for x, y in zip(before[2:], after[2:]):
            y[pid, :, slot // block] = x[pid, :, slot // block]
    for x, y in zip(before, after):
        assert torch.equal(x.view(torch.uint8 if x.dtype == torch.uint8 else I32),
                           y.view(torch.uint8 if y.dtype == torch.uint8 else I32))


def test_q8_append_special_values():
    """Infinities saturate and do not count for the scale, NaN stays NaN, zeros take the least
    scale, huge and tiny values the ends of its range; values at a border of two scales."""
    k = torch.zeros(6, 1, 64, dtype=BF)
    k[0, 0, :4] = torch.tensor([math.inf, -math.inf, NAN, 2.0]).to(BF)
    k[2, 0, :2] = torch.tensor([1e38, -3e20]).to(BF)
    k[3, 0, :2] = torch.tensor([1e-38, 1e-17]).to(BF)
    k[4, 0, 0], k[5, 0, 0] = 448.0, 450.0
    pages = torch.zeros(6, 16, 1, 64, dtype=BF, device="cuda").to(F8)
    sc = torch.full((6, 1, 1), NAN, device="cuda")
    table = torch.arange(6, dtype=I32, device="cuda")[:, None].contiguous()
    lens = torch.ones(6, dtype=I32, device="cuda")
    nsa.nsa_paged_q8_append(k.cuda().view(6, 1, 1, 64), k.cuda().view(6, 1, 1, 64), pages, pages.clone(), sc, sc.clone(),
                            table, lens)
    got, s = pages[:, 0, 0].float().cpu(), sc.view(6).cpu()
    assert s.tolist() == [2.0 ** -7, 2.0 ** -60, 2.0 ** 60, 2.0 ** -60, 1.0, 2.0]
    assert got[0, :2].tolist() == [448.0, -448.0] and math.isnan(got[0, 2]) and got[0, 3] == 256.0
    assert (got[1] == 0).all() and got[2, 0] == 448.0
    assert got[2, 1] == ref8.code(torch.tensor(float(k[2, 0, 1]) / 2.0 ** 60))
    assert got[3, 0] == 0.0 and got[3, 1] == ref8.code(torch.tensor(float(k[3, 0, 1]) * 2.0 ** 60))
    assert got[4, 0] == 448.0 and got[5, 0] == 224.0  # 225 to the even one of 224 and 240's neighbours


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (16, False)])
def test_q8_append_rotated(rot, interleaved):
    lens, q_lens, hk, d, H = [700, 90], [301, 90], 2, 128, 6
    c = Cache8(lens, hk, d, 64, 64, 31)
    k, cu = _queries(q_lens, hk, d, 32)
    v, _ = _queries(q_lens, hk, d, 33)
    q, _ = _queries(q_lens, H, d, 34)
    pos = torch.randint(0, 1 << 24, (int(cu[-1]),), generator=_gen(35)).to(I32)
    inv = _inv_freq(rot, 500000.0)
    out = nsa.nsa_paged_q8_append(k.cuda(), v.cuda(), *c.args, q=q.cuda(), inv_freq=inv.cuda(), positions=pos.cuda(),
                                  interleaved=interleaved, cu_seqlens=cu.cuda(), max_seqlen=max(q_lens))
    rq, eq = ref8.rotate(q.double(), inv, pos, interleaved)
    ref.within(out, rq, eq + ref.B * (rq.abs() + eq), "q")
    rk, ek = ref8.rotate(k.double(), inv, pos, interleaved)
    for b in range(2):
        a, e = int(cu[b]), int(cu[b + 1])
        (kc, ks), (vc, vs) = _cached8(c, b)
        (wk, wks), (wv, wvs) = _plain_store(c, b, q_lens[b], rk[a:e], v[a:e].double())
        assert torch.equal(vc, wv) and torch.equal(vs, wvs) and torch.equal(ks, wks)
        first = lens[b] - q_lens[b]
        assert torch.equal(kc[:first], wk[:first])
        s = ks[first:, :, None]
        # half a step of the code at the exact value, which the fp32 rotation may miss by ek
        half = torch.maximum(2.0 ** -4 * (rk[a:e].abs() + ek[a:e]), 2.0 ** -10 * s)
        ref.within(kc[first:] * s, rk[a:e], half + ek[a:e], f"k of sequence {b}")


def test_a_block_filled_token_by_token():
    """A run of single appends (with growing values, so that the scale grows), each read by the
    attention; and the codes never further than a step from the values."""
    c = Cache8([0, 0], 2, 64, 32, 32, 36, spare=8)
    table = torch.tensor(c.free[:8], dtype=I32).view(2, 4)
    c.dev_table, c.table = table.cuda(), table
    k, v = _bf((2, 70, 2, 64), _gen(37)), _bf((2, 70, 2, 64), _gen(38))
    ramp = torch.exp2(torch.linspace(-6, 6, 70))[None, :, None, None].to(BF)
    k, v = k * ramp, v * ramp
    c.codes = [torch.zeros(2, 0, 2, 64, dtype=torch.float64) for _ in range(2)]
    for t in range(70):
        lens = torch.tensor([t + 1, max(1, t)], dtype=I32, device="cuda")  # (the second writes its last token again)
        rows = [t, max(0, t - 1)]
        nsa.nsa_paged_q8_append(torch.stack([k[b, rows[b]] for b in range(2)])[:, None].cuda(),
                                torch.stack([v[b, rows[b]] for b in range(2)])[:, None].cuda(),
                                c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.dev_table, lens)
        if t % 13 == 5:
            c.lens = lens.tolist()
            q, cu = _queries([1, 1], 8, 64, 39 + t)
            lse = torch.empty(2, 8, device="cuda")
            o = nsa.nsa_paged_q8_attn_fwd(q.view(2, 1, 8, 64).cuda(), c.k_pages, c.v_pages, c.k_scales, c.v_scales,
                                          c.dev_table, lens, lse=lse, scale=0.01)
            for b in range(2):
                held = _cached8(c, b)
                for (codes, scales), x in zip(held, (k, v)):
                    err = (codes * scales[..., None] - x[b, :c.lens[b]].double()).abs()
                    # one rounding of the value, and half a subnormal step for every time a scale grew
                    bound = 2.0 ** -4 * x[b, :c.lens[b]].double().abs() + 2.0 ** -9 * scales[..., None]
                    assert (err <= bound).all()
                see = ref.visible([c.lens[b] - 1], c.lens[b], 0, 0)
                ro, rl, eo, el = ref8.attend(q[b:b + 1].double(), held[0][0], held[0][1], held[1][0], held[1][1], see, 0.01)
                ref.within(o[b], ro, eo, f"o at {t}")
                ref.within(lse[b:b + 1], rl, el, f"lse at {t}")
