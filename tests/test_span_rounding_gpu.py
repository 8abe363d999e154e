"""Rows with few keys in the sink-window training pair, and rows of the attention that one key makes
up: there no single rounding averages out, so these are held to tighter bounds than
tests/test_span_gpu.py's (which grant the gradient of q the rounding of the stored o everywhere, and
P and dS a rounding to bf16)."""
import math

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from tests import span_reference as ref

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32


def _bf(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF)


def _train(lens, H, hk, d, window, n_sink):
    """(the kernel's gradients; per sequence its rows, lse, mask, exact inputs, exact gradients and bounds)."""
    cu = torch.tensor([0] + lens).cumsum(0).to(I32)
    n = int(cu[-1])
    x = [_bf((n, h, d), 200 + i) for i, h in enumerate((H, hk, hk, H))]
    q, k, v, do = (t.cuda() for t in x)
    lse = torch.empty(n, H, device="cuda")
    kw = dict(cu_seqlens=cu.cuda(), max_seqlen=max(lens))
    o = nsa.nsa_swa_sink_fwd(q, k, v, window, n_sink, lse=lse, **kw)
    grads = nsa.nsa_swa_sink_bwd(q, k, v, o, lse, do, window, n_sink, **kw)
    assert nsa.nsa_device_status() == 0
    seqs = []
    for b, L in enumerate(lens):
        a, e = int(cu[b]), int(cu[b + 1])
        see = ref.visible(range(L), L, window, n_sink)
        y = [t[a:e].double() for t in x]
        ro = ref.attend(*y[:3], see, 1 / math.sqrt(d))[0]
        kept = lse[a:e].cpu().double()
        seqs.append((a, e, kept, see, y, ref.gradients(*y, ro, kept, see, 1 / math.sqrt(d))))
    return grads, seqs


# Sequences of a few tokens, and long ones whose window and sinks hold at most 32 keys.
FEW = [
    ([1, 2, 3, 4, 5, 6, 7, 8], 2, 2, 64, 100, 0), ([8, 7, 3, 2, 1], 16, 2, 128, 100, 4), ([5, 8, 16], 6, 2, 64, 3, 2),
    ([2, 31, 4], 128, 1, 128, 100, 0), ([300], 2, 2, 128, 1, 0), ([300], 2, 2, 128, 1, 1), ([300, 129], 2, 2, 64, 2, 0),
    ([257], 1, 1, 128, 3, 4), ([300], 4, 2, 64, 4, 2), ([400], 8, 1, 128, 2, 2), ([700], 3, 3, 64, 20, 12),
    ([600], 2, 1, 128, 28, 4), ([520], 3, 1, 64, 32, 0), ([390], 24, 2, 128, 4, 28), ([300], 2, 2, 64, 1, 31),
]


@pytest.mark.parametrize("lens,H,hk,d,window,n_sink", FEW)
def test_gradients_of_few_keys_carry_no_rounding_of_o(lens, H, hk, d, window, n_sink):
    """The bounds without the term of o's distance from the exact one: D is the sum of p dp."""
    assert max(min(L, window + n_sink) for L in lens) <= 32
    grads, seqs = _train(lens, H, hk, d, window, n_sink)
    for b, (a, e, _, _, _, (want, bounds)) in enumerate(seqs):
        for name, got, w, bd in zip(("dq", "dk", "dv"), grads, want, bounds):
            ref.within(got[a:e], w, bd, f"{name} of sequence {b}")


# A value and its remainder, both bf16: the remainder is at most 2^-8 of the value and is itself
# rounded by at most 2^-8 of that.
BB = ref.B * ref.B


def _bounds(q, k, v, do, o, lse, see, scale):
    """ref.gradients' bounds with P and dS carried as value and remainder and D summed as p dp."""
    Q, H, d = q.shape
    n, hk = k.shape[:2]
    r, U, B = H // hk, ref.U, ref.B
    grads, _ = ref.gradients(q, k, v, do, o, lse, see, scale)
    eq, ek, ev = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for h in range(H):
        g = h // r
        kk, vv, qq, dd = k[:, g], v[:, g], q[:, h], do[:, h]
        p = torch.where(see, torch.exp(qq @ kk.T * scale - lse[:, h][:, None]), 0.0)
        dp = dd @ vv.T
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        arg = (d + 8) * U * (qq.abs() @ kk.abs().T) * scale + 4 * U * lse[:, h].abs()[:, None] + 2.0 ** -20
        mag = dd.abs() @ vv.abs().T
        ed = ((arg + n * U) * p * mag).sum(1, keepdim=True) + (dd * o[:, h]).abs().sum(1, keepdim=True) * (d + n) * U
        eds = ds.abs() * (BB + arg) + p * ((d + 4) * U * mag + ed)
        eq[:, h] = scale * (eds + 2 * n * U * ds.abs()) @ kk.abs()
        ek[:, g] += scale * (eds + 2 * Q * r * U * ds.abs()).T @ qq.abs()
        ev[:, g] += (p * (BB + arg + 2 * Q * r * U)).T @ dd.abs()
    return tuple(e + B * x.abs() * (1 + 2 * B) for e, x in zip((eq, ek, ev), grads))


def _hold(grads, seqs, names=("dq", "dk", "dv"), rows=None):
    """Within _bounds (rows: the first ones alone)."""
    for b, (a, e, lse, see, x, (want, _)) in enumerate(seqs):
        ro = ref.attend(*x[:3], see, 1 / math.sqrt(x[0].shape[2]))[0]
        bounds = _bounds(*x, ro, lse, see, 1 / math.sqrt(x[0].shape[2]))
        for name, got, w, bd in zip(("dq", "dk", "dv"), grads, want, bounds):
            if name in names:
                ref.within(got[a:e][:rows], w[:rows], bd[:rows], f"{name} of sequence {b}")


@pytest.mark.parametrize("lens,H,hk,d,window,n_sink", FEW)
def test_gradients_of_rows_with_few_keys(lens, H, hk, d, window, n_sink):
    assert max(min(L, window + n_sink) for L in lens) <= 32
    grads, seqs = _train(lens, H, hk, d, window, n_sink)
    _hold(grads, seqs)


@pytest.mark.parametrize("T,H,hk,d,window,n_sink", [(500, 2, 2, 64, 300, 0), (260, 16, 2, 128, 100, 4)])
def test_gradients_of_a_sequence_s_first_rows(T, H, hk, d, window, n_sink):
    grads, seqs = _train([T], H, hk, d, window, n_sink)
    _hold(grads, seqs, names=("dq",), rows=32)


@pytest.mark.parametrize("q_len,bound", [(64, None), (64, 1 << 20), (1, None)])  # short, long and few-row forms
def test_a_late_key_that_outweighs_the_others(q_len, bound):
    """The weight of a key that holds two thirds of a row, or nearly all, is not rounded more than
    the row's o: with the row's own maximum it is 1, which bf16 holds.  Others' weights may be."""
    n, H, d, page = 640, 64, 128, 64
    k, v, q = _bf((n, 1, d), 210), _bf((n, 1, d), 211), _bf((q_len, H, d), 212)
    u = torch.zeros(d)
    u[0] = 1.0  # the late key's direction: scores of the other keys keep their size
    k[:, 0, 0], q[..., 0] = 0.0, 16.0
    k[550, 0] = (u * 1.0).to(BF)
    rise = torch.linspace(4.0, 13.0, q_len * H)  # how far its score lies above the others' mean
    q[..., 0] = (rise.view(q_len, H) * math.sqrt(d)).to(BF)
    pages = torch.zeros(n // page, page, 1, d, dtype=BF)
    k_pages, v_pages = pages.clone().cuda(), pages.clone().cuda()
    k_pages.view(n, 1, d).copy_(k)
    v_pages.view(n, 1, d).copy_(v)
    table = torch.arange(n // page, dtype=I32, device="cuda")[None]
    lens = torch.tensor([n], dtype=I32, device="cuda")
    o = nsa.nsa_paged_attn_fwd(q[None].cuda(), k_pages, v_pages, table, lens, max_cache_len=bound)[0]
    see = ref.visible(range(n - q_len, n), n, 0, 0)
    ro, lse, _, _ = ref.attend(q.double(), k.double(), v.double(), see, 1 / math.sqrt(d))
    s = torch.einsum("qhd,kd->qhk", q.double(), k[:, 0].double()) / math.sqrt(d)
    p = torch.where(see[:, None], torch.exp(s - lse[..., None]), 0.0)
    heavy = p[..., 550] > 0.6
    assert int(heavy.sum()) >= 0.4 * heavy.numel()
    mag = torch.einsum("qhd,kd->qhk", q.double().abs(), k[:, 0].double().abs()).amax(-1) / math.sqrt(d)
    rel = 2 * (d + 8) * ref.U * mag + 2.0 ** -20 + n * ref.U
    p[..., 550] = 0.0
    # (its weight next to the maximum in fp32: the exponent's error is in rel)
    bound = torch.einsum("qhk,kd->qhd", p, v[:, 0].double().abs()) * ref.B \
        + rel[..., None] * v.double().abs().max() + ref.B * ro.abs() * (1 + ref.B)
    ref.within(o[heavy], ro[heavy], bound[heavy], "o of rows with a heavy key")
