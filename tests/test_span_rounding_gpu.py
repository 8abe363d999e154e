"""Rows with few keys in the sink-window training pair: there no single rounding averages out, so these
are held to tighter bounds than tests/test_span_gpu.py's (which grant the gradient of q the
rounding of the stored o everywhere)."""
import math

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from tests import span_reference as ref

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
def _bf(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF)


def _train(lens, H, hk, d, window, n_sink, q_scale=1.0):
    """(kernel's o, lse and gradients, and per sequence the exact inputs, masks and slices)."""
    cu = torch.tensor([0] + lens).cumsum(0).to(I32)
    n = int(cu[-1])
    x = [_bf((n, h, d), 200 + i, s) for i, (h, s) in enumerate(((H, q_scale), (hk, 1.0), (hk, 1.0), (H, 1.0)))]
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
        seqs.append((a, e, see, y, ro, ref.gradients(*y, ro, lse[a:e].cpu().double(), see, 1 / math.sqrt(d))))
    return o, lse, grads, seqs


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
    _, _, grads, seqs = _train(lens, H, hk, d, window, n_sink)
    for b, (a, e, _, _, _, (want, bounds)) in enumerate(seqs):
        for name, got, w, bd in zip(("dq", "dk", "dv"), grads, want, bounds):
            ref.within(got[a:e], w, bd, f"{name} of sequence {b}")
