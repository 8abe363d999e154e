"""How exact the 8-bit cache's attention is in each of its forms (up to 32 rows a kv-head, up to 256, more): queries whose
elements lie far apart, weights of the form that holds them in f16."""
import math

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from tests.test_q8_gpu import BF, F8, Cache8, _check, _gen

pytestmark = pytest.mark.gpu


def _set_keys(c, codes):
    """Codes [n, d] of the keys of a cache of one sequence and kv-head, with scales of 1."""
    n = codes.shape[0]
    at = torch.arange(n)
    pid, slot = c.table[0].long()[at // c.page], at % c.page
    pages = c.k_pages.view(torch.uint8).cpu()
    pages[pid, slot, 0] = codes.to(F8).view(torch.uint8)
    c.k_pages = pages.cuda().view(F8)
    c.k_scales.fill_(1.0)
    c.codes[0][0, :, 0] = codes.double()
    c.scales[0][0] = 1.0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 4, 20, 70])  # 8, 16, 32, 160 and 560 rows
def test_elements_far_below_a_rows_largest(n, d):
    """An element of 128 where every key has nothing, the others 2^13 to 2^20 times smaller and equal within a row, so
    that what is cut of them adds up over a key of equal codes: at most 2^-24 of the largest each."""
    g = _gen(200 + n)
    c = Cache8([150], 1, d, 64, 64, 201)
    codes = torch.where(torch.rand(150, d, generator=g) < 0.5, 448.0, -448.0)
    codes[0], codes[149] = 448.0, -448.0
    codes[:, 5] = 0.0
    _set_keys(c, codes)
    cu = torch.tensor([0, n], dtype=torch.int32)
    for e in range(-13, -5):
        m = 1.0 + (2 * torch.randint(0, 64, (n, 8), generator=g) + 1) / 128.0  # all eight significant bits
        m[0, 0] = 1.125  # (with e = -11: 5.49e-4)
        q = (m * 2.0 ** e)[..., None].expand(n, 8, d).contiguous().to(BF)
        q[..., 5] = 128.0
        for scale in (0.02, 0.1):
            lse = torch.empty(n, 8, device="cuda")
            o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, scale=scale, cu_seqlens=cu.cuda(), max_seqlen=n, lse=lse)
            assert nsa.nsa_device_status() == 0
            _check(c, q, cu, o, lse, 0, 0, scale)


@pytest.mark.parametrize("n", [1, 2, 4, 20])  # 8, 16, 32 and 160 rows
@pytest.mark.parametrize("first", [60, -60])
def test_value_scales_at_both_ends_of_their_range(n, first):
    """Value scales of 2^60 in one half of a cache and 2^-60 in the other, scores near one another: every key counts in
    the row's sum, also where the parts of a row have one kind of scale alone."""
    c = Cache8([6000], 1, 128, 64, 64, 210)
    half = 6000 // 128 * 64
    at = torch.arange(6000)
    scales = torch.where(at < half, 2.0 ** first, 2.0 ** -first).double()
    c.scales[0][1] = scales[:, None]
    vs = c.v_scales.cpu()
    vs[c.table[0].long()[at // 64], 0, 0] = scales.float()
    c.v_scales = vs.cuda()
    q = (torch.randn(n, 8, 128, generator=_gen(211)) * 0.01).to(BF)
    cu = torch.tensor([0, n], dtype=torch.int32)
    lse = torch.empty(n, 8, device="cuda")
    o = nsa.nsa_paged_q8_attn_fwd(q.cuda(), *c.args, cu_seqlens=cu.cuda(), max_seqlen=n, lse=lse)
    assert nsa.nsa_device_status() == 0
    _check(c, q, cu, o, lse, 0, 0, 1 / math.sqrt(128))
