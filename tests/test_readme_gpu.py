"""README's examples of the paged caches, run as they are printed."""
import math
import os
import re

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from tests import q8_reference as ref8
from tests import span_reference as ref

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _blocks():
    with open(README) as f:
        return re.findall(r"```python\n(.*?)```", f.read(), re.S)


def test_the_rotating_examples_turn_queries_once():
    T, H, Hkv, d, n_pages = 100, 8, 2, 128, 4
    g = torch.Generator().manual_seed(1)
    rand = lambda h: torch.randn(1, T, h, d, generator=g).to(torch.bfloat16)  # noqa: E731
    q, k, v = rand(H), rand(Hkv), rand(Hkv)
    names = dict(torch=torch, nsa=nsa, H=H, Hkv=Hkv, d=d, n_pages=n_pages, q=q.cuda(), k_new=k.cuda(), v_new=v.cuda(),
                 k_pages=torch.zeros(n_pages, 64, Hkv, d, dtype=torch.bfloat16, device="cuda"),
                 v_pages=torch.zeros(n_pages, 64, Hkv, d, dtype=torch.bfloat16, device="cuda"),
                 table=torch.tensor([[3, 1]], dtype=torch.int32, device="cuda"),
                 lens=torch.tensor([T], dtype=torch.int32, device="cuda"))
    blocks = _blocks()
    first = next(i for i, b in enumerate(blocks) if b.startswith("inv_freq ="))
    last = next(i for i, b in enumerate(blocks) if "nsa_paged_q8_attn_fwd" in b)
    rotated = None
    for code in blocks[first:last + 1]:
        exec(code, names)
        inv, pos = names["inv_freq"].cpu(), torch.arange(T)
        if rotated is None:
            rotated = [ref8.rotate(x[0].double(), inv, pos, False)[0] for x in (q, k)]
            o, _, _, _ = ref.attend(*rotated, v[0].double(), ref.visible(pos, T, 0, 0), 1 / math.sqrt(d))
        off = names["o"][0].cpu().double() - o
        # 8 bits: K and V in 4 significant bits are off by at most 2^-4 of a value, a few percent in the mean, which is what
        # scores (of about 1) and outputs are off by; queries turned twice give scores that have nothing to do with these
        assert float(off.norm() / o.norm()) < (0.06 if "q8" in code else 0.01)
