"""Numbers past 32 bits in the paged-cache and sink-window calls: refused, not cut to their low bits."""
import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib

BIG = ((1 << 32) + 5, 1 << 31, -(1 << 31) - 1, -(1 << 32) + 5)


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _calls(**kw):
    """Every call that takes one of the keywords (the numbers are looked at before the tensors)."""
    q, pages, i32 = _z(1, 4, 64), _z(2, 16, 2, 64), torch.int32
    table, lens, lse = _z(1, 2, dtype=i32), _z(1, dtype=i32), _z(1, 4, dtype=torch.float32)
    shape = nsa.make_shape(1, 4, 2, 64, _lib.NSA_BF16)
    evict = dict(budget=8) | kw
    yield lambda: nsa.nsa_paged_evict(pages, pages, _z(2, 2, 16, dtype=torch.float32), table, lens, table, **evict)
    if "window" in kw or "n_sink" in kw:
        yield lambda: nsa.nsa_paged_attn_fwd(q, pages, pages, table, lens, **kw)
        yield lambda: nsa.nsa_paged_attn_weights(q, pages, lse, table, lens, **kw)
        yield lambda: nsa.nsa_swa_sink_fwd(q, q, q, **kw)
        yield lambda: nsa.nsa_swa_sink_bwd(q, q, q, q, lse, q, **kw)
        yield lambda: nsa.nsa_paged_attn_fwd_workspace_size(shape, 64, **kw)
        yield lambda: nsa.nsa_swa_sink_fwd_workspace_size(shape, **kw)
        yield lambda: nsa.nsa_swa_sink_bwd_workspace_size(shape, **kw)


@pytest.mark.parametrize("value", BIG)
@pytest.mark.parametrize("name", ["window", "n_sink", "budget", "n_recent"])
def test_numbers_past_32_bits_are_refused(name, value):
    for i, call in enumerate(_calls(**{name: value})):
        if i == 0 and name == "window":
            continue  # (an eviction has no window)
        with pytest.raises(ValueError, match=f"{name} = {value}"):
            call()


@pytest.mark.parametrize("value", BIG)
def test_a_longest_length_past_32_bits_is_refused(value):
    q, cu = _z(5, 4, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_seqlen"):
        _lib._span_shape("f", q, 2, 64, q.device, cu, value)
