"""Selected attention from several host threads with block lists of other lengths, as prepared C calls
(ctypes lets go of the interpreter's lock during a call)."""
import ctypes
import threading

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib

pytestmark = pytest.mark.gpu

CALLS = 1500


def _idx(T, hk, S, bs):
    """Block lists [T, hk, S]: the query's own block and those before it."""
    own = torch.arange(T) // bs
    idx = own[:, None] - torch.arange(S)[None]
    return torch.where(idx >= 0, idx, -1).to(torch.int32)[:, None].expand(T, hk, S).contiguous().cuda()


class Forward:
    """fp32: shared memory for S * block_size keys."""

    def __init__(self, T, S, bs):
        g = torch.Generator().manual_seed(S)
        self.q, self.k, self.v = (torch.randn(T, h, 64, generator=g).cuda() for h in (4, 1, 1))
        self.idx, self.o, self.stream = _idx(T, 1, S, bs), torch.empty_like(self.q), torch.cuda.Stream()
        self.shape = nsa.make_shape(T, 4, 1, 64, _lib.NSA_F32)
        self.call = nsa.load().nsa_sparse_fwd
        self.args = (ctypes.byref(self.shape), self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.idx.data_ptr(),
                     S, bs, 0.0, self.o.data_ptr(), None, self.stream.cuda_stream)

    def out(self):
        self.stream.synchronize()
        return (self.o.clone(),)


class Backward:
    """Lists turned round, in shared memory for the sequence's blocks."""

    def __init__(self, T, S):
        g = torch.Generator().manual_seed(T)
        self.q, self.k, self.v, self.do = (torch.randn(T, h, 128, generator=g).to(torch.bfloat16).cuda() for h in (16, 1, 1, 16))
        self.idx, self.stream = _idx(T, 1, S, 64), torch.cuda.Stream()
        self.lse = torch.empty(T, 16, device="cuda")
        self.o = nsa.nsa_sparse_fwd(self.q, self.k, self.v, self.idx, 64, lse=self.lse)
        self.shape = nsa.make_shape(T, 16, 1, 128, _lib.NSA_BF16)
        size = nsa.nsa_sparse_bwd_workspace_size(self.shape, S)
        self.ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
        self.g = [torch.empty_like(x) for x in (self.q, self.k, self.v)]
        torch.cuda.synchronize()
        self.call = nsa.load().nsa_sparse_bwd
        self.args = (ctypes.byref(self.shape), self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.idx.data_ptr(),
                     S, 64, 0.0, self.o.data_ptr(), self.lse.data_ptr(), self.do.data_ptr(),
                     *(x.data_ptr() for x in self.g), self.ws.data_ptr(), size, self.stream.cuda_stream)

    def out(self):
        self.stream.synchronize()
        return tuple(x.clone() for x in self.g)


@pytest.mark.parametrize("make", [lambda: [Forward(8, 2, 16), Forward(8, 64, 64), Forward(8, 20, 32)],
                                  lambda: [Backward(64, 1), Backward(4096, 2)]], ids=["forward_fp32", "backward"])
def test_block_lists_of_other_lengths_from_several_threads(make):
    work = make()
    want = []
    for w in work:
        assert w.call(*w.args) == 0
        want.append(w.out())
    errors, start = [], threading.Barrier(len(work))

    def run(w):
        w.stream.synchronize()  # (the device's context is this thread's from here on)
        start.wait()
        for _ in range(CALLS):
            if w.call(*w.args):
                errors.append(nsa.load().nsa_last_error())
                return

    threads = [threading.Thread(target=run, args=(w,)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    got = [w.out() for w in work]
    assert not errors, errors
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)
