"""Paged-cache calls from several host threads.  ctypes lets go of the interpreter's lock during a
call; with the arguments made beforehand the threads are inside the library at the same time."""
import ctypes
import threading

import pytest
import torch

import sparse_attention_compress_gb300 as nsa
from sparse_attention_compress_gb300 import _lib

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
CALLS = 2000


def _bf(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


class Work:
    """Attention and weights of one sequence's `t` new tokens, as prepared C calls."""

    def __init__(self, h, hk, t, d, seed):
        n, page = 512, 64
        self.q, self.k, self.v = _bf((1, t, h, d), seed), *(_bf((n // page, page, hk, d), seed + i) for i in (1, 2))
        self.table, self.lens = torch.arange(n // page, dtype=I32, device="cuda"), torch.tensor([n], dtype=I32, device="cuda")
        self.stream = torch.cuda.Stream()
        self.o, self.lse = torch.empty_like(self.q), torch.empty(t, h, device="cuda")
        self.w = torch.zeros(n // page, hk, page, device="cuda")
        self.shape = nsa.make_shape(t, h, hk, d, _lib.NSA_BF16)
        self.cache = _lib.NsaPagedCache(self.k.data_ptr(), self.v.data_ptr(), None, self.table.data_ptr(),
                                        self.lens.data_ptr(), n // page, page, n // page, page * hk * d)
        size = nsa.nsa_paged_attn_fwd_workspace_size(self.shape, n)
        self.ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
        lib, s, c = nsa.load(), ctypes.byref(self.shape), ctypes.byref(self.cache)
        st = self.stream.cuda_stream
        self.calls = [
            (lib.nsa_paged_attn_fwd, (s, self.q.data_ptr(), c, n, 0, 0, 0.0, self.o.data_ptr(), self.lse.data_ptr(),
                                      self.ws.data_ptr(), size, st)),
            (lib.nsa_paged_attn_weights, (s, self.q.data_ptr(), c, self.lse.data_ptr(), 0, 0, 0.0, 1.0,
                                          self.w.data_ptr(), st))]

    def run(self, times=1):
        for _ in range(times):
            for f, args in self.calls:
                rc = f(*args)
                if rc:
                    raise RuntimeError(f"{f.__name__}: {rc}: {nsa.load().nsa_last_error().decode()}")

    def out(self):
        self.stream.synchronize()
        return self.o.clone(), self.lse.clone(), self.w.clone()


# (heads, kv-heads, tokens) of the threads' calls: 8, 48 and 16 rows a kv-head take the few-row forms,
# 320, 128 and 100 the others (of the weights: 128, 128 and 112 columns)
@pytest.mark.parametrize("sizes", [((16, 2, 1), (16, 2, 6), (32, 2, 1)), ((16, 1, 20), (8, 1, 16), (100, 1, 1))])
@pytest.mark.parametrize("d", [64, 128])
def test_calls_of_other_row_counts_from_several_threads(sizes, d):
    work = [Work(*x, d, 300 + 10 * i) for i, x in enumerate(sizes)]
    torch.cuda.synchronize()
    want = []
    for w in work:
        w.run()
        want.append(w.out())
    errors, start = [], threading.Barrier(len(work))

    def run(w):
        try:
            w.stream.synchronize()  # (the device's context is this thread's from here on)
            start.wait()
            w.run(CALLS)
        except BaseException as e:  # noqa: BLE001  (reported below, in the test's own thread)
            errors.append(e)

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


@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_a_call_without_queries_at_the_largest_group(d):
    """No query, one token's heads a tile: the widest launch of the few-row form."""
    k, lse = _bf((4, 64, 1, d), 330), torch.empty(0, 128, device="cuda")
    table, lens = torch.arange(4, dtype=I32, device="cuda")[None], torch.tensor([200], dtype=I32, device="cuda")
    w = torch.rand(4, 1, 64, device="cuda")
    out = nsa.nsa_paged_attn_weights(_bf((1, 0, 128, d), 331), k, lse, table, lens, weights=w, decay=0.5,
                                     out=torch.full_like(w, 7.0))
    assert torch.equal(out.view(-1)[:200], 0.5 * w.view(-1)[:200]) and (out.view(-1)[200:] == 7.0).all()


@pytest.mark.parametrize("size", [(16, 2, 1), (16, 1, 20)])
def test_a_thread_whose_first_cuda_call_it_is(size):
    w = Work(*size, 128, 340)
    torch.cuda.synchronize()
    w.run()
    want, errors = w.out(), []
    w.o.zero_()
    torch.cuda.synchronize()

    def run():
        try:
            w.run()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not errors, errors
    for a, b in zip(w.out(), want):
        assert torch.equal(a, b)
