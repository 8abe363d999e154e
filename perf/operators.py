"""Cases of the paged-cache and sink-window operators: inputs, plain forms, exact values.

Five operators that a server or trainer of this library uses together:

  append   the keys and values of new tokens written into a paged cache
  attn     attention of a chunk of new tokens (or of one token a sequence) over the
           paged cache, causal, with an optional sliding window and n_sink first
           tokens that stay visible
  weights  the attention weight that the chunk gave to every cached key, summed over
           the queries and the heads of a kv-group, added to an accumulator
  evict    the cache cut to a budget of keys by accumulated weight (first and last
           tokens kept), the kept rows copied to new pages in order
  train    sliding-window attention with sinks on packed sequences, forward and backward

A case's lengths follow from the case alone; the seed decides the values and the pages.
With `own` false, run() computes the plain forms: elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one sequence, one new token over a short chat: the smallest call, latency counts
        dict(name="attn_token_1x4096", op="attn", seqs=1, q=1, ctx=4096, spread=0.0, h=16, h_kv=2, d=128, page=64,
             window=0, sink=0),
        # a decode step of 32 users at up to 32768 tokens, as the decode benchmark's cache
        dict(name="attn_token_32x32768", op="attn", seqs=32, q=1, ctx=32768, spread=0.5, h=16, h_kv=2, d=128, page=64,
             window=0, sink=0),
        # ragged chunks of eight prompts in small pages, a streaming window with sinks, an odd group
        dict(name="attn_chunk_8x509_window", op="attn", seqs=8, q=509, ctx=8191, spread=0.7, h=12, h_kv=4, d=64,
             page=16, window=1024, sink=4),
        # a long prompt prefilled in chunks: 2048 new tokens at the end of 32768, the layer's heads
        dict(name="attn_chunk_1x2048_at_32768", op="attn", seqs=1, q=2048, ctx=32768, spread=0.0, h=64, h_kv=4, d=128,
             page=64, window=0, sink=0),
        # weights of a decode step, for eviction between steps
        dict(name="weights_token_32x32768", op="weights", seqs=32, q=1, ctx=32768, spread=0.5, h=16, h_kv=2, d=128,
             page=64, window=0, sink=0),
        # weights of a prompt's last chunk, which decide what of the prompt stays
        dict(name="weights_chunk_2x1000_at_16384", op="weights", seqs=2, q=1000, ctx=16384, spread=0.1, h=16, h_kv=2,
             d=128, page=64, window=0, sink=0),
        # one short cache cut to a quarter
        dict(name="evict_1x4096_to_1024", op="evict", seqs=1, ctx=4096, spread=0.0, h_kv=2, d=128, page=64,
             budget=1024, sink=4, recent=256),
        # a batch at the memory limit cut to 4096 keys each
        dict(name="evict_16x32768_to_4096", op="evict", seqs=16, ctx=32768, spread=0.5, h_kv=4, d=128, page=64,
             budget=4096, sink=4, recent=1024),
        # the new token of 32 users
        dict(name="append_token_32", op="append", seqs=32, q=1, ctx=1024, spread=0.5, h_kv=2, d=128, page=64),
        # prompt chunks of four users
        dict(name="append_chunk_4x2048", op="append", seqs=4, q=2048, ctx=4096, spread=0.4, h_kv=4, d=128, page=64),
        # a packed batch of short documents, odd lengths
        dict(name="train_3x1001_window_256", op="train", seqs=3, t=1001, spread=0.8, h=16, h_kv=2, d=128, window=256,
             sink=4),
        # the three-branch layer's sequence and heads with its window of 512
        dict(name="train_1x65536_window_512", op="train", seqs=1, t=65536, spread=0.0, h=64, h_kv=4, d=128, window=512,
             sink=4),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "weights", "evict", "append", "train"])
    d = rng.choice([64, 128])
    h_kv = rng.choice([1, 2, 4, 8])
    h = h_kv * rng.choice([1, 2, 3, 4, 6, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    spread = round(rng.uniform(0.0, 0.9), 2)
    if op in ("attn", "weights"):
        seqs = _log_int(rng, 1, 32)
        q = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2048)
        ctx = _log_int(rng, max(16, q), 32768)
        # score elements of the padded batch are bounded by the largest listed case's
        while seqs * q * h * ctx > 64 * 2048 * 32768 // 2 or seqs * ctx * h_kv * d > 32 * 32768 * 2 * 128:
            seqs, q, ctx = max(1, seqs // 2), max(1, q * 2 // 3), max(16, ctx * 3 // 4)
        q = min(q, ctx)
        window = 0 if rng.random() < 0.5 else _log_int(rng, 1, 4096)
        return dict(op=op, seqs=seqs, q=q, ctx=ctx, spread=spread, h=h, h_kv=h_kv, d=d, page=page, window=window,
                    sink=rng.randrange(0, 65) if window else 0)
    if op == "evict":
        seqs, ctx = _log_int(rng, 1, 16), _log_int(rng, 64, 32768)
        while seqs * ctx * h_kv * d > 16 * 32768 * 4 * 128:
            seqs, ctx = max(1, seqs // 2), max(64, ctx * 3 // 4)
        budget = _log_int(rng, 16, min(ctx, 8192))
        sink = rng.randrange(0, min(64, budget // 2) + 1)
        return dict(op=op, seqs=seqs, ctx=ctx, spread=spread, h_kv=h_kv, d=d, page=page, budget=budget, sink=sink,
                    recent=rng.randrange(0, budget - sink + 1))
    if op == "append":
        seqs, ctx = _log_int(rng, 1, 64), _log_int(rng, 16, 8192)
        while seqs * ctx * h_kv * d > 64 * 1024 * 4 * 128:
            seqs, ctx = max(1, seqs // 2), max(16, ctx * 3 // 4)
        q = 1 if rng.random() < 0.4 else _log_int(rng, 1, min(2048, ctx))
        return dict(op=op, seqs=seqs, q=q, ctx=ctx, spread=spread, h_kv=h_kv, d=d, page=page)
    seqs, t = _log_int(rng, 1, 8), _log_int(rng, 1, 32768)
    while seqs * t * h > 65536 * 32:
        seqs, t = max(1, seqs // 2), max(1, t * 3 // 4)
    return dict(op=op, seqs=seqs, t=t, spread=spread, h=h, h_kv=h_kv, d=128, window=_log_int(rng, 1, 1024),
                sink=rng.randrange(0, 65))


def _ragged(longest, shortest, seqs, spread):
    """Lengths from `longest` down by the share `spread`, never below `shortest`."""
    return [max(shortest, longest - int(spread * longest * b / max(1, seqs - 1))) if seqs > 1 else longest
            for b in range(seqs)]


def _q_lens(case):
    return _ragged(case["q"], 1, case["seqs"], case["spread"])


def _lens(case):
    """Cache lengths, the new tokens included."""
    q = _q_lens(case) if "q" in case else [1] * case["seqs"]
    return [max(a, b) for a, b in zip(_ragged(case["ctx"], 1, case["seqs"], case["spread"]), q)]


def _t_lens(case):
    return _ragged(case["t"], 1, case["seqs"], case["spread"])


def _pairs(L, Q, window, sink):
    """(visible (query, key) pairs, keys that some query sees) of the last Q positions of L."""
    p = np.arange(L - Q, L, dtype=np.int64)
    lo = np.maximum(p - window + 1, 0) if window else np.zeros_like(p)
    n = p + 1 - lo + np.minimum(lo, sink)
    first = int(lo[0])
    return int(n.sum()), L - first + min(first, sink)


def work(case):
    op, hk, d = case["op"], case["h_kv"], case["d"]
    if op == "train":
        L = _t_lens(case)
        n, h = sum(L), case["h"]
        pairs = sum(_pairs(x, x, case["window"], case["sink"])[0] for x in L)
        # q, dO read, o, dq written; k, v read, dk, dv written
        return {"bytes": n * 4 * (h + hk) * d * 2, "flops": 14 * d * h * pairs}
    L = _lens(case)
    if op == "append":
        n = sum(_q_lens(case))
        return {"bytes": 4 * n * hk * d * 2 + 4 * n * hk, "flops": 0}
    if op == "evict":
        kept = sum(min(x, case["budget"]) for x in L)
        return {"bytes": 4 * hk * (sum(L) + 2 * kept) + 4 * kept * hk * d * 2, "flops": 0}
    Q, h = _q_lens(case), case["h"]
    both = [_pairs(a, b, case["window"], case["sink"]) for a, b in zip(L, Q)]
    pairs, keys = sum(x[0] for x in both), sum(x[1] for x in both)
    if op == "attn":
        return {"bytes": 2 * sum(Q) * h * d * 2 + 4 * sum(Q) * h + 2 * keys * hk * d * 2, "flops": 4 * d * h * pairs}
    return {"bytes": sum(Q) * h * (d * 2 + 4) + keys * hk * d * 2 + 8 * sum(L) * hk, "flops": 2 * d * h * pairs}


# ----------------------------------------------------------------------------- inputs
def _normal(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def _prefix(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    op, hk, d = case["op"], case["h_kv"], case["d"]
    st = dict(case=dict(case))
    if op == "train":
        L = _t_lens(case)
        n = sum(L)
        st.update(q=_normal((n, case["h"], d), gen), k=_normal((n, hk, d), gen), v=_normal((n, hk, d), gen),
                  d_o=_normal((n, case["h"], d), gen), cu=_prefix(L), longest=max(L),
                  lse=torch.empty((n, case["h"]), dtype=torch.float32, device="cuda"))
        return st
    L, page = _lens(case), case["page"]
    need = [-(-x // page) for x in L]
    # an allocator hands out pages in no order; recycled pages hold earlier tokens
    budget_pages = -(-case["budget"] // page) * len(L) if op == "evict" else 0
    n_pages = sum(need) + budget_pages + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(L), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st.update(k_pages=_normal((n_pages, page, hk, d), gen), v_pages=_normal((n_pages, page, hk, d), gen),
              table=table, lens=torch.tensor(L, dtype=torch.int32, device="cuda"))
    if op == "evict":
        # accumulated weight: most keys little, a few much; rounded, so that some are equal
        w = torch.rand((n_pages, hk, page), generator=gen, device="cuda").pow(8) * 64.0
        st["weights"] = (w * 4096).round() / 4096
        st["new_table"] = order[at:at + budget_pages].reshape(len(L), -1).contiguous()
        return st
    Q = _q_lens(case)
    st.update(cu=_prefix(Q), longest=max(Q))
    n = sum(Q)
    if op == "append":
        st.update(k=_normal((n, hk, d), gen), v=_normal((n, hk, d), gen),
                  weights=torch.rand((n_pages, hk, page), generator=gen, device="cuda"))
        return st
    st.update(q=_normal((n, case["h"], d), gen), lse=torch.empty((n, case["h"]), dtype=torch.float32, device="cuda"))
    if op == "weights":
        st["weights"] = torch.rand((n_pages, hk, page), generator=gen, device="cuda")
        st["weights_out"] = st["weights"].clone()
        st["lse"] = _attn_lse(st)
    return st


# ----------------------------------------------------------------------------- plain forms
def _padded(st):
    """Row of every (sequence, chunk position), its position in the cache and whether it exists."""
    cu, lens = st["cu"].long(), st["lens"].long()
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(st["longest"], device=cu.device)
    rows = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1 if "q" in st else st["k"].shape[0] - 1)
    pos = (lens - q_len)[:, None] + i
    return rows, pos, i < q_len[:, None]


def _packed(st, n):
    """(sequence, chunk position) of every packed row."""
    cu = st["cu"].long()
    b = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=cu.device), cu[1:] - cu[:-1], output_size=n)
    return b, torch.arange(n, device=cu.device) - cu[b]


def _gathered(pages, table):
    """Pages of each sequence one after another: [seqs, h_kv, slots, d] in 32 bits."""
    t = pages[table.long().clamp(min=0)]
    return t.reshape(t.shape[0], -1, t.shape[3], t.shape[4]).permute(0, 2, 1, 3).float()


def _scores(st):
    """Scaled scores [seqs, h_kv, queries * group, slots], -inf where a key is not visible."""
    c = st["case"]
    rows, pos, valid = _padded(st)
    B, Q = rows.shape
    hk, r, d = c["h_kv"], c["h"] // c["h_kv"], c["d"]
    k = _gathered(st["k_pages"], st["table"])
    q = st["q"][rows].reshape(B, Q, hk, r, d).permute(0, 2, 1, 3, 4).reshape(B, hk, Q * r, d).float()
    s = torch.matmul(q * (1.0 / math.sqrt(d)), k.transpose(2, 3))
    key = torch.arange(k.shape[2], device=s.device)
    see = key <= pos[..., None]
    if c["window"]:
        see &= (key > pos[..., None] - c["window"]) | (key < c["sink"])
    see &= valid[..., None]
    return s.view(B, hk, Q, r, -1).masked_fill_(~see[:, None, :, None, :], NEG).view(B, hk, Q * r, -1)


def _attn_lse(st):
    s = _scores(st)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    lse = m[..., 0] + s.sub_(m).exp_().sum(-1).log()
    return _rows_of(st, lse.unsqueeze(-1))[..., 0].contiguous()


def _rows_of(st, x):
    """[seqs, h_kv, queries * group, e] -> packed [tokens, h, e]."""
    c = st["case"]
    r = c["h"] // c["h_kv"]
    b, i = _packed(st, st["q"].shape[0])
    x = x.reshape(x.shape[0], c["h_kv"], -1, r, x.shape[-1]).permute(0, 2, 1, 3, 4)
    return x[b, i].reshape(b.numel(), c["h"], -1)


def _plain_attn(st):
    s = _scores(st)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gathered(st["v_pages"], st["table"])) / torch.where(l > 0, l, torch.ones_like(l))
    return _rows_of(st, o).to(torch.bfloat16), _rows_of(st, m + l.log())[..., 0].contiguous()


def _slots(st):
    """Flat slot (page * page_size + offset) of every (sequence, cache position)."""
    page = st["case"]["page"]
    t = st["table"].long().clamp(min=0)
    return (t[..., None] * page + torch.arange(page, device=t.device)).reshape(t.shape[0], -1)


def _plain_weights(st):
    c = st["case"]
    hk, page = c["h_kv"], c["page"]
    s = _scores(st)
    B, Q = s.shape[0], st["longest"]
    rows, _, _ = _padded(st)
    lse = st["lse"][rows].reshape(B, Q, hk, -1).permute(0, 2, 1, 3).reshape(B, hk, -1, 1)
    add = s.sub_(lse).exp_().sum(2).permute(0, 2, 1)                             # [seqs, slots, h_kv]
    slot = _slots(st)
    have = torch.arange(slot.shape[1], device=slot.device) < st["lens"].long()[:, None]
    # one row of spare slots takes what lies past a sequence's length
    total = st["weights"].shape[0] * page
    flat = torch.cat([st["weights"].permute(0, 2, 1).reshape(total, hk), torch.zeros_like(add[0, :1])])
    out = torch.cat([st["weights_out"].permute(0, 2, 1).reshape(total, hk), torch.zeros_like(add[0, :1])])
    to = torch.where(have, slot, total).reshape(-1)
    out[to] = flat[to] + add.reshape(-1, hk)
    st["weights_out"].copy_(out[:total].reshape(-1, page, hk).permute(0, 2, 1))
    return st["weights_out"]


def _plain_evict(st):
    c = st["case"]
    hk, page, d, budget = c["h_kv"], c["page"], c["d"], c["budget"]
    slot, lens = _slots(st), st["lens"].long()[:, None, None]
    w = st["weights"][st["table"].long().clamp(min=0)].permute(0, 2, 1, 3).reshape(slot.shape[0], hk, -1)
    i = torch.arange(w.shape[2], device=w.device)
    w = w.masked_fill((i < c["sink"]) | (i >= lens - c["recent"]), math.inf).masked_fill(i >= lens, NEG)
    best = torch.sort(w, dim=2, descending=True, stable=True).indices[..., :budget]
    best = torch.where(best < lens, best, w.shape[2])                            # past the length: last
    keep = torch.sort(best, dim=2).values
    keep = torch.nn.functional.pad(keep, (0, budget - keep.shape[2]), value=w.shape[2])
    kept = keep < w.shape[2]
    new = (st["new_table"].long()[..., None] * page + torch.arange(page, device=w.device)).reshape(w.shape[0], -1)
    dst = new[:, None, :budget].expand_as(keep)
    src = torch.where(kept, torch.gather(slot[:, None].expand(-1, hk, -1), 2, keep.clamp(max=w.shape[2] - 1)), dst)
    g = torch.arange(hk, device=w.device)[None, :, None].expand_as(keep)
    k, v = st["k_pages"].view(-1, hk, d), st["v_pages"].view(-1, hk, d)
    k[dst, g] = k[src, g]
    v[dst, g] = v[src, g]
    ws = st["weights"]
    ws[dst // page, g, dst % page] = ws[src // page, g, src % page]
    new_lens = st["lens"].clamp(max=budget)
    return dict(keep=torch.where(kept, keep, -1).to(torch.int32), lens=new_lens, k_pages=st["k_pages"],
                v_pages=st["v_pages"], weights=ws)


def _plain_append(st):
    c = st["case"]
    page, hk, d = c["page"], c["h_kv"], c["d"]
    b, i = _packed(st, st["k"].shape[0])
    cu = st["cu"].long()
    pos = st["lens"].long()[b] - (cu[1:] - cu[:-1])[b] + i
    at = st["table"].long()[b, pos // page] * page + pos % page
    st["k_pages"].view(-1, hk, d)[at] = st["k"]
    st["v_pages"].view(-1, hk, d)[at] = st["v"]
    st["weights"][at // page, :, at % page] = 0.0
    return dict(k_pages=st["k_pages"], v_pages=st["v_pages"], weights=st["weights"])


def _plain_train(st):
    """Query blocks of `width` >= window tokens against the sinks, the block before and their
    own, every sequence padded to whole blocks."""
    c = st["case"]
    h, hk, d, window, sink = c["h"], c["h_kv"], c["d"], c["window"], c["sink"]
    r, width, dev = h // hk, max(window, 128), st["q"].device
    cu = st["cu"].long()
    L = cu[1:] - cu[:-1]
    B, nb = L.numel(), -(-st["longest"] // width)
    i = torch.arange(nb * width, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    valid = i < L[:, None]

    def heads(x):  # [B, h_kv, blocks, width * group, d]
        x = x[rows].masked_fill(~valid[..., None, None], 0).view(B, nb, width, hk, -1, d)
        return x.permute(0, 3, 1, 2, 4, 5).reshape(B, hk, nb, -1, d).float()

    q, do = heads(st["q"]), heads(st["d_o"])
    first = rows[:, :1] + torch.arange(sink, device=dev)

    def spans(x):  # [B, h_kv, blocks, sink + 2 * width, d]
        t = x[rows].masked_fill(~valid[..., None, None], 0).permute(0, 2, 1, 3).reshape(B, hk, nb, width, d).float()
        before = torch.cat([torch.zeros_like(t[:, :, :1]), t[:, :, :-1]], 2)
        s = x[first.clamp(max=x.shape[0] - 1)].permute(0, 2, 1, 3).float()
        return torch.cat([s[:, :, None].expand(-1, -1, nb, -1, -1), before, t], 3)

    k, v = spans(st["k"]), spans(st["v"])
    start = torch.arange(nb, device=dev) * width
    tq = i.view(nb, width)
    span = start[:, None] - width + torch.arange(2 * width, device=dev)
    near = (span[:, None] <= tq[..., None]) & (span[:, None] > tq[..., None] - window) & (span[:, None] >= 0)
    far = torch.arange(sink, device=dev) <= tq[..., None] - window
    see = torch.cat([far, near], 2)                                             # [blocks, width, keys]
    see = see & valid.view(B, 1, nb, width, 1)                                  # [B, 1, blocks, width, keys]
    see = see[:, :, :, :, None].expand(-1, -1, -1, -1, r, -1).reshape(B, 1, nb, width * r, -1)
    scale = 1.0 / math.sqrt(d)
    s = torch.matmul(q * scale, k.transpose(3, 4)).masked_fill_(~see, NEG)
    del see
    p = s.sub_(s.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l > 0, l, torch.ones_like(l)))
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(3, 4), do)
    ds = torch.matmul(do, v.transpose(3, 4)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(3, 4), q) * scale
    b, at = _packed(st, st["q"].shape[0])

    def rows_of(x):
        x = x.view(B, hk, nb, width, r, d).permute(0, 2, 3, 1, 4, 5).reshape(B, nb * width, h, d)
        return x[b, at].to(torch.bfloat16)

    def keys_of(x):  # own block + the next block's "before" + every block's sinks
        t = x[:, :, :, sink + width:].clone()
        t[:, :, :-1] += x[:, :, 1:, sink:sink + width]
        t = t.reshape(B, hk, nb * width, d)
        n = min(sink, nb * width)
        t[:, :, :n] += x[:, :, :, :n].sum(2)
        return t.permute(0, 2, 1, 3)[b, at].to(torch.bfloat16)

    return rows_of(o), rows_of(dq), keys_of(dk), keys_of(dv)


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import sparse_attention_compress_gb300 as nsa

        if op == "attn":
            o = nsa.nsa_paged_attn_fwd(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                       window=c["window"], n_sink=c["sink"], cu_seqlens=st["cu"],
                                       max_seqlen=st["longest"], lse=st["lse"])
            return o, st["lse"]
        if op == "weights":
            return nsa.nsa_paged_attn_weights(st["q"], st["k_pages"], st["lse"], st["table"], st["lens"],
                                              window=c["window"], n_sink=c["sink"], cu_seqlens=st["cu"],
                                              max_seqlen=st["longest"], weights=st["weights"], out=st["weights_out"])
        if op == "evict":
            keep, lens = nsa.nsa_paged_evict(st["k_pages"], st["v_pages"], st["weights"], st["table"], st["lens"],
                                             st["new_table"], c["budget"], n_sink=c["sink"], n_recent=c["recent"])
            return dict(keep=keep, lens=lens, k_pages=st["k_pages"], v_pages=st["v_pages"], weights=st["weights"])
        if op == "append":
            nsa.nsa_paged_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                 weights=st["weights"], cu_seqlens=st["cu"], max_seqlen=st["longest"])
            return dict(k_pages=st["k_pages"], v_pages=st["v_pages"], weights=st["weights"])
        o = nsa.nsa_swa_sink_fwd(st["q"], st["k"], st["v"], c["window"], c["sink"], cu_seqlens=st["cu"],
                                 max_seqlen=st["longest"], lse=st["lse"])
        dq, dk, dv = nsa.nsa_swa_sink_bwd(st["q"], st["k"], st["v"], o, st["lse"], st["d_o"], c["window"], c["sink"],
                                          cu_seqlens=st["cu"], max_seqlen=st["longest"])
        return o, dq, dk, dv
    return dict(attn=_plain_attn, weights=_plain_weights, evict=_plain_evict, append=_plain_append,
                train=_plain_train)[op](st)


# ----------------------------------------------------------------------------- exact values
def _sees(pos, n_keys, window, sink):
    key = torch.arange(n_keys, device=pos.device)[None, :]
    t = pos[:, None]
    return (key <= t) & ((t - key < window) | (key < sink)) if window else key <= t


def _cached(pages, table_row, n):
    """The first n cached rows of one sequence, [n, h_kv, d] in 64 bits."""
    used = table_row[:-(-n // pages.shape[1])].long()
    return torch.cat([pages[int(u)] for u in used.tolist()])[:n].double()


def exact(case, seed):
    op = case["op"]
    if op in ("append", "evict"):
        return None  # copies and choices: nothing is computed
    w = work(case)
    if w["flops"] > 1e12:
        return None
    st = prepare(case, seed)
    h, hk, d = case["h"], case["h_kv"], case["d"]
    r, scale = h // hk, 1.0 / math.sqrt(d)
    cu = st["cu"].tolist()
    if op == "train":
        outs = [torch.zeros_like(st[x], dtype=torch.float64) for x in ("q", "q", "k", "k")]
        step = min(2048, max(256, case["window"]))
        for a, e in zip(cu[:-1], cu[1:]):
            for g in range(hk):
                kk, vv = st["k"][a:e, g].double(), st["v"][a:e, g].double()
                for hh in range(g * r, (g + 1) * r):
                    for t0 in range(0, e - a, step):
                        t1 = min(e - a, t0 + step)
                        lo = max(0, t0 - case["window"] + 1)
                        ns = min(case["sink"], lo)
                        at = torch.cat([torch.arange(ns), torch.arange(lo, t1)]).to(kk.device)
                        qq, dd = st["q"][a + t0:a + t1, hh].double(), st["d_o"][a + t0:a + t1, hh].double()
                        see = _sees(torch.arange(t0, t1, device=kk.device), e - a, case["window"], case["sink"])[:, at]
                        p = torch.softmax((qq @ kk[at].T * scale).masked_fill(~see, NEG), -1)
                        o = p @ vv[at]
                        dp = dd @ vv[at].T
                        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
                        outs[0][a + t0:a + t1, hh] = o
                        outs[1][a + t0:a + t1, hh] = ds @ kk[at]
                        outs[2][a + at, g] += ds.T @ qq
                        outs[3][a + at, g] += p.T @ dd
        return tuple(outs)
    page = case["page"]
    o = torch.zeros_like(st["q"], dtype=torch.float64)
    lse = torch.full(st["lse"].shape, NEG, dtype=torch.float64, device="cuda")
    acc = st["weights_out"].double() if op == "weights" else None
    for b, (n, a, e) in enumerate(zip(st["lens"].tolist(), cu[:-1], cu[1:])):
        kk, vv = _cached(st["k_pages"], st["table"][b], n), _cached(st["v_pages"], st["table"][b], n)
        at = torch.arange(n, device="cuda")
        pg, sl = st["table"][b].long()[at // page], at % page
        for g in range(hk):
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for t0 in range(a, e, 512):
                t1 = min(e, t0 + 512)
                see = _sees(torch.arange(n - e + t0, n - e + t1, device="cuda"), n, case["window"], case["sink"])
                x = torch.einsum("qhd,kd->hqk", st["q"][t0:t1, g * r:(g + 1) * r].double(), kk[:, g]) * scale
                x = x.masked_fill(~see, NEG)
                if op == "attn":
                    o[t0:t1, g * r:(g + 1) * r] = torch.einsum("hqk,kd->qhd", torch.softmax(x, -1), vv[:, g])
                    lse[t0:t1, g * r:(g + 1) * r] = torch.logsumexp(x, -1).T
                else:
                    got += torch.exp(x - st["lse"][t0:t1, g * r:(g + 1) * r].double().T[..., None]).sum((0, 1))
            if op == "weights":
                acc[pg, g, sl] = st["weights"][pg, g, sl].double() + got
    return (o, lse) if op == "attn" else acc
