"""Cases of the rotating append and of the 8-bit paged cache: inputs, plain forms, exact values.

Three operators that a server of this library uses together:

  rope    keys and values of new tokens written into a paged bf16 cache, K (and the tokens'
          queries) rotated by position on the way
  q8      the same into a cache held in 8 bits (e4m3) with a scale, a power of two, for each
          block of tokens and kv-head: a block's scale grows when a larger value arrives and
          its earlier codes are then rounded again
  attn    attention of a chunk of new tokens (or of one token a sequence) over that 8-bit
          cache, causal, with an optional sliding window and n_sink first tokens that stay
          visible

A case's lengths follow from the case alone; the seed decides the values and the pages.
With `own` false, run() computes the plain forms: elementary torch operations in 32 bits, the
angles of the rotation in 64.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")
TOP = 448.0           # the largest e4m3 value
E_MIN, E_MAX = -60, 60  # exponents of the scales


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # the new token of 32 users: latency counts
        dict(name="rope_token_32", op="rope", seqs=32, q=1, ctx=1024, spread=0.5, h=16, h_kv=2, d=128, page=64, rot=128,
             pairs="halves", far=0),
        # prompt chunks of four users
        dict(name="rope_chunk_4x2048", op="rope", seqs=4, q=2048, ctx=4096, spread=0.4, h=16, h_kv=4, d=128, page=64,
             rot=128, pairs="halves", far=0),
        # odd chunks after an eviction: true positions far past the cache's own, half of each head rotated, neighbours
        dict(name="rope_chunk_7x333_far", op="rope", seqs=7, q=333, ctx=1500, spread=0.6, h=12, h_kv=4, d=64, page=16,
             rot=32, pairs="neighbours", far=1000000),
        # the same token and chunks into the 8-bit cache
        dict(name="q8_token_32", op="q8", seqs=32, q=1, ctx=1024, spread=0.5, h=16, h_kv=2, d=128, page=64, block=64,
             rot=128, pairs="halves", far=0),
        dict(name="q8_chunk_4x2048", op="q8", seqs=4, q=2048, ctx=4096, spread=0.4, h=16, h_kv=4, d=128, page=64,
             block=64, rot=128, pairs="halves", far=0),
        # odd chunks, small blocks, no rotation (keys that a model rotated itself)
        dict(name="q8_chunk_5x777_plain", op="q8", seqs=5, q=777, ctx=3001, spread=0.7, h=12, h_kv=4, d=64, page=32,
             block=16, rot=0, pairs="halves", far=0),
        # one sequence, one new token over a short chat: the smallest attention call
        dict(name="attn_token_1x4096", op="attn", seqs=1, q=1, ctx=4096, spread=0.0, h=16, h_kv=2, d=128, page=64,
             block=64, window=0, sink=0),
        # a decode step of 32 users at up to 32768 tokens, as the decode benchmark's cache
        dict(name="attn_token_32x32768", op="attn", seqs=32, q=1, ctx=32768, spread=0.5, h=16, h_kv=2, d=128, page=64,
             block=64, window=0, sink=0),
        # drafted tokens of six users in small pages and blocks, odd lengths, an odd group
        dict(name="attn_draft_6x5_at_16001", op="attn", seqs=6, q=5, ctx=16001, spread=0.5, h=12, h_kv=4, d=64, page=16,
             block=16, window=0, sink=0),
        # eight drafted tokens with large groups: 128 rows a kv-head
        dict(name="attn_draft_16x8_at_8192", op="attn", seqs=16, q=8, ctx=8192, spread=0.4, h=64, h_kv=4, d=128, page=64,
             block=32, window=0, sink=0),
        # ragged chunks of eight prompts, a streaming window with sinks
        dict(name="attn_chunk_8x509_window", op="attn", seqs=8, q=509, ctx=8191, spread=0.7, h=12, h_kv=4, d=64, page=16,
             block=16, window=1024, sink=4),
        # a long prompt prefilled in chunks: 2048 new tokens at the end of 32768, the layer's heads
        dict(name="attn_chunk_1x2048_at_32768", op="attn", seqs=1, q=2048, ctx=32768, spread=0.0, h=64, h_kv=4, d=128,
             page=64, block=64, window=0, sink=0),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "q8", "q8", "attn", "attn", "attn"])
    d = rng.choice([64, 128])
    h_kv = rng.choice([1, 2, 4, 8])
    h = h_kv * rng.choice([1, 2, 3, 4, 6, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    spread = round(rng.uniform(0.0, 0.9), 2)
    if op == "attn":
        seqs = _log_int(rng, 1, 32)
        q = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2048)
        ctx = _log_int(rng, max(16, q), 32768)
        # score elements of the padded batch are bounded by the largest listed case's
        while seqs * q * h * ctx > 64 * 2048 * 32768 // 2 or seqs * ctx * h_kv * d > 32 * 32768 * 2 * 128:
            seqs, q, ctx = max(1, seqs // 2), max(1, q * 2 // 3), max(16, ctx * 3 // 4)
        q = min(q, ctx)
        window = 0 if rng.random() < 0.5 else _log_int(rng, 1, 4096)
        return dict(op=op, seqs=seqs, q=q, ctx=ctx, spread=spread, h=h, h_kv=h_kv, d=d, page=page, block=block,
                    window=window, sink=rng.randrange(0, 65) if window else 0)
    seqs, ctx = _log_int(rng, 1, 64), _log_int(rng, 16, 8192)
    while seqs * ctx * (h + 2 * h_kv) * d > 4 * 4096 * 24 * 128:
        seqs, ctx = max(1, seqs // 2), max(16, ctx * 3 // 4)
    q = 1 if rng.random() < 0.4 else _log_int(rng, 1, min(2048, ctx))
    rot = rng.choice([0, 16, d // 2, d, d]) if op == "q8" else rng.choice([16, d // 2, d, d])
    c = dict(op=op, seqs=seqs, q=q, ctx=ctx, spread=spread, h=h, h_kv=h_kv, d=d, page=page, rot=rot,
             pairs=rng.choice(["halves", "neighbours"]), far=rng.choice([0, 0, _log_int(rng, 1, 4000000)]))
    return dict(c, block=block) if op == "q8" else c


def _ragged(longest, shortest, seqs, spread):
    """Lengths from `longest` down by the share `spread`, never below `shortest`."""
    return [max(shortest, longest - int(spread * longest * b / max(1, seqs - 1))) if seqs > 1 else longest
            for b in range(seqs)]


def _q_lens(case):
    return _ragged(case["q"], 1, case["seqs"], case["spread"])


def _lens(case):
    """Cache lengths, the new tokens included."""
    return [max(a, b) for a, b in zip(_ragged(case["ctx"], 1, case["seqs"], case["spread"]), _q_lens(case))]


def _pairs(L, Q, window, sink):
    """(visible (query, key) pairs, keys that some query sees) of the last Q positions of L."""
    p = np.arange(L - Q, L, dtype=np.int64)
    lo = np.maximum(p - window + 1, 0) if window else np.zeros_like(p)
    n = p + 1 - lo + np.minimum(lo, sink)
    first = int(lo[0])
    return int(n.sum()), L - first + min(first, sink)


def work(case):
    op, h, hk, d = case["op"], case["h"], case["h_kv"], case["d"]
    L, Q = _lens(case), _q_lens(case)
    n = sum(Q)
    if op == "attn":
        both = [_pairs(a, b, case["window"], case["sink"]) for a, b in zip(L, Q)]
        pairs, keys = sum(x[0] for x in both), sum(x[1] for x in both)
        return {"bytes": 2 * n * h * d * 2 + 4 * n * h + 2 * keys * hk * d + 8 * keys * hk // case["block"],
                "flops": 4 * d * h * pairs}
    rotated = n * (h + hk) * (case["rot"] // 2) * 6
    queries = 2 * n * h * d * 2 if case["rot"] else 0
    if op == "rope":
        return {"bytes": queries + 4 * n * hk * d * 2, "flops": rotated}
    return {"bytes": queries + 2 * n * hk * d * 3 + 8 * n * hk // case["block"], "flops": rotated + 4 * n * hk * d}


# ----------------------------------------------------------------------------- inputs
def _normal(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def _prefix(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _keys(shape, gen):
    """Keys as models have them: some channels larger than the others, tokens of several sizes."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= 1.0 + 3.0 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.06)
    x *= torch.exp(0.4 * torch.randn(shape[:-2] + (1, 1), generator=gen, device="cuda"))
    return x.to(torch.bfloat16)


def _exponent(top):
    """Least e in [E_MIN, E_MAX] with top <= 448 * 2^e."""
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875)
    return torch.where(top > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _codes(x):
    return x.clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _pool(x, block):
    """(codes, scales) of a pool [n_pages, page, h_kv, d] of values: [n_pages, h_kv, page / block] scales."""
    n, page, hk, d = x.shape
    t = x.float().view(n, page // block, block, hk, d)
    s = torch.ldexp(torch.ones((), device=x.device), _exponent(t.abs().amax((2, 4))))
    return _codes(t / s[:, :, None, :, None]).view(n, page, hk, d), s.permute(0, 2, 1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 17)
    op, h, hk, d, page = case["op"], case["h"], case["h_kv"], case["d"], case["page"]
    L, Q = _lens(case), _q_lens(case)
    need = [-(-x // page) for x in L]
    # an allocator hands out pages in no order; recycled pages hold earlier tokens
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(L), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    n = sum(Q)
    k_pages, v_pages = _keys((n_pages, page, hk, d), gen), _normal((n_pages, page, hk, d), gen)
    st = dict(case=dict(case), table=table, lens=torch.tensor(L, dtype=torch.int32, device="cuda"), cu=_prefix(Q),
              longest=max(Q), q=_normal((n, h, d), gen))
    if op == "rope":
        st.update(k_pages=k_pages, v_pages=v_pages)
    else:
        st["k_pages"], st["k_scales"] = _pool(k_pages, case["block"])
        st["v_pages"], st["v_scales"] = _pool(v_pages, case["block"])
    if op == "attn":
        st["lse"] = torch.empty((n, h), dtype=torch.float32, device="cuda")
        return st
    st.update(k=_keys((n, hk, d), gen), v=_normal((n, hk, d), gen), q_out=torch.empty_like(st["q"]), inv_freq=None,
              positions=None)
    if case["rot"]:
        i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
        st["inv_freq"] = torch.pow(500000.0, -i / case["rot"]).float()
    if case["far"]:
        # tokens of a cache that was cut: their positions are those of the whole text
        b, i = _packed(st, n)
        st["positions"] = (case["far"] + 977 * b + i).to(torch.int32)
    return st


# ----------------------------------------------------------------------------- plain forms
def _padded(st):
    """Row of every (sequence, chunk position), its position in the cache and whether it exists."""
    cu, lens = st["cu"].long(), st["lens"].long()
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(st["longest"], device=cu.device)
    rows = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    return rows, (lens - q_len)[:, None] + i, i < q_len[:, None]


def _packed(st, n):
    """(sequence, chunk position) of every packed row."""
    cu = st["cu"].long()
    b = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=cu.device), cu[1:] - cu[:-1], output_size=n)
    return b, torch.arange(n, device=cu.device) - cu[b]


def _places(st):
    """Cache position of every packed row."""
    cu = st["cu"].long()
    b, i = _packed(st, st["q"].shape[0])
    return b, st["lens"].long()[b] - (cu[1:] - cu[:-1])[b] + i


def _rotate(st, x, pos):
    """x [tokens, heads, d] in 32 bits, its first rot dimensions rotated by position."""
    c = st["case"]
    x, n = x.float(), c["rot"] // 2
    if not n:
        return x
    a = pos.double()[:, None] * st["inv_freq"].double()
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    if c["pairs"] == "halves":
        u, v = x[..., :n], x[..., n:2 * n]
        both = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    else:
        u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        both = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    return torch.cat([both, x[..., 2 * n:]], -1)


def _plain_rope(st):
    c = st["case"]
    page, hk, d = c["page"], c["h_kv"], c["d"]
    b, place = _places(st)
    pos = place if st["positions"] is None else st["positions"]
    at = st["table"].long()[b, place // page] * page + place % page
    st["k_pages"].view(-1, hk, d)[at] = _rotate(st, st["k"], pos).to(torch.bfloat16)
    st["v_pages"].view(-1, hk, d)[at] = st["v"]
    return dict(q=_rotate(st, st["q"], pos).to(torch.bfloat16), k_pages=st["k_pages"], v_pages=st["v_pages"])


def _store(st, pages, scales, x):
    """New values x [tokens, h_kv, d] in 32 bits into the 8-bit pages, block by block."""
    c = st["case"]
    page, block, hk, d = c["page"], c["block"], c["h_kv"], c["d"]
    cu, lens = st["cu"].long(), st["lens"].long()
    first = lens - (cu[1:] - cu[:-1])                                            # the first new position
    nb = st["longest"] // block + 2                                              # blocks that new tokens can touch
    start = (first // block)[:, None] * block + torch.arange(nb, device=x.device) * block
    pos = start[..., None] + torch.arange(block, device=x.device)                # [seqs, blocks, block]
    new = (pos >= first[:, None, None]) & (pos < lens[:, None, None])
    row = (cu[:-1] - first)[:, None, None] + pos
    v = x[row.clamp(0, x.shape[0] - 1)].masked_fill(~new[..., None, None], 0)    # [seqs, blocks, block, h_kv, d]
    touched = new.any(-1)
    slots = st["table"].shape[1] * page
    pid = torch.gather(st["table"].long(), 1, (start.clamp(max=slots - 1) // page))
    part = start % page // block
    old = (pos < first[:, None, None]) & touched[..., None]
    was = scales[pid, :, part]                                                   # [seqs, blocks, h_kv]
    need = torch.ldexp(torch.ones((), device=x.device), _exponent(v.abs().amax((2, 4))))
    s = torch.where(old.any(-1, keepdim=True), torch.maximum(was, need), need)
    flat = pages.view(torch.uint8).view(-1, hk, d)
    at = (pid * page + part * block)[..., None] + torch.arange(block, device=x.device)
    held = flat[at].view(torch.float8_e4m3fn).float() * (was / s)[:, :, None, :, None]
    codes = _codes(torch.where(new[..., None, None], v / s[:, :, None, :, None], held)).view(torch.uint8)
    write = new | old
    flat[at[write]] = codes[write]
    scales[pid[touched], :, part[touched]] = s[touched]


def _plain_q8(st):
    _, place = _places(st)
    pos = place if st["positions"] is None else st["positions"]
    _store(st, st["k_pages"], st["k_scales"], _rotate(st, st["k"], pos))
    _store(st, st["v_pages"], st["v_scales"], st["v"].float())
    out = {x: st[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")}
    if st["case"]["rot"]:
        out["q"] = _rotate(st, st["q"], pos).to(torch.bfloat16)
    return out


def _gathered(pages, scales, table, block):
    """Values of each sequence's pages one after another: [seqs, h_kv, slots, d] in 32 bits."""
    t = table.long().clamp(min=0)
    x = pages.view(torch.uint8)[t].view(torch.float8_e4m3fn).float()             # [seqs, pages, page, h_kv, d]
    x = x * scales[t].repeat_interleave(block, 3).permute(0, 1, 3, 2)[..., None]
    return x.reshape(x.shape[0], -1, x.shape[3], x.shape[4]).permute(0, 2, 1, 3)


def _plain_attn(st):
    c = st["case"]
    rows, pos, valid = _padded(st)
    B, Q = rows.shape
    h, hk, d = c["h"], c["h_kv"], c["d"]
    r = h // hk
    k = _gathered(st["k_pages"], st["k_scales"], st["table"], c["block"])
    q = st["q"][rows].reshape(B, Q, hk, r, d).permute(0, 2, 1, 3, 4).reshape(B, hk, Q * r, d).float()
    s = torch.matmul(q * (1.0 / math.sqrt(d)), k.transpose(2, 3))
    del k
    key = torch.arange(s.shape[3], device=s.device)
    see = key <= pos[..., None]
    if c["window"]:
        see &= (key > pos[..., None] - c["window"]) | (key < c["sink"])
    see &= valid[..., None]
    s = s.view(B, hk, Q, r, -1).masked_fill_(~see[:, None, :, None, :], NEG).view(B, hk, Q * r, -1)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = _gathered(st["v_pages"], st["v_scales"], st["table"], c["block"])
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    b, i = _packed(st, st["q"].shape[0])

    def rows_of(x):  # [seqs, h_kv, queries * group, e] -> packed [tokens, h, e]
        x = x.reshape(B, hk, Q, r, x.shape[-1]).permute(0, 2, 1, 3, 4)
        return x[b, i].reshape(b.numel(), h, -1)

    return rows_of(o).to(torch.bfloat16), rows_of(m + l.log())[..., 0].contiguous()


def run(st):
    c = st["case"]
    if own:
        import sparse_attention_compress_gb300 as nsa

        packed = dict(cu_seqlens=st["cu"], max_seqlen=st["longest"])
        if c["op"] == "attn":
            o = nsa.nsa_paged_q8_attn_fwd(st["q"], st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"],
                                          st["table"], st["lens"], window=c["window"], n_sink=c["sink"], lse=st["lse"],
                                          **packed)
            return o, st["lse"]
        turn = {}
        if c["rot"]:
            turn = dict(q=st["q"], q_out=st["q_out"], inv_freq=st["inv_freq"], positions=st["positions"],
                        interleaved=c["pairs"] == "neighbours")
        if c["op"] == "rope":
            q = nsa.nsa_paged_append_rope(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                          **turn, **packed)
            return dict(q=q, k_pages=st["k_pages"], v_pages=st["v_pages"])
        q = nsa.nsa_paged_q8_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"],
                                    st["table"], st["lens"], **turn, **packed)
        out = {x: st[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")}
        return dict(out, q=q) if c["rot"] else out
    return dict(rope=_plain_rope, q8=_plain_q8, attn=_plain_attn)[c["op"]](st)


# ----------------------------------------------------------------------------- exact values
def _turned(case, inv_freq, x, pos):
    """The rotation in 64 bits as a product of complex numbers."""
    x, n = x.double(), case["rot"] // 2
    if not n:
        return x
    turn = torch.polar(torch.ones(pos.numel(), n, dtype=torch.float64, device=x.device),
                       torch.outer(pos.double(), inv_freq.double()))[:, None]
    head = x[..., :2 * n]
    z = torch.complex(head[..., :n].contiguous(), head[..., n:].contiguous()) if case["pairs"] == "halves" else \
        torch.view_as_complex(head.reshape(*head.shape[:-1], n, 2).contiguous())
    z = z * turn
    head = torch.cat([z.real, z.imag], -1) if case["pairs"] == "halves" else torch.view_as_real(z).flatten(-2)
    return torch.cat([head, x[..., 2 * n:]], -1)


def _least(top):
    """Least power of two s with top <= 448 s, within the scales' range."""
    e = E_MIN
    while e < E_MAX and top > TOP * 2.0 ** e:
        e += 1
    return 2.0 ** e


def exact(case, seed):
    w = work(case)
    if w["flops"] > 1e12:
        return None
    st = prepare(case, seed)
    h, hk, d, page = case["h"], case["h_kv"], case["d"], case["page"]
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    if case["op"] != "attn":
        out = {x: st[x].double() for x in ("k_pages", "v_pages", "k_scales", "v_scales") if x in st}
        if case["rot"]:
            out["q"] = torch.zeros_like(st["q"], dtype=torch.float64)
        for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
            first = lens[b] - (e - a)
            pos = torch.arange(first, lens[b], device="cuda") if st["positions"] is None else st["positions"][a:e]
            if case["rot"]:
                out["q"][a:e] = _turned(case, st["inv_freq"], st["q"][a:e], pos)
            new = {"k": _turned(case, st["inv_freq"], st["k"][a:e], pos), "v": st["v"][a:e].double()}
            step = case.get("block", page)
            for p0 in range(first // step * step, lens[b], step):
                lo, hi = max(p0, first), min(p0 + step, lens[b])
                pid, at = int(st["table"][b, p0 // page]), p0 % page
                for x in "kv":
                    pages, part = out[x + "_pages"], new[x][lo - first:hi - first]
                    if case["op"] == "rope":
                        pages[pid, at + lo - p0:at + hi - p0] = part
                        continue
                    was = st[x + "_scales"][pid, :, at // step].tolist()
                    for g, top in enumerate(part.abs().amax((0, 2)).tolist()):
                        # what a code stands for before it is rounded
                        s = max(was[g], _least(top)) if lo > p0 else _least(top)
                        pages[pid, at:at + lo - p0, g] *= was[g] / s
                        pages[pid, at + lo - p0:at + hi - p0, g] = part[:, g] / s
                        out[x + "_scales"][pid, g, at // step] = s
        return out
    r, scale, block = h // hk, 1.0 / math.sqrt(d), case["block"]
    o = torch.zeros_like(st["q"], dtype=torch.float64)
    lse = torch.full(st["lse"].shape, NEG, dtype=torch.float64, device="cuda")
    for b, (n, a, e) in enumerate(zip(lens, cu[:-1], cu[1:])):
        at = torch.arange(n, device="cuda")
        pid, slot = st["table"][b].long()[at // page], at % page
        for g in range(hk):
            kk, vv = (st[x + "_pages"].view(torch.uint8)[pid, slot, g].view(torch.float8_e4m3fn).double()
                      * st[x + "_scales"][pid, g, slot // block].double()[:, None] for x in "kv")
            for t0 in range(a, e, 512):
                t1 = min(e, t0 + 512)
                t = torch.arange(n - e + t0, n - e + t1, device="cuda")[:, None]
                see = at <= t
                if case["window"]:
                    see &= (t - at < case["window"]) | (at < case["sink"])
                x = torch.einsum("qhd,kd->hqk", st["q"][t0:t1, g * r:(g + 1) * r].double(), kk) * scale
                x = x.masked_fill(~see, NEG)
                o[t0:t1, g * r:(g + 1) * r] = torch.einsum("hqk,kd->qhd", torch.softmax(x, -1), vv)
                lse[t0:t1, g * r:(g + 1) * r] = torch.logsumexp(x, -1).T
    return o, lse
