"""Cases and plain forms of the paged key/value cache operators.

Four operators that a serving loop runs on one cache:

  write   the new tokens' K and V rows go to their sequences' pages
  attend  attention of the new tokens (one a sequence, or a chunk) over the
          paged cache: o and the log-sum-exp
  score   each cached key gains the attention weight that the new tokens'
          queries give it, summed over the query heads of its kv head
  evict   a sequence longer than a budget keeps its newest keys and, of the
          others, those of largest accumulated weight, moved to its front

Keys and values lie in pages: a cache tensor is [pages, kv heads, page size,
head dim] by shape, stored rows-before-heads ("nhd") or heads-before-rows
("hnd"); position p of sequence b is row p % page_size of page
page_table[b, p // page_size].  Queries are packed [tokens, heads, head dim]
with cu_seqlens; the last tokens of a batch may belong to no sequence.
"""
import math
import random

import torch

own = False

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
BYTES = {"float32": 4, "float16": 2, "bfloat16": 2}


# ------------------------------------------------------------------- cases
def _case(op, batch, q_len, kv_len, hq, hkv, dim, dtype, page, layout="nhd", ragged=False, pad=0,
          sinks=False, keep=0, recent=0, mix=0, **kw):
    return dict(op=op, batch=batch, q_len=q_len, kv_len=kv_len, hq=hq, hkv=hkv, dim=dim,
                dtype=dtype, page=page, layout=layout, ragged=ragged, pad=pad, sinks=sinks,
                keep=keep, recent=recent, mix=mix, **kw)


def listed():
    return [
        # one new token for each of 64 running sequences: the cache write of a decode step
        _case("write", 64, 1, 2048, 32, 8, 128, "bfloat16", 16, ragged=True, name="write_step_b64"),
        # prompts' chunks written to pages; the batch is padded to a fixed size
        _case("write", 4, 2048, 8192, 32, 8, 128, "float16", 64, "hnd", ragged=True, pad=37,
              name="write_chunks_b4"),
        # a decode step of a few short sequences: latency counts
        _case("attend", 4, 1, 1000, 32, 8, 128, "bfloat16", 16, ragged=True,
              name="attend_step_short"),
        # the long decode's sizes (8 sequences of 32768 keys), on pages
        _case("attend", 8, 1, 32768, 32, 8, 128, "bfloat16", 64, name="attend_step_long"),
        # a full batch of unequal sequences with sink logits, head dim 64
        _case("attend", 64, 1, 8192, 16, 2, 64, "float16", 32, "hnd", ragged=True, sinks=True,
              name="attend_step_ragged"),
        # chunked prefill: unequal chunks of four prompts over what was cached before
        _case("attend", 4, 700, 5000, 32, 8, 128, "bfloat16", 16, ragged=True, pad=11,
              name="attend_chunks_b4"),
        # one large chunk at the end of a long prompt
        _case("attend", 1, 4096, 32768, 32, 8, 128, "bfloat16", 128, name="attend_chunk_long"),
        # full precision, a page size that is no power of two
        _case("attend", 2, 301, 2001, 8, 8, 64, "float32", 48, ragged=True,
              name="attend_chunks_f32"),
        # weights of one decode step added to every cached key's
        _case("score", 8, 1, 16384, 32, 8, 128, "bfloat16", 64, name="score_step_b8"),
        # weights of a prompt's chunk
        _case("score", 2, 2048, 8192, 32, 8, 128, "float16", 16, ragged=True,
              name="score_chunks_b2"),
        # a small cache cut back: latency counts
        _case("evict", 2, 1, 1500, 8, 8, 64, "float32", 16, ragged=True, keep=1024, recent=100,
              name="evict_small"),
        # eight long sequences cut to a quarter
        _case("evict", 8, 1, 16384, 32, 8, 128, "bfloat16", 64, keep=4096, recent=512,
              name="evict_b8"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "score", "evict"])
    hq, hkv = rng.choice([(32, 8), (16, 2), (8, 8), (12, 4), (16, 1), (38, 38), (24, 8)])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bfloat16", "float16", "bfloat16", "float16", "float32"])
    page = rng.choice([16, 16, 32, 64, 128, 8, 48, 256])
    layout = rng.choice(["nhd", "hnd"])
    kv = _log_int(rng, 1, 32768)
    q = 1 if (op != "write" and rng.random() < 0.5) else _log_int(rng, 1, min(kv, 4096))
    if op == "evict":
        q = 1
    batch = _log_int(rng, 1, 64)
    # no dearer than the largest listed cases: query-key pairs, keys, tokens
    f32 = 8 if dtype == "float32" else 1
    while batch > 1 and (batch * q * kv * hq * dim * f32 > 2 ** 38 or batch * kv * hkv > 2 ** 21):
        batch -= 1
    while q > 1 and (batch * q * kv * hq * dim * f32 > 2 ** 38):
        q = max(1, q // 2)
    keep = recent = 0
    if op == "evict":
        keep = max(1, int(kv * rng.uniform(0.1, 0.9)))
        recent = int(keep * rng.uniform(0.0, 0.5))
    return _case(op, batch, q, kv, hq, hkv, dim, dtype, page, layout,
                 ragged=rng.random() < 0.7, pad=rng.choice([0, 0, 5]) if op != "evict" else 0,
                 sinks=op == "attend" and rng.random() < 0.3, keep=keep, recent=recent,
                 mix=rng.randrange(1 << 16))


def _lengths(c):
    """Query and key counts of each sequence; the keys include the new tokens."""
    r = random.Random(c["mix"])
    qs, ks = [], []
    for b in range(c["batch"]):
        q, k = c["q_len"], c["kv_len"]
        if c["ragged"] and b > 0:  # the first sequence has the full length
            k = max(1, int(k * r.uniform(0.05, 1.0)))
            q = 1 if q == 1 else max(1, min(k, int(q * r.uniform(0.1, 1.0))))
        qs.append(min(q, k))
        ks.append(k)
    return qs, ks


def _pairs(c):
    """Query-key pairs under the causal rule: query i of q sees k - q + i + 1 keys."""
    return sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(*_lengths(c)))


def work(c):
    qs, ks = _lengths(c)
    es, d, hq, hkv = BYTES[c["dtype"]], c["dim"], c["hq"], c["hkv"]
    t, keys = sum(qs), sum(ks)
    if c["op"] == "write":  # K and V rows in and out
        return {"bytes": 4 * t * hkv * d * es, "flops": 0}
    if c["op"] == "attend":  # Q, O, LSE; K and V of every key once
        return {"bytes": 2 * t * hq * d * es + 4 * t * hq + 2 * keys * hkv * d * es,
                "flops": 4 * d * hq * _pairs(c)}
    if c["op"] == "score":  # Q, LSE; K of every key once; the weights in and out
        return {"bytes": t * hq * d * es + 4 * t * hq + keys * hkv * (d * es + 8),
                "flops": 2 * d * hq * _pairs(c)}
    cut = [k for k in ks if k > c["keep"]]
    moved = len(cut) * c["keep"] * hkv
    # weights of every key in and out, kept rows of K and V in and out, their positions out
    return {"bytes": 8 * keys * hkv + moved * (4 * d * es + 4), "flops": 0}


# ------------------------------------------------------------------ inputs
def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    qs, ks = _lengths(c)
    B, d, hq, hkv, ps = c["batch"], c["dim"], c["hq"], c["hkv"], c["page"]
    T = sum(qs) + c["pad"]
    need = [-(-k // ps) for k in ks]
    cols, pages = max(need), sum(need) + 3

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def cache():
        if c["layout"] == "nhd":
            return normal(pages, ps, hkv, d).transpose(1, 2)
        return normal(pages, hkv, ps, d)

    # pages in random order, as a pool hands them out; unused columns hold 0
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    need_t = torch.tensor(need, device=dev)
    start = torch.cumsum(need_t, 0) - need_t
    col = torch.arange(cols, device=dev)[None, :]
    table = torch.where(col < need_t[:, None], order[(start[:, None] + col).clamp(max=pages - 1)],
                        torch.zeros((), dtype=torch.int32, device=dev)).contiguous()
    s = dict(op=c["op"], scale=1.0 / math.sqrt(d), page=ps, max_q=max(qs), max_kv=max(ks),
             keep=c["keep"], recent=c["recent"], table=table,
             lens=torch.tensor(ks, dtype=torch.int32, device=dev),
             cu=torch.tensor([sum(qs[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev),
             k_pages=cache(), v_pages=cache(), sinks=None)
    if c["op"] == "write":
        s["k"], s["v"] = normal(T, hkv, d), normal(T, hkv, d)
    if c["op"] in ("attend", "score"):
        s["q"] = normal(T, hq, d)
        s["out"] = torch.zeros(T, hq, d, device=dev, dtype=dt)
        s["lse"] = torch.zeros(T, hq, device=dev)
        if c["sinks"]:
            s["sinks"] = torch.randn(hq, generator=g, device=dev)
    if c["op"] == "score":  # the log-sum-exp that the attention of these queries left
        s["lse"] = _attend(s)[1].clone()
    if c["op"] in ("score", "evict"):
        w = torch.rand(B, hkv, cols * ps, generator=g, device=dev)
        s["scores"] = -torch.log(1.0 - w) ** 3 if c["op"] == "evict" else w
        if c["op"] == "evict":  # a few heavy keys among many light ones, some of no weight
            s["scores"] = torch.where(w < 0.02, torch.zeros_like(w), s["scores"].abs())
    return s


# ------------------------------------------------------------- plain forms
def _rows(s):
    """For each packed token: its sequence, its place in it, and whether it has one."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    valid = b < cu.numel() - 1
    b = b.clamp(max=cu.numel() - 2)
    return b, t - cu[b], valid


def _gather(pages, s, dtype):
    """The cache rows of every sequence, [B, kv heads, max_kv, D]."""
    x = pages[s["table"].long()]  # [B, columns, heads, page, D]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, : s["max_kv"]]
    return x.to(dtype)


def _scores_of(s, dtype=torch.float32):
    """Scaled scores [B, kv heads, G, max_q, max_kv], -inf where not visible."""
    q, cu, lens = s["q"], s["cu"].long(), s["lens"].long()
    k = _gather(s["k_pages"], s, dtype)
    B, hkv = k.shape[0], k.shape[1]
    i = torch.arange(s["max_q"], device=q.device)
    tok = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[tok].to(dtype) * s["scale"]  # [B, max_q, Hq, D]
    x = x.unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4)
    sc = (x.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (x.shape[2], x.shape[3]))
    nq = cu[1:] - cu[:-1]
    last = (lens - nq)[:, None] + i  # last key that query i sees
    j = torch.arange(s["max_kv"], device=q.device)
    hidden = (j > last[:, :, None]) | (j >= lens[:, None, None]) | (i >= nq[:, None])[:, :, None]
    return sc.masked_fill_(hidden[:, None, None], -math.inf)


def _attend(s):
    s = dict(s, T=s["q"].shape[0])
    sc = _scores_of(s)
    m = sc.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, sc.shape[1], sc.shape[2], 1, 1)
        m = torch.maximum(m, sink)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        l = l + (sink - m).exp()
    o = p.flatten(2, 3) @ _gather(s["v_pages"], s, torch.float32)
    o = o.unflatten(2, (p.shape[2], p.shape[3])) / l.clamp(min=1e-38)
    lse = (m + l.log())[..., 0]
    b, i, valid = _rows(s)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i.clamp(max=s["max_q"] - 1)]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[b, i.clamp(max=s["max_q"] - 1)]
    return (torch.where(valid[:, None, None], o.to(s["q"].dtype), s["out"]),
            torch.where(valid[:, None], lse, s["lse"]))


def _write(s):
    s = dict(s, T=s["k"].shape[0])
    b, i, valid = _rows(s)
    cu, lens = s["cu"].long(), s["lens"].long()
    nq = cu[1:] - cu[:-1]
    pos = (lens - nq)[b] + i
    # a token of no sequence repeats the first token's write
    src = torch.where(valid, torch.arange(s["T"], device=b.device), 0)
    pos, b = pos[src], b[src]
    page = s["table"][b, pos // s["page"]].long()
    s["k_pages"][page, :, pos % s["page"]] = s["k"][src]
    s["v_pages"][page, :, pos % s["page"]] = s["v"][src]
    return s["k_pages"], s["v_pages"]


def _score(s):
    s = dict(s, T=s["q"].shape[0])
    sc = _scores_of(s)
    cu = s["cu"].long()
    i = torch.arange(s["max_q"], device=cu.device)
    lse = s["lse"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)]  # [B, max_q, Hq]
    lse = lse.unflatten(2, (sc.shape[1], sc.shape[2])).permute(0, 2, 3, 1)
    s["scores"][:, :, : s["max_kv"]] += sc.sub_(lse[..., None]).exp_().sum((2, 3))
    return s["scores"]


def _evict(s):
    scores, lens, keep, ps = s["scores"], s["lens"].long(), s["keep"], s["page"]
    C = scores.shape[2]
    j = torch.arange(C, device=scores.device)
    n = lens[:, None, None]
    x = scores.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    x = x.masked_fill(j >= n - min(s["recent"], keep), math.inf).masked_fill(j >= n, -math.inf)
    top = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(top, dim=-1).values
    j = j[:keep]
    kept = torch.where(n > keep, kept, torch.where(j < n, j, -1))
    new = lens.clamp(max=keep)
    # the rows move to positions 0, 1, ...; where there is none the first row's move is repeated
    dst = torch.where(kept >= 0, j, 0)
    src = torch.where(kept >= 0, kept, kept[..., :1])
    b = torch.arange(lens.numel(), device=lens.device)[:, None, None]
    h = torch.arange(scores.shape[1], device=lens.device)[None, :, None]
    table = s["table"].long()
    ps_src, ps_dst = table[b, src // ps], table[b, dst // ps]
    s["k_pages"][ps_dst, h, dst % ps] = s["k_pages"][ps_src, h, src % ps]
    s["v_pages"][ps_dst, h, dst % ps] = s["v_pages"][ps_src, h, src % ps]
    out = torch.zeros_like(scores)
    out[..., :keep] = torch.where(kept >= 0, scores.gather(2, kept.clamp(min=0)), 0.0)
    return kept.to(torch.int32), new.to(torch.int32), out, s["k_pages"], s["v_pages"]


PLAIN = {"write": _write, "attend": _attend, "score": _score, "evict": _evict}


# --------------------------------------------------------- the framework's
def _own(s):
    import scaled_dot_product_fwd_gb300 as S
    if s["op"] == "write":
        S.sdpa_paged_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                           cu_seqlens_q=s["cu"])
        return s["k_pages"], s["v_pages"]
    if s["op"] == "attend":
        return S.sdpa_paged_forward(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                    cu_seqlens_q=s["cu"], scale=s["scale"], sinks=s["sinks"],
                                    out=s["out"], lse=s["lse"])
    if s["op"] == "score":
        return S.sdpa_paged_scores(s["q"], s["k_pages"], s["lse"], s["scores"], s["table"],
                                   s["lens"], cu_seqlens_q=s["cu"], scale=s["scale"])
    kept, lens, scores = S.sdpa_paged_evict(s["k_pages"], s["v_pages"], s["scores"], s["table"],
                                            s["lens"], keep=s["keep"], recent=s["recent"])
    return kept, lens, scores, s["k_pages"], s["v_pages"]


def run(s):
    if own:
        return _own(s)
    return PLAIN[s["op"]](s)


# ------------------------------------------------------------------- exact
def exact(c, seed):
    """The definitions in 64 bits, sequence by sequence and kv head by kv head."""
    if c["op"] in ("write", "evict"):  # copies and whole numbers: the plain form is the value
        return None
    if 4 * c["dim"] * c["hq"] * _pairs(c) > 8e12:  # too long in 64 bits
        return None
    s = prepare(c, seed)
    qs, ks = _lengths(c)
    G, ps = c["hq"] // c["hkv"], c["page"]
    o = s["out"].double()
    lse = s["lse"].double()
    add = s["scores"].double() if c["op"] == "score" else None
    t0 = 0
    for b, (nq, nk) in enumerate(zip(qs, ks)):
        rows = torch.arange(nk, device="cuda")
        page = s["table"][b].long()[rows // ps]
        i = torch.arange(nq, device="cuda")
        hidden = rows[None, :] > (nk - nq + i)[:, None]
        for h in range(c["hkv"]):
            k = s["k_pages"][page, h, rows % ps].double()
            for e in range(G):
                hh = h * G + e
                x = s["q"][t0:t0 + nq, hh].double() @ k.T * s["scale"]
                x = x.masked_fill(hidden, -math.inf)
                if c["op"] == "score":
                    add[b, h, :nk] += (x - s["lse"][t0:t0 + nq, hh, None].double()).exp().sum(0)
                    continue
                if s["sinks"] is not None:
                    x = torch.cat([x, s["sinks"][hh].double().expand(nq, 1)], 1)
                z = torch.logsumexp(x, 1)
                w = (x[:, :nk] - z[:, None]).exp()
                o[t0:t0 + nq, hh] = w @ s["v_pages"][page, h, rows % ps].double()
                lse[t0:t0 + nq, hh] = z
        t0 += nq
    return add if c["op"] == "score" else (o, lse)
