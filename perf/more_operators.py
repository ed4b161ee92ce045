"""Cases and plain forms of the rotary operators and of the 4-bit paged cache.

Four operators around the attention of a serving or training loop:

  rope     rotary positions of q and k [batch, heads, length, dim], or, for the
           gradients, the transposed rotation
  append   a serving step's rotation on the way to the paged cache: the new
           tokens' q rotated, their k rotated and written to pages, v written
  append4  the same into a cache held in 4 bits
  attend4  attention of the new tokens (one a sequence, or a chunk) over the
           4-bit cache: o and the log-sum-exp

The rotation table is float32 [positions, R / 2, 2]: cosine and sine of every
position and frequency, R <= dim the rotated elements of a head.  Pair i of a
head is (i, i + R / 2), or (2i, 2i + 1) where `interleaved`; a pair (x, y)
turns to (x cos - y sin, y cos + x sin).

The 4-bit cache keeps a row of dim elements as dim / 2 bytes, two 4-bit floats
(1 sign, 2 exponent, 1 mantissa bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6) each, the
even element in the low half, and a scale of 8 bits (e4m3) for every 16
elements.  Element = code * scale * g, g a float32 of the kv head (1 without).
With y = x / g in 32 bits, the scale is max |y| / 6 rounded to e4m3 (at most
448, at least 2^-9), a code y / scale rounded to the nearest, ties to even.
x is the row in its own type: k is rounded to it after the rotation.

Pages, page tables, packed tokens and lengths are those of the paged cache:
[pages, kv heads, page size, ...] by shape, stored rows-before-heads ("nhd")
or heads-before-rows ("hnd"); position p of sequence b is row p % page_size of
page page_table[b, p // page_size]; the last tokens of a batch may belong to no
sequence.
"""
import math
import random

import torch

own = False

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
BYTES = {"float32": 4, "float16": 2, "bfloat16": 2}
# the 16 values of a 4-bit code
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------- cases
def _case(op, batch, q_len, kv_len, hq, hkv, dim, dtype, page=16, layout="nhd", ragged=False,
          pad=0, sinks=False, rot=0, interleaved=False, shift=0, backward=False, gains=False,
          mix=0, **kw):
    return dict(op=op, batch=batch, q_len=q_len, kv_len=kv_len, hq=hq, hkv=hkv, dim=dim,
                dtype=dtype, page=page, layout=layout, ragged=ragged, pad=pad, sinks=sinks,
                rot=rot or dim, interleaved=interleaved, shift=shift, backward=backward,
                gains=gains, mix=mix, **kw)


def listed():
    return [
        # q and k of the image transformer (2 x 38 heads x 4250 x 64), heads before rows
        _case("rope", 2, 4250, 4250, 38, 38, 64, "float16", layout="hnd", interleaved=True,
              name="rope_dit"),
        # gradients of q and k of a long training sequence, grouped heads, rows before heads
        _case("rope", 1, 8192, 8192, 32, 8, 128, "bfloat16", shift=1000, backward=True,
              name="rope_backward_gqa"),
        # one new token for each of 64 running sequences: latency counts
        _case("append", 64, 1, 2048, 32, 8, 128, "bfloat16", 16, ragged=True,
              name="append_step_b64"),
        # prompts' chunks, half of each head rotated, positions of their own
        _case("append", 4, 2048, 8192, 32, 8, 128, "float16", 64, "hnd", ragged=True, pad=37,
              rot=64, shift=500, name="append_chunks_b4"),
        # the decode step into the 4-bit cache
        _case("append4", 64, 1, 2048, 32, 8, 128, "bfloat16", 16, ragged=True,
              name="append4_step_b64"),
        # prompts' chunks into the 4-bit cache, with a gain for each kv head
        _case("append4", 4, 2048, 8192, 32, 8, 128, "float16", 64, "hnd", ragged=True, pad=37,
              interleaved=True, gains=True, name="append4_chunks_b4"),
        # a decode step of a few short sequences: latency counts
        _case("attend4", 4, 1, 1000, 32, 8, 128, "bfloat16", 16, ragged=True,
              name="attend4_step_short"),
        # the long decode's sizes (8 sequences of 32768 keys)
        _case("attend4", 8, 1, 32768, 32, 8, 128, "bfloat16", 64, name="attend4_step_long"),
        # a full batch of unequal sequences with sink logits, head dim 64
        _case("attend4", 64, 1, 8192, 16, 2, 64, "float16", 32, "hnd", ragged=True, sinks=True,
              gains=True, name="attend4_step_ragged"),
        # chunked prefill: unequal chunks of four prompts over what was cached before
        _case("attend4", 4, 700, 5000, 32, 8, 128, "bfloat16", 16, ragged=True, pad=11,
              name="attend4_chunks_b4"),
        # one large chunk at the end of a long prompt
        _case("attend4", 1, 4096, 32768, 32, 8, 128, "bfloat16", 128, name="attend4_chunk_long"),
        # full-precision queries, a page size that is no power of two
        _case("attend4", 2, 301, 2001, 8, 8, 64, "float32", 48, ragged=True, gains=True,
              name="attend4_chunks_f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append4", "attend4", "attend4"])
    hq, hkv = rng.choice([(32, 8), (16, 2), (8, 8), (12, 4), (16, 1), (38, 38), (24, 8)])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bfloat16", "float16", "bfloat16", "float16", "float32"])
    kv = _log_int(rng, 1, 32768)
    q = 1 if rng.random() < 0.5 else _log_int(rng, 1, min(kv, 4096))
    batch = _log_int(rng, 1, 64)
    # no dearer than the largest listed cases: query-key pairs, keys, tokens
    f32 = 8 if dtype == "float32" else 1
    while batch > 1 and (op == "attend4" and batch * q * kv * hq * dim * f32 > 2 ** 38
                         or batch * kv * hkv > 2 ** 21 or batch * q > 8192):
        batch -= 1
    while op == "attend4" and q > 1 and batch * q * kv * hq * dim * f32 > 2 ** 38:
        q = max(1, q // 2)
    return _case(op, batch, q, kv, hq, hkv, dim, dtype,
                 rng.choice([16, 16, 32, 64, 128, 8, 48, 256]), rng.choice(["nhd", "hnd"]),
                 ragged=op != "rope" and rng.random() < 0.7,
                 pad=rng.choice([0, 0, 5]) if op != "rope" else 0,
                 sinks=op == "attend4" and rng.random() < 0.3,
                 rot=rng.choice([dim, dim, dim // 2, 16]), interleaved=rng.random() < 0.4,
                 shift=rng.choice([0, rng.randrange(1, 4000)]),
                 backward=op == "rope" and rng.random() < 0.5, gains=rng.random() < 0.4,
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
    es, d, hq, hkv, r = BYTES[c["dtype"]], c["dim"], c["hq"], c["hkv"], c["rot"]
    t, keys, row4 = sum(qs), sum(ks), c["dim"] // 2 + c["dim"] // 16
    if c["op"] == "rope":  # q and k in and out; the table's rows once
        t = c["batch"] * c["q_len"]
        return {"bytes": 2 * t * (hq + hkv) * d * es + 4 * r * c["q_len"],
                "flops": 3 * t * (hq + hkv) * r}
    if c["op"] == "append":  # q, k and v in and out; a row of the table a token
        return {"bytes": 2 * t * (hq + 2 * hkv) * d * es + 4 * r * t,
                "flops": 3 * t * (hq + hkv) * r}
    if c["op"] == "append4":  # the same, the rows' codes and scales out, and what they stand for
        return {"bytes": t * (2 * hq + 4 * hkv) * d * es + 2 * t * hkv * row4 + 4 * r * t,
                "flops": 3 * t * (hq + hkv) * r}
    # Q, O, LSE; the codes and scales of every key once
    return {"bytes": 2 * t * hq * d * es + 4 * t * hq + 2 * keys * hkv * row4,
            "flops": 4 * d * hq * _pairs(c)}


# ------------------------------------------------------------------ inputs
def _table(length, rot, device):
    """Cosine and sine of position * 10000^(-2i / rot), from angles in 64 bits."""
    i = torch.arange(rot // 2, device=device, dtype=torch.float64)
    p = torch.arange(length, device=device, dtype=torch.float64)
    a = p[:, None] * 10000.0 ** (-2.0 * i / rot)
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _heads(x, c):
    """[batch, heads, rows, dim] by shape, stored in the case's order."""
    return x if c["layout"] == "hnd" else x.transpose(1, 2).contiguous().transpose(1, 2)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    B, d, hq, hkv, ps = c["batch"], c["dim"], c["hq"], c["hkv"], c["page"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    s = dict(op=c["op"], interleaved=c["interleaved"], backward=c["backward"], page=ps)
    if c["op"] == "rope":
        L = c["q_len"]
        s["q"], s["k"] = _heads(normal(B, hq, L, d), c), _heads(normal(B, hkv, L, d), c)
        start = torch.randint(0, c["shift"] + 1, (B, 1), generator=g, device=dev)
        s["positions"] = (start + torch.arange(L, device=dev)).to(torch.int32)
        s["rope"] = _table(L + c["shift"], c["rot"], dev)
        return s

    qs, ks = _lengths(c)
    T = sum(qs) + c["pad"]
    need = [-(-k // ps) for k in ks]
    cols, pages = max(need), sum(need) + 3
    # pages in random order, as a pool hands them out; unused columns hold 0
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    need_t = torch.tensor(need, device=dev)
    start = torch.cumsum(need_t, 0) - need_t
    col = torch.arange(cols, device=dev)[None, :]
    s["table"] = torch.where(
        col < need_t[:, None], order[(start[:, None] + col).clamp(max=pages - 1)],
        torch.zeros((), dtype=torch.int32, device=dev)).contiguous()
    s.update(scale=1.0 / math.sqrt(d), max_q=max(qs), max_kv=max(ks), T=T,
             lens=torch.tensor(ks, dtype=torch.int32, device=dev),
             cu=torch.tensor([sum(qs[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev),
             k_gain=None, v_gain=None, sinks=None, positions=None)
    if c["gains"]:  # of a calibration: the heads' magnitudes differ
        s["k_gain"] = 0.05 + torch.rand(hkv, generator=g, device=dev)
        s["v_gain"] = 0.05 + torch.rand(hkv, generator=g, device=dev)
    s["q"] = normal(T, hq, d)
    if c["op"] != "attend4":
        s["k"], s["v"] = normal(T, hkv, d), normal(T, hkv, d)
        s["rope"] = _table(max(ks) + c["shift"], c["rot"], dev)
        s["q_out"] = torch.zeros_like(s["q"])
        if c["shift"]:  # positions of their own: keys were evicted before
            b, i, valid = _rows(s)
            nq = (s["cu"][1:] - s["cu"][:-1]).long()
            p = (s["lens"].long() - nq)[b] + i + c["shift"]
            s["positions"] = torch.where(valid, p, 0).to(torch.int32)
    if c["op"] == "append":
        s["k_pages"] = _heads(normal(pages, hkv, ps, d), c)
        s["v_pages"] = _heads(normal(pages, hkv, ps, d), c)
        return s
    s["codes"] = torch.tensor(CODES, device=dev)
    if c["op"] == "append4":
        for x in "kv":
            s[x + "_out"] = torch.zeros_like(s["k"])
            s[x + "_pages"] = _heads(torch.zeros(pages, hkv, ps, d // 2, dtype=torch.uint8,
                                                 device=dev), c)
            s[x + "_scales"] = _heads(torch.zeros(pages, hkv, ps, d // 16, dtype=torch.uint8,
                                                  device=dev), c)
        return s
    for x in "kv":
        codes, scales, _ = _quantise(normal(pages, hkv, ps, d), s[x + "_gain"], 1)
        s[x + "_pages"], s[x + "_scales"] = _heads(codes, c), _heads(scales, c)
    s["out"] = torch.zeros(T, hq, d, device=dev, dtype=dt)
    s["lse"] = torch.zeros(T, hq, device=dev)
    if c["sinks"]:
        s["sinks"] = torch.randn(hq, generator=g, device=dev)
    return s


# ------------------------------------------------------------- plain forms
def _rotate(x, cs, interleaved, back=False):
    """x [..., dim] turned by the table rows cs [..., R / 2, 2]."""
    h = cs.shape[-2]
    c, s = cs[..., 0], -cs[..., 1] if back else cs[..., 1]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    ra, rb = a * c - b * s, b * c + a * s
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([r, x[..., 2 * h:]], -1)


def _rope(s):
    cs = s["rope"][s["positions"].long()][:, None]
    return tuple(_rotate(x.float(), cs, s["interleaved"], s["backward"]).to(x.dtype)
                 for x in (s["q"], s["k"]))


def _rows(s):
    """For each packed token: its sequence, its place in it, and whether it has one."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    valid = b < cu.numel() - 1
    b = b.clamp(max=cu.numel() - 2)
    return b, t - cu[b], valid


def _places(s):
    """The packed tokens that have a sequence repeat the first one's place where they have
    none: (source token, page, row in it, valid), and the tokens' rotation rows."""
    b, i, valid = _rows(s)
    cu, lens = s["cu"].long(), s["lens"].long()
    pos = (lens - (cu[1:] - cu[:-1]))[b] + i
    src = torch.where(valid, torch.arange(s["T"], device=b.device), 0)
    turn = s["positions"].long() if s["positions"] is not None else torch.where(valid, pos, 0)
    pos, b = pos[src], b[src]
    return src, s["table"][b, pos // s["page"]].long(), pos % s["page"], valid, s["rope"][turn]


def _append(s):
    src, page, row, valid, cs = _places(s)
    q = _rotate(s["q"].float(), cs[:, None], s["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cs[:, None], s["interleaved"]).to(s["k"].dtype)
    s["k_pages"][page, :, row] = k[src]
    s["v_pages"][page, :, row] = s["v"][src]
    return torch.where(valid[:, None, None], q, s["q_out"]), s["k_pages"], s["v_pages"]


def _quantise(x, gain, head_dim):
    """Codes in bytes, scales in bytes, and the values of rows x; gain of dimension head_dim."""
    y = x.float()
    if gain is not None:
        y = y / gain.view([-1 if i == head_dim else 1 for i in range(x.dim())])
    y = y.unflatten(-1, (-1, 16))
    top = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    scale = top.float().clamp(min=2.0 ** -9)
    t = y / scale
    a = t.abs().clamp(max=6.0)
    # steps of 0.5 below 2, of 1 below 4, of 2 above; round() takes ties to even
    m = torch.where(a < 2.0, (2.0 * a).round() * 0.5,
                    torch.where(a < 4.0, a.round(), (0.5 * a).round() * 2.0))
    code = torch.where(m < 2.0, 2.0 * m, torch.where(m < 4.0, m + 2.0, m * 0.5 + 4.0))
    code = code + 8.0 * torch.signbit(t)
    value = (torch.copysign(m, t) * scale).flatten(-2)
    if gain is not None:
        value = value * gain.view([-1 if i == head_dim else 1 for i in range(x.dim())])
    code = code.to(torch.uint8).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4),
            scale[..., 0].to(torch.float8_e4m3fn).view(torch.uint8), value.to(x.dtype))


def _append4(s):
    # the rotation in 64 bits: a code next to a border must not turn on its rounding
    src, page, row, valid, cs = _places(s)
    q = _rotate(s["q"].float(), cs[:, None], s["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].double(), cs[:, None].double(), s["interleaved"]).to(s["k"].dtype)
    kc, ks, kv = _quantise(k, s["k_gain"], 1)
    vc, vs, vv = _quantise(s["v"], s["v_gain"], 1)
    s["k_pages"][page, :, row], s["k_scales"][page, :, row] = kc[src], ks[src]
    s["v_pages"][page, :, row], s["v_scales"][page, :, row] = vc[src], vs[src]
    at = valid[:, None, None]
    return (torch.where(at, q, s["q_out"]), torch.where(at, kv, s["k_out"]),
            torch.where(at, vv, s["v_out"]))


def _gather(s, x):
    """The cache rows of every sequence in 32 bits, [B, kv heads, max_kv, D]."""
    t = s["table"].long()
    p, c = s[x + "_pages"][t], s[x + "_scales"][t]  # [B, columns, heads, page, ...]
    v = torch.stack([s["codes"][(p & 15).int()], s["codes"][(p >> 4).int()]], -1).flatten(-2)
    v = (v.unflatten(-1, (-1, 16)) * c.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)
    v = v.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, : s["max_kv"]]
    return v if s[x + "_gain"] is None else v * s[x + "_gain"][:, None, None]


def _scores_of(s):
    """Scaled scores [B, kv heads, G, max_q, max_kv], -inf where not visible."""
    q, cu, lens = s["q"], s["cu"].long(), s["lens"].long()
    k = _gather(s, "k")
    hkv = k.shape[1]
    i = torch.arange(s["max_q"], device=q.device)
    tok = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[tok].float() * s["scale"]  # [B, max_q, Hq, D]
    x = x.unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4)
    sc = (x.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (x.shape[2], x.shape[3]))
    nq = cu[1:] - cu[:-1]
    last = (lens - nq)[:, None] + i  # last key that query i sees
    j = torch.arange(s["max_kv"], device=q.device)
    hidden = (j > last[:, :, None]) | (j >= lens[:, None, None]) | (i >= nq[:, None])[:, :, None]
    return sc.masked_fill_(hidden[:, None, None], -math.inf)


def _attend4(s):
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
    o = p.flatten(2, 3) @ _gather(s, "v")
    o = o.unflatten(2, (p.shape[2], p.shape[3])) / l.clamp(min=1e-38)
    lse = (m + l.log())[..., 0]
    b, i, valid = _rows(s)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i.clamp(max=s["max_q"] - 1)]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[b, i.clamp(max=s["max_q"] - 1)]
    return (torch.where(valid[:, None, None], o.to(s["q"].dtype), s["out"]),
            torch.where(valid[:, None], lse, s["lse"]))


PLAIN = {"rope": _rope, "append": _append, "append4": _append4, "attend4": _attend4}


# --------------------------------------------------------- the framework's
def _own(s):
    import scaled_dot_product_fwd_gb300 as S
    if s["op"] == "rope":
        call = S.sdpa_rope_backward if s["backward"] else S.sdpa_rope
        return call(s["q"], s["k"], s["rope"], positions=s["positions"],
                    interleaved=s["interleaved"])
    if s["op"] == "append":
        q = S.sdpa_paged_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"],
                                s["lens"], s["rope"], cu_seqlens_q=s["cu"],
                                positions=s["positions"], interleaved=s["interleaved"],
                                q_out=s["q_out"])
        return q, s["k_pages"], s["v_pages"]
    if s["op"] == "append4":
        q = S.sdpa_paged_append_fp4(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"],
                                    s["k_scales"], s["v_scales"], s["table"], s["lens"],
                                    s["rope"], cu_seqlens_q=s["cu"], positions=s["positions"],
                                    interleaved=s["interleaved"], k_gain=s["k_gain"],
                                    v_gain=s["v_gain"], q_out=s["q_out"], k_out=s["k_out"],
                                    v_out=s["v_out"])
        return q, s["k_out"], s["v_out"]
    return S.sdpa_paged_forward_fp4(s["q"], s["k_pages"], s["v_pages"], s["k_scales"],
                                    s["v_scales"], s["table"], s["lens"], cu_seqlens_q=s["cu"],
                                    scale=s["scale"], sinks=s["sinks"], k_gain=s["k_gain"],
                                    v_gain=s["v_gain"], out=s["out"], lse=s["lse"])


def run(s):
    if own:
        return _own(s)
    return PLAIN[s["op"]](s)


# ------------------------------------------------------------------- exact
def _turned(x, cos, sin, interleaved):
    """x [rows, heads, dim] in 64 bits as complex numbers times cos + i sin [rows, R / 2]."""
    h = cos.shape[-1]
    turn = torch.complex(cos.double(), sin.double())[:, None]
    y = x.double().clone()
    even = torch.arange(h, device=x.device) * (2 if interleaved else 1)
    odd = even + (1 if interleaved else h)
    z = torch.complex(y[..., even], y[..., odd]) * turn
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _nearest(x, gain):
    """What rows x [rows, kv heads, dim] of their own type stand for in 4 bits, in 64 bits."""
    g = torch.ones(x.shape[1], device=x.device) if gain is None else gain
    y = (x.float() / g[:, None]).double().unflatten(-1, (-1, 16))
    scales = torch.arange(1, 127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn)
    scales = scales.double()  # ascending; the parity of a place is that of its code
    s = _round_to(y.abs().amax(-1) / 6.0, scales, 1)[..., None]
    grid = torch.tensor(CODES[:8], dtype=torch.float64, device=x.device)
    m = _round_to(y.abs() / s, grid, 0)
    return (torch.sign(y) * m * s).flatten(-2) * g.double()[:, None]


def _round_to(a, grid, odd):
    """The nearest of the ascending values `grid`; ties to the one of even code (place + odd)."""
    i = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
    lo, hi = grid[i - 1], grid[i]
    even = ((i - 1 + odd) % 2) == 0
    down = (a - lo < hi - a) | ((a - lo == hi - a) & even)
    return torch.where(down, lo, hi)


def exact(c, seed):
    """The definitions in 64 bits, sequence by sequence and kv head by kv head."""
    if c["op"] == "attend4" and 4 * c["dim"] * c["hq"] * _pairs(c) > 8e12:
        return None  # too long in 64 bits
    s = prepare(c, seed)
    if c["op"] == "rope":
        res = []
        for x in (s["q"], s["k"]):
            rows = x.transpose(1, 2).flatten(0, 1)
            cs = s["rope"][s["positions"].flatten().long()]
            y = _turned(rows, cs[..., 0], -cs[..., 1] if c["backward"] else cs[..., 1],
                        c["interleaved"])
            res.append(y.unflatten(0, (c["batch"], -1)).transpose(1, 2))
        return tuple(res)
    qs, ks = _lengths(c)
    n, ps = sum(qs), c["page"]
    if c["op"] in ("append", "append4"):
        pos = torch.cat([torch.arange(k - q, k) for q, k in zip(qs, ks)]).cuda()
        seq = torch.cat([torch.full((q,), b) for b, q in enumerate(qs)]).cuda()
        cs = s["rope"][pos + c["shift"]]
        q, k = s["q_out"].double(), _turned(s["k"][:n], cs[..., 0], cs[..., 1], c["interleaved"])
        q[:n] = _turned(s["q"][:n], cs[..., 0], cs[..., 1], c["interleaved"])
        if c["op"] == "append":
            kp, vp = s["k_pages"].double(), s["v_pages"].double()
            page = s["table"][seq, pos // ps].long()
            kp[page, :, pos % ps] = k
            vp[page, :, pos % ps] = s["v"][:n].double()
            return q, kp, vp
        ko, vo = s["k_out"].double(), s["v_out"].double()
        ko[:n] = _nearest(k.to(s["k"].dtype), s["k_gain"])
        vo[:n] = _nearest(s["v"][:n], s["v_gain"])
        return q, ko, vo
    G = c["hq"] // c["hkv"]
    o, lse = s["out"].double(), s["lse"].double()

    def rows_of(x, page, h, row):
        p = s[x + "_pages"][page, h, row].long()
        code = torch.stack([p % 16, p // 16], -1).flatten(-2)
        e, m = (code // 2) % 4, (code % 2).double()
        mag = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m) * 2.0 ** (e - 1).double())
        scale = s[x + "_scales"][page, h, row].view(torch.float8_e4m3fn).double()
        y = torch.where(code >= 8, -mag, mag) * scale.repeat_interleave(16, -1)
        return y if s[x + "_gain"] is None else y * s[x + "_gain"][h].double()

    t0 = 0
    for b, (nq, nk) in enumerate(zip(qs, ks)):
        rows = torch.arange(nk, device="cuda")
        page = s["table"][b].long()[rows // ps]
        hidden = rows[None, :] > (nk - nq + torch.arange(nq, device="cuda"))[:, None]
        for h in range(c["hkv"]):
            k, v = rows_of("k", page, h, rows % ps), rows_of("v", page, h, rows % ps)
            for hh in range(h * G, h * G + G):
                x = s["q"][t0:t0 + nq, hh].double() @ k.T * s["scale"]
                x = x.masked_fill(hidden, -math.inf)
                if s["sinks"] is not None:
                    x = torch.cat([x, s["sinks"][hh].double().expand(nq, 1)], 1)
                z = torch.logsumexp(x, 1)
                o[t0:t0 + nq, hh] = (x[:, :nk] - z[:, None]).exp() @ v
                lse[t0:t0 + nq, hh] = z
        t0 += nq
    return o, lse
