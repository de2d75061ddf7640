"""The 4-bit key/value cache for streaming inference: what is measured of it.

Five operators, which one streaming loop uses together: `append` (quantise finished keys and values into
the cache) with `read` (the values the cache holds), `fwd` (attention of new queries over the cache, joined
with the attention over the chunk's own keys), `weights` (the attention weight each cached key received) and
`evict` (keep the recent keys and the ones with most weight).

Format of the cache, per (batch element, key/value head), `capacity` token slots:
  a value is x = c * s: c a 4-bit float (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6),
  s the scale of its 16 neighbouring features, 8 bits (5 exponent and 3 mantissa bits, no sign, steps of
  2^-17 below 2^-14, at most 10240): s = round(max|x| / 6), c = round(x / s), both to nearest, ties to even.
  k_codes  [B, H, capacity, D/2]      byte i: feature 2i in the low half, 2i + 1 in the high half
  k_scales [B, H, capacity, D/16]
  v_codes  [B, H, capacity/2, D]      byte d of row p: token 2p in the low half, 2p + 1 in the high half
  v_scales [B, H, capacity/2, D/16, 2]  last axis: token 2p, 2p + 1
Keys are stored rotated and divided by their RMS (gamma_k joins the query); values as they are.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
TOP = 10240.0                  # the largest scale; 6 * TOP is the largest magnitude
TOP_BYTE = 226                 # its 8 bits


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token for each of 8 conversations of different lengths: latency
        dict(name="append_token", op="append", batch=8, n=1, heads_kv=8, dim=128, capacity=4096, rope=True, ragged=True),
        # a denoised chunk of the streaming workload (6 x 24 x 40 latent patches) joins the history
        dict(name="append_chunk", op="append", batch=1, n=5760, heads_kv=8, dim=128, capacity=92160, rope=True, ragged=False),
        # three prompts of odd lengths, padded to the longest, head_dim 64
        dict(name="append_ragged", op="append", batch=3, n=1019, heads_kv=5, dim=64, capacity=2048, rope=False, ragged=True),
        # one new token over a short history: latency
        dict(name="fwd_token_4k", op="fwd", batch=1, sq=1, heads_q=16, heads_kv=4, dim=128, length=4096, capacity=4096, rope=True, base=False, ragged=False),
        # one new token for each of 4 streams over a history of up to 16 chunks: bandwidth
        dict(name="fwd_token_92k", op="fwd", batch=4, sq=1, heads_q=24, heads_kv=8, dim=128, length=92160, capacity=92160, rope=True, base=False, ragged=True),
        # a few tokens at once, odd sizes, head_dim 64, joined with their own block
        dict(name="fwd_five_tokens", op="fwd", batch=2, sq=5, heads_q=6, heads_kv=2, dim=64, length=10007, capacity=10112, rope=False, base=True, ragged=True),
        # a chunk of the small training layout over a long history, query groups of 4
        dict(name="fwd_chunk_1k", op="fwd", batch=1, sq=1024, heads_q=16, heads_kv=4, dim=128, length=8192, capacity=8192, rope=True, base=True, ragged=False),
        # one active chunk over four clean chunks of the streaming workload, joined with its own attention
        dict(name="fwd_chunk_5k", op="fwd", batch=1, sq=5760, heads_q=24, heads_kv=8, dim=128, length=23040, capacity=23040, rope=True, base=True, ragged=False),
        # the weights of one decoding step
        dict(name="weights_token_92k", op="weights", batch=4, sq=1, heads_q=24, heads_kv=8, dim=128, length=92160, capacity=92160, rope=True, ragged=True),
        # the weights a whole chunk gives to the history
        dict(name="weights_chunk_5k", op="weights", batch=1, sq=5760, heads_q=24, heads_kv=8, dim=128, length=23040, capacity=23040, rope=True, ragged=False),
        # an odd short history cut to half
        dict(name="evict_4k", op="evict", batch=2, heads_kv=4, dim=64, length=4097, capacity=4224, keep=2049, recent=65, ragged=True),
        # 16 chunks cut to 8, the last chunk kept whole
        dict(name="evict_92k", op="evict", batch=2, heads_kv=8, dim=128, length=92160, capacity=92160, keep=46080, recent=5760, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "fwd", "fwd", "weights", "evict"])
    dim = rng.choice([64, 128])
    heads_q, heads_kv = rng.choice([(24, 8), (16, 4), (16, 2), (6, 2), (8, 8), (5, 5), (2, 1)])
    batch = rng.randint(1, 4)
    rope, ragged = rng.random() < 0.5, rng.random() < 0.5
    if op == "append":
        n = _log(rng, 1, 5760)
        capacity = -(-rng.randint(n, 4 * n + 256) // 128) * 128
        return dict(op=op, batch=batch, n=n, heads_kv=heads_kv, dim=dim, capacity=capacity, rope=rope, ragged=ragged)
    if op == "evict":
        length = _log(rng, 2, 92160)
        keep = rng.randint(1, length)
        return dict(op=op, batch=rng.randint(1, 2), heads_kv=heads_kv, dim=dim, length=length, capacity=-(-length // 128) * 128,
                    keep=keep, recent=rng.randint(0, keep), ragged=ragged)
    sq = _log(rng, 1, 5760)
    most = min(92160, int(5760 * 24 * 23040 / (batch * heads_q * sq)))
    length = _log(rng, 1, most)
    capacity = -(-rng.randint(length, length + 300) // 128) * 128
    case = dict(op=op, batch=batch, sq=sq, heads_q=heads_q, heads_kv=heads_kv, dim=dim, length=length, capacity=capacity, rope=rope, ragged=ragged)
    if op == "fwd":
        case["base"] = rng.random() < 0.5
    return case


def work(case):
    B, H, D = case["batch"], case["heads_kv"], case["dim"]
    row = D // 2 + D // 16                       # bytes of one cached key or value
    if case["op"] == "append":
        n = sum(_counts(case))
        rope = case["n"] * D // 2 * 4 if case["rope"] else 0
        # k and v in, the cache's rows out, and the values the rows hold out
        return dict(bytes=n * H * (4 * D + 2 * row) + B * case["n"] * H * 4 * D + rope, flops=n * H * 20 * D)
    lengths = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(l, case["keep"]) for l in lengths)
        return dict(bytes=sum(lengths) * H * 4 + kept * H * 2 * (2 * row) + kept * H * 8, flops=sum(lengths) * H)
    Hq, sq = case["heads_q"], case["sq"]
    rope = sq * D // 2 * 4 if case["rope"] else 0
    q = B * sq * Hq * D * 2
    if case["op"] == "fwd":
        base = q + B * Hq * sq * 4 if case["base"] else 0
        return dict(bytes=sum(lengths) * H * 2 * row + 2 * q + B * Hq * sq * 4 + base + rope, flops=4 * D * Hq * sq * sum(lengths))
    return dict(bytes=sum(lengths) * H * (row + 8) + q + B * Hq * sq * 4 + rope, flops=2 * D * Hq * sq * sum(lengths))


def _lengths(case):
    """Tokens in the cache of each batch element: the full length first, the others shorter if ragged."""
    L, B = case["length"], case["batch"]
    return [max(1, L - (b * L) // (3 * B) - (b > 0)) if case["ragged"] else L for b in range(B)]


def _counts(case):
    n, B = case["n"], case["batch"]
    return [max(1, n - (b * n) // (2 * B)) if case["ragged"] else n for b in range(B)]


# ----------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kw = dict(generator=g, device=DEV, dtype=torch.float32)
    B, H, D, cap = case["batch"], case["heads_kv"], case["dim"], case["capacity"]
    s = dict(op=case["op"])
    if case["op"] == "append":
        n = case["n"]
        # channels of unequal size and tokens of unequal size, as projections of a trained model have them
        size = torch.exp(0.5 * torch.randn(1, 1, H, D, **kw)) * torch.exp(0.3 * torch.randn(B, n, 1, 1, **kw))
        s["k"] = (torch.randn(B, n, H, D, **kw) * size).to(torch.bfloat16)
        s["v"] = (torch.randn(B, n, H, D, **kw) * size).to(torch.bfloat16)
        r = random.Random(seed)
        room = cap - n
        start = [r.randint(0, room) for _ in range(B)] if case["ragged"] else [room] * B
        s["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
        s["rope"] = _angles(max(start), n, D, g) if case["rope"] else None
        s["n"] = n
        s["cache"] = _empty(B, H, cap, D)
        return s
    lengths = _lengths(case)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    s["most"] = max(lengths)
    s["cache"] = _filled(B, H, cap, D, kw)
    if case["op"] == "evict":
        # a few keys draw most of the weight; many equal small ones (ties) among the rest
        w = torch.exp(2.0 * torch.randn(B, H, cap, **kw))
        s["w"] = torch.where(w < 0.5, torch.round(w * 16) / 16, w).contiguous()
        s["keep"], s["recent"] = case["keep"], case["recent"]
        room = -(-case["keep"] // 128) * 128
        s["to"] = _empty(B, H, room, D)
        s["to_w"] = torch.zeros(B, H, room, device=DEV)
        return s
    sq, Hq = case["sq"], case["heads_q"]
    s["q"] = torch.randn(B, sq, Hq, D, **kw).to(torch.bfloat16)
    s["gq"] = 1.0 + 0.1 * torch.randn(D, **kw)
    s["gk"] = 1.0 + 0.1 * torch.randn(D, **kw)
    s["rope"] = _angles(max(lengths), sq, D, g) if case["rope"] else None
    s["base"] = None
    if case["op"] == "fwd":
        if case["base"]:   # the active chunk's own attention, as the forward over its bf16 keys gives it
            out = (torch.randn(B, sq, Hq, D, **kw) * 0.3).to(torch.bfloat16)
            s["base"] = (out, math.log(max(2, sq)) + 0.5 * torch.randn(B, Hq, sq, **kw))
    else:
        s["lse"] = _attend(s, False)[1]
        s["w"] = torch.rand(B, H, cap, **kw) * (2 * sq * Hq / H / max(lengths))   # what a pass or two before left
    return s


def _angles(first, n, D, g):
    """Angles [n, D/2] of the positions from `first` on."""
    t = torch.arange(first, first + n, device=DEV, dtype=torch.float64)
    freq = 10000.0 ** (-torch.arange(D // 2, device=DEV, dtype=torch.float64) / (D // 2))
    jitter = 1.0 + 0.05 * torch.rand(D // 2, generator=g, device=DEV).double()   # learnt frequencies
    return (t[:, None] * freq * jitter).float()


def _empty(B, H, cap, D):
    z = dict(device=DEV, dtype=torch.uint8)
    return (torch.zeros(B, H, cap, D // 2, **z), torch.zeros(B, H, cap, D // 16, **z),
            torch.zeros(B, H, cap // 2, D, **z), torch.zeros(B, H, cap // 2, D // 16, 2, **z))


def _filled(B, H, cap, D, kw):
    """A cache as appends leave it: keys of unit RMS, values of unit size with some larger channels."""
    k = torch.randn(B, H, cap, D, **kw)
    k *= torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS)
    kc, ks = _quantise(k)
    del k
    vc, vs = _quantise(torch.randn(B, H, cap, D, **kw) * torch.exp(0.3 * torch.randn(1, H, 1, D, **kw)))
    return kc[..., 0::2] | kc[..., 1::2] << 4, ks, vc[:, :, 0::2] | vc[:, :, 1::2] << 4, torch.stack((vs[:, :, 0::2], vs[:, :, 1::2]), -1)


# ------------------------------------------------------------------------------------------ plain forms
def _quantise(x):
    """Codes [..., D] (one per byte) and scale bytes [..., D/16] of x [..., D], in x's own precision."""
    x = torch.nan_to_num(x, nan=0.0, posinf=6 * TOP, neginf=-6 * TOP).clamp(-6 * TOP, 6 * TOP)
    xb = x.unflatten(-1, (-1, 16))
    want = xb.abs().amax(-1) / 6
    e = torch.frexp(want)[1].clamp(min=-13)                                   # 2^(e-1) <= want < 2^e
    step = torch.ldexp(torch.ones_like(want), e - 4)                          # of 3 mantissa bits
    scale = (torch.round(want / step) * step).clamp(max=TOP)
    byte = (scale.half().view(torch.int16) >> 7).to(torch.uint8)              # the same exponent bits as fp16's
    y = (xb / torch.where(scale > 0, scale, 1.0).unsqueeze(-1)).clamp(-6, 6) * (scale > 0).unsqueeze(-1)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    return (code | torch.signbit(y).to(torch.uint8) << 3).flatten(-2), byte


def _values(codes, scales):
    """fp32 values of codes [..., D] (one per byte) with scale bytes [..., D/16]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    scale = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (table[codes.int()].unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)).flatten(-2)


def _k_values(cache, n):
    c = cache[0][:, :, :n]
    return _values(torch.stack((c & 15, c >> 4), -1).flatten(-2), cache[1][:, :, :n])


def _v_values(cache, n):
    c, s = cache[2], cache[3]
    m = (n + 1) // 2
    c, s = c[:, :, :m], s[:, :, :m]
    return torch.stack((_values(c & 15, s[..., 0]), _values(c >> 4, s[..., 1])), 3).flatten(2, 3)[:, :, :n]


def _rotate(x, angles):
    """x [B, n, H, D] by angles [n, D/2]: feature i with feature i + D/2."""
    if angles is None:
        return x
    c, s = torch.cos(angles.to(x.dtype))[:, None], torch.sin(angles.to(x.dtype))[:, None]
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _append(s):
    kc, ks, vc, vs = s["cache"]
    B, n, H, D = s["k"].shape
    k = s["k"].double()                                    # 64 bits: the choice of a code is a border
    k = _rotate(k, s["rope"]) * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS)
    kq, kqs = _quantise(k)
    vq, vqs = _quantise(s["v"].double())
    counts = s["counts"] if s["counts"] is not None else torch.full((B,), n, device=DEV)
    start = s["start"].long()
    bi, hi = torch.arange(B, device=DEV)[:, None, None], torch.arange(H, device=DEV)[None, None, :]
    t = torch.arange(n, device=DEV)
    at = (start[:, None] + t)[:, :, None]
    fine = (t[None] < counts[:, None])[:, :, None, None]
    kc[bi, hi, at] = torch.where(fine, kq[..., 0::2] | kq[..., 1::2] << 4, kc[bi, hi, at])
    ks[bi, hi, at] = torch.where(fine, kqs, ks[bi, hi, at])
    # values: rows of two tokens
    pair = (start // 2)[:, None] + torch.arange(n // 2 + 1, device=DEV)
    lo, hi2 = 2 * pair - start[:, None], 2 * pair + 1 - start[:, None]
    at = (pair % vc.shape[2])[:, :, None]
    b2 = torch.arange(B, device=DEV)[:, None]

    def side(t, new, old):
        ok = ((t >= 0) & (t < counts[:, None]))[:, :, None, None]
        return torch.where(ok, new[b2, t.clamp(0, n - 1)], old)

    old, olds = vc[bi, hi, at], vs[bi, hi, at]
    vc[bi, hi, at] = side(lo, vq, old & 15) | side(hi2, vq, old >> 4) << 4
    vs[bi, hi, at] = torch.stack((side(lo, vqs, olds[..., 0]), side(hi2, vqs, olds[..., 1])), -1)


def _read(s):
    kc, ks, vc, vs = s["cache"]
    B, H, n = kc.shape[0], kc.shape[1], s["n"]
    bi, hi = torch.arange(B, device=DEV)[:, None, None], torch.arange(H, device=DEV)[None, None, :]
    at = (s["start"].long()[:, None] + torch.arange(n, device=DEV))[:, :, None]
    c = kc[bi, hi, at]
    k = _values(torch.stack((c & 15, c >> 4), -1).flatten(-2), ks[bi, hi, at])
    odd = (at % 2).unsqueeze(-1).bool()
    c, sc = vc[bi, hi, at // 2], vs[bi, hi, at // 2]
    v = _values(torch.where(odd, c >> 4, c & 15), torch.where(odd, sc[..., 1], sc[..., 0]))
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _scores(s):
    """fp32 scores [B, H, G * Sq, most]; keys behind the length are -inf."""
    q = s["q"].float()
    B, sq, Hq, D = q.shape
    H = s["cache"][0].shape[1]
    q = _rotate(q, s["rope"]) * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * (s["gq"] * s["gk"] / math.sqrt(D))
    q = q.unflatten(2, (H, Hq // H)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = q @ _k_values(s["cache"], s["most"]).transpose(-1, -2)
    behind = torch.arange(s["most"], device=DEV)[None] >= s["lengths"][:, None]
    return x.masked_fill_(behind[:, None, None], -math.inf)


def _attend(s, values=True):
    B, sq, Hq, D = s["q"].shape
    H = s["cache"][0].shape[1]
    x = _scores(s)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + torch.log(l)).view(B, H, Hq // H, sq).flatten(1, 2)
    if not values:
        return None, lse
    o = (p @ _v_values(s["cache"], s["most"])) / torch.where(l > 0, l, 1.0)
    o = o.view(B, H, Hq // H, sq, D).permute(0, 3, 1, 2, 4).flatten(2, 3)
    if s["base"] is not None:
        base, base_lse = s["base"]
        top = torch.maximum(lse, base_lse)
        top = torch.where(top == -math.inf, 0.0, top)
        a, b = torch.exp(lse - top), torch.exp(base_lse - top)
        both = a + b
        part = lambda w: (w / torch.where(both > 0, both, 1.0)).transpose(1, 2).unsqueeze(-1)  # noqa: E731
        o = o * part(a) + base.float() * part(b)
        lse = top + torch.log(both)
    return o.to(torch.bfloat16), lse


def _weigh(s):
    B, sq, Hq, _ = s["q"].shape
    H, n = s["cache"][0].shape[1], s["most"]
    p = _scores(s).sub_(s["lse"].view(B, H, -1, 1)).exp_().sum(2)
    inside = (torch.arange(n, device=DEV)[None] < s["lengths"][:, None])[:, None]
    w = s["w"]
    w[:, :, :n] = torch.where(inside, w[:, :, :n] + p, w[:, :, :n])
    return w


def _evict(s):
    kc, ks, vc, vs = s["cache"]
    tk, tks, tv, tvs = s["to"]
    n, keep, recent = s["most"], s["keep"], s["recent"]
    lengths = s["lengths"][:, None, None]
    w = s["w"][:, :, :n]
    t = torch.arange(n, device=DEV)[None, None]
    order = torch.where(torch.isnan(w), -math.inf, w).sort(dim=-1, descending=True, stable=True)[1]
    rank = torch.where(t >= lengths, 2, torch.where(t >= lengths - recent, 0, 1)).expand(w.shape)
    order = order.gather(-1, rank.gather(-1, order).sort(dim=-1, stable=True)[1])
    left = torch.clamp(s["lengths"], max=keep)
    m = min(keep, n)
    at = torch.where(torch.arange(m, device=DEV) < left[:, None, None], order[..., :m], n).sort(-1)[0]
    fine = at < n
    src = at.clamp(max=n - 1)
    row = lambda x, i: x.gather(2, i.unsqueeze(-1).expand(-1, -1, -1, x.shape[-1]))  # noqa: E731
    put = lambda x, new: x.copy_(torch.where(fine.unsqueeze(-1), new, x))  # noqa: E731
    put(tk[:, :, :m], row(kc, src))
    put(tks[:, :, :m], row(ks, src))
    s["to_w"][:, :, :m] = torch.where(fine, w.gather(-1, src), s["to_w"][:, :, :m])
    # values: unpack the two tokens of a row, choose, pack
    odd = (src % 2).unsqueeze(-1).bool()
    c, sc = row(vc, src // 2), row(vs.flatten(3), src // 2).unflatten(-1, (-1, 2))
    new, news = torch.where(odd, c >> 4, c & 15), torch.where(odd, sc[..., 1], sc[..., 0])
    old = torch.stack((tv & 15, tv >> 4), 3).flatten(2, 3)
    olds = tvs.transpose(3, 4).flatten(2, 3).contiguous()
    put(old[:, :, :m], new)
    put(olds[:, :, :m], news)
    tv.copy_(old[:, :, 0::2] | old[:, :, 1::2] << 4)
    tvs.copy_(torch.stack((olds[:, :, 0::2], olds[:, :, 1::2]), -1))
    index = torch.full((*at.shape[:2], keep), -1, device=DEV, dtype=torch.int32)
    index[..., :m] = torch.where(fine, at, -1).int()
    return left.int(), index


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "append":
        _append(s)
        return _read(s)
    if s["op"] == "fwd":
        return _attend(s)
    if s["op"] == "weights":
        return _weigh(s)
    left, index = _evict(s)
    # rows move and are not computed: their bytes have to be equal
    return (*s["to"], s["to_w"], left, index)


def _run_own(s):
    import block_causal_attention_gqa_b200 as bca
    if s["op"] == "append":
        bca.magi_bca_kv4_append(s["cache"], s["k"], s["v"], s["start"], counts=s["counts"], rope_k=s["rope"], rms_eps=EPS)
        return bca.magi_bca_kv4_read(s["cache"], s["start"], s["n"])
    if s["op"] == "fwd":
        base, base_lse = s["base"] if s["base"] is not None else (None, None)
        return bca.magi_bca_kv4_fwd(s["q"], s["cache"], s["lengths"], s["gq"], s["gk"], rope_q=s["rope"], base_out=base,
                                    base_lse=base_lse, rms_eps=EPS)
    if s["op"] == "weights":
        return bca.magi_bca_kv4_weights(s["q"], s["cache"], s["lengths"], s["lse"], s["gq"], s["gk"], s["w"], rope_q=s["rope"],
                                        rms_eps=EPS)
    left, index = bca.magi_bca_kv4_evict(s["cache"], s["w"], s["lengths"], s["keep"], s["recent"], s["to"], s["to_w"])
    return (*s["to"], s["to_w"], left, index)


# ------------------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        return _exact_append(s)
    if s["op"] == "evict":
        return _exact_evict(s)
    k, v = _exact_cache(s["cache"])
    B, sq, Hq, D = s["q"].shape
    H = k.shape[1]
    G = Hq // H
    out = torch.zeros(B, sq, Hq, D, device=DEV, dtype=torch.float64)
    lse = torch.full((B, Hq, sq), -math.inf, device=DEV, dtype=torch.float64)
    w = s["w"].double() if s["op"] == "weights" else None
    for b in range(B):
        n = int(s["lengths"][b])
        for h in range(Hq):
            q = s["q"][b, :, h].double()
            norm = torch.sqrt(q.pow(2).sum(-1, keepdim=True) / D + EPS)
            if s["rope"] is not None:
                z = torch.complex(q[:, : D // 2], q[:, D // 2:]) * torch.polar(torch.ones((), device=DEV, dtype=torch.float64), s["rope"].double())
                q = torch.cat((z.real, z.imag), -1)
            q = q / norm * s["gq"].double() * s["gk"].double()
            x = torch.einsum("id,jd->ij", q, k[b, h // G, :n].double()) / math.sqrt(D)
            if w is not None:
                w[b, h // G, :n] += torch.exp(x - s["lse"][b, h].double()[:, None]).sum(0)
                continue
            if s["base"] is not None:   # one more key: the base's value, with its log of the sum as score
                x = torch.cat((x, s["base"][1][b, h].double()[:, None]), 1)
            lse[b, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b, h][:, None])
            out[b, :, h] = p[:, :n] @ v[b, h // G, :n].double()
            if s["base"] is not None:
                out[b, :, h] += p[:, n:] * s["base"][0][b, :, h].double()
    return w if w is not None else (out, lse)


def _grid():
    """The scale of each byte, and the eight magnitudes of a code."""
    scales = [(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 18) for e in range(32) for m in range(8)][: TOP_BYTE + 1]
    return torch.tensor(scales, dtype=torch.float64, device=DEV), torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)


def _nearest(x, grid):
    """The grid's value nearest to x >= 0; of two as near, the one of even place."""
    i = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    below, above = x - grid[i - 1], grid[i] - x
    up = (above < below) | ((above == below) & (i % 2 == 0))
    return grid[torch.where(up, i, i - 1)]


def _exact_rows(x):
    scales, mags = _grid()
    out = torch.empty_like(x)
    for j in range(0, x.shape[-1], 16):
        b = x[..., j:j + 16]
        s = _nearest(b.abs().amax(-1, keepdim=True) / 6, scales)
        out[..., j:j + 16] = torch.where(s > 0, torch.sign(b) * _nearest(b.abs() / torch.where(s > 0, s, 1.0), mags) * s, 0.0)
    return out


def _exact_append(s):
    B, n, H, D = s["k"].shape
    x = s["k"].double()
    norm = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
    if s["rope"] is not None:
        z = torch.complex(x[..., : D // 2], x[..., D // 2:]) * torch.polar(torch.ones((), device=DEV, dtype=torch.float64), s["rope"].double())[:, None]
        x = torch.cat((z.real, z.imag), -1)
    k, v = _exact_rows(x / norm), _exact_rows(s["v"].double())
    if s["counts"] is not None:
        for b in range(B):
            k[b, int(s["counts"][b]):] = 0
            v[b, int(s["counts"][b]):] = 0
    return k, v


def _exact_cache(cache):
    scales, mags = _grid()
    kc, ks, vc, vs = cache
    signed = torch.cat((mags, -mags)).float()
    scales = scales.float()
    k = torch.empty(*kc.shape[:3], 2 * kc.shape[3], device=DEV)
    k[..., 0::2], k[..., 1::2] = signed[(kc % 16).int()], signed[(kc // 16).int()]
    v = torch.empty(*vc.shape[:2], 2 * vc.shape[2], vc.shape[3], device=DEV)
    v[:, :, 0::2], v[:, :, 1::2] = signed[(vc % 16).int()], signed[(vc // 16).int()]
    k *= scales[ks.int()].repeat_interleave(16, -1)
    for odd in (0, 1):
        v[:, :, odd::2] *= scales[vs[..., odd].int()].repeat_interleave(16, -1)
    return k, v


def _exact_evict(s):
    """Only the weights are computed numbers; which rows stay is compared as it is."""
    w, lengths = s["w"].cpu().numpy().astype(np.float64), s["lengths"].tolist()
    out = np.zeros(tuple(s["to_w"].shape))
    for b, n in enumerate(lengths):
        for h in range(w.shape[1]):
            first = max(0, n - s["recent"])
            old = np.lexsort((np.arange(first), -w[b, h, :first]))[: max(0, min(s["keep"], n) - (n - first))]
            at = np.concatenate((np.sort(old), np.arange(first, n)[-s["keep"]:]))
            out[b, h, : len(at)] = w[b, h, at]
    return None, None, None, None, out, None, None
