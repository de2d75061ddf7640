"""The 4-bit key/value cache on the GPU, against the fp64 reference.

Tolerances.
  append, read: the cached values are the definition's exactly (a code is a
    decision, and rows near a border are decided in fp64).
  scores: sum_d |Q^_d K^_d| <= |Q^| |K^|, in log2 units at most
    S = sqrt(D) gq gk 1.4427 |K^| / sqrt(D) with |K^| <= 1.25 sqrt(D) after
    quantisation (a code is off by at most a sixth of its block's maximum, far
    less on average) and gains below 1.4 in product: S <= 30 at D = 128.
  few rows (and weights): queries are two fp16 numbers, 2^-22 relative, and up
    to 32 fp32 accumulations of 2^-23 each: |ds| <= 30 (2^-22 + 32 2^-23) <
    1.3e-4 log2 units, 9e-5 natural.  lse: that plus its own rounding, 1e-4.
    Weights: each term relative 9e-5 + 2^-22 (exponential): 1e-4 relative.
    out: twice that times max|v| for the shift of the weights, plus half a
    bf16 step, 2^-8 relative.
  many rows: queries are one fp16 number, 2^-11 relative: |ds| <= 30 2^-11 =
    1.5e-2 log2 units at the very worst, where every product has one sign and
    every rounding goes the same way.  lse 1.1e-2.  The roundings are
    independent, so relative L2 is held to 4e-3: bf16's own (uniform within
    half a step, at most 2^-8 / sqrt 3 = 2.3e-3), P's 2^-11 and the
    exponential's 7.5e-5 included.
"""
import math

import pytest
import torch

import block_causal_attention_gqa_b200 as bca
from tests import kv4_reference as ref
from tests._helpers import assert_close, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def angles(g, *shape, far=3000.0):
    return far * torch.rand(*shape, generator=g, device=DEV) - far / 4


def filled(g, B, H, D, cap, lengths, behind=True):
    """A cache holding random keys of unit RMS and values; slots behind a length
    hold bytes that decode to NaN and infinities if `behind`."""
    k = ref.keys(randn(g, B, cap, H, D)).transpose(1, 2)
    v = randn(g, B, H, cap, D).double() * torch.exp(0.5 * randn(g, 1, H, 1, D)).double()
    _, kc, kb = ref.quantise(k)
    _, vc, vb = ref.quantise(v)
    if behind:
        for b, n in enumerate(lengths):
            kc[b, :, n:] = 15
            vc[b, :, n:] = 15
            kb[b, :, n:] = 255
            vb[b, :, n:] = 255
    return bca.Kv4Cache(*ref.pack(kc, kb, vc, vb))


def gains(g, D):
    return 1 + 0.1 * randn(g, D), 1 + 0.1 * randn(g, D)


def check_attention(got, want, few, vmax):
    (out, lse), (o, l) = got, want
    assert torch.equal(torch.isinf(lse), torch.isinf(l))
    fin = torch.isfinite(l)
    d = (lse.double() - l)[fin].abs()
    assert d.numel() == 0 or d.max() <= (1e-4 if few else 1.1e-2), d.max()
    err = (out.double() - o).abs()
    if few:
        assert (err <= 2.0 ** -8 * o.abs() + 2e-4 * vmax).all(), (err - 2.0 ** -8 * o.abs()).max()
    else:
        assert_close("out", to_np(out), o.cpu().numpy(), rel=4e-3)


# ---------------------------------------------------------------- append, read
@pytest.mark.parametrize("B,n,H,D,start,counts,rope", [
    (1, 1, 1, 64, [0], None, False), (1, 1, 3, 128, [127], None, True), (2, 2, 2, 64, [1, 254], None, True),
    (3, 5, 2, 128, [7, 0, 123], [5, 0, 2], True), (2, 131, 5, 64, [3, 100], [131, 77], False),
    (1, 300, 8, 128, [84], None, True), (4, 17, 1, 128, [0, 1, 2, 3], [17, 16, 1, 0], False)])
def test_append_stores_the_definitions_values(B, n, H, D, start, counts, rope):
    g = gen(n * 7 + B)
    cap = 384
    k = (randn(g, B, n, H, D) * torch.exp(randn(g, B, n, 1, 1))).bfloat16()
    v = (randn(g, B, n, H, D) * torch.exp(2 * randn(g, 1, 1, H, D))).bfloat16()
    ang = angles(g, B, n, D // 2) if rope and B > 1 else angles(g, n, D // 2) if rope else None
    cache = bca.Kv4Cache(*[torch.randint(0, 200, t.shape, generator=g, device=DEV, dtype=torch.uint8)
                           for t in bca.magi_bca_kv4_cache(B, H, D, cap)])
    before = [x.clone() for x in ref.unpack(cache)]
    bca.magi_bca_kv4_append(cache, k, v, ints(*start), None if counts is None else ints(*counts), rope_k=ang)
    want_k, want_v = ref.quantise(ref.keys(k, ang))[0], ref.quantise(v.double())[0]
    got_k, got_v = ref.unpack(cache)
    for b in range(B):
        m = n if counts is None else counts[b]
        before[0][b, :, start[b]:start[b] + m] = want_k[b, :m].transpose(0, 1)
        before[1][b, :, start[b]:start[b] + m] = want_v[b, :m].transpose(0, 1)
    assert torch.equal(got_k, before[0]) and torch.equal(got_v, before[1])   # and nothing else has changed
    rk, rv = bca.magi_bca_kv4_read(cache, ints(*start), n)
    for b in range(B):
        sl = slice(start[b], start[b] + n)
        assert torch.equal(rk[b].double(), got_k[b, :, sl].transpose(0, 1))
        assert torch.equal(rv[b].double(), got_v[b, :, sl].transpose(0, 1))
    assert bca.magi_bca_last_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_append_on_borders_and_odd_values(D):
    """Values on the borders between codes and scales, zeros, infinities, NaN, tiny and huge ones."""
    n = 64
    v = torch.zeros(1, n, 1, D, device=DEV)
    grid = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -2.5], device=DEV)
    for t in range(n):
        v[0, t, 0, :16] = grid * 2.0 ** (t - 40)
        v[0, t, 0, 16:32] = grid * (1 + t / 64) * (1 if t % 2 else -1)
        v[0, t, 0, 32:48] = 6.0 * (2 * t + 17) * 2.0 ** -20 * (torch.arange(16, device=DEV) == t % 16)   # scale midpoints
    v[0, 0, 0, 48], v[0, 1, 0, 49], v[0, 2, 0, 50], v[0, 3, 0, 51] = math.inf, -math.inf, math.nan, 3e38
    v = v.bfloat16()
    k = torch.randn(1, n, 1, D, device=DEV).bfloat16()
    k[0, 0], k[0, 1, 0, 3], k[0, 2, 0, 5] = 0, math.inf, math.nan
    cache = bca.magi_bca_kv4_cache(1, 1, D, 128)
    bca.magi_bca_kv4_append(cache, k, v, ints(0))
    gk, gv = ref.unpack(cache)
    assert torch.equal(gv[0, :, :n].transpose(0, 1), ref.quantise(v[0].double())[0])
    assert (gk[0, 0, :3] == 0).all()
    assert torch.equal(gk[0, 0, 3:n], ref.quantise(ref.keys(k[:, 3:]))[0][0, :, 0])


def test_append_decides_a_large_sample_exactly():
    """1.5 million keys' values with far angles: every code as in fp64."""
    g = gen(5)
    k = randn(g, 2, 1500, 4, 128).bfloat16()
    ang = angles(g, 1500, 64, far=2e5)
    cache = bca.magi_bca_kv4_cache(2, 4, 128, 1536)
    bca.magi_bca_kv4_append(cache, k, k, ints(11, 36), rope_k=ang)
    got, _ = bca.magi_bca_kv4_read(cache, ints(11, 36), 1500)
    assert torch.equal(got.double(), ref.quantise(ref.keys(k, ang))[0])


def test_append_outside_the_cache_is_skipped_and_reported():
    g = gen(1)
    k = randn(g, 3, 4, 2, 64).bfloat16()
    cache = bca.magi_bca_kv4_cache(3, 2, 64, 128)
    assert bca.magi_bca_last_device_status() == 0
    bca.magi_bca_kv4_append(cache, k, k, ints(126, -3, 1 << 30))
    want = ref.quantise(k.double())[0]
    _, v = ref.unpack(cache)
    assert torch.equal(v[0, :, 126:].transpose(0, 1), want[0, :2])
    assert torch.equal(v[1, :, :1].transpose(0, 1), want[1, 3:])
    assert (v[0, :, :126] == 0).all() and (v[1, :, 1:] == 0).all() and (v[2] == 0).all()
    assert bca.magi_bca_last_device_status() == -7
    assert bca.magi_bca_last_device_status() == 0
    rk, rv = bca.magi_bca_kv4_read(cache, ints(126, -3, 1 << 30), 4)
    assert torch.equal(rv[0, :2].double(), want[0, :2]) and (rv[0, 2:] == 0).all()
    assert (rv[1, :3] == 0).all() and (rv[2] == 0).all() and (rk[2] == 0).all()


# ----------------------------------------------------------------- attention
FEW = [(1, 1, 1, 1, 64, 128, [1]), (1, 1, 2, 1, 128, 128, [33]), (2, 1, 4, 2, 128, 512, [512, 0]),
       (3, 1, 8, 8, 64, 256, [255, 1, 129]), (1, 3, 6, 2, 128, 1408, [1301]), (2, 5, 6, 2, 64, 384, [31, 384]),
       (1, 8, 4, 1, 128, 640, [600]), (1, 1, 24, 8, 128, 9216, [9001]), (4, 2, 10, 5, 64, 128, [5, 64, 65, 128]),
       # histories long enough to be laid end to end over the CTAs (the others take a cluster each)
       (1, 1, 2, 1, 128, 20480, [20001]), (3, 2, 4, 1, 64, 17536, [17, 0, 17500]), (2, 1, 3, 1, 64, 65536, [65536, 40000]),
       (5, 1, 2, 2, 128, 16512, [1, 16512, 0, 9000, 333]), (1, 5, 6, 1, 128, 16640, [16639]),
       (1, 64, 1, 1, 128, 33024, [32900]), (1, 33, 1, 1, 64, 128, [1]), (1, 40, 2, 1, 128, 384, [257]),
       (1, 90, 4, 2, 64, 256, [255])]
MANY = [(1, 193, 1, 1, 64, 128, [1]), (1, 97, 2, 1, 128, 384, [257]), (2, 129, 4, 2, 128, 512, [512, 0]),
        (1, 100, 24, 8, 128, 1152, [1050]), (3, 200, 3, 3, 64, 256, [255, 128, 7]), (1, 513, 4, 2, 64, 2560, [2433]),
        (1, 300, 16, 4, 128, 4096, [4096])]


@pytest.mark.parametrize("base", [False, True])
@pytest.mark.parametrize("few,case", [(True, c) for c in FEW] + [(False, c) for c in MANY])
def test_attention(few, case, base):
    B, Sq, Hq, H, D, cap, lengths = case
    g = gen(sum(case[:6]))
    cache = filled(g, B, H, D, cap, lengths)
    q = randn(g, B, Sq, Hq, D).bfloat16()
    gq, gk = gains(g, D)
    ang = angles(g, B, Sq, D // 2) if base and B > 1 else angles(g, Sq, D // 2) if base else None
    bo = bl = None
    if base:
        bo, bl = randn(g, B, Sq, Hq, D).bfloat16(), 2 * randn(g, B, Hq, Sq) + math.log(cap) / 2
        bl[:, 0, 0] = -math.inf                      # a row without keys of its own
        bo[:, 0, 0] = math.nan                       # whose output must not be read
    got = bca.magi_bca_kv4_fwd(q, cache, ints(*lengths), gq, gk, rope_q=ang, base_out=bo, base_lse=bl)
    bo2 = torch.nan_to_num(bo) if base else None
    want = ref.attention(q, cache, torch.tensor(lengths), gq, gk, ang, bo2, bl)
    vmax = max(ref.unpack(cache)[1].nan_to_num(0, 0, 0).abs().max().item(), bo2.abs().max().item() if base else 0)
    check_attention(got, want, few, vmax)
    if not base and 0 in lengths:
        b = lengths.index(0)
        assert (got[0][b] == 0).all() and (got[1][b] == -math.inf).all()
    again = bca.magi_bca_kv4_fwd(q, cache, ints(*lengths), gq, gk, rope_q=ang, base_out=bo, base_lse=bl)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    only, none = bca.magi_bca_kv4_fwd(q, cache, ints(*lengths), gq, gk, rope_q=ang, base_out=bo, base_lse=bl, want_lse=False)
    assert none is None and torch.equal(only, got[0])
    assert bca.magi_bca_last_device_status() == 0


@pytest.mark.parametrize("Sq", [2, 64])
def test_attention_with_scores_that_grow_along_the_history(Sq):
    """Rising scores move the running reference many times; a scale of 4 makes
    the softmax peaked.  The bound on the scores grows with the scale."""
    g = gen(3)
    D, cap = 128, 1024
    lengths = [1000]
    q = randn(g, 1, Sq, 4, D).bfloat16()
    gq, gk = torch.ones(D, device=DEV), torch.ones(D, device=DEV)
    d = ref.keys(q)[0, 0, 0]
    mix = torch.linspace(-1, 1, cap, device=DEV).double()[:, None]
    k = mix * d + (1 - mix.abs()) * randn(g, cap, D).double()
    _, kc, kb = ref.quantise(k[None, None])
    _, vc, vb = ref.quantise(randn(g, 1, 1, cap, D).double())
    cache = bca.Kv4Cache(*ref.pack(kc, kb, vc, vb))
    kw = dict(softmax_scale=0.35)
    out, lse = bca.magi_bca_kv4_fwd(q, cache, ints(*lengths), gq, gk, **kw)
    o, l = ref.attention(q, cache, torch.tensor(lengths), gq, gk, scale=0.35)
    few = Sq == 2
    assert (lse.double() - l).abs().max() <= (4e-4 if few else 4.4e-2)
    assert (out.double() - o).norm() <= (3e-3 if few else 6e-3) * o.norm()


def test_a_query_that_is_nan_gives_nan_and_no_other_row_does():
    g = gen(9)
    for Sq in (3, 200):
        cache = filled(g, 1, 2, 128, 256, [200])
        q = randn(g, 1, Sq, 4, 128).bfloat16()
        q[0, 1, 2, 5] = math.nan
        gq, gk = gains(g, 128)
        out, lse = bca.magi_bca_kv4_fwd(q, cache, ints(200), gq, gk)
        bad = torch.isnan(lse)
        assert bad[0, 2, 1] and bad.sum() == 1
        assert torch.isnan(out[0, 1, 2]).all() and torch.isnan(out).sum() == 128


def test_lengths_beyond_the_cache_are_clamped():
    g = gen(2)
    cache = filled(g, 2, 1, 64, 128, [128, 128])
    q = randn(g, 2, 1, 2, 64).bfloat16()
    gq, gk = gains(g, 64)
    a = bca.magi_bca_kv4_fwd(q, cache, ints(1 << 30, -5), gq, gk)
    b = bca.magi_bca_kv4_fwd(q, cache, ints(128, 0), gq, gk)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------- weights
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.5])
@pytest.mark.parametrize("case", FEW + MANY)
def test_weights(case, decay):
    B, Sq, Hq, H, D, cap, lengths = case
    g = gen(sum(case[:6]) + 1)
    cache = filled(g, B, H, D, cap, lengths)
    q = randn(g, B, Sq, Hq, D).bfloat16()
    gq, gk = gains(g, D)
    ang = angles(g, Sq, D // 2)
    _, lse = ref.attention(q, cache, torch.tensor(lengths), gq, gk, ang)
    lse = torch.where(torch.isinf(lse), 0.0, lse).float() + 0.3 * torch.rand(B, Hq, Sq, generator=g, device=DEV)
    lse[:, -1, -1] = -math.inf
    old = torch.rand(B, H, cap, generator=g, device=DEV) / cap
    if decay == 0:
        old[:] = math.nan
    w = old.clone()
    r = bca.magi_bca_kv4_weights(q, cache, ints(*lengths), lse, gq, gk, w, rope_q=ang, decay=decay)
    assert r is w
    want = ref.weights(q, cache, torch.tensor(lengths), lse, gq, gk, old, ang, decay)
    for b, n in enumerate(lengths):
        assert torch.equal(w[b, :, n:].nan_to_num(-1), old[b, :, n:].nan_to_num(-1))
        err = (w[b, :, :n].double() - want[b, :, :n]).abs()
        assert (err <= 1e-4 * want[b, :, :n] + 1e-30).all(), (err / want[b, :, :n]).max()
    w2 = old.clone()
    bca.magi_bca_kv4_weights(q, cache, ints(*lengths), lse, gq, gk, w2, rope_q=ang, decay=decay)
    assert torch.equal(w.nan_to_num(-1), w2.nan_to_num(-1))
    assert bca.magi_bca_last_device_status() == 0


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("B,H,D,cap,lengths,keep,recent,dst_cap", [
    (1, 1, 64, 128, [1], 1, 0, 128), (1, 2, 128, 128, [128], 1, 1, 128), (2, 2, 64, 256, [200, 3], 100, 7, 128),
    (3, 1, 128, 384, [0, 384, 77], 77, 0, 128), (1, 3, 64, 1280, [1279], 1278, 1278, 1280),
    (2, 4, 128, 5120, [5001, 4000], 2049, 65, 2176), (1, 2, 64, 512, [512], 512, 3, 512),
    (1, 1, 128, 40960, [40001], 20003, 128, 20096)])
@pytest.mark.parametrize("kind", ["distinct", "ties", "odd"])
def test_evict(B, H, D, cap, lengths, keep, recent, dst_cap, kind):
    g = gen(keep + cap)
    cache = filled(g, B, H, D, cap, [cap] * B, behind=False)
    w = torch.exp(2 * randn(g, B, H, cap))
    if kind == "ties":
        w = torch.round(w * 2) / 2
    elif kind == "odd":
        w[..., ::7], w[..., 1::11], w[..., 2::13] = math.nan, math.inf, -math.inf
        w[..., 3::5], w[..., 4::5] = -0.0, 0.0
    to = bca.Kv4Cache(*[torch.randint(0, 255, t.shape, generator=g, device=DEV, dtype=torch.uint8)
                        for t in bca.magi_bca_kv4_cache(B, H, D, dst_cap)])
    was = [t.clone() for t in to]
    tw = torch.full((B, H, dst_cap), 7.0, device=DEV)
    n, index = bca.magi_bca_kv4_evict(cache, w, ints(*lengths), keep, recent, to, tw)
    assert n.tolist() == [min(x, keep) for x in lengths]
    nib = lambda t: torch.stack((t & 15, t >> 4), 3).flatten(2, 3)  # noqa: E731  value codes by token
    side = lambda t: t.transpose(3, 4).flatten(2, 3)  # noqa: E731  value scales by token
    for b in range(B):
        for h in range(H):
            at = ref.kept(w[b, h].tolist(), lengths[b], keep, recent)
            m = len(at)
            assert index[b, h].tolist() == at + [-1] * (keep - m)
            src = torch.tensor(at, device=DEV, dtype=torch.long)
            for new, old, first in ((to[0], cache[0], was[0]), (to[1], cache[1], was[1]),
                                    (nib(to[2]), nib(cache[2]), nib(was[2])),
                                    (side(to[3]), side(cache[3]), side(was[3]))):
                assert torch.equal(new[b, h, :m], old[b, h, src])
                assert torch.equal(new[b, h, m:], first[b, h, m:])      # slots behind are left as they were
            assert torch.equal(tw[b, h, :m].nan_to_num(-1, 2e38, -2e38), w[b, h, src].nan_to_num(-1, 2e38, -2e38))
            assert (tw[b, h, m:] == 7).all()


def test_evict_from_a_history_longer_than_shared_memory_holds():
    g = gen(41)
    n, keep = 330001, 5001
    cap = -(-n // 128) * 128
    cache = bca.magi_bca_kv4_cache(1, 1, 64, cap)
    cache.k_codes.random_(0, 256, generator=g)
    w = torch.round(torch.exp(2 * randn(g, 1, 1, cap)) * 64) / 64
    to, tw = bca.magi_bca_kv4_cache(1, 1, 64, keep), torch.zeros(1, 1, -(-keep // 128) * 128, device=DEV)
    _, index = bca.magi_bca_kv4_evict(cache, w, ints(n), keep, 100, to, tw)
    at = ref.kept(w[0, 0].tolist(), n, keep, 100)
    assert index[0, 0].tolist() == at
    assert torch.equal(to.k_codes[0, 0, :keep], cache.k_codes[0, 0, torch.tensor(at, device=DEV)])


# ----------------------------------------------------- together, as it is used
@pytest.mark.parametrize("D,Hq,H", [(128, 6, 2), (64, 4, 4)])
def test_a_streaming_loop(D, Hq, H):
    """Chunks attend among themselves through magi_bca_fwd and to the 4-bit
    history through the cache, joined; finished chunks are appended; when the
    history is full it is cut to the keys with most weight."""
    g = gen(17)
    B, L, cap, keep = 2, 96, 384, 160
    gq, gk = gains(g, D)
    cache, spare = bca.magi_bca_kv4_cache(B, H, D, cap), bca.magi_bca_kv4_cache(B, H, D, cap)
    w, spare_w = torch.zeros(B, H, cap, device=DEV), torch.zeros(B, H, cap, device=DEV)
    n = ints(0, 0)
    ref_w, host_n, evicted = w.double(), 0, 0
    for step in range(7):
        q, k, v = (randn(g, B, L, h, D).bfloat16() for h in (Hq, H, H))
        ang = angles(g, L, D // 2)
        own = bca.magi_bca_fwd_rope(q, k, v, [0, L], [0, L], gq, gk, ang, ang)
        out, lse = bca.magi_bca_kv4_fwd(q, cache, n, gq, gk, rope_q=ang, base_out=own[0], base_lse=own[1])
        # the whole in fp64: history and own keys in one softmax
        K, V = ref.unpack(cache)
        K2 = torch.cat((K[:, :, :host_n], ref.keys(k, ang).transpose(1, 2)), 2)
        V2 = torch.cat((V[:, :, :host_n], v.double().transpose(1, 2)), 2)
        s = ref.scores(q, K2, torch.tensor([host_n + L] * B), gq, gk, ang)
        want_lse = torch.logsumexp(s, -1).flatten(1, 2)
        want = torch.einsum("bhgij,bhjd->bhgid", torch.softmax(s, -1), V2).flatten(1, 2).transpose(1, 2)
        # own part: the forward's stated bounds; it enters rounded to bf16 once more
        assert_close(f"out {step}", to_np(out), want.cpu().numpy(), rel=8e-3)
        assert (lse.double() - want_lse).abs().max() <= 1.1e-2
        bca.magi_bca_kv4_weights(q, cache, n, lse, gq, gk, w, rope_q=ang)
        ref_w = ref.weights(q, cache, torch.tensor([host_n] * B), lse, gq, gk, ref_w, ang)
        assert torch.allclose(w[:, :, :host_n].double(), ref_w[:, :, :host_n], rtol=2e-4, atol=0)
        bca.magi_bca_kv4_append(cache, k, v, n, rope_k=ang)
        w[:, :, host_n:host_n + L] = 0
        ref_w[:, :, host_n:host_n + L] = 0
        n = n + L
        host_n += L
        if host_n + L > cap:
            n, index = bca.magi_bca_kv4_evict(cache, w, n, keep, L, spare, spare_w)
            ref_w = torch.zeros_like(ref_w).scatter_(2, torch.arange(keep, device=DEV).expand(B, H, keep),
                                                     ref_w.gather(2, index.long()))
            cache, spare, w, spare_w = spare, cache, spare_w, w
            host_n = keep
            evicted += 1
            assert n.tolist() == [keep] * B
    assert evicted >= 2 and bca.magi_bca_last_device_status() == 0


def test_a_captured_decoding_step_replays_while_the_history_grows():
    g = gen(23)
    B, Hq, H, D, cap = 2, 8, 2, 128, 256
    gq, gk = gains(g, D)
    cache = bca.magi_bca_kv4_cache(B, H, D, cap)
    n, one = ints(0, 5), ints(1, 1)
    q, k, v = (torch.zeros(B, 1, h, D, device=DEV, dtype=torch.bfloat16) for h in (Hq, H, H))
    w = torch.zeros(B, H, cap, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device=DEV)

    def step():
        bca.magi_bca_kv4_append(cache, k, v, n)
        n.add_(one)
        bca.magi_bca_kv4_fwd(q, cache, n, gq, gk, out=out, lse=lse)
        bca.magi_bca_kv4_weights(q, cache, n, lse, gq, gk, w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    total = torch.zeros_like(w, dtype=torch.float64)
    for i in range(40):
        for t, h in ((q, Hq), (k, H), (v, H)):
            t.copy_(randn(g, B, 1, h, D))
        graph.replay()
        o, l = ref.attention(q, cache, n.cpu(), gq, gk)
        check_attention((out, lse), (o, l), True, v.abs().max().item() * 2 + 4)
        total = ref.weights(q, cache, n.cpu(), lse, gq, gk, total)
    assert n.tolist() == [40, 45]
    assert torch.allclose(w.double(), total, rtol=2e-4, atol=1e-12)
    assert bca.magi_bca_last_device_status() == 0


def test_two_captured_chunk_steps_do_not_share_a_workspace():
    """Two graphs of the chunk kernels, replayed at the same time on two streams."""
    g = gen(37)
    D, cap, Sq = 128, 2048, 300
    gq, gk = gains(g, D)
    jobs = []
    for i in range(2):
        cache = filled(g, 1, 2, D, cap, [1900 + i])
        q = randn(g, 1, Sq, 4, D).bfloat16()
        jobs.append((cache, q, ints(1900 + i), torch.zeros(1, 2, cap, device=DEV)))

    def step(cache, q, n, w):
        out, lse = bca.magi_bca_kv4_fwd(q, cache, n, gq, gk)
        return out, lse, bca.magi_bca_kv4_weights(q, cache, n, lse, gq, gk, w, decay=0.0)

    want = [[t.clone() for t in step(*j)] for j in jobs]
    torch.cuda.synchronize()
    streams, graphs, got = [torch.cuda.Stream() for _ in jobs], [], []
    for s, j in zip(streams, jobs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got.append(step(*j))
        graphs.append(graph)
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        n = 1900
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2][..., :n], b[2][..., :n])
    assert bca.magi_bca_last_device_status() == 0


def test_calls_on_another_stream():
    g = gen(29)
    D, cap = 128, 1024
    cache = filled(g, 1, 2, D, cap, [1000])
    q = randn(g, 1, 200, 4, D).bfloat16()
    gq, gk = gains(g, D)
    n = ints(1000)
    want = bca.magi_bca_kv4_fwd(q, cache, n, gq, gk)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [bca.magi_bca_kv4_fwd(q, cache, n, gq, gk, stream=side) for _ in range(4)]
    noise = [torch.full((1 << 22,), 3.0, device=DEV) for _ in range(4)]   # would reuse a workspace freed too early
    side.synchronize()
    assert all(torch.equal(a[0], want[0]) and torch.equal(a[1], want[1]) for a in got) and len(noise) == 4


def test_binding_refusals():
    g = gen(31)
    c = bca.magi_bca_kv4_cache(2, 2, 64, 128)
    q = randn(g, 2, 1, 4, 64).bfloat16()
    k = randn(g, 2, 3, 2, 64).bfloat16()
    one = torch.ones(64, device=DEV)
    n = ints(1, 1)
    w = torch.zeros(2, 2, 128, device=DEV)
    lse = torch.zeros(2, 4, 1, device=DEV)
    for bad in (lambda: bca.magi_bca_kv4_append(c, k.float(), k, n), lambda: bca.magi_bca_kv4_append(c, k, k, n.long()),
                lambda: bca.magi_bca_kv4_append(c, k.transpose(1, 2), k, n),
                lambda: bca.magi_bca_kv4_fwd(q, c, n, one.double(), one),
                lambda: bca.magi_bca_kv4_fwd(q, c, n.cpu(), one, one),
                lambda: bca.magi_bca_kv4_weights(q, c, n, lse, one, one, w.half()),
                lambda: bca.magi_bca_kv4_fwd(q, (c[0].int(), *c[1:]), n, one, one)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: bca.magi_bca_kv4_append(c, k[:1].contiguous(), k[:1].contiguous(), n),
                lambda: bca.magi_bca_kv4_append(c, k, k[:, :2].contiguous(), n),
                lambda: bca.magi_bca_kv4_append(c, k, k, ints(1)),
                lambda: bca.magi_bca_kv4_append(c, k, k, n, rope_k=torch.zeros(2, 32, device=DEV)),
                lambda: bca.magi_bca_kv4_fwd(q, c, n, one, one, base_out=q),
                lambda: bca.magi_bca_kv4_fwd(q, c, n, one[:32].contiguous(), one),
                lambda: bca.magi_bca_kv4_weights(q, c, n, lse, one, one, w[:, :, :64].contiguous()),
                lambda: bca.magi_bca_kv4_evict(c, w, n, 129, 0, c, w),
                lambda: bca.magi_bca_kv4_evict(c, w, n, 5, 6, c, w),
                lambda: bca.magi_bca_kv4_fwd(q, (c[0], c[1][:, :, :64].contiguous(), *c[2:]), n, one, one)):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: bca.magi_bca_kv4_fwd(q, c, n, one, one, base_out=q, base_lse=lse, lse=lse), -1),
                        (lambda: bca.magi_bca_kv4_evict(c, w, n, 5, 0, c, w), -1),
                        (lambda: bca.magi_bca_kv4_fwd(q[:, :, :3].contiguous(), c, n, one, one), -2),
                        (lambda: bca.magi_bca_kv4_fwd(q.expand(2, 300, 4, 64).contiguous(), c, n, one, one,
                                                      workspace=torch.empty(256, device=DEV)), -4)):
        with pytest.raises(bca.MagiBcaError) as e:
            bad()
        assert e.value.status == status


def test_binding_refusals_say_what_was_expected():
    c = bca.magi_bca_kv4_cache(2, 2, 64, 128)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device=DEV)
    n, one = ints(1, 1), torch.ones(64, device=DEV)
    w = torch.zeros(2, 2, 128, device=DEV)
    to = bca.magi_bca_kv4_cache(2, 2, 64, 128)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    for bad, kind, text in (
            (lambda: bca.magi_bca_kv4_append(c, k, k, ints(1)), ValueError, r"start has shape \(1,\), expected \(2,\)"),
            (lambda: bca.magi_bca_kv4_append(c, k, k.float(), n), TypeError, "v must be a contiguous bfloat16 CUDA tensor"),
            (lambda: bca.magi_bca_kv4_append(c, k[0], k[0], n), ValueError, r"k has shape \(3, 2, 64\), expected 4 dimensions"),
            (lambda: bca.magi_bca_kv4_append(c, k, k, n, rms_eps="x"), TypeError, "real number"),
            (lambda: bca.magi_bca_kv4_read(c, n, -1), ValueError, "n is negative"),
            (lambda: bca.magi_bca_kv4_read(c, n, 1 << 40), ValueError, "n is out of range"),
            (lambda: bca.magi_bca_kv4_read(c, n, 3, k=k[:, :2].contiguous()), ValueError, r"k has shape \(2, 2, 2, 64\)"),
            (lambda: bca.magi_bca_kv4_fwd(q, (c[0], c[1][..., :2].contiguous(), *c[2:]), n, one, one), ValueError,
             r"cache.k_scales has shape \(2, 2, 128, 2\), expected \(2, 2, 128, 4\)"),
            (lambda: bca.magi_bca_kv4_fwd(q, c, n, one, one, workspace=torch.zeros(8)), TypeError, "workspace must be"),
            (lambda: bca.magi_bca_kv4_fwd(q, c, n, one, one, stream=5), AttributeError, "cuda_stream"),
            (lambda: bca.magi_bca_kv4_evict(c, w, n, 5, 6, to, w.clone()), ValueError, r"0 <= recent <= keep \(got 5, 6\)"),
            (lambda: bca.magi_bca_kv4_evict(c, w, n, 1 << 70, 0, to, w.clone()), ValueError, "keep is out of range")):
        with pytest.raises(kind, match=text):
            bad()
    # what was refused left the calls usable, and given outputs come back as themselves
    out, lse = torch.empty_like(q), torch.empty(2, 4, 1, device=DEV)
    got = bca.magi_bca_kv4_fwd(q, c, n, one, one, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert bca.magi_bca_kv4_fwd(q, c, n, one, one, want_lse=False)[1] is None
    assert bca.magi_bca_kv4_weights(q, c, n, lse, one, one, w) is w
    assert all(x.shape == (2, 0, 2, 64) for x in bca.magi_bca_kv4_read(c, n, 0))
    assert bca.magi_bca_last_device_status() == 0


def test_calls_from_several_threads():
    """Each thread on its own stream; the answers are those of one thread."""
    import threading
    g = gen(37)
    D, cap = 64, 2048
    cache = filled(g, 1, 2, D, cap, [2000])
    q = randn(g, 1, 2, 4, D).bfloat16()
    gq, gk = gains(g, D)
    n = ints(2000)
    want = bca.magi_bca_kv4_fwd(q, cache, n, gq, gk)
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = bca.magi_bca_kv4_fwd(q, cache, n, gq, gk)
                s.synchronize()
                if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                    wrong.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# the forms of the kernel for few rows: clusters whose CTAs have an SM each and
# twice the warps (of 16 CTAs, of 8), clusters of small CTAs, histories laid end to end
FORMS = [(1, 1, 4, 1, 128, 24576, [24001]), (1, 1, 8, 8, 64, 2176, [2049]), (2, 2, 6, 2, 128, 4224, [4200, 2]),
         (2, 5, 6, 2, 64, 10112, [0, 10007]), (1, 9, 3, 1, 128, 12288, [12287]), (2, 1, 16, 8, 64, 2176, [2100, 1]),
         (3, 2, 12, 4, 128, 1152, [1100, 0, 64]), (1, 3, 10, 10, 128, 12288, [12200]), (18, 1, 4, 1, 64, 1280, [70 * i for i in range(18)]),
         (4, 1, 8, 8, 128, 8192, [8192, 31, 0, 5000]), (1, 2, 40, 20, 64, 4096, [4000]),
         (2, 1, 6, 3, 128, 32896, [32800, 5]), (1, 1, 16, 16, 64, 20480, [20333]), (1, 5, 8, 4, 128, 32768, [32111])]


@pytest.mark.parametrize("base", [False, True])
@pytest.mark.parametrize("case", FORMS)
def test_attention_forms(case, base):
    test_attention(True, case, base)


@pytest.mark.parametrize("case", FORMS[:8])
def test_attention_forms_repeat_the_same_bits(case):
    B, Sq, Hq, H, D, cap, lengths = case
    g = gen(cap + Hq)
    cache = filled(g, B, H, D, cap, lengths)
    q = randn(g, B, Sq, Hq, D).bfloat16()
    gq, gk = gains(g, D)
    n = ints(*lengths)
    first = bca.magi_bca_kv4_fwd(q, cache, n, gq, gk)
    for _ in range(20):
        out, lse = bca.magi_bca_kv4_fwd(q, cache, n, gq, gk)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("kind", ["one value", "two values", "denormal", "steps", "negative"])
def test_evict_weights_of_few_values(kind):
    """Thresholds in a full bin, in the lowest and in the highest bits."""
    g = gen(41)
    B, H, D, cap, n, keep, recent = 1, 3, 64, 4352, 4300, 2000, 9
    cache = filled(g, B, H, D, cap, [cap], behind=False)
    r = torch.rand(B, H, cap, generator=g, device=DEV)
    w = {"one value": torch.full_like(r, 0.25), "two values": (r < 0.3).float() * 2 - 1,
         "denormal": (r * 1000).round() * 2.0 ** -149, "steps": 1 + (r * 300).round() * 2.0 ** -23,
         "negative": -torch.exp(20 * r - 10)}[kind].contiguous()
    to, to_w = bca.magi_bca_kv4_cache(B, H, D, 2048), torch.zeros(B, H, 2048, device=DEV)
    left, index = bca.magi_bca_kv4_evict(cache, w, ints(n), keep, recent, to, to_w)
    assert left.item() == keep
    cand = w[0, :, :n - recent].double().cpu()
    order = torch.sort(-cand, dim=-1, stable=True)[1][:, :keep - recent].sort(-1)[0]
    want = torch.cat((order, torch.arange(n - recent, n).expand(H, recent)), -1)
    assert torch.equal(index[0].cpu().long(), want)
    assert torch.equal(to_w[0, :, :keep].cpu(), torch.gather(w[0].cpu(), 1, want))
    assert bca.magi_bca_last_device_status() == 0
