"""The 4-bit key/value cache in fp64, for the tests: format, attention, weights
and eviction written from their definitions, on whatever device the tensors
are on.  Shares no code with the package."""
import math

import torch

MAGS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
# value of each scale byte: 5 exponent and 3 mantissa bits, steps of 2^-17 below 2^-14; 226 = 10240
SCALES = torch.tensor([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 18) for e in range(32) for m in range(8)],
                      dtype=torch.float64)
TOP_BYTE = 226
TOP = 6 * 10240.0


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0, the even index of two as near."""
    mids = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(mids.to(x.device), x.contiguous())             # mids below x
    tie = (i < len(mids)) & (mids.to(x.device)[i.clamp(max=len(mids) - 1)] == x) & (i % 2 == 1)
    return torch.where(tie, i + 1, i)


def quantise(x):
    """(values, codes, scale bytes) of x [..., D] fp64 with D a multiple of 16."""
    x = torch.nan_to_num(x, nan=0.0, posinf=TOP, neginf=-TOP).clamp(-TOP, TOP)
    b = x.unflatten(-1, (-1, 16))
    byte = nearest(b.abs().amax(-1) / 6, SCALES[: TOP_BYTE + 1])
    s = SCALES.to(x.device)[byte].unsqueeze(-1)
    code = torch.where(s > 0, nearest(b.abs() / torch.where(s > 0, s, 1.0), MAGS), 0)
    val = torch.where(b < 0, -1.0, 1.0) * MAGS.to(x.device)[code] * s
    return val.flatten(-2), (code | (torch.signbit(b) & (s > 0)) * 8).flatten(-2), byte


def rotate(x, angles):
    """x [..., n, H, D] by angles [..., n, D/2]: feature i with i + D/2."""
    if angles is None:
        return x
    c, s = torch.cos(angles.double()).unsqueeze(-2), torch.sin(angles.double()).unsqueeze(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def keys(k, angles=None, eps=1e-6):
    """K^ of k [B, n, H, D]."""
    k = k.double()
    return rotate(k, angles) / torch.sqrt(k.square().mean(-1, keepdim=True) + eps)


def unpack(cache):
    """fp64 (K, V) [B, H, capacity, D] that the four tensors stand for."""
    kc, ks, vc, vs = [t.long() for t in cache]
    signed = torch.cat((MAGS, -MAGS)).to(kc.device)
    scales = SCALES.to(kc.device)
    k = signed[torch.stack((kc % 16, kc // 16), -1).flatten(-2)] * scales[ks].repeat_interleave(16, -1)
    v = signed[torch.stack((vc % 16, vc // 16), 3).flatten(2, 3)]
    return k, v * scales[vs.transpose(3, 4).flatten(2, 3)].repeat_interleave(16, -1)


def pack(kcode, kbyte, vcode, vbyte):
    """The four tensors from codes [B, H, capacity, D] and scale bytes."""
    u = torch.uint8
    return ((kcode[..., 0::2] | kcode[..., 1::2] << 4).to(u).contiguous(), kbyte.to(u).contiguous(),
            (vcode[:, :, 0::2] | vcode[:, :, 1::2] << 4).to(u).contiguous(),
            torch.stack((vbyte[:, :, 0::2], vbyte[:, :, 1::2]), -1).to(u).contiguous())


def scores(q, K, lengths, gq, gk, angles=None, scale=0.0, eps=1e-6):
    """Natural-log scores [B, H, G, Sq, capacity]; -inf behind the length."""
    B, Sq, Hq, D = q.shape
    H = K.shape[1]
    x = q.double()
    x = rotate(x, angles) / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * (gq.double() * gk.double())
    x = x.unflatten(2, (H, Hq // H)).permute(0, 2, 3, 1, 4)
    s = torch.einsum("bhgid,bhjd->bhgij", x, K) * (scale if scale > 0 else 1 / math.sqrt(D))
    behind = torch.arange(K.shape[2], device=q.device) >= lengths.to(q.device)[:, None]
    return s.masked_fill(behind[:, None, None, None], -math.inf)


def attention(q, cache, lengths, gq, gk, angles=None, base_out=None, base_lse=None, scale=0.0, eps=1e-6):
    """(out [B, Sq, Hq, D], lse [B, Hq, Sq]) in fp64."""
    K, V = unpack(cache)
    V = torch.nan_to_num(V, nan=0.0, posinf=0.0, neginf=0.0)      # only slots behind the length can hold those
    K = torch.nan_to_num(K, nan=0.0, posinf=0.0, neginf=0.0)
    s = scores(q, K, lengths, gq, gk, angles, scale, eps)
    if base_out is not None:   # the base part is one more key, whose value differs from row to row
        B, H, G, Sq, _ = s.shape
        s = torch.cat((s, base_lse.double().view(B, H, G, Sq, 1)), -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    lse = (torch.where(m == -math.inf, 0.0, m) + torch.log(l)).squeeze(-1).flatten(1, 2)
    p = p / torch.where(l > 0, l, 1.0)
    o = torch.einsum("bhgij,bhjd->bhgid", p[..., : K.shape[2]], V)
    o = o.flatten(1, 2).transpose(1, 2)
    if base_out is not None:
        share = p[..., -1].flatten(1, 2).transpose(1, 2).unsqueeze(-1)
        o = o + torch.where(share > 0, share * base_out.double(), 0.0)
    return o, lse


def weights(q, cache, lengths, lse, gq, gk, old, angles=None, decay=1.0, scale=0.0, eps=1e-6):
    K, _ = unpack(cache)
    K = torch.nan_to_num(K, nan=0.0, posinf=0.0, neginf=0.0)
    s = scores(q, K, lengths, gq, gk, angles, scale, eps)
    B, H, G, Sq, cap = s.shape
    x = lse.double().view(B, H, G, Sq, 1)
    p = torch.where(x == -math.inf, 0.0, torch.exp(s - x)).sum((2, 3))
    new = (decay * old.double() if decay else 0.0) + p
    inside = (torch.arange(cap, device=q.device) < lengths.to(q.device)[:, None])[:, None]
    return torch.where(inside, new, old.double())


def kept(w, length, keep, recent):
    """The slots that stay of one (batch element, head), in order (w: list of floats)."""
    left = min(length, keep)
    rec = min(recent, left)
    old = range(length - rec)
    key = lambda j: -math.inf if math.isnan(w[j]) else w[j]  # noqa: E731
    best = sorted(old, key=lambda j: (-key(j), j))[: left - rec]
    return sorted(best) + list(range(length - rec, length))
