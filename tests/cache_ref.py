"""Plain 64-bit forms of the cache calls (torch on the CPU), and the inputs of
their tests.  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn
BF = torch.bfloat16


def random_parents(B, N, rs, max_depth=64, back=8):
    parents = np.full((B, N), -1, dtype=np.int32)
    depth = np.zeros((B, N), dtype=np.int32)
    for b in range(B):
        for n in range(1, N):
            p = rs.randint(max(0, n - back), n)
            if depth[b, p] >= max_depth:
                p = 0
            parents[b, n], depth[b, n] = p, depth[b, p] + 1
    return parents


def plan(parents, lengths):
    """Positions and masks of one valid batch, node by node."""
    B, N = parents.shape
    W = (N + 31) // 32
    pos = np.full((B, N), -1, dtype=np.int32)
    words = np.zeros((B, N, W), dtype=np.uint32)
    for b in range(B):
        if lengths[b] < 0:
            continue
        for n in range(N):
            cur, d = n, -1
            while cur >= 0:
                words[b, n, cur // 32] |= np.uint32(1 << (cur % 32))
                cur, d = parents[b, cur], d + 1
            pos[b, n] = lengths[b] + d
    return pos, words.view(np.int32)


def unpack(words, N):
    """[B, N, W] int32 -> [B, N, N] bool."""
    w = words.cpu().numpy().view(np.uint32)
    bits = (w[..., None] >> np.arange(32, dtype=np.uint32)) & 1
    return torch.from_numpy(bits.reshape(*w.shape[:2], -1)[..., :N].astype(bool))


def pack(mask):
    """[B, N, N] bool -> [B, N, W] int32."""
    m = mask.numpy()
    B, N, _ = m.shape
    W = (N + 31) // 32
    p = np.zeros((B, N, W * 32), dtype=bool)
    p[..., :N] = m
    return torch.from_numpy(np.packbits(p.reshape(B, N, W, 32), axis=-1, bitorder="little").view(np.int32)
                            .reshape(B, N, W).copy())


def norm_rope(x, pos, inv_freq, weight, eps, interleaved):
    """x [..., H, D] f64 at pos [...]; returns the rows and, per element, |a| + |b| of its pair."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    y, mag = x.clone(), x.abs()
    if inv_freq is not None:
        h = inv_freq.numel()
        a = slice(0, 2 * h, 2) if interleaved else slice(0, h)
        b = slice(1, 2 * h, 2) if interleaved else slice(h, 2 * h)
        ang = pos.double()[..., None, None] * inv_freq.double()
        c, s = torch.cos(ang), torch.sin(ang)
        xa, xb = x[..., a].clone(), x[..., b].clone()
        y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
        mag[..., a] = mag[..., b] = xa.abs() + xb.abs()
    return y, mag


def block_scale(amax):
    m, e = math.frexp(float(amax))
    if m == 0:
        return 1.0
    return 2.0 ** max(e - 9 + (m > 0.875), -126)


def e4m3(x):
    """Bytes of f64 values that are at most 448 in magnitude (nearest, ties to even), NaN 0x7F."""
    out = x.float().to(F8).view(torch.uint8)
    return torch.where(torch.isfinite(x), out, torch.full_like(out, 0x7F))


class Cache:
    """The cache on the CPU: token rows as bf16 per sequence, blocks quantised when full."""

    def __init__(self, B, Hkv, D, page):
        self.B, self.H, self.D, self.page = B, Hkv, D, page
        self.rows = [[torch.zeros(0, Hkv, D, dtype=BF) for _ in range(B)] for _ in range(2)]

    def append(self, b, k, v):
        for which, x in enumerate((k, v)):
            self.rows[which][b] = torch.cat((self.rows[which][b], x.to(BF)))

    def length(self, b):
        return self.rows[0][b].shape[0]

    def blocks(self, b, which):
        """(bytes, scale) of every full block: [n, H, page, D] uint8, [n, H] f32."""
        n = self.length(b) // self.page
        x = self.rows[which][b][:n * self.page].view(n, self.page, self.H, self.D).transpose(1, 2).double()
        fin = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax((2, 3)) if n else torch.zeros(0, self.H)
        scale = torch.tensor([[block_scale(a) for a in r] for r in fin.tolist()], dtype=torch.float64).view(n, self.H)
        return e4m3(x / scale[..., None, None]), scale

    def open_rows(self, b, which):
        n = self.length(b) // self.page * self.page
        return self.rows[which][b][n:]


def row_scale(x):
    """[.., D] -> [..]: the power of two at or below the row's largest finite magnitude (1 for zeros)."""
    a = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(-1)
    m, e = torch.frexp(a)
    return torch.where(a > 0, torch.ldexp(torch.ones_like(a), e - 1), torch.ones_like(a))


def small_part(x):
    """Per element, what a row loses when it is held as two e4m3 rows after its largest magnitude was brought to
    [2^7, 2^8): 2^-10 of that scale, for elements below 2^-2 of it only (the others have their eight bits)."""
    unit = row_scale(x) * 2.0 ** -7
    a = torch.nan_to_num(x, 0, 0, 0).abs()
    return torch.where(a < unit[..., None] * 0.25, torch.minimum(a, unit[..., None] * 2.0 ** -10), torch.zeros_like(a))


def attention(q, k, v, keys, values, mask, scale, vscale, full):
    """One sequence: q [N, Hq, D], nodes k/v [N, Hkv, D], cached keys/values [L, Hkv, D], mask [N, N],
    vscale [L, Hkv] the scales of the cached values, full: the tokens in 8-bit blocks.  All f64.  Returns
    out, lse, sum p |v|, max over keys of scale * sum |q| |k|, max p s * sum |v| / s over the keys' value
    scales s, and max over keys of scale * (what the rows' small elements can lose)."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    K = torch.cat((keys, k)).repeat_interleave(G, 1)          # [T, Hq, D]
    V = torch.cat((values, v)).repeat_interleave(G, 1)
    loss = torch.cat((torch.zeros_like(K[:full]), small_part(K[full:])))
    lost = (torch.einsum("nhd,thd->nht", small_part(q), K.abs()) + torch.einsum("nhd,thd->nht", q.abs(), loss)) * scale
    see = torch.cat((torch.ones(N, keys.shape[0], dtype=torch.bool), mask), 1)[:, None].expand(N, Hq, -1)
    s = torch.einsum("nhd,thd->nht", q, K) * scale
    mag = torch.einsum("nhd,thd->nht", q.abs(), K.abs()) * scale
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    mag = torch.where(see, mag, torch.zeros_like(mag)).amax(-1)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.where(see, torch.exp(s - top), torch.zeros_like(s))
    total = p.sum(-1, keepdim=True)
    w = torch.where(total > 0, p / total, torch.zeros_like(p))
    # a masked key's value takes no part, whatever it holds
    out = torch.einsum("nht,thd->nhd", w, torch.nan_to_num(V, 0, 0, 0))
    vabs = torch.nan_to_num(V, 0, 0, 0).abs()
    S = torch.cat((vscale, row_scale(v))).repeat_interleave(G, 1)     # [T, Hq]
    lead = (w * S.T).amax(-1)                                         # [N, Hq]
    small = lead[..., None] * torch.einsum("nht,thd->nhd", see.double(), vabs / S[..., None])
    lost = torch.where(see, lost, torch.zeros_like(lost)).amax(-1)
    return out, (torch.log(total) + top)[..., 0], torch.einsum("nht,thd->nhd", w, vabs), mag, small, lost


def inv_freq(rot, base=1e6):
    return torch.exp(torch.arange(0, rot, 2, dtype=torch.float64) * (-math.log(base) / rot)).float()
