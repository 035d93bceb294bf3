"""Plain 64-bit forms of the history-cache operators for the tests (CPU, torch double), written from the definitions."""
import math

import numpy as np
import torch


def rope_angles(max_pos, rot, base=10000.0):
    i = np.arange(rot // 2)
    return np.arange(max_pos)[:, None] * base ** (-2.0 * i / rot)


def rotate(x, cs, rot, interleaved):
    """x [n, heads, dh] double; cs [n, rot]: cosines, then sines."""
    y = x.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = cs[:, i, None], cs[:, rot // 2 + i, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def norm(x, kind, gamma, beta, eps):
    if kind == "none":
        return x
    mean = x.mean(-1, keepdim=True) if kind == "layernorm" else 0.0
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y


def quantise(x):
    """x [..., dh] double -> (codes [..., dh] int64, step [...], minimum [...]) with the format's roundings; NaN rows for
    rows with values that are not finite."""
    lo, hi = x.amin(-1), x.amax(-1)
    fine = torch.isfinite(x).all(-1)
    step = torch.where(fine, ((hi - lo) / 15).to(torch.bfloat16).double(), math.nan)
    mn = torch.where(fine, lo.to(torch.bfloat16).double(), math.nan)
    c = torch.where((step > 0)[..., None], ((x - mn[..., None]) / step[..., None]).round().clamp(0, 15), 0.0)
    return c.long(), step, mn


def channel_shift(dh):
    """Bit position of each channel's nibble in its 32-bit word."""
    ch = torch.arange(dh) % 8
    return 4 * (ch // 2) + 16 * (ch % 2)


def codes_of(packed):
    """bytes [..., dh/2] -> codes [..., dh] int64."""
    b = packed.cpu().long()
    w = b[..., 0::4] | b[..., 1::4] << 8 | b[..., 2::4] << 16 | b[..., 3::4] << 24
    w = w.repeat_interleave(8, -1)
    return w >> channel_shift(w.shape[-1]) & 15


def pack(codes):
    """codes [..., dh] int64 -> bytes [..., dh/2] uint8."""
    dh = codes.shape[-1]
    w = (codes << channel_shift(dh)).unflatten(-1, (dh // 8, 8)).sum(-1)
    return torch.stack([w >> 8 * k & 255 for k in range(4)], -1).flatten(-2).to(torch.uint8)


def values(packed, scale):
    """The values of cache rows in 64 bits: packed [..., dh/2], scale [..., 2] bf16."""
    s = scale.cpu().double()
    return s[..., 1:] + s[..., :1] * codes_of(packed).double()


def make_cache(pages, page, heads, dh, gen, std=1.0):
    """(k_codes, v_codes, k_scale, v_scale) on the CPU from normal K and V."""
    out = []
    for _ in range(2):
        c, step, mn = quantise(std * torch.randn(pages, heads, page, dh, generator=gen).double())
        out.append((pack(c), torch.stack((step, mn), -1).to(torch.bfloat16)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def gather(codes, scale, table_row, n, page):
    """Values [n, heads, dh] of the first n tokens of one request."""
    j = torch.arange(n)
    at = table_row.cpu().long()[j // page]
    return values(codes.cpu()[at, :, j % page], scale.cpu()[at, :, j % page])


def attend(q, cache, table, lens, cand_off, q_tokens, scale, limit=None):
    """(o [C*q, H, dh], lse [C*q, H]) in 64 bits."""
    k_codes, v_codes, k_scale, v_scale = cache
    heads, page, dh = k_codes.shape[1], k_codes.shape[2], 2 * k_codes.shape[3]
    H = q.shape[1]
    q = q.cpu().double()
    o = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    for r in range(len(cand_off) - 1):
        a, b, n = int(cand_off[r]) * q_tokens, int(cand_off[r + 1]) * q_tokens, int(lens[r])
        if a == b or n == 0:
            continue
        k = gather(k_codes, k_scale, table[r], n, page).repeat_interleave(H // heads, 1)
        v = gather(v_codes, v_scale, table[r], n, page).repeat_interleave(H // heads, 1)
        s = torch.einsum("ihd,jhd->ihj", q[a:b], k) * scale
        if limit is not None:
            lim = limit.cpu().long()[a // q_tokens:b // q_tokens].repeat_interleave(q_tokens)
            masked = torch.arange(n)[None, :] >= lim[:, None]
            s = s.masked_fill(masked[:, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
        l = p.sum(-1, keepdim=True)
        # a masked key counts for nothing, whatever it holds
        pv = torch.stack([torch.einsum("hj,jhd->hd", p[i][:, p[i].sum(0) != 0], v[p[i].sum(0) != 0]) for i in range(b - a)])
        o[a:b] = pv / torch.where(l == 0, 1.0, l)
        lse[a:b] = (m + torch.log(l))[..., 0]
    return o, lse


def attend_rows(q, cache, table, lens, cand_off, q_tokens, scale, limit=None):
    """:func:`attend` on the device of ``q`` and ``cache`` (64 bits), request by request, with each row's own sums:
    (o, lse, mag, spread) with mag = sum_j p_j (|v_j| + |minimum_j|) and spread = sqrt(sum_j (p_j v_j)^2), [C*q, H, dh] each.
    A masked key counts for nothing, a visible row that is held as NaN makes o (keys: lse too) NaN."""
    k_codes, v_codes, k_scale, v_scale = cache
    dev, hk, page, dh = q.device, k_codes.shape[1], k_codes.shape[2], 2 * k_codes.shape[3]
    H = q.shape[1]
    shift = channel_shift(dh).to(dev)

    def rows(codes, scales, at, within):
        b = codes[at, :, within].long()
        w = (b[..., 0::4] | b[..., 1::4] << 8 | b[..., 2::4] << 16 | b[..., 3::4] << 24).repeat_interleave(8, -1)
        s = scales[at, :, within].double()
        return (s[..., 1:] + s[..., :1] * (w >> shift & 15).double()).transpose(0, 1), s[..., 1].abs().transpose(0, 1)

    o, mag, spread = (torch.zeros(q.shape, dtype=torch.float64, device=dev) for _ in range(3))
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=dev)
    for r in range(len(cand_off) - 1):
        a, b, n = int(cand_off[r]) * q_tokens, int(cand_off[r + 1]) * q_tokens, int(lens[r])
        if a == b or n == 0:
            continue
        j = torch.arange(n, device=dev)
        at, within = table[r].to(dev).long()[j // page], j % page
        k, _ = rows(k_codes, k_scale, at, within)  # [hk, n, dh]
        v, mn = rows(v_codes, v_scale, at, within)
        s = q[a:b].double().view(b - a, hk, H // hk, dh).permute(1, 2, 0, 3).reshape(hk, -1, dh) @ k.transpose(1, 2) * scale
        if limit is not None:
            lim = limit[a // q_tokens:b // q_tokens].long().repeat_interleave(q_tokens).repeat(H // hk)
            s = s.masked_fill(j >= lim[:, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l == 0, 1.0, l)
        bad = torch.isnan(v).any(-1)  # [hk, n]
        seen = (s > -math.inf).double() @ bad.double()[..., None] > 0
        clean, least = v.masked_fill(bad[..., None], 0.0), mn.masked_fill(bad, 0.0)
        back = lambda t: t.view(hk, H // hk, b - a, -1).permute(2, 0, 1, 3).reshape(b - a, H, -1)  # noqa: E731
        o[a:b] = back((p @ clean).masked_fill(seen, math.nan))
        mag[a:b] = back(p @ (clean.abs() + least[..., None]))
        spread[a:b] = back(((p * p) @ (clean * clean)).sqrt())
        lse[a:b] = back(m + l.log())[..., 0]
    return o, lse, mag, spread
