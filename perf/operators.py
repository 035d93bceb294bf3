"""Work that the history-cache operators are timed and compared on: plain forms, the framework's calls, exact values.

Three operators of a request's cached history (its keys and values held once per request and read by all of the
request's candidates):

* ``norm_rope``  per-head norm of queries and keys with the position rotation in the same pass;
* ``append``     new keys and values into a paged 4-bit cache, keys rotated on the way, and the read-back of the
                 appended rows as bf16 (the cache's contents as the values that they stand for);
* ``attend``     every candidate's queries over its request's paged 4-bit keys and values.

4-bit rows: one (token, head) row of dh values is held as codes c in 0..15 with a bf16 step and minimum, value =
minimum + step * c.  In every 32-bit word (8 channels) nibble i of the low half is channel 2i, nibble i of the high
half channel 2i + 1.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------- cases
def _nr(name, nq, nk, hq, hk, dh, rot, norm, style, dtype, max_pos):
    return {"name": name, "op": "norm_rope", "nq": nq, "nk": nk, "hq": hq, "hk": hk, "dh": dh, "rot": rot, "norm": norm,
            "style": style, "dtype": dtype, "max_pos": max_pos}


def _ap(name, R, new_lo, new_hi, base_lo, base_hi, hk, dh, rot, style, page):
    return {"name": name, "op": "append", "R": R, "new_lo": new_lo, "new_hi": new_hi, "base_lo": base_lo,
            "base_hi": base_hi, "hk": hk, "dh": dh, "rot": rot, "style": style, "page": page}


def _at(name, R, n_lo, n_hi, q, l_lo, l_hi, h, hk, dh, page, limits=False):
    return {"name": name, "op": "attend", "R": R, "n_lo": n_lo, "n_hi": n_hi, "q": q, "l_lo": l_lo, "l_hi": l_hi,
            "h": h, "hk": hk, "dh": dh, "page": page, "limits": limits}


def listed():
    return [
        # one candidate of 4 query tokens and one new history event: the smallest call, latency counts
        _nr("norm_rope_step", 4, 1, 8, 8, 128, 128, "rmsnorm", "half", "bf16", 8192),
        # queries of 32 x 512 candidates and the keys of 32 histories of 2048 events, both normed and rotated
        _nr("norm_rope_batch", 16384, 65536, 8, 8, 128, 128, "rmsnorm", "half", "bf16", 2049),
        # fp32, odd counts, half of the channels rotated in interleaved pairs, LayerNorm with an offset
        _nr("norm_rope_fp32_odd", 1999, 7001, 5, 3, 64, 32, "layernorm", "interleaved", "fp32", 5000),
        # one new event in each of 64 running histories: the serving step
        _ap("append_step", 64, 1, 1, 500, 8000, 8, 128, 128, "half", 64),
        # 8 whole histories of 4096 to 8192 events put into an empty cache
        _ap("append_histories", 8, 4096, 8192, 0, 0, 4, 128, 128, "half", 128),
        # ragged additions behind histories that end inside pages; small pages, narrow heads
        _ap("append_ragged", 32, 1, 700, 0, 2000, 16, 64, 64, "interleaved", 16),
        # one query token over one history: the smallest call
        _at("attend_one", 1, 1, 1, 1, 1000, 1000, 8, 8, 128, 64),
        # a few query tokens over many long histories: the cache's bytes count
        _at("attend_few_long", 32, 1, 1, 4, 8192, 16384, 8, 8, 128, 64),
        # heads that share keys, narrow heads, small pages, a handful of candidates
        _at("attend_shared_heads", 16, 2, 8, 2, 1024, 4096, 16, 4, 64, 16),
        # 512 candidates for each of 32 histories of 2048 events: the ordinary batch
        _at("attend_batch", 32, 512, 512, 1, 2048, 2048, 8, 8, 128, 64),
        # 2048 candidates of 4 tokens over 8 histories of 4096 to 8192 events: the largest
        _at("attend_long", 8, 2048, 2048, 4, 4096, 8192, 4, 4, 128, 128),
        # ragged candidates, each allowed to see its own prefix of the history (some of them nothing), three query
        # heads to a key head, histories that may be empty
        _at("attend_limits", 24, 0, 300, 1, 0, 2500, 6, 2, 128, 32, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "attend", "attend"))
    dh = rng.choice((64, 128))
    if op == "norm_rope":
        return {k: v for k, v in _nr("", _log(rng, 1, 20000), _log(rng, 1, 60000), rng.randint(1, 16), rng.randint(1, 8),
                                     dh, rng.choice((dh, dh // 2)), rng.choice(("rmsnorm", "layernorm", "none")),
                                     rng.choice(("half", "interleaved")), rng.choice(("bf16", "bf16", "fp32")),
                                     _log(rng, 100, 20000)).items() if k != "name"}
    page = rng.choice((16, 32, 64, 128))
    hk = rng.choice((1, 2, 3, 4, 8))
    if op == "append":
        R = _log(rng, 1, 128)
        new = _log(rng, 1, 40000 // R)
        base = _log(rng, 1, 4000)
        return {k: v for k, v in _ap("", R, max(1, new // 3), new, base // 3, base, hk, dh, rng.choice((dh, dh // 2)),
                                     rng.choice(("half", "interleaved")), page).items() if k != "name"}
    R = _log(rng, 1, 32)
    L = _log(rng, 1, 12000)
    g = rng.choice((1, 1, 2, 3, 4, 8))
    q = rng.choice((1, 2, 4))
    # rows x keys of all requests and heads stays within the largest listed case
    n = max(1, min(_log(rng, 1, 2000), int(1.0e9 / (R * L * hk * g * q))))
    return {k: v for k, v in _at("", R, n // 3, n, q, L // 2, L, hk * g, hk, dh, page, rng.random() < 0.3).items()
            if k != "name"}


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, the same for every seed: ragged, both ends among them from n = 2 on."""
    if n == 1:
        return np.array([hi], np.int64)
    f = (np.arange(n) * 0.6180339887498949) % 1.0
    v = np.floor(lo + (hi - lo + 1) * f).astype(np.int64).clip(lo, hi)
    v[0], v[1] = lo, hi
    return v


def _off(counts):
    o = np.zeros(len(counts) + 1, np.int32)
    o[1:] = np.cumsum(counts)
    return o


# -------------------------------------------------------------------------------------------------------- prepare
def _rope_table(max_pos, rot):
    """[max_pos, rot] fp32: the cosines of position * 10000^(-2i/rot), then the sines; angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float().contiguous()


def _pages(g, lens, page):
    """Page table [R, max pages] over a pool with its pages in random order; entries past a history are -1."""
    need = -(-lens // page)
    cols, total = max(1, int(need.max())), max(1, int(need.sum()))
    order = torch.randperm(total + 3, generator=g, device=DEV)[:total].to(torch.int32)
    table = torch.full((len(lens), cols), -1, dtype=torch.int32, device=DEV)
    first = torch.as_tensor(np.concatenate(([0], np.cumsum(need)[:-1])), device=DEV)
    k = torch.arange(cols, device=DEV)[None, :]
    have = k < torch.as_tensor(need, device=DEV)[:, None]
    table[have] = order[(first[:, None] + k)[have]]
    return table, total + 3


def _quantise(x):
    """x [..., dh] fp32 -> codes [..., dh] uint8, step and minimum [...] bf16."""
    lo, hi = x.amin(-1), x.amax(-1)
    step, mn = ((hi - lo) / 15).to(torch.bfloat16), lo.to(torch.bfloat16)
    s = step.float()[..., None]
    c = torch.where(s > 0, ((x - mn.float()[..., None]) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15), 0.0)
    return c.to(torch.uint8), step, mn


def _pack(c):
    """codes [..., dh] -> bytes [..., dh / 2]"""
    w = c.view(*c.shape[:-1], -1, 2, 2, 2)  # word, byte of its half, channels (2i, 2i + 2), (even, odd)
    b = w[..., 0, :] | (w[..., 1, :] << 4)  # [word, byte, (even, odd)]
    return b.transpose(-1, -2).reshape(*c.shape[:-1], -1).contiguous()


def _unpack(b):
    """bytes [..., dh / 2] -> codes [..., dh]"""
    w = b.view(*b.shape[:-1], -1, 2, 2)  # word, (even, odd), byte of its half
    n = torch.stack((w & 15, w >> 4), -1)  # word, (even, odd), byte, nibble
    return n.flatten(-2).transpose(-1, -2).reshape(*b.shape[:-1], -1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    dh = case["dh"]
    if case["op"] == "norm_rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s = {"q": randn(case["nq"], case["hq"], dh).to(dt), "k": (1.5 * randn(case["nk"], case["hk"], dh) + 0.2).to(dt)}
        for x, n in (("q", case["nq"]), ("k", case["nk"])):
            s["pos_" + x] = torch.randint(0, case["max_pos"], (n,), generator=g, device=DEV, dtype=torch.int32)
            s["gamma_" + x] = 1 + 0.2 * randn(dh)
            s["beta_" + x] = 0.1 * randn(dh) if case["norm"] == "layernorm" else None
        s["rope"] = _rope_table(case["max_pos"], case["rot"])
        return {"case": case, **s}
    hk, page, R = case["hk"], case["page"], case["R"]
    if case["op"] == "append":
        new, base = _spread(case["new_lo"], case["new_hi"], R), _spread(case["base_lo"], case["base_hi"], R)[::-1].copy()
        off, T = _off(new), int(new.sum())
        table, pool = _pages(g, base + new, page)
        req = np.repeat(np.arange(R), new)
        return {"case": case, "k": (randn(T, hk, dh) * torch.exp(0.5 * randn(hk, dh))).bfloat16(),
                "v": randn(T, hk, dh).bfloat16(), "tok_off": (torch.from_numpy(off).to(DEV), off),
                "base": torch.from_numpy(base.astype(np.int32)).to(DEV), "table": table,
                "rope": _rope_table(int((base + new).max()), case["rot"]), "req": torch.from_numpy(req).to(DEV),
                "k_codes": torch.zeros(pool, hk, page, dh // 2, dtype=torch.uint8, device=DEV),
                "v_codes": torch.zeros(pool, hk, page, dh // 2, dtype=torch.uint8, device=DEV),
                "k_scale": torch.zeros(pool, hk, page, 2, dtype=torch.bfloat16, device=DEV),
                "v_scale": torch.zeros(pool, hk, page, 2, dtype=torch.bfloat16, device=DEV)}
    lens, cnt = _spread(case["l_lo"], case["l_hi"], R), _spread(case["n_lo"], case["n_hi"], R)[::-1].copy()
    off = _off(cnt)
    C, q = int(off[-1]), case["q"]
    table, pool = _pages(g, lens, page)
    s = {"case": case, "table": table, "lens": torch.from_numpy(lens.astype(np.int32)).to(DEV), "limit": None,
         "cand_off": (torch.from_numpy(off).to(DEV), off), "q": (1.5 * randn(C * q, case["h"], dh)).bfloat16(),
         "scale": 1.0 / math.sqrt(dh), "l_max": int(lens.max()), "n_max": int(cnt.max()) * q}
    for x in "kv":
        codes, step, mn = _quantise(randn(pool, hk, page, dh))
        s[x + "_codes"], s[x + "_scale"] = _pack(codes), torch.stack((step, mn), -1).contiguous()
        del codes
    if case["limits"]:
        u = torch.rand(C, generator=g, device=DEV) * 1.2 - 0.1  # a twelfth of the candidates see nothing, as many all
        of = torch.from_numpy(np.repeat(lens, cnt)).to(DEV)
        s["limit"] = (u * of).floor().clamp(min=0).to(torch.int32)
    return s


# ------------------------------------------------------------------------------------------------------------ run
def _norm(x, norm, gamma, beta, eps=1e-6):
    if norm == "none":
        return x
    if norm == "layernorm":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gamma
    return y if beta is None else y + beta


def _rotate(x, cs, rot, style):
    """x [n, heads, dh]; cs [n, rot]: cosines, then sines"""
    c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    a, b = (x[..., : rot // 2], x[..., rot // 2: rot]) if style == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    y, z = a * c - b * s, b * c + a * s
    r = torch.cat((y, z), -1) if style == "half" else torch.stack((y, z), -1).flatten(-2)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_norm_rope(s):
    c = s["case"]

    def side(x):
        y = _norm(s[x].float(), c["norm"], s["gamma_" + x], s["beta_" + x])
        return _rotate(y, s["rope"][s["pos_" + x].long()], c["rot"], c["style"]).to(s[x].dtype)

    return {"q": side("q"), "k": side("k")}


def _plain_append(s):
    c = s["case"]
    page, req = c["page"], s["req"]
    slot = torch.arange(len(req), device=DEV) - s["tok_off"][0].long()[req] + s["base"].long()[req]
    at, within = s["table"].long()[req, slot // page], slot % page
    k = _rotate(s["k"].float(), s["rope"][slot], c["rot"], c["style"])

    def side(x, y):
        codes, step, mn = _quantise(y)
        s[x + "_codes"][at, :, within] = _pack(codes)
        s[x + "_scale"][at, :, within] = torch.stack((step, mn), -1)
        held = s[x + "_scale"][at, :, within].float()
        return (held[..., 1:] + held[..., :1] * _unpack(s[x + "_codes"][at, :, within]).float()).bfloat16()

    return {"k": side("k", k), "v": side("v", s["v"].float())}


def _plain_attend(s):
    c = s["case"]
    R, page, q, h, hk, dh = c["R"], c["page"], c["q"], c["h"], c["hk"], c["dh"]
    off, lens = s["cand_off"][0].long() * q, s["lens"].long()
    n = torch.arange(max(1, s["n_max"]), device=DEV)
    have = n < (off[1:] - off[:-1])[:, None]
    tok = torch.where(have, off[:-1, None] + n, 0)
    j = torch.arange(max(1, s["l_max"]), device=DEV)
    seen = j < lens[:, None]
    at = torch.where(seen, s["table"].long()[:, j // page], 0)

    def side(x):
        held = s[x + "_scale"][at, :, j % page].float()
        y = held[..., 1:] + held[..., :1] * _unpack(s[x + "_codes"][at, :, j % page]).float()
        return torch.where(seen[..., None, None], y, 0.0).transpose(1, 2)  # [R, hk, keys, dh]

    qs = s["q"][tok].float().view(R, len(n), hk, h // hk, dh).transpose(1, 2).reshape(R, hk, -1, dh)
    x = qs @ side("k").transpose(-1, -2) * s["scale"]
    if s["limit"] is not None:
        lim = torch.minimum(s["limit"].long()[tok // q], lens[:, None]).repeat_interleave(h // hk, 1)
        x.masked_fill_(~(j < lim[..., None])[:, None], -math.inf)
    else:
        x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x @ side("v")) / torch.where(l > 0, l, 1.0)
    o = o.view(R, hk, len(n), h // hk, dh).transpose(1, 2).reshape(R, len(n), h, dh)
    lse = (m + l.log()).view(R, hk, len(n), h // hk).transpose(1, 2).reshape(R, len(n), h)
    return {"o": o[have].bfloat16(), "lse": lse[have]}


def run(state):
    s, c = state, state["case"]
    if own:
        import attention_ikbo_b200 as ikbo

        if c["op"] == "norm_rope":
            q, k = ikbo.rocs_qk_norm_rope_forward(s["q"], s["k"], s["pos_q"], s["pos_k"], s["rope"], norm=c["norm"],
                                                  gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], beta_q=s["beta_q"],
                                                  beta_k=s["beta_k"], eps=1e-6, interleaved=c["style"] == "interleaved")
            return {"q": q, "k": k}
        cache = ikbo.CacheQ4(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        if c["op"] == "append":
            ikbo.rocs_cache_append(cache, s["k"], s["v"], s["tok_off"], s["base"], s["table"], rope=s["rope"],
                                   interleaved=c["style"] == "interleaved")
            k, v = ikbo.rocs_cache_read(cache, s["tok_off"], s["base"], s["table"])
            return {"k": k, "v": v}
        o, lse = ikbo.rocs_dca_cache_forward(s["q"], cache, s["table"], s["lens"], s["cand_off"], c["q"], s["scale"],
                                             key_limit=s["limit"])
        return {"o": o, "lse": lse}
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "attend": _plain_attend}[c["op"]](s)


# ------------------------------------------------------------------------------------------------ work and exactness
def work(case):
    dh, op = case["dh"], case["op"]
    if op == "norm_rope":
        e = 2 if case["dtype"] == "bf16" else 4
        values = (case["nq"] * case["hq"] + case["nk"] * case["hk"]) * dh
        n = case["nq"] + case["nk"]
        rows = case["max_pos"] * (1 - (1 - 1 / case["max_pos"]) ** n)  # different positions among n
        return {"bytes": 2 * values * e + 4 * n + 4 * rows * case["rot"], "flops": 10 * values}
    hk, R = case["hk"], case["R"]
    row = dh + 8  # codes, step and minimum of one token's key and value, a head
    if op == "append":
        new, base = _spread(case["new_lo"], case["new_hi"], R), _spread(case["base_lo"], case["base_hi"], R)[::-1]
        T = int(new.sum())
        table = len(np.unique(np.concatenate([np.arange(b, b + n) for b, n in zip(base, new)]))) * case["rot"] * 4
        pages = int((-(-(base + new) // case["page"])).sum())
        # keys and values in; rows out; rows in and bf16 keys and values out
        return {"bytes": T * hk * (4 * dh + row + row + 4 * dh) + table + 4 * (pages + 2 * R + 1), "flops": T * hk * dh * 16}
    lens, cnt = _spread(case["l_lo"], case["l_hi"], R), _spread(case["n_lo"], case["n_hi"], R)[::-1]
    rows = cnt * case["q"] * case["h"]
    C = int(cnt.sum())
    read = lens * (cnt > 0)
    return {"bytes": int(read.sum()) * hk * row + int(rows.sum()) * (4 * dh + 4) + 4 * int((-(-read // case["page"])).sum())
            + 4 * (2 * R + 1) + (4 * C if case["limits"] else 0), "flops": 4 * dh * int((rows * lens).sum())}


def _exact_values(codes, scale):
    """The values of packed rows, in 64 bits, from the format's definition: codes [n, dh / 2], scale [n, 2]."""
    n, half = codes.shape
    words = codes.reshape(n, half // 4, 4).long()
    word = words[..., 0] | words[..., 1] << 8 | words[..., 2] << 16 | words[..., 3] << 24
    out = torch.empty(n, half // 4, 8, dtype=torch.float64, device=codes.device)
    for ch in range(8):
        out[..., ch] = (word >> (4 * (ch // 2) + 16 * (ch % 2)) & 15).double()
    return out.reshape(n, 2 * half) * scale[:, :1].double() + scale[:, 1:].double()


def _exact_rotation(x, angle_cos, angle_sin, style):
    """Channel pairs as complex numbers times cos + i sin; x [n, heads, dh] in 64 bits."""
    half = angle_cos.shape[1]
    i = torch.arange(half, device=x.device)
    a, b = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., a], x[..., b]) * torch.complex(angle_cos, angle_sin)[:, None]
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    rot = case.get("rot", 0) // 2
    if case["op"] == "norm_rope":
        out = {}
        for x in "qk":
            y, g = s[x].double(), s["gamma_" + x].double()
            if case["norm"] != "none":
                if case["norm"] == "layernorm":
                    y = (y - y.mean(-1, keepdim=True)) / torch.sqrt(y.var(-1, unbiased=False, keepdim=True) + 1e-6) * g
                else:
                    y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["dh"] + 1e-6) * g
                if s["beta_" + x] is not None:
                    y = y + s["beta_" + x].double()
            cs = s["rope"].double()[s["pos_" + x].long()]
            out[x] = _exact_rotation(y, cs[:, :rot], cs[:, rot:], case["style"])
        return out
    hk, dh, page, R = case["hk"], case["dh"], case["page"], case["R"]
    if case["op"] == "append":
        off, base = s["tok_off"][1], s["base"].cpu().numpy()
        slot = torch.from_numpy(np.concatenate([base[r] + np.arange(off[r + 1] - off[r]) for r in range(R)])).to(DEV)
        cs = s["rope"].double()[slot]
        out = {}
        for x in "kv":
            y = s[x].double()
            y = _exact_rotation(y, cs[:, :rot], cs[:, rot:], case["style"]) if x == "k" else y
            lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
            step, mn = ((hi - lo) / 15).bfloat16().double(), lo.bfloat16().double()
            code = torch.nan_to_num((y - mn) / step, nan=0.0, posinf=0.0, neginf=0.0).round().clamp(0, 15)
            out[x] = mn + step * code
        return out
    off, lens = s["cand_off"][1], s["lens"].cpu().numpy()
    q, h = case["q"], case["h"]
    n = int(off[-1]) * q
    o = torch.zeros(n, h, dh, dtype=torch.float64, device=DEV)
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device=DEV)
    for r in range(R):
        a, b, L = int(off[r]) * q, int(off[r + 1]) * q, int(lens[r])
        if a == b or L == 0:
            continue
        j = torch.arange(L, device=DEV)
        at = s["table"][r].long()[j // page]
        for head in range(h):
            kh = head // (h // hk)
            k = _exact_values(s["k_codes"][at, kh, j % page], s["k_scale"][at, kh, j % page])
            v = _exact_values(s["v_codes"][at, kh, j % page], s["v_scale"][at, kh, j % page])
            x = s["q"][a:b, head].double() @ k.T * s["scale"]
            if s["limit"] is not None:
                lim = s["limit"][a // q: b // q].repeat_interleave(q)
                x = x.masked_fill(j >= lim[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None])
            o[a:b, head], lse[a:b, head] = p @ v, z
    return {"o": o, "lse": lse}
