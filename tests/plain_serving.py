"""The operators around the paged cache written out in 64 bits on the CPU, for the tests."""
import math

import torch

QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "int8": torch.int8}
SCALE_LO, SCALE_HI = -50, 50


def values(codes):
    """Codes (a tensor of an 8-bit cache type) as the numbers they stand for, in units of the scale."""
    return codes.cpu().float().double()


def half_step(x, kind):
    """Half the distance between representable numbers around x, for codes in units of the scale."""
    if kind == "int8":
        return torch.full_like(x, 0.5)
    eps, low = {"e4m3": (2.0 ** -4, 2.0 ** -6), "e5m2": (2.0 ** -3, 2.0 ** -14)}[kind]
    return x.abs().clamp(min=low) * eps


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    x = x.double()
    d, r = x.shape[-1], cos_sin.shape[1]
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps) * weight.double()
    out = y.clone()
    cs = cos_sin.double()[positions]
    c, s = cs[:, None, : r // 2], cs[:, None, r // 2:]
    if interleaved:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., : r // 2], y[..., r // 2: r]
        out[..., : r // 2], out[..., r // 2: r] = a * c - b * s, b * c + a * s
    return out


def nearest_code(x, kind):
    """x (in units of the scale) rounded to the nearest code, ties to even, saturated; NaN stays (INT8: 0)."""
    q = QMAX[kind]
    nan = torch.isnan(x)
    y = torch.where(nan, torch.zeros_like(x), x).clamp(-q, q)
    if kind == "int8":
        return y.round()
    mant, low = (3, -6) if kind == "e4m3" else (2, -14)
    _, e = torch.frexp(y)                                   # |y| in [2^(e-1), 2^e)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), (e - 1).clamp(min=low).double() - mant)
    y = (y / step).round() * step
    return torch.where(nan, x, y)


def scale_for(absmax, kind):
    for e in range(SCALE_LO, SCALE_HI):
        if absmax <= QMAX[kind] * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** SCALE_HI


def append_block_scales(rows, codes, scales, table, lens, offsets, block, kind):
    """codes [blocks, heads, block, d] float64 in units of the scale, scales [blocks, heads] float64;
    both changed in place."""
    for s, L in enumerate(lens):
        a, b = offsets[s], offsets[s + 1]
        first = L - (b - a)
        if b == a:
            continue
        for j in range(first // block, (L - 1) // block + 1):
            lo, hi = max(0, first - j * block), min(block, L - j * block)
            p = int(table[s, j])
            for h in range(codes.shape[1]):
                x = rows[a + j * block + lo - first: a + j * block + hi - first, h].double()
                ok = x[torch.isfinite(x)]
                need = scale_for(float(ok.abs().max()) if ok.numel() else 0.0, kind)
                before = float(scales[p, h])
                after = max(need, before) if lo > 0 else need
                if lo > 0 and after > before:
                    codes[p, h, :lo] = nearest_code(codes[p, h, :lo] * before / after, kind)
                codes[p, h, lo:hi] = nearest_code(x / after, kind)
                scales[p, h] = after


def attend(q, k, v, scale):
    """softmax(scale q k^T) v and the same with |v|, for q [G, d], k and v [T, d] in float64."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
        return z, z
    p = torch.softmax(q @ k.T * scale, -1)
    return p @ v, p @ v.abs()


def decode(q, k, v, table, lens, scale, block, selected=None, ks=None, vs=None):
    """q [S, Hq, d]; k, v [blocks, heads, block, d] values in units of the scales; (out, its terms' size)."""
    S, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    q, k, v = q.cpu().double(), k.cpu().double(), v.cpu().double()
    out = torch.zeros(S, Hq, d, dtype=torch.float64)
    size = torch.zeros_like(out)
    for s, L in enumerate(lens):
        n = -(-L // block)
        for h in range(Hkv):
            js = range(n) if selected is None else [j for j in selected[s][h][:n] if 0 <= j < n]
            kk, vv = [], []
            for j in js:
                p, t = int(table[s, j]), min(block, L - j * block)
                fk = 1.0 if ks is None else float(ks[p, h])
                fv = 1.0 if vs is None else float(vs[p, h])
                kk.append(k[p, h, :t] * fk)
                vv.append(v[p, h, :t] * fv)
            kk = torch.cat(kk) if kk else torch.zeros(0, d, dtype=torch.float64)
            vv = torch.cat(vv) if vv else torch.zeros(0, d, dtype=torch.float64)
            o, a = attend(q[s, h * G:(h + 1) * G], kk, vv, scale)
            out[s, h * G:(h + 1) * G], size[s, h * G:(h + 1) * G] = o, a
    return out, size


def select(q, bounds, table, lens, block, keep, sink, recent):
    """Lists of lists [S][heads] of the kept blocks, -1 padded to `keep`."""
    S, Hq, d = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    q, bounds = q.cpu().double(), bounds.cpu().double()
    out = []
    for s, L in enumerate(lens):
        n = -(-L // block)
        row = []
        for h in range(Hkv):
            if n <= keep:
                row.append(list(range(n)) + [-1] * (keep - n))
                continue
            x = bounds[table[s, :n].long().clamp(min=0), h]                       # [n, 2, d]
            qq = q[s, h * G:(h + 1) * G]
            sc = torch.maximum(qq[:, None] * x[None, :, 0], qq[:, None] * x[None, :, 1]).sum(-1).amax(0)
            sc = torch.where(torch.isfinite(sc), sc, torch.full_like(sc, math.inf))
            sc = torch.where(table[s, :n].cpu() >= 0, sc, torch.full_like(sc, -math.inf))
            rank = [(0 if j < sink or j >= n - recent else 1, -float(sc[j]), j) for j in range(n)]
            row.append(sorted(j for _, _, j in sorted(rank)[:keep]))
        out.append(row)
    return out


def tables(lens, block, gen, spare=3):
    """Scattered block tables over a pool a little larger than needed: (table int32 [S, MB], pool size)."""
    n = [-(-L // block) for L in lens]
    pool = sum(n) + spare
    order = torch.randperm(pool, generator=gen).to(torch.int32)
    t = torch.full((len(lens), max(1, max(n, default=1)) + 1), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(n):
        t[s, :c] = order[at:at + c]
        at += c
    return t, pool
