"""64-bit references of the 8-bit pool, of the decode with weights and of the eviction.

Plain loops and numpy / torch float64, written from the header's definitions; no library code.
"""
from __future__ import annotations

import math

import numpy as np
import torch

BS = 16
E_MIN, E_MAX = -100, 119


def e4m3_values() -> np.ndarray:
    """The 256 values of e4m3 (1 sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f, 0xff NaN)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v[c] = math.nan if (c & 0x7f) == 0x7f else (-x if c & 0x80 else x)
    return v


VALUES = e4m3_values()
GRID = VALUES[:0x7f]  # 0 .. 448, rising with the code


def encode(x: np.ndarray) -> np.ndarray:
    """Codes of x rounded to the nearest e4m3, ties to the even code, saturating; NaN -> 0x7f."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(GRID, a), 0, 0x7e)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - GRID[lo], GRID[hi] - a
    pick = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    pick = np.where(np.isnan(x), 0x7f, pick)
    return (pick | np.where(np.signbit(x) & ~np.isnan(x), 0x80, 0)).astype(np.uint8)


def scale_exponent(amax: float) -> int:
    k = E_MIN
    while k < E_MAX and amax > math.ldexp(448.0, k):
        k += 1
    return k


def append(codes: np.ndarray, exps: np.ndarray, new: np.ndarray, slots) -> None:
    """One tensor (K or V): codes [nb, H, 16, D] uint8 and exps [nb, H] uint8 in place, new [T, H, D] float64."""
    blocks = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0] * BS:
            blocks.setdefault(s // BS, {})[s % BS] = t
    for blk, rows in blocks.items():
        for h in range(codes.shape[1]):
            x = {o: new[t, h] for o, t in rows.items()}
            amax = max((float(np.abs(r[np.isfinite(r)]).max(initial=0.0)) for r in x.values()), default=0.0)
            k = scale_exponent(amax)
            if 0 not in rows:
                k_old = int(exps[blk, h]) - 127
                if k > k_old:
                    for o in range(BS):
                        if o not in rows:
                            codes[blk, h, o] = encode(VALUES[codes[blk, h, o]] * 2.0 ** (k_old - k))
                k = max(k, k_old)
            for o, r in x.items():
                codes[blk, h, o] = encode(r * 2.0 ** -k)
            exps[blk, h] = k + 127


def dequant(codes: torch.Tensor, exps: torch.Tensor) -> torch.Tensor:
    """float64 values of codes [nb, H, 16, D] and exps [nb, H] (uint8 tensors)."""
    table = torch.tensor(VALUES, dtype=torch.float64, device=codes.device)
    return table[codes.long()] * torch.exp2(exps.double() - 127)[..., None, None]


def attention(q, k_pool, v_pool, tables, lens, scale, cu=None):
    """Causal attention of the last queries of every sequence in float64.

    q [rows, Hq, D]; k_pool, v_pool [nb, Hkv, 16, D]; cu [B + 1] (None: one query each).  Returns out,
    spread = sum_t p_t |V_t| (what a relative error of the weights is worth), per sequence
    the weights [Hkv, blocks] summed over the group's heads, the queries and each block's keys, and
    the largest log2(e) |scale| sum_d |q_d K_d| of a visible key (what a relative error of the
    scores' sums is worth).
    """
    dev = q.device
    q = q.double()
    rows, hq, d = q.shape
    hkv = k_pool.shape[1]
    g = hq // hkv
    out = torch.zeros(rows, hq, d, dtype=torch.float64, device=dev)
    spread = torch.zeros_like(out)
    weights, mag = [], 0.0
    for b, n in enumerate(lens):
        q0, q1 = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
        c = q1 - q0
        nb = (n + BS - 1) // BS
        if n == 0 or c == 0:
            weights.append(torch.zeros(hkv, nb, dtype=torch.float64, device=dev))
            continue
        ids = torch.tensor(tables[b][:nb], device=dev)
        k = k_pool[ids].double().transpose(0, 1).reshape(hkv, nb * BS, d)[:, :n]
        v = v_pool[ids].double().transpose(0, 1).reshape(hkv, nb * BS, d)[:, :n]
        qq = q[q0:q1].reshape(c, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * c, d)
        x = qq @ k.transpose(1, 2) * scale
        last = n - c + torch.arange(c, device=dev).repeat(g)
        x = x.masked_fill(torch.arange(n, device=dev)[None, None] > last[None, :, None], -math.inf)
        p = torch.softmax(x, dim=2)
        mag = max(mag, float((qq.abs() @ k.abs().transpose(1, 2)).amax()) * abs(scale) * math.log2(math.e))
        o, s = p @ v, p @ v.abs()
        out[q0:q1] = o.reshape(hkv, g, c, d).permute(2, 0, 1, 3).reshape(c, hq, d)
        spread[q0:q1] = s.reshape(hkv, g, c, d).permute(2, 0, 1, 3).reshape(c, hq, d)
        per = torch.nn.functional.pad(p.sum(1), (0, nb * BS - n)).view(hkv, nb, BS).sum(2)
        weights.append(per)
    return out, spread, weights, mag


def evict(tables, lens, weights, keep, sink, recent):
    """Lists in, lists out: tables [B][W], lens [B], weights [B][H][W] floats."""
    res = [], [], [], [], []
    for b, n in enumerate(lens):
        width, nb = len(tables[b]), (n + BS - 1) // BS
        gone = max(0, nb - keep)
        total = []
        for j in range(width):
            w = float(np.float32(math.fsum(weights[b][h][j] for h in range(len(weights[b])))))
            total.append(-math.inf if math.isnan(w) else w)
        out = set(sorted(range(sink, max(sink, nb - recent)), key=lambda j: (total[j], j))[:gone])
        kept = [j for j in range(width) if j not in out]
        res[0].append([tables[b][j] for j in kept] + [-1] * gone)
        res[1].append(n - BS * gone)
        res[2].append([[row[j] for j in kept] + [0.0] * gone for row in weights[b]])
        res[3].append([tables[b][j] for j in sorted(out)] + [-1] * (width - gone))
        res[4].append(gone)
    return res
