"""64-bit references of packed prompts, of the tables built on the GPU and of linear attention.

Plain loops and torch float64, written from the header's definitions; no library code.
"""
from __future__ import annotations

import math

import torch

BS = 16


def blocks(n: int) -> int:
    return (n + BS - 1) // BS


def packed_rows(lens, heads, kvh, d, seed, before=0, behind=0, strided=True, device="cuda"):
    """q, k, v [before + sum(lens) + behind, heads, d]: views of one fused tensor, or tensors of their own."""
    gen = torch.Generator(device=device).manual_seed(seed)
    rows = before + sum(lens) + behind
    if strided:
        qkv = torch.randn(rows, heads + 2 * kvh, d, device=device, generator=gen).bfloat16()
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kvh], qkv[:, heads + kvh:]
    else:
        q, k, v = (torch.randn(rows, h, d, device=device, generator=gen).bfloat16() for h in (heads, kvh, kvh))
    cu = [before]
    for n in lens:
        cu.append(cu[-1] + n)
    return q, k, v, torch.tensor(cu, dtype=torch.int32, device=device)


def packed(q, k, v, cu, scale):
    """(o, sum of the weights' |v|) per row, fp64; rows outside every sequence are NaN."""
    cu = cu.tolist()
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    size = out.clone()
    for a, b in zip(cu[:-1], cu[1:]):
        n = b - a
        seen = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        for h in range(heads):
            x, y, z = q[a:b, h].double(), k[a:b, h // group].double(), v[a:b, h // group].double()
            p = torch.softmax((x @ y.T * scale).masked_fill(~seen, -math.inf), 1)
            # a masked key has weight zero whatever its value
            mixed = lambda w: torch.where(seen[:, :, None], p[:, :, None] * w, 0.0).sum(1) if not bool(  # noqa: E731
                torch.isfinite(w).all()) else p @ w
            out[a:b, h] = mixed(z)
            size[a:b, h] = mixed(z.abs())
    return out, size


def packed_bound(ref, size):
    """Half a bf16 step of the result (2^-8 of it), and the weights as bf16 against their own sum: 2^-8 of
    sum w (|v| + |o|); 2^-12 for scores, exponentials and sums in fp32 (their errors are below 2^-14 for the
    sizes tested: |scores| up to 2^5, 2^-22 a step of the sums)."""
    return 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * (size + ref.abs()) + 1e-30


CHUNK = 128  # tokens that a prefill takes at a time: q reads the state that its chunk begins with


def linear(state, slots, q, k, v, log_decay, cu, lens, scale):
    """(o, its terms' size, new state, its terms' size), fp64; rows outside every sequence are NaN.
    A term of o is a score of its chunk times v, or an element of q times one of the state that the chunk
    begins with; a term of the state k times v, or what it was, with their decays."""
    kvh, d = k.shape[1], q.shape[2]
    group = q.shape[1] // kvh
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    size = out.clone()
    new = state.double().clone()
    new_size = state.double().abs().clone()
    la = log_decay.double().clamp(-1e4, 0.0)
    for b, (c0, c1) in enumerate(zip(cu[:-1], cu[1:])):
        n = c1 - c0
        if n == 0:
            continue
        if slots[b] < 0:
            out[c0:c1] = size[c0:c1] = 0.0
            continue
        i = torch.arange(n, device=q.device, dtype=torch.float64)
        apart = i[:, None] - i
        for h in range(kvh):
            a = la[h]
            x, y = k[c0:c1, h].double(), v[c0:c1, h].double()
            old = state[slots[b], h].double() if lens[b] > n else torch.zeros(d, d, dtype=torch.float64, device=q.device)
            far = torch.where(apart >= 0, torch.exp(a * apart.clamp(min=0)), torch.zeros_like(apart))
            lead = torch.exp(a * (i + 1))[:, None]
            rest = torch.exp(a * (n - 1 - i))[:, None]
            for hq in range(h * group, (h + 1) * group):
                z = q[c0:c1, hq].double()
                out[c0:c1, hq] = ((z @ x.T * far) @ y + lead * (z @ old)) * scale
                near = far * (i[:, None] // CHUNK == i // CHUNK)
                size[c0:c1, hq] = ((z @ x.T * near).abs() @ y.abs()) * abs(scale)
                begin = old
                for p in range(0, n, CHUNK):
                    e = min(p + CHUNK, n)
                    size[c0 + p:c0 + e, hq] += lead[:e - p] * (z[p:e].abs() @ begin.abs()) * abs(scale)
                    begin = torch.exp(a * (e - p)) * begin + (x[p:e] * rest[n - (e - p):]).T @ y[p:e]
            new[slots[b], h] = torch.exp(a * n) * old + (x * rest).T @ y
            new_size[slots[b], h] = torch.exp(a * n) * old.abs() + (x.abs() * rest).T @ y.abs()
    return out, size, new, new_size


def linear_bounds(ref, size, new_size, n, one_token=False):
    """Outputs: half a bf16 step of the result; the scores, and S where q reads it, as bf16 (2^-8 of every term)
    unless the call is for one token; the error that S itself has (below 2^-16 of sum a^.. |k| |v|, taken as 2^-12
    of the terms), and fp32 sums (each of n + 2 d additions up to 2^-22 of the terms' size).
    State: the decays' exponents, products of two fp32 numbers and up to 126 where the term does not vanish, 2^-16 of
    every term, and the sums."""
    sums = (n + 256) * 2.0 ** -22
    out = 2.0 ** -8 * ref.abs() + ((0 if one_token else 2.0 ** -8 + 2.0 ** -12) + sums) * size + 1e-30
    return out, ((0 if one_token else 2.0 ** -16) + sums) * new_size + 1e-30


def grow(tables, lens, new, free, have, max_tokens):
    """pa_kv_grow on lists; (tables, lens, blocks left, cu, slots, positions, token_seqs, bad)."""
    tables, lens = [list(r) for r in tables], list(lens)
    width = len(tables[0]) if tables else 0
    cu, slots, pos, seqs, bad = [0], [], [], [], False
    have = min(max(have, 0), len(free))
    left, asked_blocks, asked_rows = have, 0, 0
    for b in range(len(lens)):
        n, m = lens[b], new[b]
        if n < 0 or m < 0 or n + m > width * BS:
            bad = True
            cu.append(cu[-1])
            continue
        need = blocks(n + m) - blocks(n)
        asked_blocks += need
        asked_rows += m
        if (need == 0 or asked_blocks <= have) and asked_rows <= max_tokens:
            for j in range(blocks(n), blocks(n + m)):
                left -= 1
                tables[b][j] = free[left]
            for p in range(n, n + m):
                slots.append(tables[b][p // BS] * BS + p % BS)
                pos.append(p)
                seqs.append(b)
            lens[b] += m
        cu.append(len(slots))
    more = max_tokens - len(slots)
    return tables, lens, left, cu, slots + [-1] * more, pos + [0] * more, seqs + [-1] * more, bad


def give_back(ids, counts, free, have):
    """pa_kv_free on lists; (free list, blocks free, bad)."""
    free = list(free)
    at = min(max(have, 0), len(free))
    bad = at != have
    width = len(ids[0]) if ids else 0
    for row, c in zip(ids, counts):
        bad |= not 0 <= c <= width
        for x in row[:min(max(c, 0), width)]:
            if x >= 0:
                if at < len(free):
                    free[at] = x
                    at += 1
                else:
                    bad = True
    return free, at, bad
