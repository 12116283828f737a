"""The 8-bit pool, the weights and the eviction where values, scales or arguments are at their ends."""
import numpy as np
import pytest
import torch

import kv8_ref as R
import paged_kv_gqa_slot_gb300 as pa
from test_kv8 import NAN_CODE, Case, check, clean, make_pool

gpu = pytest.mark.gpu


# ----------------------------------------------------------------------------- V scales far apart in one row's walk
FAR = {  # exponent byte of V, block by block (repeated over the sequence)
    "large first": [127 + 30] * 4 + [27] * 4,
    "small first": [27] * 4 + [127 + 30] * 4,
    "both ends": [127 + 112] * 4 + [27] * 4 + [127 - 7] * 4,
    "both ends, small first": [27] * 4 + [127 + 112] * 4,
    "just over": [127 + 20] * 4 + [127 - 70] * 4,
}


def far_apart(c, how):
    for row, n in zip(c.tables_h, c.lens_h):
        for j in range((n + 15) // 16):
            e = FAR[how][j % len(FAR[how])]
            c.exps[row[j], :, 1] = e
            if e == 27:  # what the append stores for a block of zeros
                codes = c.v[row[j]]
                c.v[row[j]] = torch.where(codes & 0x7f == NAN_CODE, codes, torch.zeros_like(codes))


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("how", FAR)
def test_decode_v_scales_far_apart_in_one_warp(how, d):
    """Sequences of which one CTA walks all, several blocks a warp: the keys of a block count in the
    normaliser whatever the scale of its V beside the others'."""
    lens = [192, 250, 129] * 20 + [17]
    c = Case(81, lens, 16, 8, d, spread=0.0)
    far_apart(c, how)
    ref, spread, want, mag = c.reference()
    out = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    check(out, ref, spread, 250, mag)
    w = torch.zeros(len(lens), 8, c.tables.shape[1], device="cuda")
    out = pa.pa_decode8_weights(c.pool, c.q, c.tables, c.lens, c.scale, w)
    check(out, ref, spread, 250, mag)
    assert torch.allclose(w.sum(2).double(), torch.stack([x.sum(1) for x in want]), rtol=2.0 ** -11)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("how", FAR)
def test_decode_v_scales_far_apart_in_a_cluster(how, d):
    c = Case(82, [3000, 700], 14, 2, d, spread=0.0)
    far_apart(c, how)
    ref, spread, _, mag = c.reference()
    out = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    check(out, ref, spread, 3000, mag)
    clean()


@gpu
@pytest.mark.parametrize("chunks", [[64, 150], [4, 3]])
@pytest.mark.parametrize("how", FAR)
def test_prefill_v_scales_far_apart(how, chunks):
    for d in (64, 128):
        c = Case(83, [400, 333], 8, 2, d, chunks, spread=0.0)
        far_apart(c, how)
        ref, spread, _, mag = c.reference()
        out = pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, c.max_chunk)
        check(out, ref, spread, 400, mag)
    clean()


# ----------------------------------------------------------------------------- one dominant key with no value
def sink_case(seed, n, d, where, chunk, code):
    """Keys of ordinary scores and positive values, and one key (position `where`) that takes nearly all
    of every row's weight and has V = 0.  All scales are 2^-7, so its score is q_0 code / 128 * scale above 0."""
    c = Case(seed, [n], 8, 2, d, [chunk] if chunk else None, spread=0.0)
    c.exps[...] = 127 - 7
    c.q[..., 0] = 64.0
    c.k[..., 0] = 0                       # (the rows behind the end stay NaN in their other columns)
    blk, row = c.tables_h[0][where // 16], where % 16
    c.k[blk, :, row] = 0
    c.k[blk, :, row, 0] = torch.tensor([float(code)]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    used = torch.tensor(c.tables_h[0][:(n + 15) // 16], device="cuda")
    c.v[used] = torch.where(c.v[used] & 0x7f == NAN_CODE, c.v[used], c.v[used] & 0x7f)
    c.v[blk, :, row] = 0
    return c


def sink_check(c, out):
    """The bounds of test_kv8.tolerance, but with the flush counted where f16 has it.  A row's base lies at
    least 7 log2 units below its largest contribution, so a weight's u = p 2^7 / p_max or more, its rounding to f16
    is at most 2^-11 of it or, below 2^-14, half of f16's smallest step, 2^-25: in p at most 2^-32 a key, and the
    keys' |V| average at most V_mean."""
    ref, spread, _, mag = c.reference()
    n = c.lens_h[0]
    ids = torch.tensor(c.tables_h[0][:(n + 15) // 16], device="cuda")
    v = R.dequant(c.v, c.exps[..., 1])[ids].transpose(0, 1).reshape(2, -1, c.q.shape[2])[:, :n].abs().sum(1)  # [hkv, d]
    flush = 2.0 ** -32 * v.repeat_interleave(4, 0)[None]
    rel = 2.0 ** -11 + 2 * mag * 2.0 ** -19 + 2.0 ** -13
    tol = 2.0 ** -8 * ref.abs() + rel * spread + flush
    assert float((tol / ref.abs()).median()) < 0.015  # the sink leaves a result to speak of
    assert torch.isfinite(out.float()).all()
    assert bool(((out.double() - ref).abs() <= tol).all()), f"worst {float(((out.double() - ref).abs() / tol).max()):.2f} of the bound"


@gpu
@pytest.mark.parametrize("d,code", [(128, 352), (128, 384), (64, 256), (64, 240)])
@pytest.mark.parametrize("where", [0, 3, 2100, 4095])
def test_decode_with_a_sink(where, d, code):
    c = sink_case(91, 4096, d, where, 0, code)
    sink_check(c, pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale))
    # the same where one CTA walks the whole sequence
    many = 60 * 8
    tables, q, lens = c.tables.repeat(many, 1), c.q.repeat(many, 1, 1), c.lens.repeat(many)
    out = pa.pa_decode8(c.pool, q, tables, lens, c.scale)
    assert torch.equal(out, out[:1].expand_as(out))
    sink_check(c, out[:1])
    clean()


@gpu
@pytest.mark.parametrize("d,code", [(128, 352), (128, 384), (64, 256), (64, 240)])
@pytest.mark.parametrize("where,chunk", [(0, 100), (3, 300), (2100, 64), (3000, 4)])
def test_prefill_with_a_sink(where, chunk, d, code):
    c = sink_case(92, 4096, d, where, chunk, code)
    sink_check(c, pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, c.max_chunk))
    clean()
