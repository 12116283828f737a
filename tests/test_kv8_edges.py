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
