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
    """The bounds of test_kv8.tolerance, but with the flush counted where f16 has it.  The dominant
    key stands alone, so a row's base lies at least 7 log2 units below its contribution, and a weight's u = p 2^7 / p_max or more, its rounding to f16
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


# ----------------------------------------------------------------------------- NaN among the scores
@gpu
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_nan_in_a_query_row(d, many):
    """A NaN in q makes the result of that (sequence, head) NaN, adds nothing to the weights, and concerns no other."""
    lens = [40, 700, 17, 3, 0] * (30 if many else 1)
    c = Case(101, lens, 16, 4, d)
    ref, spread, want, mag = c.reference()
    q = c.q.clone()
    bad = [(0, 0, 5), (1, 7, d - 1), (2, 15, 0), (3, 4, 9)]
    for b, h, i in bad:
        q[b, h, i] = float("nan")
    w = torch.zeros(len(lens), 4, c.tables.shape[1], device="cuda")
    out8 = pa.pa_decode8(c.pool, q, c.tables, c.lens, c.scale)
    out = pa.pa_decode8_weights(c.pool, q, c.tables, c.lens, c.scale, w)
    k, v = R.dequant(c.k, c.exps[..., 0]), R.dequant(c.v, c.exps[..., 1])
    w16 = torch.zeros_like(w)
    out16 = pa.pa_decode_weights(pa.PaPool(k.to(torch.bfloat16), v.to(torch.bfloat16)), q, c.tables, c.lens, c.scale, w16)
    for o in (out8, out, out16):
        for b, h, _ in bad:
            assert torch.isnan(o[b, h]).all()
            o[b, h] = ref[b, h].to(o.dtype)
        check(o, ref, spread, 700, mag)
    heads = torch.full((len(lens), 4), 4.0, device="cuda")
    for b, h, _ in bad:
        heads[b, h // 4] -= 1
    heads[[b for b, n in enumerate(lens) if n == 0]] = 0
    for got in (w, w16):
        assert torch.allclose(got.sum(2), heads, rtol=2.0 ** -11)
    clean()


@gpu
@pytest.mark.parametrize("n", [17, 33, 700 * 16 + 1])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_nan_in_a_key_that_is_alone_in_its_block(d, n):
    """The last block holds one key, whose K has a NaN: every head of its kv head sees it, whichever warp and
    split the block falls to.  Its weights get the decay and nothing else."""
    c = Case(102, [n, 50], 8, 2, d)
    ref, spread, want, mag = c.reference()
    c.k[c.tables_h[0][n // 16], 1, 0, 3] = NAN_CODE
    w0 = torch.rand(2, 2, c.tables.shape[1], device="cuda")
    w = w0.clone()
    out8 = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    out = pa.pa_decode8_weights(c.pool, c.q, c.tables, c.lens, c.scale, w, 0.5)
    for o in (out8, out):
        assert torch.isnan(o[0, 4:]).all()
        o[0, 4:] = ref[0, 4:].to(o.dtype)
        check(o, ref, spread, n, mag)
    nb = (n + 15) // 16
    assert torch.equal(w[0, 1, :nb], w0[0, 1, :nb] * 0.5) and torch.isfinite(w).all()
    assert torch.allclose(w[0, 0, :nb].double(), w0[0, 0, :nb].double() * 0.5 + want[0][0], rtol=2.0 ** -11)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_short_prefill_nan_in_a_query_row(d):
    c = Case(103, [100, 3, 700], 8, 2, d, [4, 1, 3])
    ref, spread, _, mag = c.reference()
    q = c.q.clone()
    bad = [(0, 1), (2, 7), (4, 0), (7, 5)]
    for r, h in bad:
        q[r, h, 11] = float("nan")
    out = pa.pa_prefill_chunked8(c.pool, q, c.cu, c.tables, c.lens, c.scale, c.max_chunk)
    for r, h in bad:
        assert torch.isnan(out[r, h]).all()
        out[r, h] = ref[r, h].to(out.dtype)
    check(out, ref, spread, 700, mag)
    clean()


# ----------------------------------------------------------------------------- NaN in the V of a later key
@gpu
@pytest.mark.parametrize("cached,chunks,hq,hkv", [
    ([100, 0], [40, 300], 8, 2), ([16, 770], [17, 129], 32, 8), ([5, 60], [200, 31], 6, 2), ([0, 31], [130, 64], 2, 2),
    ([700, 0] * 4, [130, 257] * 4, 64, 8),          # two tiles a CTA
    ([100, 0, 31], [4, 4, 2], 16, 4), ([29, 1000], [8, 5], 4, 2),  # the short form
])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_nan_in_later_values_stays_with_those_that_see_it(d, cached, chunks, hq, hkv):
    """V's NaN at a position reaches exactly the queries at or past it, in its column."""
    lens = [a + b for a, b in zip(cached, chunks)]
    c = Case(111, lens, hq, hkv, d, chunks)
    ref, spread, _, mag = c.reference()
    rng = np.random.RandomState(7)
    g = hq // hkv
    nan = torch.zeros(c.q.shape, dtype=torch.bool, device="cuda")
    for b, (n, m) in enumerate(zip(lens, chunks)):
        for i in range(3):
            pos = n - 1 - int(rng.randint(0, m)) if i else n - 1
            h, col = int(rng.randint(hkv)), slice(None) if i == 1 else slice(int(rng.randint(d)), None, 37)
            codes = c.v[c.tables_h[b][pos // 16], h, pos % 16]
            codes[col] = NAN_CODE if i else 0xff
            nan[c.cu_h[b] + pos - (n - m):c.cu_h[b + 1], h * g:(h + 1) * g, col] = True
    out = pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, c.max_chunk)
    assert torch.equal(torch.isnan(out), nan)
    out[nan] = ref[nan].to(out.dtype)
    check(out, ref, spread, max(lens), mag)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("chunks", [[40, 300], [4, 2]])
def test_prefill_nan_in_cached_values_reaches_every_query(d, chunks):
    c = Case(112, [360, 500], 8, 2, d, chunks)
    ref, spread, _, mag = c.reference()
    for pos in (0, 100, 200 - 1):
        c.v[c.tables_h[1][pos // 16], 1, pos % 16, 5] = NAN_CODE
    out = pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, c.max_chunk)
    rows = slice(c.cu_h[1], c.cu_h[2])
    assert torch.isnan(out[rows, 4:, 5]).all()
    out[rows, 4:, 5] = ref[rows, 4:, 5].to(out.dtype)
    check(out, ref, spread, 500, mag)
    clean()


# ----------------------------------------------------------------------------- exponent bytes outside the range
@gpu
@pytest.mark.parametrize("byte,size", [(255, 2.0 ** 120), (247, 2.0 ** 121), (0, 2.0 ** -92), (20, 2.0 ** -95), (0, 0.0)])
def test_append_takes_an_exponent_as_it_is_read(byte, size):
    """Rows behind offset 0 of a block whose exponent byte is outside 27 .. 246: the append goes by the
    nearer end, as the reading calls do, for the codes that stay and for the new ones."""
    hkv, d = 2, 64
    k, v, exps = make_pool(121, 3, hkv, d)
    exps[:] = byte
    pool = pa.PaPool8(k, v, exps)
    kh, vh = k.cpu().numpy(), v.cpu().numpy()
    eh = np.clip(exps.cpu().numpy(), 27, 246)
    gen = torch.Generator().manual_seed(5)
    new = [(torch.randn(3, hkv, d, generator=gen) * size).to(torch.bfloat16) for _ in range(2)]
    slots = [5, 6, 16 + 9]
    pa.pa_kv_append8(pool, new[0].cuda(), new[1].cuda(), torch.tensor(slots, device="cuda"))
    for i, codes in enumerate((kh, vh)):
        R.append(codes, eh[:, :, i], new[i].double().numpy(), slots)
    got = exps.cpu().numpy()
    assert np.array_equal(got[:2], eh[:2]) and (got[2] == byte).all()
    for g, w in ((k, kh), (v, vh)):
        assert np.array_equal(R.VALUES[g.cpu().numpy()], R.VALUES[w], equal_nan=True)
    clean()


# ----------------------------------------------------------------------------- sums of the eviction
@gpu
@pytest.mark.parametrize("width", [12, 600, 30000])
def test_evict_sums_at_a_rounding_border(width):
    """W is the fp64 sum rounded once: 1 + 2^-24 + 2^-49 lies just above the middle of two fp32 numbers and
    counts as the upper one, 1 + 2^-24 as the lower; sums whose terms cancel keep fp64's remainder."""
    w = np.full((1, 3, width), 9.0, np.float32)
    w[0, :, 3] = 1.0, 2.0 ** -24, 2.0 ** -49       # 1 + 2^-23
    w[0, :, 5] = 1.0, 0.0, 0.0                     # 1: the lowest of these
    w[0, :, 6] = 1.0, 2.0 ** -24, 0.0              # 1 again (to even)
    w[0, :, 7] = 2.0 ** -24, 1.0, -(2.0 ** -49)    # 1 again (below the middle)
    w[0, :, 8] = 2.0 ** 40, 2.0 ** -20, -(2.0 ** 40)  # 0 in fp64, 2^-20 in exact arithmetic
    w[0, :, 9] = 2.0 ** 40, 2.0 ** -10, -(2.0 ** 40)  # 2^-10
    tables = np.arange(width, dtype=np.int32)[None]
    order = [8, 9, 5, 6, 7, 3]
    for e in range(1, 7):
        t, _, _, evicted, num = pa.pa_kv_evict(*(torch.tensor(x, device="cuda") for x in (tables, np.array([width * 16], np.int32), w)),
                                               width - e, 0, 1)
        assert num.tolist() == [e] and evicted[0, :e].tolist() == sorted(order[:e]), e
    clean()


@gpu
def test_evict_many_heads_of_mixed_signs():
    rng = np.random.RandomState(8)
    b, h, width = 3, 70, 300
    w = (rng.randn(b, h, width) * np.exp2(rng.uniform(-30, 30, size=(b, h, width)))).astype(np.float32)
    lens = [width * 16, width * 16 - 5, 2000]
    tables = rng.permutation(b * width).reshape(b, width).astype(np.int32)
    total = np.zeros((b, width))
    for i in range(h):
        total = total + w[:, i].astype(np.float64)
    one = total.astype(np.float32)[:, None]        # the same ranking from sums that need no rounding
    got = pa.pa_kv_evict(*(torch.tensor(x, device="cuda") for x in (tables, np.array(lens, np.int32), w)), 100, 2, 3)
    want = R.evict(tables.tolist(), lens, one.tolist(), 100, 2, 3)
    assert got[0].tolist() == want[0] and got[3].tolist() == want[3]
    clean()


# ----------------------------------------------------------------------------- tables of no width
@gpu
def test_decode_with_weights_over_tables_of_no_width_is_refused():
    """As the decode without weights: there is no row to read, and no result to give."""
    c = Case(131, [40, 50], 8, 2, 128)
    none = c.tables[:, :0].contiguous()
    w = torch.zeros(2, 2, 0, device="cuda")
    bf16 = pa.PaPool(torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(pa.PagedAttnError):
        pa.pa_decode8(c.pool, c.q, none, c.lens, c.scale)
    for call, pool in ((pa.pa_decode8_weights, c.pool), (pa.pa_decode_weights, bf16)):
        with pytest.raises(pa.PagedAttnError):
            call(pool, c.q, none, c.lens, c.scale, w)
        with pytest.raises(pa.PagedAttnError):
            call(pool, c.q, none, c.lens, c.scale, w, stream=torch.cuda.current_stream())
        assert call(pool, c.q[:0], none[:0], c.lens[:0], c.scale, w[:0]).shape == (0, 8, 128)


# ----------------------------------------------------------------------------- weights under large V scales
@gpu
@pytest.mark.parametrize("lens", [[300, 1000], [300, 250] * 30])  # a cluster a sequence; one CTA, five blocks a warp
@pytest.mark.parametrize("byte", [27, 127 - 7, 127 + 100, 246])
def test_weights_do_not_depend_on_the_scale_of_v(byte, lens):
    """Blocks of very different weight, V at any scale: the weights follow K alone."""
    for d in (64, 128):
        c = Case(141, lens, 16, 8, d, scale=1.2, spread=0.0)
        c.exps[..., 1] = byte
        if byte == 246:  # 448 * 2^119 is the end of the range; keep the sums inside it
            c.v[:] = torch.where(c.v & 0x7f == NAN_CODE, c.v, c.v & 0x9f)
        ref, spread, want, mag = c.reference()
        w = torch.zeros(len(lens), 8, c.tables.shape[1], device="cuda")
        out = pa.pa_decode8_weights(c.pool, c.q, c.tables, c.lens, c.scale, w)
        check(out, ref, spread, max(lens), mag)
        least = 1.0
        rel = 2 * mag * 2.0 ** -19 + 2.0 ** -13
        for b, n in enumerate(lens):
            nb = (n + 15) // 16
            big = want[b] > 2.0 ** -60
            least = min(least, float(want[b][big].min()))
            assert bool(((w[b, :, :nb].double() - want[b]).abs()[big] <= rel * want[b][big]).all())
        assert least < 2.0 ** -16
        clean()
