"""The 8-bit pool: quantising append, decode, chunked prefill, and their refusals."""
import ctypes

import numpy as np
import pytest
import torch

import kv8_ref as R
import paged_kv_gqa_slot_gb300 as pa
from paged_kv_gqa_slot_gb300 import build as pbuild

gpu = pytest.mark.gpu
FAKE = 0x40000
NAN_CODE = 0x7f


# ----------------------------------------------------------------------------- without a GPU
@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.library()


def _pool8(nb=16, bs=16, hkv=2, d=128, k=0x10000, v=0x20000, e=0x30000):
    return ctypes.byref(pa._PaPool8C(k, v, e, nb, bs, hkv, d))


def test_header_and_binding_agree_on_the_new_symbols(lib):
    for name in ("pa_kv_append8", "pa_decode8", "pa_prefill_chunked8", "pa_decode_weights", "pa_decode8_weights",
                 "pa_weights_workspace_bytes", "pa_kv_evict", "pa_bm_evict"):
        assert hasattr(lib, name) and name in pa.EXPORTED_SYMBOLS


def test_refusals_before_any_launch(lib):
    bad, unsup = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    dec = lambda pool, q=FAKE, bt=FAKE, mb=4, sl=FAKE, b=1, h=4, s=0.1, o=FAKE: lib.pa_decode8(  # noqa: E731
        pool, q, bt, mb, sl, b, h, s, o, None)
    for pool in (None, _pool8(k=0), _pool8(v=0), _pool8(e=0), _pool8(k=0x10008), _pool8(e=0x30001), _pool8(nb=0),
                 _pool8(hkv=0)):
        assert dec(pool) == bad
        assert lib.pa_kv_append8(pool, FAKE, FAKE, FAKE, 1, None) == bad
        assert lib.pa_prefill_chunked8(pool, FAKE, FAKE, FAKE, 4, FAKE, 1, 4, 8, 0.1, FAKE, None) == bad
    for pool in (_pool8(bs=8), _pool8(d=96)):
        assert dec(pool) == unsup
    ok = _pool8()
    assert dec(ok, h=5) == bad and dec(ok, h=0) == bad and dec(ok, h=64) == unsup
    assert dec(ok, q=FAKE + 2) == bad and dec(ok, o=None) == bad and dec(ok, mb=0) == bad and dec(ok, b=-1) == bad
    assert dec(ok, b=70000) == bad and dec(ok, s=float("inf")) == bad and dec(ok, b=0) == pa.PA_OK
    assert lib.pa_kv_append8(ok, FAKE, FAKE, None, 3, None) == bad
    assert lib.pa_kv_append8(ok, FAKE, FAKE + 8, FAKE, 3, None) == bad
    assert lib.pa_kv_append8(ok, FAKE, FAKE, FAKE, -1, None) == bad
    assert lib.pa_kv_append8(ok, None, None, None, 0, None) == pa.PA_OK
    pre = lambda cu=FAKE, mc=16: lib.pa_prefill_chunked8(ok, FAKE, cu, FAKE, 4, FAKE, 1, 4, mc, 0.1, FAKE, None)  # noqa: E731
    assert pre(cu=None) == bad and pre(mc=-1) == bad and pre(mc=1 << 30) == bad and pre(mc=0) == pa.PA_OK


def test_cpu_tensors_and_shapes_are_refused():
    codes = torch.zeros(2, 1, 16, 64, dtype=torch.uint8)
    exps = torch.zeros(2, 1, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pa.PaPool8(codes, codes, exps)  # not on a GPU
    with pytest.raises(ValueError):
        pa.PaPool8(codes, codes[:1], exps)
    with pytest.raises(ValueError):
        pa.PaPool8(codes.float(), codes.float(), exps)
    with pytest.raises(ValueError):
        pa.PaPool8(codes, codes, exps[:, :, :1])


def test_reference_rounding_is_nearest_even():
    # every code is its own rounding, and every midpoint of neighbours goes to the even code
    assert np.array_equal(R.encode(R.GRID), np.arange(0x7f))
    mid = (R.GRID[1:] + R.GRID[:-1]) / 2
    got = R.encode(mid)
    assert np.all(got % 2 == 0) and np.all(np.abs(got.astype(int) - np.arange(0x7e) - 0.5) == 0.5)
    assert R.encode(np.array([1e9, -np.inf, np.nan])).tolist() == [0x7e, 0xfe, 0x7f]
    for a in (1.0, 448.0, 448.5, 1e-3, 2.0 ** 127):
        k = R.scale_exponent(a)
        assert a <= 448 * 2.0 ** k and (k == R.E_MIN or a > 448 * 2.0 ** (k - 1)) or k == R.E_MAX


# ----------------------------------------------------------------------------- helpers
def make_pool(seed, nb, hkv, d, spread=2.0):
    """Codes and exponents of a pool whose blocks differ in size; values up to a few 2^spread."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pools = []
    for _ in range(2):
        x = torch.randn(nb, hkv, 16, d, generator=gen, device="cuda")
        c = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        e = torch.randn(nb, hkv, generator=gen, device="cuda") * spread
        pools.append((c, (e.round() - 7 + 127).to(torch.uint8)))  # 100 * 2^-7 is about 0.8
    exps = torch.stack([pools[0][1], pools[1][1]], -1).contiguous()
    return pools[0][0], pools[1][0], exps


class Case:
    """Sequences over a shuffled 8-bit pool; NaN codes behind every sequence's end and in every unused
    block, garbage behind the tables' used entries."""

    def __init__(self, seed, lens, hq, hkv, d, chunks=None, scale=None, spread=2.0, extra_width=2):
        rng = np.random.RandomState(seed)
        need = [(n + 15) // 16 for n in lens]
        nb = sum(need) + 5
        self.k, self.v, self.exps = make_pool(seed, nb, hkv, d, spread)
        perm = rng.permutation(nb)
        width = max(need + [1]) + extra_width
        tables = np.full((len(lens), width), -7, dtype=np.int32)
        at = 0
        for b, m in enumerate(need):
            tables[b, :m] = perm[at:at + m]
            at += m
            if lens[b] % 16:
                for pool in (self.k, self.v):
                    pool[int(tables[b, m - 1]), :, lens[b] % 16:] = NAN_CODE
        for blk in perm[at:]:
            self.k[int(blk)] = NAN_CODE
            self.v[int(blk)] = NAN_CODE
            self.exps[int(blk)] = 255
        self.tables_h, self.lens_h = tables.tolist(), list(lens)
        self.tables = torch.tensor(tables, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu_h = None
        rows = len(lens)
        if chunks is not None:
            self.cu_h = [0] + np.cumsum(chunks).tolist()
            self.cu = torch.tensor(self.cu_h, dtype=torch.int32, device="cuda")
            self.max_chunk = max(chunks)
            rows = self.cu_h[-1]
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.q = torch.randn(rows, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
        self.scale = d ** -0.5 if scale is None else scale
        self.pool = pa.PaPool8(self.k, self.v, self.exps)

    def reference(self):
        k, v = R.dequant(self.k, self.exps[..., 0]), R.dequant(self.v, self.exps[..., 1])
        return R.attention(self.q, k, v, self.tables_h, self.lens_h, self.scale, self.cu_h)


def tolerance(ref, spread, lens_max, mag):
    """Per element.  The result's rounding to bf16: 2^-8 |o|.  Each weight's rounding to f16: 2^-11.  The
    scores: products are exact, the fp32 sum over d loses at most 8 MMA steps x 2^-22 of the sum of
    magnitudes, `mag` in log2 units, so a weight moves by less than mag * 2^-19 of itself, in numerator
    and normaliser; ex2, the sum over the keys and the merge add less than 2^-13.  f16 flushes weights
    below 2^-25 of the largest contribution (at most every key's)."""
    rel = 2.0 ** -11 + 2 * mag * 2.0 ** -19 + 2.0 ** -13
    return 2.0 ** -8 * ref.abs() + rel * spread + lens_max * 2.0 ** -25 * spread.amax(-1, keepdim=True) + 1e-30


def check(out, ref, spread, lens_max, mag):
    assert torch.isfinite(out.float()).all()
    err = (out.double() - ref).abs() - tolerance(ref, spread, lens_max, mag)
    assert (err <= 0).all(), f"{int((err > 0).sum())} elements past the bound, worst by {float(err.max()):.3e}"


def clean():
    assert pa.pa_device_status(clear=True) == 0


# ----------------------------------------------------------------------------- append
APPENDS = [  # seed, kv heads, d, slot lists (one per call)
    (1, 2, 128, [[0, 1, 2, 3], [4], [5, 6]]),
    (2, 3, 64, [list(range(32, 64)), [64], [65]]),
    (3, 1, 128, [[3, 4, 5, -1, 6], [16 + 15], [-1, -1], [7]]),
    (4, 8, 128, [[16 * b + o for b, o in enumerate([0, 1, 7, 15, 8, 0])]]),
    (5, 4, 64, [list(range(5, 150)), list(range(150, 170))]),
    (6, 2, 128, [[33, 32, 35, 34], [40, 40, 41]]),       # any order in a block, the last of equal slots
    (7, 8, 128, [[16 * 20 + i for i in range(333)]]),     # many windows
    (8, 2, 128, [[5] + [-1] * 70 + [6] + [-1] * 40 + [200]]),  # padding between the rows of a block
]


@gpu
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_is_exact(case):
    seed, hkv, d, calls = APPENDS[case]
    nb = 48
    k, v, exps = make_pool(seed, nb, hkv, d)
    pool = pa.PaPool8(k, v, exps)
    kh, vh, eh = k.cpu().numpy(), v.cpu().numpy(), exps.cpu().numpy().copy()
    rng = np.random.RandomState(seed)
    for n, slots in enumerate(calls):
        size = np.exp2(rng.uniform(-6, 6, size=(len(slots), hkv, 1)))
        new = [torch.tensor(rng.randn(len(slots), hkv, d) * size, dtype=torch.float32).to(torch.bfloat16) for _ in range(2)]
        pa.pa_kv_append8(pool, new[0].cuda(), new[1].cuda(), torch.tensor(slots, device="cuda"))
        for i, codes in enumerate((kh, vh)):
            R.append(codes, eh[:, :, i], new[i].double().numpy(), slots)
        assert np.array_equal(exps.cpu().numpy(), eh), f"call {n}: exponents"
        for got, want in ((k, kh), (v, vh)):
            assert np.array_equal(R.VALUES[got.cpu().numpy()], R.VALUES[want], equal_nan=True), f"call {n}: codes"
    clean()


@gpu
@pytest.mark.parametrize("hkv,d,rows", [(8, 128, 9900), (16, 64, 5100)])
def test_append_of_many_rows_is_exact(hkv, d, rows):
    """More units than the few-unit form takes: several sequences, the first of each ending inside a block,
    padding between them."""
    seed, nb = 9, rows // 16 + 8
    k, v, exps = make_pool(seed, nb, hkv, d)
    pool = pa.PaPool8(k, v, exps)
    kh, vh, eh = k.cpu().numpy(), v.cpu().numpy(), exps.cpu().numpy().copy()
    rng = np.random.RandomState(seed)
    perm, slots = rng.permutation(nb), []
    for i in range(4):
        blocks = perm[i * (nb // 4):(i + 1) * (nb // 4)]
        line = [int(b) * 16 + o for b in blocks for o in range(16)][3 + 2 * i:]
        slots += line[:rows // 4 - 5 * i] + [-1] * (5 * i)
    new = [torch.tensor(rng.randn(len(slots), hkv, d) * np.exp2(rng.uniform(-6, 6, size=(len(slots), hkv, 1))),
                        dtype=torch.float32).to(torch.bfloat16) for _ in range(2)]
    pa.pa_kv_append8(pool, new[0].cuda(), new[1].cuda(), torch.tensor(slots, device="cuda"))
    for i, codes in enumerate((kh, vh)):
        R.append(codes, eh[:, :, i], new[i].double().numpy(), slots)
    assert np.array_equal(exps.cpu().numpy(), eh)
    for got, want in ((k, kh), (v, vh)):
        assert np.array_equal(R.VALUES[got.cpu().numpy()], R.VALUES[want], equal_nan=True)
    clean()


@gpu
def test_append_special_values():
    pool = pa.PaPool8.zeros(4, 1, 64)
    x = torch.zeros(7, 1, 64)
    x[0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 3.0])
    x[1] = 0.0                                   # an all-zero row
    x[2, 0, 0], x[2, 0, 1] = 3.3e38, -1.0         # past 448 * 2^119: saturates
    x[3, 0, 0] = 2.0 ** -130                     # below every scale
    x[4, 0, 0] = 448.0
    x[5, 0, 0] = 450.0                           # one bf16 step past 448 * 2^0
    x[6, 0, :2] = torch.tensor([1.0, -0.0])
    x = x.to(torch.bfloat16)
    slots = [0, 16, 17, 32, 48, 49, 50]
    kh = np.zeros((4, 1, 16, 64), np.uint8)
    eh = np.zeros((4, 1, 2), np.uint8)
    pa.pa_kv_append8(pool, x.cuda(), x.cuda(), torch.tensor(slots, device="cuda"))
    R.append(kh, eh[:, :, 0], x.double().numpy(), slots)
    assert np.array_equal(pool.exps.cpu().numpy()[..., 0], eh[..., 0])
    assert np.array_equal(pool.exps.cpu().numpy()[..., 1], eh[..., 0])
    assert np.array_equal(R.VALUES[pool.k_cache.cpu().numpy()], R.VALUES[kh], equal_nan=True)
    clean()


@gpu
def test_append_skips_and_reports_slots_past_the_pool():
    pool = pa.PaPool8.zeros(2, 2, 128)
    new = torch.ones(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pa.pa_kv_append8(pool, new, new, torch.tensor([0, 32, 1 << 40, 1], device="cuda"))
    assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    got = R.dequant(pool.k_cache, pool.exps[..., 0])
    assert (got[0, :, :2] == 1).all() and (got[0, :, 2:] == 0).all() and (got[1] == 0).all()


@gpu
def test_append_empty_and_argument_checks():
    pool = pa.PaPool8.zeros(2, 2, 128)
    none = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    pa.pa_kv_append8(pool, none, none, torch.empty(0, dtype=torch.int64, device="cuda"))
    one = torch.ones(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        pa.pa_kv_append8(pool, one, one, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        pa.pa_kv_append8(pool, one.float(), one, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        pa.pa_kv_append8(pool, one[:, :1], one, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        pa.pa_kv_append8(pool, one.cpu(), one, torch.zeros(1, dtype=torch.int64, device="cuda"))
    clean()


# ----------------------------------------------------------------------------- decode
DECODES = [  # seed, lens, q heads, kv heads, d
    (11, [1], 4, 1, 64),
    (12, [0, 1, 15, 16, 17, 0], 8, 2, 128),
    (13, [37, 64, 65, 200], 8, 8, 128),
    (14, [33, 500, 7], 12, 4, 64),        # group 3
    (15, [1000, 3, 129], 14, 2, 128),     # group 7
    (16, [90, 300], 32, 2, 128),          # group 16: two column tiles
    (17, [90, 300, 1], 22, 2, 64),        # group 11
    (18, [1152], 32, 8, 128),
    (19, [5000], 16, 2, 128),             # long, split over a cluster
    (20, [300 + 7 * i for i in range(40)], 8, 4, 64),   # one CTA a sequence
    (21, [2000 + 131 * i for i in range(20)], 8, 8, 64),  # more than 32 blocks a warp, one CTA
    (22, [2048, 4096 - 15, 2049] * 13, 16, 4, 128),
]


@gpu
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_decode(case):
    seed, lens, hq, hkv, d = DECODES[case]
    c = Case(seed, lens, hq, hkv, d)
    out = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    ref, spread, _, mag = c.reference()
    check(out, ref, spread, max(lens), mag)
    again = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale, out=torch.empty_like(out))
    assert torch.equal(out, again), "the same call gives the same bits"
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_decode_blocks_of_very_different_size(d):
    """Scales 2^-40 .. 2^40 from block to block, a block of zeros at the smallest scale, tiny and huge q."""
    c = Case(31, [160, 640, 20], 8, 2, d, spread=0.0)
    rng = np.random.RandomState(3)
    c.exps[..., 1] = torch.tensor(127 + rng.randint(-40, 41, size=tuple(c.exps.shape[:2])), dtype=torch.uint8, device="cuda")
    zero = c.tables_h[0][2]
    c.v[zero] = 0
    c.exps[zero, :, 1] = 27
    c.q[0] *= 2.0 ** -60
    c.exps[c.tables_h[1][:40], :, 0] = 127 - 7 - 60
    c.q[1] = (c.q[1].float() * 2.0 ** 60).to(torch.bfloat16)
    ref, spread, _, mag = c.reference()
    out = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    check(out, ref, spread, 640, mag)
    clean()


@gpu
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_decode_scales(scale):
    c = Case(32, [40, 333], 8, 2, 128, scale=scale, spread=0.5)
    ref, spread, _, mag = c.reference()
    out = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    check(out, ref, spread, 333, mag)
    clean()


@gpu
def test_decode_reports_bad_blocks_and_lengths():
    c = Case(33, [100, 100, 100], 8, 2, 128)
    ref, spread, _, mag = c.reference()
    c.tables[0, 2] = -1
    c.tables[1, 0] = 10 ** 6
    c.lens[1] = -5
    out = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    check(out[2:], ref[2:], spread[2:], 100, mag)
    assert (out[1] == 0).all()


@gpu
def test_decode_nan_in_a_valid_row_reaches_only_its_sequence_and_head():
    c = Case(34, [50, 60], 4, 2, 128)
    ref, spread, _, mag = c.reference()
    c.v[c.tables_h[0][1], 1, 3, 5] = NAN_CODE
    out = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    assert torch.isnan(out[0, 2:, 5]).all()
    out[0, 2:, 5] = ref[0, 2:, 5].to(torch.bfloat16)
    check(out, ref, spread, 60, mag)
    clean()


# ----------------------------------------------------------------------------- prefill
PREFILLS = [  # seed, cached lengths, chunks, q heads, kv heads, d
    (41, [0], [1], 4, 1, 64),
    (42, [0, 16, 5], [16, 1, 40], 8, 2, 128),
    (43, [0, 100, 768], [300, 0, 129], 32, 8, 128),
    (44, [30, 0, 77], [65, 200, 3], 12, 4, 64),         # group 3
    (45, [17, 600], [150, 90], 14, 2, 128),             # group 7
    (46, [20, 0], [33, 260], 48, 2, 128),               # group 24
    (47, [2500], [20], 16, 2, 128),                     # more than 32 blocks, several score rings
    (48, [1023, 1, 0, 64], [64, 63, 1, 128], 2, 2, 64),  # group 1
    (49, [100, 0, 1000], [4, 1, 3], 16, 4, 128),        # short chunks: the decode form, 16 columns
    (50, [100, 0, 40], [2, 2, 0], 6, 2, 64),            # 6 columns
    (51, [700] * 6, [130] * 6, 64, 8, 128),
]


@gpu
@pytest.mark.parametrize("case", range(len(PREFILLS)))
def test_prefill(case):
    seed, cached, chunks, hq, hkv, d = PREFILLS[case]
    lens = [a + b for a, b in zip(cached, chunks)]
    c = Case(seed, lens, hq, hkv, d, chunks)
    out = pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, c.max_chunk)
    ref, spread, _, mag = c.reference()
    check(out, ref, spread, max(lens), mag)
    clean()


@gpu
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.5])
def test_prefill_scales(scale):
    c = Case(52, [400, 90], 8, 2, 128, [120, 90], scale=scale, spread=0.5)
    ref, spread, _, mag = c.reference()
    out = pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, 120)
    check(out, ref, spread, 400, mag)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_rising_scores_move_the_base(d):
    """Keys whose scores grow along the sequence, stage after stage, so O is rescaled again and again;
    V of very different size."""
    c = Case(53, [640], 8, 1, d, [64], spread=0.0)
    ids = c.tables_h[0][:40]
    c.k[ids] = c.k[ids[0]].clone()[None]  # every block the same codes, under growing scales
    c.exps[ids, 0, 0] = torch.tensor([127 - 11 + i // 5 for i in range(40)], dtype=torch.uint8, device="cuda")
    c.exps[ids, 0, 1] = torch.tensor([127 - 7 + (i * 7) % 23 - 11 for i in range(40)], dtype=torch.uint8, device="cuda")
    ref, spread, _, mag = c.reference()
    out = pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, 64)
    check(out, ref, spread, 640, mag)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_rows_of_any_size_and_with_nan(d):
    """Rows of q down to 2^-100, zero rows, and rows with a NaN or an infinity, which concern their own
    (query, head) alone."""
    c = Case(56, [300, 70], 6, 2, d, [150, 70])
    size = torch.exp2(torch.randint(-100, 3, c.q.shape[:2], device="cuda").float())
    c.q = (c.q.float() * size[..., None]).to(torch.bfloat16)
    c.q[5, 1] = 0
    c.q[7, 2] *= -0.0
    ref, spread, _, mag = c.reference()
    q = c.q.clone()
    bad = [(3, 0, 5, float("nan")), (149, 5, d - 1, float("inf")), (150, 2, 0, float("-inf")), (219, 4, 17, float("nan"))]
    for r, h, i, x in bad:
        q[r, h, i] = x
    out = pa.pa_prefill_chunked8(c.pool, q, c.cu, c.tables, c.lens, c.scale, c.max_chunk)
    for r, h, i, x in bad:
        if x != x:
            assert torch.isnan(out[r, h]).all()
        out[r, h] = ref[r, h].to(out.dtype)
    check(out, ref, spread, 300, mag)
    clean()


@gpu
def test_prefill_many_rounds_back_to_back():
    """Several CTAs an SM one after another, tiles of one CTA with different stage counts, and launches that
    start before the one before them has ended."""
    c = Case(57, [500, 1030, 64, 777, 0, 130] * 4, 32, 8, 128, [70, 130, 64, 1, 0, 129] * 4)
    ref, spread, _, mag = c.reference()
    outs = [torch.full_like(c.q, 7.0) for _ in range(4)]
    for out in outs:
        pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, c.max_chunk, out=out)
    for out in outs:
        check(out, ref, spread, 1030, mag)
    clean()


@gpu
def test_prefill_reports_and_skips():
    c = Case(54, [200, 300, 90], 8, 2, 128, [50, 60, 70])
    ref, spread, _, mag = c.reference()
    c.lens[0] = 20                       # shorter than its chunk
    c.tables[1, 4] = 1 << 30             # outside the pool
    out = torch.full_like(c.q, 7.0)
    pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, 70, out=out)
    assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    assert (out[:50] == 7.0).all()       # the skipped sequence's rows stay as they were
    check(out[110:], ref[110:], spread[110:], 90, mag)
    # a chunk longer than max_chunk: covered rows are right, the others stay
    c = Case(55, [200, 90], 8, 2, 128, [150, 40])
    ref, spread, _, mag = c.reference()
    out = torch.full_like(c.q, 7.0)
    pa.pa_prefill_chunked8(c.pool, c.q, c.cu, c.tables, c.lens, c.scale, 40, out=out)
    assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    check(out[150:], ref[150:], spread[150:], 200, mag)


# ----------------------------------------------------------------------------- as they are used
@gpu
def test_rows_behind_the_batch_and_unused_blocks_stay():
    c = Case(61, [40, 100], 8, 2, 128, [20, 30])
    before = [t.clone() for t in (c.k, c.v, c.exps)]
    out = torch.full((60, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    q = torch.cat([c.q, torch.full((10, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    pa.pa_prefill_chunked8(c.pool, q, c.cu, c.tables, c.lens, c.scale, 30, out=out)
    assert (out[50:] == 5.0).all()
    assert all(torch.equal(a, b) for a, b in zip(before, (c.k, c.v, c.exps)))
    clean()


@gpu
def test_graph_capture_and_another_stream():
    c = Case(62, [700, 90], 8, 2, 128)
    ref, spread, _, mag = c.reference()
    out = torch.empty_like(c.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale, out=out, stream=side)
    fresh = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale, stream=side.cuda_stream)
    side.synchronize()
    check(out, ref, spread, 700, mag)
    assert torch.equal(out, fresh)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale, out=out)
    c.lens[0] = 333  # the replay reads the tensors as they are then
    out.zero_()
    graph.replay()
    want = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    assert torch.equal(out, want)
    clean()


@gpu
def test_append_then_prefill_then_decode_follow_a_growing_sequence():
    """A prompt in two chunks, then single tokens: every step's output against float64 on the pool as
    the reference append leaves it."""
    hkv, g, d, nb = 2, 4, 128, 24
    pool = pa.PaPool8.zeros(nb, hkv, d)
    kh = np.zeros((nb, hkv, 16, d), np.uint8)
    vh, eh = kh.copy(), np.zeros((nb, hkv, 2), np.uint8)
    rng = np.random.RandomState(9)
    table = rng.permutation(nb).astype(np.int32)
    tables = torch.tensor(table[None], device="cuda")
    n = 0
    for c in (150, 37, 1, 1, 1, 1, 1, 1):
        pos = np.arange(n, n + c)
        slots = (table[pos // 16].astype(np.int64) * 16 + pos % 16).tolist()
        new = [torch.tensor(rng.randn(c, hkv, d) * 2.0 ** rng.uniform(-2, 2), dtype=torch.float32).to(torch.bfloat16) for _ in range(2)]
        pa.pa_kv_append8(pool, new[0].cuda(), new[1].cuda(), torch.tensor(slots, device="cuda"))
        R.append(kh, eh[:, :, 0], new[0].double().numpy(), slots)
        R.append(vh, eh[:, :, 1], new[1].double().numpy(), slots)
        n += c
        q = torch.tensor(rng.randn(c, hkv * g, d), dtype=torch.float32).to(torch.bfloat16).cuda()
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        if c > 1:
            cu = torch.tensor([0, c], dtype=torch.int32, device="cuda")
            out = pa.pa_prefill_chunked8(pool, q, cu, tables, lens, d ** -0.5, c)
        else:
            out = pa.pa_decode8(pool, q, tables, lens, d ** -0.5)
        k = R.dequant(torch.tensor(kh).cuda(), torch.tensor(eh[:, :, 0]).cuda())
        v = R.dequant(torch.tensor(vh).cuda(), torch.tensor(eh[:, :, 1]).cuda())
        ref, spread, _, mag = R.attention(q, k, v, [table.tolist()], [n], d ** -0.5, [0, c])
        check(out, ref, spread, n, mag)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("how", ["k first", "v first", "one tensor", "same tensor"])
def test_any_placement_of_the_two_pools(how, d):
    """K and V of a block come by one copy over the distance of the pools, or by two where the pools are one."""
    c = Case(71, [333, 50, 16], 8, 2, d)
    nb = c.k.shape[0]
    both = torch.empty(2 * nb + 3, *c.k.shape[1:], dtype=torch.uint8, device="cuda")
    if how == "k first":
        k, v = both[:nb], both[nb + 3:]
    elif how == "v first":
        k, v = both[nb + 1:2 * nb + 1], both[:nb]
    elif how == "one tensor":
        k, v = both[:2 * nb].view(2, nb, *c.k.shape[1:]).unbind(0)
    else:
        k = v = both[:nb]
    k.copy_(c.k)
    if how == "same tensor":
        c.k, c.v = k, k
    else:
        v.copy_(c.v)
    c.pool = pa.PaPool8(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), c.exps)
    ref, spread, _, mag = c.reference()
    check(pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale), ref, spread, 333, mag)
    clean()


@gpu
def test_offsets_past_4_gb():
    """Blocks whose codes lie more than 2^32 bytes into the pools."""
    hkv, d, lens = 8, 128, [100, 777]
    nb = (1 << 32) // (hkv * 16 * d) + 64
    c = Case(72, lens, 16, hkv, d, [20, 17])
    far = np.random.RandomState(1).permutation(64)[:c.k.shape[0]] + nb - 64
    far_t = torch.tensor(far, device="cuda")
    k, v = (torch.empty(nb, hkv, 16, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    exps = torch.zeros(nb, hkv, 2, dtype=torch.uint8, device="cuda")
    used = len(far)
    k[far_t], v[far_t], exps[far_t] = c.k[:used], c.v[:used], c.exps[:used]
    remap = {old: int(far[old]) for old in range(used)}
    tables = [[remap.get(x, -7) if x >= 0 else x for x in row] for row in c.tables_h]
    c.tables = torch.tensor(tables, dtype=torch.int32, device="cuda")
    ref, spread, _, mag = c.reference()
    pool = pa.PaPool8(k, v, exps)
    out = pa.pa_prefill_chunked8(pool, c.q, c.cu, c.tables, c.lens, c.scale, c.max_chunk)
    check(out, ref, spread, 777, mag)
    last = torch.stack([c.q[19], c.q[36]])
    out = pa.pa_decode8(pool, last, c.tables, c.lens, c.scale)
    check(out, ref[[19, 36]], spread[[19, 36]], 777, mag)
    new = torch.randn(3, hkv, d, device="cuda").to(torch.bfloat16)
    blk = int(far[0])
    pa.pa_kv_append8(pool, new, new, torch.tensor([blk * 16, blk * 16 + 1, blk * 16 + 2], device="cuda"))
    kh, eh = np.zeros((1, hkv, 16, d), np.uint8), np.zeros((1, hkv, 1), np.uint8)
    R.append(kh, eh[:, :, 0], new.double().cpu().numpy(), [0, 1, 2])
    assert np.array_equal(R.VALUES[k[blk, :, :3].cpu().numpy()], R.VALUES[kh[0, :, :3]])
    assert np.array_equal(exps[blk, :, 0].cpu().numpy(), eh[0, :, 0])
    clean()


@gpu
def test_blocks_of_a_zeroed_pool_that_were_never_written():
    """A sequence over two written blocks and two of zeros (exponent byte 0) beside them."""
    hkv, d, nb = 2, 128, 8
    pool = pa.PaPool8.zeros(nb, hkv, d)
    new = torch.randn(32, hkv, d, device="cuda").to(torch.bfloat16)
    pa.pa_kv_append8(pool, new, new, torch.arange(16, 48, device="cuda"))
    tables = torch.tensor([[0, 1, 2, 5], [4, 3, 0, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([64, 30], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 8, d, device="cuda").to(torch.bfloat16)
    k, v = R.dequant(pool.k_cache, pool.exps[..., 0]), R.dequant(pool.v_cache, pool.exps[..., 1])
    ref, spread, _, mag = R.attention(q, k, v, tables.tolist(), [64, 30], d ** -0.5)
    out = pa.pa_decode8(pool, q, tables, lens, d ** -0.5)
    check(out, ref, spread, 64, mag)
    assert (out[1] == 0).all()
    cu = torch.tensor([0, 17, 47], dtype=torch.int32, device="cuda")
    q = torch.randn(47, 8, d, device="cuda").to(torch.bfloat16)
    ref, spread, _, mag = R.attention(q, k, v, tables.tolist(), [64, 30], d ** -0.5, [0, 17, 47])
    out = pa.pa_prefill_chunked8(pool, q, cu, tables, lens, d ** -0.5, 30)
    check(out, ref, spread, 64, mag)
    clean()


@gpu
def test_other_streams_handles_and_devices():
    c = Case(73, [100, 20], 8, 2, 128)
    want = pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale)
    torch.cuda.synchronize()
    assert torch.equal(pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale, stream=0), want)  # the legacy default stream
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q.cpu(), c.tables, c.lens, c.scale)
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q, c.tables.cpu(), c.lens, c.scale)
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q, c.tables, c.lens, c.scale, out=want[:1])
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q.transpose(0, 1).contiguous().transpose(0, 1), c.tables, c.lens, c.scale)
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q, c.tables[:1], c.lens, c.scale)
    with pytest.raises(ValueError):
        pa.pa_prefill_chunked8(c.pool, c.q, c.lens, c.tables, c.lens, c.scale, 1)
    clean()
