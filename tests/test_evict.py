"""Decode with accumulated block weights, eviction, and the block manager's side of it."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv8_ref as R
import paged_kv_gqa_slot_gb300 as pa
from paged_kv_gqa_slot_gb300 import build as pbuild
from test_kv8 import Case, _pool8, check, clean

gpu = pytest.mark.gpu
FAKE = 0x40000


# ----------------------------------------------------------------------------- without a GPU
@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.library()


def test_refusals_before_any_launch(lib):
    bad, unsup = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    pool = ctypes.byref(pa._PaPoolC(0x10000, 0x20000, 16, 16, 2, 128))
    for fn, p in ((lib.pa_decode_weights, pool), (lib.pa_decode8_weights, _pool8())):
        call = lambda w=FAKE, ws=FAKE, decay=1.0, h=4, b=1: fn(p, FAKE, FAKE, 4, FAKE, b, h, 0.1, decay, w, ws, FAKE, None)  # noqa: E731
        assert call(w=None) == bad and call(ws=None) == bad and call(w=FAKE + 2) == bad
        assert call(decay=math.nan) == bad and call(h=3) == bad and call(h=64) == unsup and call(b=0) == pa.PA_OK
    ev = lambda b=1, mb=8, h=2, keep=4, sink=1, recent=1, bt=FAKE, out=FAKE: lib.pa_kv_evict(  # noqa: E731
        bt, FAKE, FAKE, b, mb, h, keep, sink, recent, out, FAKE, FAKE, FAKE, FAKE, None)
    assert ev(bt=None) == bad and ev(out=None) == bad and ev(bt=FAKE + 1) == bad
    assert ev(b=-1) == bad and ev(mb=0) == bad and ev(h=0) == bad and ev(sink=-1) == bad and ev(recent=0) == bad
    assert ev(keep=1) == bad and ev(mb=50000) == unsup and ev(b=0) == pa.PA_OK
    assert pa.pa_weights_workspace_bytes(3, 32, 8, 10) == 3 * 8 * 10 * 8 * 4
    assert pa.pa_weights_workspace_bytes(3, 72, 8, 10) == 3 * 8 * 10 * 16 * 4
    assert pa.pa_weights_workspace_bytes(-1, 32, 8, 10) == 0


def test_block_manager_evict_returns_blocks_and_shortens_the_request(lib):
    bm = pa.BlockManager(16, prefix_cache=False)
    table, _ = bm.admit(1, list(range(70)), 26)  # 96 tokens: 6 blocks
    assert bm.stats()[0] == 10
    bm.evict(1, [int(table[1]), int(table[3]), -1, -1])
    assert bm.stats() == (12, 0, 4)
    left = [int(table[i]) for i in (0, 2, 4, 5)]
    slots = bm.slots(1, 0, 64)
    assert [int(s) // 16 for s in slots[::16]] == left
    with pytest.raises(pa.PagedAttnError):
        bm.slots(1, 60, 5)          # the lifetime is 64 tokens now
    bm.commit(1, list(range(26)), 64)
    with pytest.raises(pa.PagedAttnError):
        bm.commit(1, [1], 64)       # and it is full
    bm.release(1)
    assert bm.stats() == (16, 0, 0)


def test_block_manager_evict_refuses_what_the_request_does_not_hold(lib):
    bm = pa.BlockManager(8, prefix_cache=False)
    table, _ = bm.admit(1, list(range(40)), 24)  # 2 full blocks, one half, one reserved
    other, _ = bm.admit(2, list(range(16)), 0)
    for ids in ([int(other[0])], [int(table[2])], [int(table[3])], [int(table[1]), int(table[0])],
                [int(table[0]), int(table[0])]):
        with pytest.raises(pa.PagedAttnError):
            bm.evict(1, ids)
    with pytest.raises(pa.PagedAttnError):
        bm.evict(9, [int(table[0])])
    assert bm.stats()[2] == 5
    bm.evict(1, [])
    assert [int(s) // 16 for s in bm.slots(1, 0, 64)[::16]] == [int(t) for t in table]


def test_block_manager_evict_keeps_the_prefix_cache_sound(lib):
    bm = pa.BlockManager(16)
    prompt = list(range(64)) + [7]
    table, cached = bm.admit(1, prompt, 31)
    assert cached == 0
    bm.commit(1, [], 65)
    _, cached = bm.admit(2, prompt, 15)
    assert cached == 64                                   # shares four blocks
    bm.evict(1, [int(table[1]), int(table[2])])
    bm.commit(1, list(range(100, 131)), 64)               # what follows saw part of the prompt only
    again, cached = bm.admit(3, prompt, 15)
    assert cached == 64 and [int(t) for t in again[:4]] == [int(t) for t in table[:4]]
    bm.release(2)
    bm.release(3)
    bm.release(1)
    free, idle, used = bm.stats()
    assert used == 0 and idle == 4                        # only the prompt's own blocks are cached


# ----------------------------------------------------------------------------- decode with weights
WEIGHTS = [  # seed, lens, q heads, kv heads, d
    (1, [1, 0, 17, 48], 8, 2, 128),
    (2, [700, 33], 12, 4, 64),
    (3, [500, 16, 90], 32, 2, 128),
    (4, [6000], 16, 2, 128),
    (5, [1000 + 97 * i for i in range(40)], 8, 4, 64),
    (6, [80, 200], 22, 2, 64),
    (7, [1152, 1030], 32, 8, 128),
]


def weights_close(got, before, want, decay, lens, mag):
    for b, n in enumerate(lens):
        nb = (n + 15) // 16
        # a weight moves by mag * 2^-19 (its score's fp32 sum, as in the outputs' tolerance), the
        # normaliser too, and by less than 2^-13 (ex2, log2 and the sums)
        rel = 2 * mag * 2.0 ** -19 + 2.0 ** -13
        ref = before[b, :, :nb].double() * decay + want[b]
        err = (got[b, :, :nb].double() - ref).abs() - (rel * want[b] + 2.0 ** -22 * ref + 1e-30)
        assert (err <= 0).all(), f"sequence {b}: worst by {float(err.max()):.3e}"
        assert torch.equal(got[b, :, nb:], before[b, :, nb:]), "entries past the sequence stay"


@gpu
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_decode_weights(case, bits):
    seed, lens, hq, hkv, d = WEIGHTS[case]
    c = Case(seed, lens, hq, hkv, d)
    k, v = R.dequant(c.k, c.exps[..., 0]), R.dequant(c.v, c.exps[..., 1])
    if bits == 16:  # the same values as a bf16 pool, NaN where the codes are NaN
        pool = pa.PaPool(k.to(torch.bfloat16), v.to(torch.bfloat16))
        call = pa.pa_decode_weights
    else:
        pool, call = c.pool, pa.pa_decode8_weights
    ref, spread, want, mag = c.reference()
    w0 = torch.rand(len(lens), hkv, c.tables.shape[1], device="cuda")
    w = w0.clone()
    out = call(pool, c.q, c.tables, c.lens, c.scale, w, 0.75)
    check(out, ref, spread, max(lens), mag)
    weights_close(w, w0, want, 0.75, lens, mag)
    w2 = w0.clone()
    out2 = call(pool, c.q, c.tables, c.lens, c.scale, w2, 0.75,
                workspace=torch.full((pa.pa_weights_workspace_bytes(len(lens), hq, hkv, c.tables.shape[1]) // 4,), float("nan"), device="cuda"))
    assert torch.equal(w, w2) and torch.equal(out, out2), "the same call gives the same bits"
    if bits == 8:
        assert torch.equal(out, pa.pa_decode8(pool, c.q, c.tables, c.lens, c.scale))
    clean()


@gpu
def test_decode_weights_argument_checks():
    c = Case(9, [40, 50], 8, 2, 128)
    w = torch.zeros(2, 2, c.tables.shape[1], device="cuda")
    with pytest.raises(ValueError):
        pa.pa_decode8_weights(c.pool, c.q, c.tables, c.lens, c.scale, w[:, :1])
    with pytest.raises(ValueError):
        pa.pa_decode8_weights(c.pool, c.q, c.tables, c.lens, c.scale, w.double())
    with pytest.raises(ValueError):
        pa.pa_decode8_weights(c.pool, c.q, c.tables, c.lens, c.scale, w, workspace=torch.empty(3, device="cuda"))
    with pytest.raises(ValueError):
        pa.pa_decode8_weights(c.pool, c.q[:, :, :64], c.tables, c.lens, c.scale, w)
    with pytest.raises(pa.PagedAttnError):
        pa.pa_decode8_weights(c.pool, c.q, c.tables, c.lens, c.scale, w, decay=float("nan"))


# ----------------------------------------------------------------------------- eviction
def run_evict(tables, lens, w, keep, sink, recent, in_place=False):
    args = (torch.tensor(tables, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            torch.tensor(w, dtype=torch.float32, device="cuda"))
    got = pa.pa_kv_evict(*args, keep, sink, recent, in_place=in_place)
    if in_place:
        assert all(a is b for a, b in zip(got, args))
    return [t.cpu().numpy() for t in got]


EVICTS = [  # seed, batch, kv heads, width, longest, keep, sink, recent
    (1, 3, 2, 12, 180, 4, 1, 1),
    (2, 5, 1, 9, 144, 9, 0, 1),
    (3, 4, 8, 80, 1270, 64, 1, 4),
    (4, 2, 8, 2050, 32768, 1536, 4, 64),
    (5, 3, 3, 700, 11200, 5, 2, 3),
    (6, 2, 9, 600, 9600, 599, 0, 1),
    (7, 1, 1, 1, 16, 1, 0, 1),
    (8, 6, 4, 513, 8208, 100, 10, 20),
]


@gpu
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(EVICTS)))
def test_evict(case, in_place, ties):
    seed, batch, hkv, width, longest, keep, sink, recent = EVICTS[case]
    rng = np.random.RandomState(seed)
    lens = [longest] + [int(rng.randint(0, longest + 1)) for _ in range(batch - 1)]
    tables = rng.permutation(batch * width).reshape(batch, width).astype(np.int32)
    w = np.exp(2 * rng.randn(batch, hkv, width)).astype(np.float32)
    if ties:
        w = np.floor(np.minimum(w, 3)).astype(np.float32) * np.where(rng.rand(batch, hkv, width) < 0.1, -0.0, 1).astype(np.float32)
    got = run_evict(tables, lens, w, keep, sink, recent, in_place)
    want = R.evict(tables.tolist(), lens, w.tolist(), keep, sink, recent)
    for name, g, r in zip(("tables", "lens", "weights", "evicted", "count"), got, want):
        assert np.array_equal(g, np.array(r, dtype=g.dtype)), name
    clean()


@gpu
def test_evict_special_weights():
    w = np.ones((1, 2, 10), np.float32)
    w[0, :, 2] = math.inf
    w[0, 1, 5] = math.nan           # counts as the lowest
    w[0, :, 7] = -3.0
    w[0, :, 3] = 1e-45              # subnormal, above zero
    tables = np.arange(10, dtype=np.int32)[None]
    for keep in (9, 8, 7, 6, 3):
        got = run_evict(tables, [160], w, keep, 0, 1)
        want = R.evict(tables.tolist(), [160], w.tolist(), keep, 0, 1)
        assert got[0].tolist() == want[0] and got[3].tolist() == want[3], keep
        assert np.array_equal(got[2], np.array(want[2], np.float32), equal_nan=True)
    assert run_evict(tables, [160], w, 9, 0, 1)[3][0, 0] == 5
    clean()


@gpu
def test_evict_reports_lengths_past_the_table():
    w = np.ones((3, 1, 4), np.float32)
    tables = np.arange(12, dtype=np.int32).reshape(3, 4)
    got = run_evict(tables, [65, -1, 20], w, 2, 0, 1)
    assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    assert got[1].tolist() == [32, 0, 20] and got[4].tolist() == [2, 0, 0]


@gpu
def test_evict_argument_checks():
    t = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 3, 4, device="cuda")
    for args in ((t[:, :3], n, w), (t, n[:1], w), (t, n, w[:1]), (t.long(), n, w), (t, n, w.half()), (t, n, w[0])):
        with pytest.raises(ValueError):
            pa.pa_kv_evict(*args, 2)
    with pytest.raises(pa.PagedAttnError):
        pa.pa_kv_evict(t, n, w, 2, 1, 2)


# ----------------------------------------------------------------------------- as they are used
@gpu
@pytest.mark.parametrize("bits", [8, 16])
def test_serving_with_a_block_budget(bits):
    """Two requests under one block manager decode with weights; whenever one passes its budget the
    lowest blocks leave the device tables (in place) and go back to the manager.  Every step's
    output is checked in float64 on what the tables hold, and the manager's slots stay in step."""
    hkv, g, d, nb, keep = 2, 4, 128, 40, 6
    bm = pa.BlockManager(nb, prefix_cache=False)
    rng = np.random.RandomState(4)
    if bits == 8:
        pool, append, decode = pa.PaPool8.zeros(nb, hkv, d), pa.pa_kv_append8, pa.pa_decode8_weights
    else:
        zeros = lambda: torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        pool, append, decode = pa.PaPool(zeros(), zeros()), pa.pa_kv_append, pa.pa_decode_weights
    lens = [60, 90]
    width = 12
    rows = []
    for r, n in enumerate(lens):
        table, _ = bm.admit(r, rng.randint(0, 1000, n).tolist(), width * 16 - n)
        rows.append(table)
    tables = torch.tensor(np.stack(rows), device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    weights = torch.zeros(2, hkv, width, device="cuda")

    def fresh(n):
        return torch.tensor(rng.randn(n, hkv, d), dtype=torch.float32).to(torch.bfloat16).cuda()

    for r, n in enumerate(lens):
        append(pool, fresh(n), fresh(n), torch.tensor(bm.slots(r, 0, n), device="cuda"))
    dropped = 0
    for step in range(50):
        now = seq.tolist()
        slots = [int(bm.slots(r, n, 1)[0]) for r, n in enumerate(now)]
        append(pool, fresh(2), fresh(2), torch.tensor(slots, device="cuda"))
        for r, n in enumerate(now):
            bm.commit(r, [step], n + 1)
        seq += 1
        q = torch.tensor(rng.randn(2, hkv * g, d), dtype=torch.float32).to(torch.bfloat16).cuda()
        before = weights.clone()
        out = decode(pool, q, tables, seq, d ** -0.5, weights, 0.9)
        if bits == 8:
            k, v = R.dequant(pool.k_cache, pool.exps[..., 0]), R.dequant(pool.v_cache, pool.exps[..., 1])
        else:
            k, v = pool.k_cache.double(), pool.v_cache.double()
        now = seq.tolist()
        ref, spread, want, mag = R.attention(q, k, v, tables.tolist(), now, d ** -0.5)
        check(out, ref, spread, max(now), mag)
        weights_close(weights, before, want, 0.9, now, mag)
        args = (tables.tolist(), now, weights.tolist(), keep, 1, 2)
        expect = R.evict(*args)
        _, _, _, evicted, num = pa.pa_kv_evict(tables, seq, weights, keep, 1, 2, in_place=True)
        assert tables.tolist() == expect[0] and seq.tolist() == expect[1] and evicted.tolist() == expect[3]
        for r, count in enumerate(num.tolist()):
            if count:
                bm.evict(r, evicted[r].tolist())
                dropped += count
    # a sequence loses a block each time it reaches 97 tokens: once from 60, three times from 90
    assert dropped == 4 and bm.stats()[2] == 2 * width - dropped
    for r in range(2):
        bm.release(r)
    assert bm.stats()[0] == nb
    clean()


@gpu
def test_weights_and_eviction_in_a_graph():
    c = Case(12, [600, 200], 8, 2, 128)
    w = torch.zeros(2, 2, c.tables.shape[1], device="cuda")
    ws = torch.empty(pa.pa_weights_workspace_bytes(2, 8, 2, c.tables.shape[1]) // 4, device="cuda")
    out = torch.empty_like(c.q)
    tables, lens = c.tables.clone(), c.lens.clone()
    pa.pa_decode8_weights(c.pool, c.q, tables, lens, c.scale, w, 1.0, workspace=ws, out=out)
    pa.pa_kv_evict(tables, lens, w, 20, 1, 1)
    graph = torch.cuda.CUDAGraph()
    w.zero_()
    with torch.cuda.graph(graph):
        pa.pa_decode8_weights(c.pool, c.q, tables, lens, c.scale, w, 1.0, workspace=ws, out=out)
        _, _, _, evicted, num = pa.pa_kv_evict(tables, lens, w, 20, 1, 1, in_place=True)
    graph.replay()
    graph.replay()  # the second finds the shortened sequences
    w2 = torch.zeros_like(w)
    t2, l2 = c.tables.clone(), c.lens.clone()
    for _ in range(2):
        o2 = pa.pa_decode8_weights(c.pool, c.q, t2, l2, c.scale, w2, 1.0)
        _, _, _, e2, n2 = pa.pa_kv_evict(t2, l2, w2, 20, 1, 1, in_place=True)
    for a, b in ((out, o2), (w, w2), (tables, t2), (lens, l2), (evicted, e2), (num, n2)):
        assert torch.equal(a, b)
    assert lens.tolist()[0] == 600 - 18 * 16
    clean()
