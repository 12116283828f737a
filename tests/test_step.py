"""Tables, lengths and slots built on the GPU, blocks given back, and a hybrid stack's step as a whole."""
import math
import random

import pytest
import torch

import paged_kv_gqa_slot_gb300 as pa
import step_ref as R
from paged_kv_gqa_slot_gb300 import build as pbuild
from test_linear import within
from test_packed import check, clean

gpu = pytest.mark.gpu
FAKE = 0x40000


# ----------------------------------------------------------------------------- without a GPU
@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.library()


def test_refusals_before_any_launch(lib):
    bad, unsup = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    grow = lambda bt=FAKE, mb=8, sl=FAKE, nl=FAKE, b=3, fr=FAKE, cap=9, nf=FAKE, mt=64, lo=FAKE, no=FAKE, cu=FAKE, sm=FAKE, ps=FAKE, ts=FAKE: (  # noqa: E731,E501
        lib.pa_kv_grow(bt, mb, sl, nl, b, fr, cap, nf, mt, lo, no, cu, sm, ps, ts, None))
    for name in ("bt", "sl", "nl", "fr", "nf", "lo", "no", "cu", "sm", "ps", "ts"):
        assert grow(**{name: None}) == bad, name
        assert grow(**{name: FAKE + 1}) == bad, name
    assert grow(sm=FAKE + 4) == bad
    assert grow(mb=0) == bad and grow(mb=1 << 28) == bad and grow(b=-1) == bad and grow(b=65536) == bad
    assert grow(cap=-1) == bad and grow(mt=-1) == bad
    free = lambda ids=FAKE, c=FAKE, r=3, w=8, fr=FAKE, cap=9, nf=FAKE, no=FAKE: lib.pa_kv_free(ids, c, r, w, fr, cap, nf, no, None)  # noqa: E731,E501
    for name in ("ids", "c", "fr", "nf", "no"):
        assert free(**{name: None}) == bad, name
        assert free(**{name: FAKE + 2}) == bad, name
    assert free(r=-1) == bad and free(w=-1) == bad and free(cap=-1) == bad and free(w=1 << 22) == unsup


def test_binding_refuses_shapes():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for args in ((i(3, 4), i(3), i(3), i(9), i(1)), (i(3), i(3), i(3), i(9), i(1)), (i(3, 4), i(2), i(3), i(9), i(1)),
                 (i(3, 4), i(3), i(3), i(9), i(2))):
        with pytest.raises(ValueError):
            pa.pa_kv_grow(*args, 64)
    for args in ((i(3, 4), i(3), i(9), i(1)), (i(3, 4), i(4), i(9), i(1)), (i(3, 4), i(3), i(9), i(2))):
        with pytest.raises(ValueError):
            pa.pa_kv_free(*args)


# ----------------------------------------------------------------------------- tables
def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


GROW = {
    "one": ([0], [1], 4, 5, 5, 64),
    "nothing new": ([5, 16, 0], [0, 0, 0], 4, 5, 5, 64),
    "block ends": ([0, 15, 16, 17, 31, 32, 1, 0], [16, 1, 1, 15, 1, 16, 14, 17], 5, 40, 33, 100),
    "one long": ([100], [5000], 400, 500, 400, 5001),
    "no blocks": ([3, 16, 10, 15, 40], [5, 1, 2, 2, 8], 6, 5, 0, 64),
    "the list runs out": ([3, 16, 10, 16, 40, 0], [5, 100, 2, 1, 8, 1], 12, 50, 6, 200),
    "the rows run out": ([3, 16, 10, 15, 40], [5, 10, 20, 2, 8], 6, 50, 50, 16),
    "no rows": ([3, 16], [5, 1], 6, 50, 50, 0),
    "past the table": ([3, 60, 10], [5, 5, 20], 4, 50, 50, 64),
    "negative": ([3, -1, 10, 5], [5, 5, -20, 2], 4, 50, 50, 64),
    "list too long": ([3, 20], [20, 20], 4, 8, 11, 64),
    "list negative": ([3, 20], [2, 20], 4, 8, -4, 64),
    "int32 ends": ([3, 2 ** 31 - 1, 7], [5, 2 ** 31 - 1, 2 ** 31 - 1], 4, 8, 8, 64),
}


def run_grow(lens, new, width, cap, have, rows, seed=1, in_place=False):
    rng = random.Random(seed)
    ids = rng.sample(range(10 ** 6), len(lens) * width + cap)
    tables = [ids[i * width:(i + 1) * width] for i in range(len(lens))]
    free = ids[len(lens) * width:]
    want = R.grow(tables, lens, new, free, have, rows)
    t, n, f, h = ints(tables).view(len(lens), width), ints(lens), ints(free), ints([have])
    got = pa.pa_kv_grow(t, n, ints(new), f, h, rows, in_place=in_place)
    assert got[0] is t and (got[1] is n) == in_place and (got[2] is h) == in_place
    for name, x, y in zip(("tables", "lens", "num_free", "cu", "slots", "positions", "seqs"), got, want):
        assert x.flatten().tolist() == ([z for r in y for z in r] if name == "tables" else [y] if name == "num_free" else y), name
    assert f.tolist() == free
    assert in_place or (n.tolist() == list(lens) and h.tolist() == [have])
    assert pa.pa_device_status(clear=True) == (pa.PA_DEV_OUT_OF_RANGE if want[7] or not 0 <= have <= cap else 0)


@gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", GROW)
def test_grow(case, in_place):
    run_grow(*GROW[case], in_place=in_place)


@gpu
@pytest.mark.parametrize("batch", [1, 31, 64, 511, 512, 513, 1025, 3000])
def test_grow_many(batch):
    """Batches around the size of a tile of sequences, lists and rows that suffice or run out midway."""
    rng = random.Random(batch)
    for new_most, enough in ((1, 1.0), (40, 1.0), (40, 0.5), (3, 0.4)):
        lens = [rng.choice([0, rng.randint(0, 300)]) for _ in range(batch)]
        new = [rng.randint(0, new_most) for _ in range(batch)]
        need = sum(R.blocks(a + b) - R.blocks(a) for a, b in zip(lens, new))
        for rows in (sum(new) + 37, int(sum(new) * 0.7)):
            run_grow(lens, new, 22, need + 5, int(need * enough), rows, seed=batch)


@gpu
def test_grow_with_no_sequences_and_largest_batch():
    empty = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    got = pa.pa_kv_grow(empty, ints([]), ints([]), ints([1, 2]), ints([2]), 5)
    assert got[3].tolist() == [0] and got[4].tolist() == [-1] * 5 and got[5].tolist() == [0] * 5 and got[2].tolist() == [2]
    batch = 65535
    t = torch.full((batch, 2), -9, dtype=torch.int32, device="cuda")
    n = torch.arange(batch, device="cuda").int() % 32
    free = torch.randperm(batch, device="cuda").int()
    _, lens, left, cu, slots, pos, seqs = pa.pa_kv_grow(t, n, torch.ones_like(n), free, ints([batch]), 65600)
    assert torch.equal(lens, n + 1) and torch.equal(cu, torch.arange(batch + 1, device="cuda").int())
    fresh = n % 16 == 0
    assert left.item() == batch - int(fresh.sum())
    at = batch - fresh.long().cumsum(0)
    ids = torch.where(fresh, free[at.clamp(max=batch - 1)], torch.full_like(n, -9))
    assert torch.equal(t[torch.arange(batch), (n // 16).long()], ids)
    assert torch.equal(slots[:batch], ids.long() * 16 + n % 16) and torch.equal(pos[:batch], n)
    assert torch.equal(seqs[:batch], torch.arange(batch, device="cuda").int()) and bool((slots[batch:] == -1).all())
    clean()


@gpu
@pytest.mark.parametrize("rows,width,negatives", [(1, 1, 0), (3, 8, 0.5), (64, 72, 0), (511, 5, 0.2), (512, 33, 0.9),
                                                  (513, 7, 0), (1300, 40, 0.1), (2, 9000, 0.3), (32, 2048, 0)])
def test_free(rows, width, negatives):
    rng = random.Random(rows * 7 + width)
    for full, have in ((1.0, 0), (0.5, 17), (0.0, 3), (0.7, 40)):
        counts = [rng.randint(0, width) if rng.random() < 0.9 else (0 if full < 0.9 else width) for _ in range(rows)]
        counts = [int(c * full) for c in counts]
        ids = [[-1 - rng.randint(0, 5) if rng.random() < negatives else rng.randint(0, 2 ** 31 - 1) for _ in range(width)]
               for _ in range(rows)]
        cap = have + sum(counts) + 3 if full != 0.7 else have + sum(counts) // 2
        free = [rng.randint(0, 1000) for _ in range(cap)]
        want, at, bad = R.give_back(ids, counts, free, have)
        f, h = ints(free), ints([have])
        left = pa.pa_kv_free(ints(ids), ints(counts), f, h, in_place=full == 0.5)
        assert f.tolist() == want and left.tolist() == [at] and (left is h) == (full == 0.5)
        assert pa.pa_device_status(clear=True) == (pa.PA_DEV_OUT_OF_RANGE if bad else 0)


@gpu
def test_free_reports_counts_and_lists_out_of_range():
    ids = [[1, 2, 3], [4, 5, 6], [7, 8, 9]]
    for counts, have in (([2, 4, 1], 1), ([2, -4, 1], 1), ([1, 1, 1], -2), ([1, 1, 1], 30)):
        want, at, bad = R.give_back(ids, counts, [0] * 8, have)
        assert bad
        f = ints([0] * 8)
        assert pa.pa_kv_free(ints(ids), ints(counts), f, ints([have])).tolist() == [at] and f.tolist() == want
        assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    assert pa.pa_kv_free(none, ints([]), ints([5]), ints([1])).tolist() == [1]
    assert pa.pa_kv_free(torch.zeros(3, 0, dtype=torch.int32, device="cuda"), ints([0, 0, 0]), ints([5]), ints([1])).tolist() == [1]
    clean()


@gpu
def test_what_grow_takes_and_eviction_gives_comes_back():
    """Blocks go round: every id is in a table or on the list, once, whatever happens in between."""
    rng = random.Random(3)
    B, width, nb = 24, 40, 400
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens, free, left = ints([0] * B), torch.randperm(nb, device="cuda").int(), ints([nb])
    for step in range(60):
        new = ints([rng.choice([0, 1, 1, 1, rng.randint(1, 60)]) for _ in range(B)])
        new = torch.minimum(new, width * 16 - lens)
        pa.pa_kv_grow(tables, lens, new, free, left, 500, in_place=True)
        if step % 3 == 0:
            done = torch.rand(B, device="cuda") < 0.15
            pa.pa_kv_free(tables, torch.where(done, (lens + 15) // 16, 0).int(), free, left, in_place=True)
            lens.masked_fill_(done, 0)
        if step % 4 == 1:
            weights = torch.rand(B, 2, width, device="cuda")
            _, _, _, gone, count = pa.pa_kv_evict(tables, lens, weights, 20, 1, 2, in_place=True)
            pa.pa_kv_free(gone, count, free, left, in_place=True)
        held = [x for row, n in zip(tables.tolist(), lens.tolist()) for x in row[:R.blocks(n)]]
        assert sorted(held + free.tolist()[:left.item()]) == list(range(nb)), step
    clean()


# ----------------------------------------------------------------------------- the step as a whole
@gpu
def test_a_hybrid_stacks_steps():
    """Prompts arrive, grow token by token and leave, in one captured decode step and eager prompt steps:
    tables from pa_kv_grow, a full-attention layer over the pool and packed prompts, a linear layer beside it."""
    B, width, nb, heads, kvh, d, kvl = 6, 20, 60, 8, 2, 128, 4
    scale = d ** -0.5
    gen = torch.Generator(device="cuda").manual_seed(5)
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens, free, left = ints([0] * B), torch.randperm(nb, device="cuda").int(), ints([nb])
    pool = pa.PaPool(*(torch.full((nb, kvh, 16, d), math.nan, device="cuda").bfloat16() for _ in range(2)))
    state, slots = torch.full((B, kvl, d, d), math.nan, device="cuda"), ints(list(range(B))[::-1])
    log_decay = -torch.exp(-torch.rand(kvl, device="cuda", generator=gen) * 5)
    history = [[] for _ in range(B)]  # every sequence's rows: (q, k, v, linear q, k, v)

    def rows(n):
        x = torch.randn(n, heads + 2 * kvh + 3 * kvl, d, device="cuda", generator=gen).bfloat16()
        return x.split([heads, kvh, kvh, kvl, kvl, kvl], 1)

    def remember(new, at):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        for b, (i, j) in enumerate(zip(cu[:-1], cu[1:])):
            history[b].append([x[i:j] for x in at])
        return cu

    def compare(new, out, lin, cu):
        for b, n in enumerate(new):
            if n == 0:
                continue
            q, k, v, lq, lk, lv = (torch.cat(x) for x in zip(*history[b]))
            total = q.shape[0]
            whole = ints([0, total])
            ref, size = R.packed(q, k, v, whole, scale)
            check(out[cu[b]:cu[b] + n], ref[-n:], size[-n:], f"attention of {b}")
            ref, size, _, _ = R.linear(state[:1], [0], lq, lk, lv, log_decay, [0, total], [total], scale)
            bound, _ = R.linear_bounds(ref, size, size, total)
            within(lin[cu[b]:cu[b] + n], ref[-n:], bound[-n:], f"linear of {b}")

    # prompts, the last of which is longer than its table: it is reported and gets nothing
    new = [40, 1, 250, 17, 130, 700]
    _, _, _, cu, slot_map, pos, seqs = pa.pa_kv_grow(tables, lens, ints(new), free, left, 1200, in_place=True)
    new[5] = 0
    assert lens.tolist() == new and pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    q, k, v, lq, lk, lv = at = rows(1200)
    pa.pa_kv_append(pool, k.contiguous(), v.contiguous(), slot_map)
    out = pa.pa_prefill_packed(q, k, v, cu, scale, 700)
    lin = pa.pa_linear_prefill(state, slots, lq, lk, lv, log_decay, cu, lens, scale, 700)
    assert cu.tolist() == remember(new, at)
    compare(new, out, lin, cu.tolist())
    # decode steps in a graph: its inputs are buffers
    q, k, v, lq, lk, lv = rows(B)
    k, v = k.contiguous(), v.contiguous()
    one = ints([1] * B)
    graph = torch.cuda.CUDAGraph()
    kept = [x.clone() for x in (tables, lens, left, state, *([pool.k_cache, pool.v_cache]))]

    def step():
        # a sequence without a token this step has no row; the rows of the others move up to the front
        _, _, _, c, sm, _, _ = pa.pa_kv_grow(tables, lens, one, free, left, B, in_place=True)
        pa.pa_kv_append(pool, k, v, sm)
        o = pa.pa_prefill_chunked(pool, q.contiguous(), c, tables, lens, scale, 1)
        return o, pa.pa_linear_prefill(state, slots, lq, lk, lv, log_decay, c, lens, scale, 1), c
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((tables, lens, left, state, pool.k_cache, pool.v_cache), kept):
        x.copy_(y)
    with torch.cuda.graph(graph):
        out, lin, cu = step()
    one[5] = 0
    for i in range(20):
        fresh = rows(B)
        for x, y in zip((q, k, v, lq, lk, lv), fresh):
            x.copy_(y)
        if i == 10:  # sequence 2 has finished, and a shorter prompt takes the place of the refused one
            pa.pa_kv_free(tables, ints([0, 0, R.blocks(lens[2].item()), 0, 0, 0]), free, left, in_place=True)
            lens[2] = 0
            one[2] = 0
            history[2] = []
            grown = pa.pa_kv_grow(tables, lens, ints([0, 0, 0, 0, 0, 200]), free, left, 200, in_place=True)
            prompt = rows(200)
            pa.pa_kv_append(pool, prompt[1].contiguous(), prompt[2].contiguous(), grown[4])
            o = pa.pa_prefill_packed(*prompt[:3], grown[3], scale, 200)
            li = pa.pa_linear_prefill(state, slots, *prompt[3:], log_decay, grown[3], lens, scale, 200)
            compare([0, 0, 0, 0, 0, 200], o, li, remember([0, 0, 0, 0, 0, 200], prompt))
            one[5] = 1
        graph.replay()
        new = one.tolist()
        assert cu.tolist() == remember(new, fresh)
        compare(new, out, lin, cu.tolist())
    # and the same token through the calls for one token
    fresh = rows(B)
    grown = pa.pa_kv_grow(tables, lens, one, free, left, B, in_place=True)
    live = [b for b in range(B) if one[b].item()]
    n = len(live)
    pa.pa_kv_append(pool, fresh[1].contiguous(), fresh[2].contiguous(), grown[4])
    at = grown[6][:n].long()
    o = pa.pa_decode(pool, fresh[0][:n].contiguous(), tables[at].contiguous(), lens[at].contiguous(), scale)
    li = pa.pa_linear_decode(state, slots[at].contiguous(), *(x[:n] for x in fresh[3:]), log_decay, lens[at].contiguous(), scale)
    compare(one.tolist(), o, li, remember(one.tolist(), fresh))
    clean()
