"""Packed prompts and linear attention where no single case looks: segments, addresses, bounds, calls at once."""
import math

import pytest
import torch

import paged_kv_gqa_slot_gb300 as pa
import step_ref as R
from test_linear import Case, within
from test_packed import check, clean

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("heads,kvh,d", [(2, 2, 128), (2, 1, 64)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_value_in_a_sequence_cut_into_segments(bad, heads, kvh, d):
    lens = [2500, 90]
    for at in (0, 127, 128, 1000, 2303, 2499, 2500):
        end = 2500 if at < 2500 else 2590
        seq = int(at >= 2500)
        c = Case(41, lens, heads, kvh, d)
        ref, size, new, new_size = c.reference()
        bound, new_bound = R.linear_bounds(ref, size, new_size, 2500)
        c.v[at, kvh - 1, 7] = bad
        out = c.prefill()
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        hit[at:end, -(heads // kvh):, 7] = True
        within(out[~hit], ref[~hit], bound[~hit], f"v {at}")
        assert not bool(torch.isfinite(out[hit]).any())
        there = torch.zeros(c.state.shape, dtype=torch.bool, device="cuda")
        there[int(c.slots[seq]), kvh - 1, :, 7] = True
        within(c.state[~there], new[~there], new_bound[~there], f"state, v {at}")
        assert not bool(torch.isfinite(c.state[there]).any())
    clean()


@gpu
def test_segments_end_in_any_order():
    """A sequence in segments replaces its state while its first segment may still be to come: the same bits
    each time, with as many segments as there are and with other sequences between them."""
    for lens, heads, d in (([3000], 1, 64), ([2100, 1, 300, 1500, 2], 3, 128)):
        c = Case(42, lens, heads, heads, d)
        start = c.state.clone()
        out = c.check(c.prefill)
        after = c.state.clone()
        for _ in range(40):
            c.state.copy_(start)
            assert torch.equal(out, c.prefill())
            assert torch.equal(after.nan_to_num(7), c.state.nan_to_num(7))
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_packed_scores_far_from_zero(d):
    """All scores of a row near one value, from -180 to 180, in stages that every row sees whole and in others; and
    keys that come by it in jumps.  (Exact operands: q and k have few bits, so the scores are those of the reference.)"""
    n, scale = 600, 1 / 64
    for steps in ([-180.0], [180.0], [-180.0, -150.0, 10.0, 12.0, 100.0], [100.0, 20.0, -60.0, 130.0, 128.0]):
        q, k, v, cu = R.packed_rows([n, 150], 4, 2, d, 49, strided=False)
        q[:] = 64.0 / d
        level = torch.tensor(steps, device="cuda")[torch.arange(n + 150, device="cuda") * len(steps) // (n + 150)]
        k[:] = (level[:, None, None] + torch.round(k.float())).bfloat16()
        out = pa.pa_prefill_packed(q, k, v, cu, scale, n)
        ref, size = R.packed(q, k, v, cu, scale)
        check(out, ref, size, str(steps))
    clean()


@gpu
@pytest.mark.parametrize("lens,d", [([640, 1], 128), ([3000], 128), ([640, 70], 64), ([2600], 64)])
def test_the_state_keeps_32_bits(lens, d):
    """Its error's size against its own: the parts of k's weighted rows 2^-24, the exponents (up to 6 where a term
    counts) 2^-21, the sums, 8 a chunk of up to 24 chunks, 2^-24 each and of either sign, 2^-20.2: below 2^-19.5
    together, where two bf16 parts would leave 2^-18 of the terms' size."""
    c = Case(48, lens, 2, 2, d, decay=-0.012)
    _, _, new, _ = c.reference()
    c.prefill()
    off, size = (c.state.double() - new)[c.slots.long()], new[c.slots.long()]
    assert float(off.square().mean().sqrt()) <= 2.0 ** -19.5 * float(size.square().mean().sqrt())
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_arrays_aligned_to_16_bytes_and_no_more(d):
    def moved(x, by):
        flat = torch.zeros(x.numel() + by, dtype=x.dtype, device="cuda")
        flat[by:].copy_(x.reshape(-1))
        return flat[by:].view(x.shape)
    lens = [130, 37, 1]
    q, k, v, cu = R.packed_rows(lens, 8, 2, d, 43, strided=False)
    q, k, v = (moved(x, 8) for x in (q, k, v))
    out = moved(torch.full(q.shape, 7.0, device="cuda").bfloat16(), 8)
    pa.pa_prefill_packed(q, k, v, cu, 0.1, 130, out=out)
    ref, size = R.packed(q, k, v, cu, 0.1)
    check(out, ref, size)
    for n in (lens, [1, 1, 1], [3, 1, 2], [1700, 2]):
        c = Case(44, n, 8, 2, d, strided=False)
        c.q, c.k, c.v, c.state = (moved(x, b) for x, b in ((c.q, 8), (c.k, 8), (c.v, 8), (c.state, 4)))
        out = moved(torch.full(c.q.shape, 7.0, device="cuda").bfloat16(), 8)
        need = pa.pa_linear_workspace_bytes(len(n), 2, d, max(n))
        ws = moved(torch.zeros(need // 4, device="cuda"), 4)
        c.check(lambda: c.prefill(out=out, workspace=ws), what=str(n))
        if max(n) == 1:
            c.check(lambda: c.decode(out=out), True, "decode")
    clean()


@gpu
@pytest.mark.parametrize("most", [5, 2000, 1 << 20, 2 ** 31 - 1])
def test_bounds_far_above_the_lengths(most):
    lens = [5, 0, 3, 1] if most == 5 else [700, 5, 0, 1300]
    q, k, v, cu = R.packed_rows(lens, 4, 2, 128, 45)
    out = pa.pa_prefill_packed(q, k, v, cu, 0.1, most)
    ref, size = R.packed(q, k, v, cu, 0.1)
    check(out, ref, size)
    c = Case(46, lens, 4, 2, 128, fresh=(1,))
    c.check(lambda: c.prefill(most=most))
    clean()


@gpu
def test_the_largest_batch():
    """65535 sequences of one row: attention gives back its value."""
    n = 65535
    gen = torch.Generator(device="cuda").manual_seed(47)
    q, k, v = (torch.randn(n, 1, 64, device="cuda", generator=gen).bfloat16() for _ in range(3))
    cu = torch.arange(n + 1, device="cuda").int()
    assert torch.equal(pa.pa_prefill_packed(q, k, v, cu, 0.1, 9), v)
    state = torch.full((3, 1, 64, 64), math.nan, device="cuda")
    slots = torch.full((n,), -1, device="cuda").int()
    at = [0, 40000, n - 1]
    slots[at] = torch.arange(3, device="cuda").int()
    lens, la = torch.ones_like(slots), torch.zeros(1, device="cuda")
    want = (q[at].double() * k[at].double()).sum(-1, keepdim=True) * v[at].double()
    size = (q[at].double() * k[at].double()).abs().sum(-1, keepdim=True) * v[at].double().abs()
    for one, run in ((True, lambda: pa.pa_linear_decode(state, slots, q, k, v, la, lens, 1.0)),
                     (True, lambda: pa.pa_linear_prefill(state, slots, q, k, v, la, cu, lens, 1.0, 1)),
                     (False, lambda: pa.pa_linear_prefill(state, slots, q, k, v, la, cu, lens, 1.0, 9))):
        state.fill_(math.nan)
        out = run()
        bound, _ = R.linear_bounds(want, size, size, 1, one)
        within(out[at], want, bound, "out")
        assert int((out != 0).any(-1).sum()) == 3
        exact = k[at, 0].double()[:, :, None] * v[at, 0].double()[:, None, :]
        within(state[:, 0], exact, R.linear_bounds(exact, exact.abs(), exact.abs(), 1, one)[1], "state")
    clean()


@gpu
def test_calls_at_once_on_two_streams():
    """A packed prompt, a sequence in segments, decode and the tables beside each other, with arrays of their own."""
    def work(seed):
        q, k, v, cu = R.packed_rows([900, 30, 411], 8, 2, 128, seed)
        c = Case(seed, [2200, 300], 4, 2, 128)
        one = Case(seed + 1, [1] * 9, 8, 4, 64)
        begin = c.state.clone(), one.state.clone()
        ws = torch.empty(pa.pa_linear_workspace_bytes(2, 2, 128, 2200) // 4, device="cuda")
        ints = lambda x: torch.tensor(x, device="cuda").int()  # noqa: E731
        tables, lens, new = torch.zeros(40, 9, dtype=torch.int32, device="cuda"), ints([5] * 40), ints([20] * 40)
        free, left = torch.arange(300, device="cuda").int(), ints([300])

        def run(stream):
            got = [pa.pa_prefill_packed(q, k, v, cu, 0.1, 900, stream=stream),
                   c.prefill(workspace=ws, stream=stream), one.decode(stream=stream),
                   *pa.pa_kv_grow(tables, lens, new, free, left, 999, stream=stream)]
            return got, [c.state, one.state]

        def reset():
            c.state.copy_(begin[0])
            one.state.copy_(begin[1])
            tables.zero_()
        return run, reset
    jobs = [work(50), work(60)]
    alone = []
    for run, reset in jobs:
        reset()
        got, states = run(None)
        alone.append([x.clone() for x in got + states])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for _, reset in jobs:
            reset()
        torch.cuda.synchronize()
        results = [run(s) for (run, _), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for (got, states), want in zip(results, alone):
            for x, y in zip(got + states, want):
                assert torch.equal(torch.nan_to_num(x, 7), torch.nan_to_num(y, 7))
    clean()
