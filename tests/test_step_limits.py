"""Packed prompts and linear attention at the limits of what they assume: the order that blocks come in, infinite
scores, values at the ends of the range, states summed over long segments."""
import math
import random

import pytest
import torch

import paged_kv_gqa_slot_gb300 as pa
import step_ref as R
from paged_kv_gqa_slot_gb300 import build as pbuild
from test_linear import Case
from test_packed import check, clean

gpu = pytest.mark.gpu
FAKE = 0x40000


# ----------------------------------------------------------------------------- without a GPU
@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.library()


def test_pair_selftest_refusals(lib):
    bad = pa.PA_ERR_INVALID_ARG
    call = lambda cu=FAKE, b=2, t=100, m=50, per=64, p=FAKE, n=3, o=FAKE: (  # noqa: E731
        lib.pa_selftest_packed_pairs(cu, b, t, m, per, p, n, o, None))
    for name in ("cu", "p", "o"):
        assert call(**{name: None}) == bad and call(**{name: FAKE + 2}) == bad, name
    assert call(b=0) == bad and call(b=65536) == bad and call(t=-1) == bad and call(m=-1) == bad and call(n=-1) == bad
    assert call(per=1) == bad and call(per=257) == bad and call(n=0, p=None, o=None) == pa.PA_OK


# ----------------------------------------------------------------------------- the order of the blocks
def pairs_of(cu, rows, most, per):
    """Every pair of the sequences, in order: [first row, length, first token]."""
    want = []
    for a, b in zip(cu[:-1], cu[1:]):
        if a < 0 or b < a or b > rows:
            continue
        n = min(b - a, most)
        want += [[a, n, at] for at in reversed(range(0, n, per))]
    return want


@gpu
@pytest.mark.parametrize("batch", [1, 2, 31, 32, 33, 64, 65, 200, 1000])
def test_pairs_are_found_in_any_order(batch):
    """Rising, falling and shuffled, with pairs past the last among them; sequences of no tokens at window ends too."""
    rng = random.Random(batch)
    for most, per in ((1, 2), (40, 64), (300, 84), (2000, 256)):
        lens = [rng.choice([0, rng.randint(0, most), most]) for _ in range(batch)]
        cu = [5]
        for n in lens:
            cu.append(cu[-1] + n)
        rows = cu[-1] + 3
        want = pairs_of(cu, rows, most, per)
        n = len(want)
        past = [n, n + 1, n + 77]
        rising = list(range(n)) + past
        orders = [rising, rising[::-1], past + rising]
        for _ in range(3):
            orders.append(rng.sample(rising, len(rising)))
        jumps = [x for i in range(min(n, 40)) for x in (i, n - 1 - i, n + i)]
        orders.append(jumps)
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for order in orders:
            if not order:
                continue
            got = pa.pa_selftest_packed_pairs(t, rows, most, per, torch.tensor(order, dtype=torch.int32, device="cuda"))
            assert got.tolist() == [want[i] if i < n else [-1] * 3 for i in order], (most, per, order[:8])
    clean()


@gpu
def test_pairs_of_sequences_that_are_skipped():
    cu, rows = [0, 100, 60, 200, 900, 300, 300], 300  # the second and the fourth are no sequences
    want = pairs_of(cu, rows, 120, 64)
    assert [w[:2] for w in want] == [[0, 100], [0, 100], [60, 120], [60, 120]]
    got = pa.pa_selftest_packed_pairs(torch.tensor(cu, dtype=torch.int32, device="cuda"), rows, 120, 64,
                                      torch.tensor([3, 0, 4, 2, 1], dtype=torch.int32, device="cuda"))
    assert got.tolist() == [want[3], want[0], [-1] * 3, want[2], want[1]]
    assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE


# ----------------------------------------------------------------------------- states summed for long
def one_signed(n, heads, d, seed):
    """k and v in [0.5, 1.5), so that every error of a sum that is always of one sign adds up."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.rand(n, heads, d, device="cuda", generator=gen) + 0.5).bfloat16() for _ in range(2))


def off_by(state, k, v, log_decay):
    """The state's relative errors against 64 bits, which has every term of one sign."""
    n = k.shape[0]
    rest = torch.exp(log_decay.double() * (n - 1 - torch.arange(n, device="cuda", dtype=torch.float64)))
    want = (k.double() * rest[:, None]).T @ v.double()
    return (state.double() - want) / want


@gpu
@pytest.mark.parametrize("decay", [0.0, -1e-5, -1e-3])
@pytest.mark.parametrize("n,heads,d", [(1 << 20, 1, 64), (20000, 75, 128), (20000, 200, 64), (9000, 32, 128)])
def test_a_state_summed_over_many_chunks(n, heads, d, decay):
    """Segments of 128, 79, all (one segment) and 6 to 9 chunks.  Errors of one sign: the 8 sums of a chunk in the tensor core,
    cut off to 2^-23 of what there is so far, half of the chunk's on average, 2^-21; the decays' 2^-22, and of their exponents 3 * 2^-24 of what is 1.44 on average, less
    than 2^-22; below 2^-20.  Errors of either sign: up to 192 sums in fp32, 2^-24 of what there is so far, 0.58 of it root mean square each, six times
    0.58 * 0.58 * 192^0.5 * 2^-24 < 2^-19: below 2^-18 with the others."""
    k, v = one_signed(n, heads, d, 71)
    q = torch.zeros(n, heads, d, device="cuda").bfloat16()
    state = torch.full((1, heads, d, d), math.nan, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    log_decay = torch.full((heads,), decay, device="cuda")
    pa.pa_linear_prefill(state, ints([0]), q, k, v, log_decay, ints([0, n]), ints([n]), 1.0, n)
    for h in {0, heads // 2, heads - 1}:
        off = off_by(state[0, h], k[:, h], v[:, h], log_decay[h])
        assert abs(float(off.mean())) <= 2.0 ** -20 and float(off.abs().max()) <= 2.0 ** -18, h
    clean()


@gpu
@pytest.mark.parametrize("step", [1, 5])
@pytest.mark.parametrize("decay", [0.0, -1e-5, -1e-3, -0.3, -0.6, -3.0])
def test_a_state_carried_token_by_token(decay, step):
    """2000 tokens by calls for one and for five.  Errors of one sign: a's, which over the tokens that count make
    1 / (1 - a) of it: of a - 1, 2^-23 of that, 2^-23; from exp2f (a < 0.61) 2^-22 a / (1 - a) < 2^-21; below 2^-20.  Errors of
    either sign: two roundings a token, 4000 at most that count, six times 0.58 * 0.58 * 4000^0.5 * 2^-24 < 2^-17."""
    n, d = 2000, 64
    k, v = one_signed(n, 1, d, 72)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    state, slot, cu = torch.full((1, 1, d, d), math.nan, device="cuda"), ints([0]), ints([0, step])
    log_decay = torch.full((1,), decay, device="cuda")
    for t in range(0, n, step):
        rows, lens = slice(t, t + step), ints([t + step])
        if step == 1:
            pa.pa_linear_decode(state, slot, k[rows], k[rows], v[rows], log_decay, lens, 1.0)
        else:
            pa.pa_linear_prefill(state, slot, k[rows], k[rows], v[rows], log_decay, cu, lens, 1.0, step)
    off = off_by(state[0, 0], k[:, 0], v[:, 0], log_decay[0])
    assert abs(float(off.mean())) <= 2.0 ** -20 and float(off.abs().max()) <= 2.0 ** -17
    clean()


# ----------------------------------------------------------------------------- infinite scores
@gpu
@pytest.mark.parametrize("heads,kvh,d", [(8, 2, 128), (3, 3, 128), (8, 2, 64), (10, 2, 64)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinite_scores_are_what_the_definition_makes_them(bad, heads, kvh, d):
    """A key of score +inf makes its rows NaN, one of score -inf has no weight, and a row whose every score is -inf is NaN:
    rows that see the value are compared like all others."""
    lens = [200, 300, 97]
    for at in (0, 1, 31, 127, 128, 140, 199, 200, 230, 499, 500, 540, 596):
        q, k, v, cu = R.packed_rows(lens, heads, kvh, d, 81)
        k[at, 0, 3] = bad
        ref, size = R.packed(q, k, v, cu, 0.1)
        check(pa.pa_prefill_packed(q, k, v, cu, 0.1, 300), ref, size, f"k {at}")
        q, k, v, cu = R.packed_rows(lens, heads, kvh, d, 82)
        q[at, 1, 0] = bad
        ref, size = R.packed(q, k, v, cu, 0.1)
        check(pa.pa_prefill_packed(q, k, v, cu, 0.1, 300), ref, size, f"q {at}")
    clean()


@gpu
@pytest.mark.parametrize("heads,kvh,d", [(4, 2, 128), (1, 1, 128), (4, 2, 64), (3, 1, 64)])
@pytest.mark.parametrize("none", [1, 127, 128, 129, 300])
def test_keys_behind_scores_of_minus_infinity(none, heads, kvh, d):
    """A sequence's first keys have scores of -inf: its first rows are NaN, and the others are those of the keys behind, however
    low or high these are (first stages that hold no weight at all, too)."""
    lens = [none + 290, 20]
    for level in (0.0, -170.0, 60.0):
        q, k, v, cu = R.packed_rows(lens, heads, kvh, d, 83, strided=False)
        q[:] = 64.0 / d
        k[:] = (level + torch.round(k.float())).bfloat16()
        k[:none, :, 1] = -math.inf
        ref, size = R.packed(q, k, v, cu, 1 / 64)
        assert bool(torch.isnan(ref[:none]).all()) and not bool(torch.isnan(ref[none:]).any())
        check(pa.pa_prefill_packed(q, k, v, cu, 1 / 64, lens[0]), ref, size, f"level {level}")
    clean()


@gpu
@pytest.mark.parametrize("heads,kvh,d", [(4, 2, 128), (1, 1, 128), (4, 2, 64), (3, 1, 64)])
@pytest.mark.parametrize("level", [6.1875, 5.0, 0.0, -9.5, -25.0, -100.0])
def test_values_at_the_ends_of_the_range(level, heads, kvh, d):
    """v of 2^111 and of 2^-100 under scores that are all alike (sums of 900 weights of up to 2^8 stay below 2^17 of them):
    the results of v of 1, times that."""
    n = 900
    q, k, v, cu = R.packed_rows([n, 70], heads, kvh, d, 84, strided=False)
    q[:] = 64.0 / d
    k[:] = level
    v[:] = v.abs() * 0.25 + 0.75
    ref, size = R.packed(q, k, v, cu, 1 / 64)
    for power in (111, -100):
        out = pa.pa_prefill_packed(q, k, (v.double() * 2.0 ** power).bfloat16(), cu, 1 / 64, n)
        check(out.double() * 2.0 ** -power, ref, size, f"2^{power}")
    clean()


# ----------------------------------------------------------------------------- bounds that int32 does not hold
@gpu
@pytest.mark.parametrize("most", [1 << 31, 1 << 32, (1 << 32) + 5, (1 << 63) - 1])
def test_bounds_past_int32_are_upper_bounds_like_others(most):
    lens = [300, 0, 41]
    q, k, v, cu = R.packed_rows(lens, 4, 2, 64, 85)
    ref, size = R.packed(q, k, v, cu, 0.1)
    check(pa.pa_prefill_packed(q, k, v, cu, 0.1, most), ref, size)
    assert pa.pa_linear_workspace_bytes(1, 2, 64, most) == pa.pa_linear_workspace_bytes(1, 2, 64, 2 ** 31 - 1) > 0
    c = Case(86, lens, 4, 2, 64, fresh=(2,))
    c.check(lambda: c.prefill(most=most))
    for refused in (-1, -(1 << 32)):
        with pytest.raises(pa.PagedAttnError):
            pa.pa_prefill_packed(q, k, v, cu, 0.1, refused)
        with pytest.raises(pa.PagedAttnError):
            c.prefill(most=refused)
