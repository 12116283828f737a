"""Linear attention with a decay for each head: one token, chunks, and the two in turn."""
import math

import pytest
import torch

import paged_kv_gqa_slot_gb300 as pa
import step_ref as R
from paged_kv_gqa_slot_gb300 import build as pbuild

gpu = pytest.mark.gpu
FAKE = 0x40000


# ----------------------------------------------------------------------------- without a GPU
@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.library()


def test_refusals_before_any_launch(lib):
    bad, unsup = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    dec = lambda st=FAKE, ns=4, sl=FAKE, q=FAKE, k=FAKE, v=FAKE, ld=FAKE, ln=FAKE, b=2, h=8, kvh=2, d=128, qs=1536, ks=1536, vs=1536, s=0.1, o=FAKE: (  # noqa: E731,E501
        lib.pa_linear_decode(st, ns, sl, q, k, v, ld, ln, b, h, kvh, d, qs, ks, vs, s, o, None))
    pre = lambda st=FAKE, ns=4, sl=FAKE, q=FAKE, k=FAKE, v=FAKE, ld=FAKE, cu=FAKE, ln=FAKE, b=2, t=9, h=8, kvh=2, d=128, qs=1536, ks=1536, vs=1536, m=5, s=0.1, ws=FAKE, o=FAKE: (  # noqa: E731,E501
        lib.pa_linear_prefill(st, ns, sl, q, k, v, ld, cu, ln, b, t, h, kvh, d, qs, ks, vs, m, s, ws, o, None))
    for call in (dec, pre):
        for name in ("st", "sl", "q", "k", "v", "ld", "ln", "o"):
            assert call(**{name: None}) == bad, name
            assert call(**{name: FAKE + 2}) == bad, name
        assert call(ns=0) == bad and call(h=7) == bad and call(kvh=0) == bad and call(b=-1) == bad and call(b=65536) == bad
        assert call(s=math.nan) == bad and call(d=96) == unsup and call(qs=1020) == bad and call(ks=248) == bad
        assert call(vs=1540) == bad and call(b=0, st=None, q=None) == pa.PA_OK
    assert pre(cu=None) == bad and pre(cu=FAKE + 1) == bad and pre(t=-1) == bad and pre(m=-1) == bad
    assert pre(t=0, q=None) == pa.PA_OK and pre(m=0) == pa.PA_OK
    assert pa.pa_linear_workspace_bytes(0, 8, 128, 100) == 0 and pa.pa_linear_workspace_bytes(2, 8, 128, -1) == 0


def test_binding_refuses_shapes():
    q, kv = torch.zeros(4, 4, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16()
    state, idx, la = torch.zeros(5, 2, 64, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(ValueError):
        pa.pa_linear_decode(state, idx, q, kv, kv, la, idx, 0.1)
    with pytest.raises(ValueError):
        pa.pa_linear_prefill(state, idx, q, kv, kv, la, torch.zeros(5, dtype=torch.int32), idx, 0.1, 4)


# ----------------------------------------------------------------------------- helpers
def clean():
    assert pa.pa_device_status(clear=True) == 0


def within(got, ref, bound, what):
    got = got.double()
    number = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), number), f"{what}: not a number in the wrong places"
    off = torch.where(number, (got - ref).abs() - bound, torch.full_like(ref, -1.0))
    if off.numel() and float(off.max()) > 0:
        at = torch.unravel_index(off.argmax(), off.shape)
        raise AssertionError(f"{what}: {int((off > 0).sum())} past the bound; at {[int(i) for i in at]} {float(got[at])} "
                             f"against {float(ref[at])}, {float(off[at])} past {float(bound[at])}")


class Case:
    """Sequences with states in shuffled slots; slots that none uses hold NaN, and so does a fresh sequence's."""

    def __init__(self, seed, lens, heads, kvh, d, fresh=(), strided=True, before=0, behind=0, decay=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.scale = list(lens), d ** -0.5
        self.q, self.k, self.v, self.cu = R.packed_rows(lens, heads, kvh, d, seed + 1, before, behind, strided)
        B = len(lens)
        order = torch.randperm(B + 3, device="cuda", generator=gen)
        self.slots = order[:B].int()
        self.state = torch.randn(B + 3, kvh, d, d, device="cuda", generator=gen) * 3
        self.state[order[B:]] = math.nan
        self.lens = torch.tensor([n + (0 if b in fresh else 5 + 11 * b) for b, n in enumerate(lens)], device="cuda").int()
        for b in fresh:
            if lens[b]:
                self.state[order[b]] = math.nan
        span = torch.rand(kvh, device="cuda", generator=gen) * 6
        self.log_decay = -torch.exp(-span) if decay is None else torch.full((kvh,), decay, device="cuda")

    def reference(self):
        return R.linear(self.state, self.slots.tolist(), self.q, self.k, self.v, self.log_decay, self.cu.tolist(),
                        self.lens.tolist(), self.scale)

    def prefill(self, most=None, **kw):
        return pa.pa_linear_prefill(self.state, self.slots, self.q, self.k, self.v, self.log_decay, self.cu, self.lens,
                                    self.scale, max(self.n) if most is None else most, **kw)

    def decode(self, **kw):
        return pa.pa_linear_decode(self.state, self.slots, self.q, self.k, self.v, self.log_decay, self.lens, self.scale,
                                   **kw)

    def check(self, run, one_token=False, what=""):
        ref, size, new, new_size = self.reference()
        out = run()
        a, b = int(self.cu[0]), int(self.cu[-1])
        bound, new_bound = R.linear_bounds(ref, size, new_size, max(self.n), one_token)
        within(out[a:b], ref[a:b], bound[a:b], what + " out")
        within(self.state, new, new_bound, what + " state")
        clean()
        return out


DECODE = {
    "one": (1, 32, 32, 128, ()),
    "one, d 64": (1, 4, 4, 64, ()),
    "few, fresh": (3, 8, 2, 128, (1,)),
    "groups": (9, 24, 2, 128, (0, 8)),
    "group 17": (5, 17, 1, 64, ()),
    "many": (70, 16, 8, 128, (3, 69)),
    "many, d 64": (200, 6, 3, 64, (7,)),
}


@gpu
@pytest.mark.parametrize("strided", [True, False])
@pytest.mark.parametrize("case", DECODE)
def test_decode(case, strided):
    batch, heads, kvh, d, fresh = DECODE[case]
    c = Case(21, [1] * batch, heads, kvh, d, fresh, strided)
    c.check(c.decode, True, case)


PREFILL = {
    "one token": ([1], 32, 32, 128, ()),
    "one token, fresh": ([1, 1, 1], 4, 2, 128, (1,)),
    "short": ([4, 7, 16, 17, 2], 8, 8, 128, (2,)),
    "tile ends": ([63, 64, 65, 127, 128, 129, 255, 256, 257], 4, 4, 128, (0, 4, 8)),
    "empty ones": ([0, 200, 0, 1, 0], 2, 2, 128, (1, 4)),
    "d 64": ([300, 64, 1, 129], 4, 4, 64, (1,)),
    "group 2": ([300, 70], 8, 4, 128, (0,)),
    "group 3, d 64": ([190, 131], 9, 3, 64, ()),
    "group 8": ([150, 260], 8, 1, 128, (1,)),
    "long": ([1700], 3, 3, 128, ()),
    "long, d 64": ([1500, 900], 2, 2, 64, (0,)),
    "many": (list(range(0, 150, 4)), 4, 4, 128, (5, 20)),
    "long beside short": ([2000, 1, 3, 40], 4, 2, 128, (0,)),
}


@gpu
@pytest.mark.parametrize("strided", [True, False])
@pytest.mark.parametrize("case", PREFILL)
def test_prefill(case, strided):
    lens, heads, kvh, d, fresh = PREFILL[case]
    c = Case(22, lens, heads, kvh, d, fresh, strided)
    c.check(c.prefill, False, case)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("decay", [0.0, -1e-5, -0.03, -0.8, -5.0, -60.0, -1e4, -math.inf, 3.0, math.nan])
def test_decays_of_every_size(decay, d):
    """None at all, hardly any, what leaves nothing; past the range its nearer end (a NaN: the lower)."""
    c = Case(23, [400, 33, 1, 150], 4, 2, d, (1,), decay=decay)
    given = c.log_decay
    c.log_decay = torch.nan_to_num(given, nan=-1e4, posinf=0.0, neginf=-1e4).clamp(-1e4, 0.0)
    ref = c.reference()
    c.reference = lambda: ref
    c.log_decay = given
    c.check(c.prefill, False, "prefill")
    c = Case(24, [1] * 5, 4, 2, d, (1,), decay=decay)
    c.log_decay = torch.nan_to_num(given, nan=-1e4, posinf=0.0, neginf=-1e4).clamp(-1e4, 0.0)
    ref1 = c.reference()
    c.reference = lambda: ref1
    c.log_decay = given
    c.check(c.decode, True, "decode")


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    c = Case(25, [140, 3], 4, 2, 128)
    c.scale = scale
    c.check(c.prefill)
    c = Case(26, [1, 1], 4, 2, 128)
    c.scale = scale
    c.check(c.decode, True)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_padding_and_rows_outside_the_sequences(d):
    c = Case(27, [50, 9, 171], 8, 2, d, before=19, behind=45)
    for x in (c.q, c.k, c.v):
        x[:19] = math.nan
        x[19 + 230:] = math.nan
    c.slots[1] = -1  # a padded sequence: zero rows, no state
    out = torch.full(c.q.shape, 7.0, device="cuda").bfloat16()
    c.check(lambda: c.prefill(out=out))
    assert bool((out[:19] == 7).all()) and bool((out[249:] == 7).all()) and bool((out[69:78] == 0).all())
    c = Case(28, [1] * 4, 8, 2, d)
    before = c.state.clone()
    c.slots[1] = -1
    c.lens[2] = 0  # no sequence there
    c.k[2] = math.nan
    out = c.decode()
    assert bool((out[1:3] == 0).all())
    kept = [int(c.slots[2]), *[i for i in range(7) if i not in c.slots.tolist()]]
    assert torch.equal(c.state[kept].nan_to_num(7), before[kept].nan_to_num(7))
    assert not torch.equal(c.state[int(c.slots[0])], before[int(c.slots[0])])
    clean()


@gpu
def test_bad_slots_offsets_and_lengths_are_reported():
    flag = pa.PA_DEV_OUT_OF_RANGE
    c = Case(29, [60, 100, 40], 4, 2, 128)
    ref, size, new, _ = c.reference()
    bound, _ = R.linear_bounds(ref, size, size, 100)
    start = c.state.clone()
    keep = c.slots.clone()
    for what, at, x, good in (("slots", 1, 99, [0, 2]), ("cu", 3, 900, [0, 1]), ("lens", 2, 39, [0, 1]), ("cu", 1, -5, [2])):
        t = getattr(c, what)
        old = t[at].clone()
        t[at] = x
        c.state.copy_(start)
        out = c.prefill(most=200)
        assert pa.pa_device_status(clear=True) == flag, what
        t[at] = old
        for b in good:
            rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
            within(out[rows], ref[rows], bound[rows], what)
        for s in range(6):
            if s not in keep.tolist():
                assert bool(torch.isnan(c.state[s]).all())
    # rows past max_chunk are not written, the state is that of the rows below it
    c.state.copy_(start)
    out = torch.full(c.q.shape, 7.0, device="cuda").bfloat16()
    c.prefill(most=64, out=out)
    assert pa.pa_device_status(clear=True) == flag
    for rows in (slice(0, 124), slice(160, 200)):
        within(out[rows], ref[rows], bound[rows], "cut")
    assert bool((out[124:160] == 7).all())
    c = Case(30, [1] * 3, 4, 2, 128)
    c.slots[0] = 1000
    out = c.decode()
    assert pa.pa_device_status(clear=True) == flag and bool((out[0] == 0).all()) and bool((out[1] != 0).any())


@gpu
@pytest.mark.parametrize("heads,kvh,d", [(4, 4, 128), (6, 2, 64), (4, 2, 128)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_value_reaches_what_follows_it_and_nothing_else(bad, heads, kvh, d):
    lens = [200, 300, 90]
    for at in (0, 31, 63, 127, 128, 199, 200, 230, 499, 500, 589):
        seq = 0 if at < 200 else 1 if at < 500 else 2
        end = [200, 500, 590][seq]
        c = Case(31, lens, heads, kvh, d, fresh=(1,))
        ref, size, new, new_size = c.reference()
        bound, new_bound = R.linear_bounds(ref, size, new_size, 300)
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
        c = Case(31, lens, heads, kvh, d, fresh=(1,))
        c.k[at, 0, 3] = bad
        out = c.prefill()
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        hit[at:end, :heads // kvh] = True
        within(out[~hit], ref[~hit], bound[~hit], f"k {at}")
        there = torch.zeros(c.state.shape, dtype=torch.bool, device="cuda")
        there[int(c.slots[seq]), 0] = True
        within(c.state[~there], new[~there], new_bound[~there], f"state, k {at}")
        assert not bool(torch.isfinite(c.state[int(c.slots[seq]), 0, 3]).any())
        c = Case(31, lens, heads, kvh, d, fresh=(1,))
        c.q[at, 1, 0] = bad
        out = c.prefill()
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        hit[at, 1] = True
        within(out[~hit], ref[~hit], bound[~hit], f"q {at}")
        within(c.state, new, new_bound, f"state, q {at}")
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_and_single_tokens_in_turn_are_one_sequence(d):
    """A prompt in chunks of any size, then token by token, against the whole at once."""
    n, heads, kvh = 700, 4, 2
    whole = Case(33, [n], heads, kvh, d, fresh=(0,))
    ref, _, new, new_size = whole.reference()
    _, new_bound = R.linear_bounds(ref, ref, new_size, n)
    carried = whole.state.double()  # the state between the calls, in 64 bits
    at = 0
    for step in (1, 130, 64, 3, 1, 300, 128, 17) + (1,) * 56:
        rows = slice(at, at + step)
        lens = torch.tensor([at + step], device="cuda").int()
        part = [x[rows] for x in (whole.q, whole.k, whole.v)]
        if step == 1 and at > 0:
            out = pa.pa_linear_decode(whole.state, whole.slots, *part, whole.log_decay, lens, whole.scale)
        else:
            cu = torch.tensor([0, step], device="cuda").int()
            out = pa.pa_linear_prefill(whole.state, whole.slots, *part, whole.log_decay, cu, lens, whole.scale, step)
        mine, size, carried, _ = R.linear(carried, whole.slots.tolist(), *part, whole.log_decay, [0, step], [at + step], whole.scale)
        bound, _ = R.linear_bounds(mine, size, size, n)
        within(out, mine, bound, f"{step} at {at}")
        within(mine, ref[rows], 1e-12 * (size + 1), "the reference's parts")
        at += step
    assert at == n
    within(whole.state, new, new_bound, "state")
    clean()


@gpu
def test_repeats_streams_and_graphs():
    c = Case(34, [700, 64, 1, 333], 8, 4, 128, fresh=(0, 2))
    start = c.state.clone()
    first = c.prefill()
    after = c.state.clone()
    for _ in range(4):
        c.state.copy_(start)
        assert torch.equal(first, c.prefill())
        assert torch.equal(after.nan_to_num(7), c.state.nan_to_num(7))
    out = torch.empty_like(first)
    need = pa.pa_linear_workspace_bytes(4, 4, 128, 800)
    ws = torch.full(((need + 3) // 4,), math.nan, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.prefill(most=800, workspace=ws, out=out)
    for new in ([700, 64, 1, 333], [1, 1, 1, 1], [800, 0, 298, 0]):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        c.cu.copy_(torch.tensor(cu))
        c.n = new
        c.lens.copy_(torch.tensor([n + 9 * (b % 2) for b, n in enumerate(new)]))
        c.state.copy_(start)
        out.fill_(5.0)

        def run():
            graph.replay()
            return out
        c.check(run, what=str(new))
        assert bool((out[cu[-1]:] == 5).all())
    side = torch.cuda.Stream()
    c.state.copy_(start)
    side.wait_stream(torch.cuda.current_stream())
    got = c.prefill(most=800, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[:1098], out[:1098])
    d1 = Case(35, [1] * 6, 8, 4, 128)
    begin = d1.state.clone()
    want = d1.decode()
    d1.state.copy_(begin)
    side.wait_stream(torch.cuda.current_stream())
    got = d1.decode(stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    clean()


@gpu
def test_states_whose_offsets_pass_32_bits():
    """9000 slots of 8 heads: 4.7 GB of state, the sequences in the last ones."""
    slots, kvh, d = 9000, 8, 128
    state = torch.zeros(slots, kvh, d, d, device="cuda")
    c = Case(36, [130, 2], 8, kvh, d)
    state[[8999, 8500]] = c.state[c.slots.long()]
    c.state, c.slots = state, torch.tensor([8999, 8500], device="cuda").int()
    ref, size, _, _ = c.reference()
    small = state[[8999, 8500]].clone()
    out = c.prefill()
    bound, _ = R.linear_bounds(ref, size, size, 130)
    within(out, ref, bound, "out")
    assert not torch.equal(state[[8999, 8500]], small)
    assert float(state[:8500].abs().max()) == 0.0
    clean()
