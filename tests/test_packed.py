"""Packed prompts: causal attention of sequences of different lengths without a cache."""
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
    call = lambda q=FAKE, k=FAKE, v=FAKE, cu=FAKE, b=2, t=100, h=8, kvh=2, d=128, qs=1536, ks=1536, vs=1536, m=50, s=0.1, o=FAKE: (  # noqa: E731,E501
        lib.pa_prefill_packed(q, k, v, cu, b, t, h, kvh, d, qs, ks, vs, m, s, o, None))
    for name in ("q", "k", "v", "cu", "o"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: FAKE + 2}) == bad, name
    assert call(h=7) == bad and call(h=0) == bad and call(kvh=0) == bad and call(b=-1) == bad and call(b=65536) == bad
    assert call(t=-1) == bad and call(m=-1) == bad and call(s=math.nan) == bad and call(s=math.inf) == bad
    assert call(d=96) == unsup and call(d=256) == unsup and call(h=131072, kvh=2) == unsup
    assert call(qs=1020) == bad and call(qs=1016) == bad and call(ks=248) == bad and call(vs=1540) == bad
    assert call(ks=-1536) == bad and call(qs=1 << 39) == bad
    assert call(b=0, q=None, cu=None) == pa.PA_OK and call(t=0, q=None) == pa.PA_OK and call(m=0) == pa.PA_OK


def test_binding_refuses_shapes_and_strides():
    q, kv, cu = torch.zeros(4, 4, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16(), torch.zeros(2, dtype=torch.int32)
    for args in ((q, kv, kv), (q.float(), kv, kv), (q[0], kv, kv), (q, kv[:3], kv), (q, kv, kv[:, :1])):
        with pytest.raises(ValueError):
            pa.pa_prefill_packed(*args, cu, 0.1, 4)


# ----------------------------------------------------------------------------- helpers
def clean():
    assert pa.pa_device_status(clear=True) == 0


def check(out, ref, size, what=""):
    """Within the bound where the reference is a number, the same infinities, NaN where it is NaN."""
    out = out.double()
    number = torch.isfinite(ref)
    assert torch.equal(torch.isnan(out), torch.isnan(ref)), f"{what}: NaN in the wrong places"
    assert torch.equal(out[~number & ~torch.isnan(ref)], ref[~number & ~torch.isnan(ref)]), what
    off = (out - ref).abs() - R.packed_bound(ref, size)
    off = torch.where(number, off, torch.full_like(off, -1.0))
    if off.numel() and float(off.max()) > 0:
        at = torch.unravel_index(off.argmax(), off.shape)
        raise AssertionError(f"{what}: {int((off > 0).sum())} past the bound; at {[int(i) for i in at]} {float(out[at])} "
                             f"against {float(ref[at])}, {float(off[at])} past it")


CASES = {
    "one token": ([1], 32, 8, 128),
    "one short": ([37], 32, 8, 128),
    "tile ends": ([127, 128, 129, 31, 32, 33, 63, 64, 65, 255, 256, 257], 8, 2, 128),
    "empty ones": ([0, 5, 0, 0, 300, 0], 8, 8, 128),
    "all ones": ([1] * 40, 16, 4, 128),
    "d 64": ([700, 1, 129, 0, 250], 8, 4, 64),
    "d 64, group 1": ([513, 66], 4, 4, 64),
    "group 1": ([900, 77], 3, 3, 128),
    "group 3": ([400, 131], 12, 4, 128),
    "group 5, d 64": ([333, 90], 15, 3, 64),
    "group 7": ([260], 14, 2, 128),
    "group 16": ([600, 13], 32, 2, 128),
    "group 17": ([100, 300], 17, 1, 128),
    "group 24": ([200, 40], 48, 2, 128),
    "group 40": ([150], 40, 1, 64),
    "long": ([3333], 4, 1, 128),
    "long, d 64": ([2900, 1000], 6, 2, 64),
    "many": (list(range(0, 130, 3)), 8, 2, 128),
}


@gpu
@pytest.mark.parametrize("strided", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_packed(case, strided):
    lens, heads, kvh, d = CASES[case]
    q, k, v, cu = R.packed_rows(lens, heads, kvh, d, 7, strided=strided)
    scale = d ** -0.5
    out = pa.pa_prefill_packed(q, k, v, cu, scale, max(lens))
    ref, size = R.packed(q, k, v, cu, scale)
    check(out, ref, size, case)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.09, 0.3, -0.5, 1e-6])
def test_scales(scale, d):
    q, k, v, cu = R.packed_rows([5, 290, 140], 8, 2, d, 8)
    out = pa.pa_prefill_packed(q, k, v, cu, scale, 290)
    ref, size = R.packed(q, k, v, cu, scale)
    check(out, ref, size)
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_climb(d):
    """Every key outweighs all before it by far, so the running maximum moves all the time; then the other way."""
    n = 700
    for sign in (1.0, -1.0):
        q, k, v, cu = R.packed_rows([n, n], 4, 2, d, 9, strided=False)
        q[:] = 1.0
        k[:] = (sign * torch.arange(2 * n, device="cuda") % n / 8).bfloat16()[:, None, None] * 0.25
        out = pa.pa_prefill_packed(q, k, v, cu, d ** -0.5, n)
        ref, size = R.packed(q, k, v, cu, d ** -0.5)
        check(out, ref, size, f"sign {sign}")
    clean()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_outside_the_sequences_stay(d):
    lens = [50, 0, 171]
    q, k, v, cu = R.packed_rows(lens, 8, 2, d, 10, before=19, behind=45)
    for x in (q, k, v):  # nobody's rows
        x[:19] = math.nan
        x[19 + 221:] = math.nan
    out = torch.full((q.shape[0], 8, d), 7.0, device="cuda").bfloat16()
    got = pa.pa_prefill_packed(q, k, v, cu, 0.1, 200, out=out)
    assert got is out
    ref, size = R.packed(q, k, v, cu, 0.1)
    check(out[19:240], ref[19:240], size[19:240])
    assert bool((out[:19] == 7).all()) and bool((out[240:] == 7).all())
    clean()


@gpu
@pytest.mark.parametrize("heads,kvh,d", [(8, 2, 128), (3, 3, 128), (8, 2, 64), (10, 2, 64)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_masked_does_not_reach_a_row(bad, heads, kvh, d):
    """A NaN or an infinity in K, V or Q reaches the rows that see it, and its column alone in V."""
    lens = [200, 300, 97]
    for at in (0, 31, 127, 128, 140, 199, 200, 230, 499, 500, 540, 596):
        q, k, v, cu = R.packed_rows(lens, heads, kvh, d, 11)
        v[at, kvh - 1, 5] = bad
        if at % 2:
            v[at, kvh - 1, d - 1] = -bad
        out = pa.pa_prefill_packed(q, k, v, cu, 0.1, 300)
        ref, size = R.packed(q, k, v, cu, 0.1)
        check(out, ref, size, f"v {at}")
        q, k, v, cu = R.packed_rows(lens, heads, kvh, d, 12)
        k[at, 0, 3] = bad
        out = pa.pa_prefill_packed(q, k, v, cu, 0.1, 300)
        seq = 0 if at < 200 else 1 if at < 500 else 2
        hit = torch.zeros(q.shape[0], heads, dtype=torch.bool, device="cuda")
        hit[at:int(cu[seq + 1]), :heads // kvh] = True
        ref, size = R.packed(q, k, v, cu, 0.1)
        check(out[~hit], ref[~hit], size[~hit], f"k {at}")
        if math.isnan(bad):
            assert bool(torch.isnan(out[hit]).all())
        q, k, v, cu = R.packed_rows(lens, heads, kvh, d, 13)
        q[at, 1, 0] = bad
        out = pa.pa_prefill_packed(q, k, v, cu, 0.1, 300)
        hit = torch.zeros(q.shape[0], heads, dtype=torch.bool, device="cuda")
        hit[at, 1] = True
        ref, size = R.packed(q, k, v, cu, 0.1)
        check(out[~hit], ref[~hit], size[~hit], f"q {at}")
        if math.isnan(bad):
            assert bool(torch.isnan(out[hit]).all())
    clean()


@gpu
def test_bad_offsets_and_lengths_are_reported():
    lens = [60, 100, 40]
    q, k, v, cu = R.packed_rows(lens, 8, 2, 128, 14)
    ref, size = R.packed(q, k, v, cu, 0.1)
    # (the last: rows 30 .. 60 are two sequences')
    for change, good in (([(1, -3)], [slice(160, 200)]), ([(3, 500)], [slice(0, 160)]), ([(2, 30)], [slice(0, 30)])):
        c = cu.clone()
        for i, x in change:
            c[i] = x
        out = torch.full((200, 8, 128), 7.0, device="cuda").bfloat16()
        pa.pa_prefill_packed(q, k, v, c, 0.1, 170, out=out)
        assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
        for rows in good:
            check(out[rows], ref[rows], size[rows])
    # a sequence longer than max_len: its first rows, at least those below it, and the others whole
    out = torch.full((200, 8, 128), 7.0, device="cuda").bfloat16()
    pa.pa_prefill_packed(q, k, v, cu, 0.1, 64, out=out)
    assert pa.pa_device_status(clear=True) == pa.PA_DEV_OUT_OF_RANGE
    for rows in (slice(0, 124), slice(160, 200)):
        check(out[rows], ref[rows], size[rows])
    assert bool((out[124:160] == 7).all())


@gpu
def test_agrees_with_prefill_over_the_pool():
    lens = [300, 17, 128]
    q, k, v, cu = R.packed_rows(lens, 8, 2, 128, 15, strided=False)
    width = 19
    pool = pa.PaPool(*(torch.zeros(64, 2, 16, 128, device="cuda").bfloat16() for _ in range(2)))
    ids = torch.randperm(64, device="cuda")[:57].int().view(3, width)
    slots = torch.cat([ids[b][torch.arange(n, device="cuda") // 16].long() * 16 + torch.arange(n, device="cuda") % 16
                       for b, n in enumerate(lens)])
    pa.pa_kv_append(pool, k, v, slots)
    want = pa.pa_prefill_chunked(pool, q, cu, ids.contiguous(), torch.tensor(lens, device="cuda").int(), 128 ** -0.5, 300)
    out = pa.pa_prefill_packed(q, k, v, cu, 128 ** -0.5, 300)
    ref, size = R.packed(q, k, v, cu, 128 ** -0.5)
    check(out, ref, size)
    check(want, ref, size)


@gpu
def test_repeats_give_the_same_bits_and_graphs_replay():
    lens = [700, 64, 1, 333]
    q, k, v, cu = R.packed_rows(lens, 16, 4, 128, 16)
    first = pa.pa_prefill_packed(q, k, v, cu, 0.1, 700)
    for _ in range(5):
        assert torch.equal(first, pa.pa_prefill_packed(q, k, v, cu, 0.1, 700))
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill_packed(q, k, v, cu, 0.1, 800, out=out)
    for new in ([700, 64, 1, 333], [1, 1, 1, 1], [800, 0, 298, 0], [300, 300, 300, 198]):
        c = [0]
        for n in new:
            c.append(c[-1] + n)
        cu.copy_(torch.tensor(c))
        out.fill_(5.0)
        graph.replay()
        ref, size = R.packed(q, k, v, cu, 0.1)
        check(out[:c[-1]], ref[:c[-1]], size[:c[-1]], str(new))
        assert bool((out[c[-1]:] == 5).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pa.pa_prefill_packed(q, k, v, cu, 0.1, 800, stream=side)
    again = pa.pa_prefill_packed(q, k, v, cu, 0.1, 800, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got[:1098], out[:1098]) and torch.equal(again[:1098], out[:1098])
    clean()


@gpu
def test_rows_whose_offsets_pass_32_bits():
    """Rows 40000 elements apart: the last lie 5 GB behind the first."""
    n, wide = 66000, 40000
    big = torch.zeros(n, wide, device="cuda", dtype=torch.bfloat16)
    q, k, v = (big[:, c:c + w].view(n, w // 128, 128) for c, w in ((0, 512), (512, 256), (39744, 256)))
    gen = torch.Generator(device="cuda").manual_seed(17)
    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
    cu = torch.tensor([0, 200], device="cuda").int()
    out = pa.pa_prefill_packed(q, k, v, cu, 0.1, 300)
    tail = torch.tensor([n - 300, n - 100, n], device="cuda").int()
    pa.pa_prefill_packed(q, k, v, tail, 0.1, 300, out=out)
    for c in (cu, tail):
        a, b = int(c[0]), int(c[-1])
        ref, size = R.packed(q[a:b], k[a:b], v[a:b], c - a, 0.1)
        check(out[a:b], ref, size)
    clean()
