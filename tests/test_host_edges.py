"""Host-side calls at their ends: the bytes of an 8-bit pool, and no memory left (no GPU)."""
import subprocess
import sys
import textwrap

import pytest

import paged_kv_gqa_slot_gb300 as pa
from paged_kv_gqa_slot_gb300 import build as pbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    pbuild.build()
    return pa.library()


@pytest.mark.parametrize("layers,heads,d", [(64, 8, 128), (1, 1, 64), (36, 8, 128)])
def test_an_8_bit_pool_fits_its_budget(layers, heads, d):
    """dtype_bytes = 1 is the 8-bit pool: codes, and an exponent byte for K and one for V per kv head."""
    per = layers * heads * (2 * 16 * d + 2)
    assert pa.pa_kv_block_bytes(layers, heads, d, dtype_bytes=1) == per
    assert pa.pa_kv_block_bytes(layers, heads, d) == layers * heads * 2 * 16 * d * 2   # bf16 as before
    for n in (1, 999, 5360):
        assert pa.pa_kv_budget_blocks(n * per, layers, heads, d, dtype_bytes=1) == n
        assert pa.pa_kv_budget_blocks(n * per - 1, layers, heads, d, dtype_bytes=1) == n - 1


NO_MEMORY = textwrap.dedent("""
    import ctypes, resource, sys
    import numpy as np
    import paged_kv_gqa_slot_gb300 as pa
    lib = pa.library()

    def limit(extra):
        used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
        resource.setrlimit(resource.RLIMIT_AS, (used + extra, resource.getrlimit(resource.RLIMIT_AS)[1]))

    n = 1 << 22                               # tokens: 16 MB
    toks = np.zeros(n, dtype=np.int32)
    bm = pa.BlockManager(1 << 19, prefix_cache=False)
    ids = np.empty(1 << 18, dtype=np.int32)
    nb, nc = ctypes.c_int32(), ctypes.c_int32()

    def admit(request, tokens, more):
        return lib.pa_bm_admit(bm._h, request, toks.ctypes.data, tokens, more, ids.ctypes.data, len(ids),
                               ctypes.byref(nb), ctypes.byref(nc))

    what = sys.argv[1]
    if what == "commit":
        assert admit(1, 16, n - 16) == 0
    if what == "evict":
        assert admit(1, n, 0) == 0
        half = ids[::2].copy()
    before = bm.stats()
    call = {"create": lambda: 0 if lib.pa_bm_create(1 << 24, 16, 1) else pa.PA_ERR_NO_MEMORY,
            "admit": lambda: admit(1, n, 0),
            "commit": lambda: lib.pa_bm_commit(bm._h, 1, toks.ctypes.data, n - 16, 0),
            "evict": lambda: lib.pa_bm_evict(bm._h, 1, half.ctypes.data, len(half))}[what]
    failed = 0
    for extra in list(range(1 << 18, 1 << 26, 1 << 18)) + [1 << 34]:
        limit(extra)                          # the allocations of the call fail one after the other
        rc = call()
        if rc == 0:
            break
        assert rc == pa.PA_ERR_NO_MEMORY and bm.stats() == before, (rc, bm.stats(), before)
        failed += 1
    after = bm.stats()
    print("rc", rc, "failed", failed > 0, "used", after[2] - before[2])
""")


@pytest.mark.parametrize("call,used", [("create", 0), ("admit", 1 << 18), ("commit", 0), ("evict", -(1 << 17))])
def test_no_memory_is_a_status(call, used):
    """A manager call that finds no memory returns (NULL or PA_ERR_NO_MEMORY) with nothing changed, and works once there
    is some; no exception crosses the C interface, where it would end the process."""
    r = subprocess.run([sys.executable, "-c", NO_MEMORY, call], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.strip() == f"rc 0 failed True used {used}", r.stdout


def test_cached_blocks_keep_their_release_order():
    """The block released longest ago is taken first, whatever was held again in between."""
    bm = pa.BlockManager(4)
    table, _ = bm.admit(1, list(range(16)) + list(range(100, 116)) + [7], 0)
    bm.commit(1, [], 33)
    bm.release(1)                                              # both cached, the second block released first
    assert bm.stats() == (2, 2, 0)
    again, cached = bm.admit(2, list(range(16)) + [9], 0)      # holds the first once more
    assert cached == 16 and again[0] == table[0]
    bm.release(2)
    wide, _ = bm.admit(3, list(range(500, 532)) + [1], 0)      # three blocks: two free ones and the second
    assert int(table[1]) in wide.tolist() and int(table[0]) not in wide.tolist()
    bm.release(3)
    _, cached = bm.admit(4, list(range(16)) + [9], 0)
    assert cached == 16
