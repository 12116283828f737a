"""Host-side calls at their ends: the bytes of an 8-bit pool (no GPU)."""
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
