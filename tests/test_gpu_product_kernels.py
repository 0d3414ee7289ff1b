"""Every kernel that the int8 products choose from, at ragged sizes, every code width, with and
without zero points, in both output types.  tests/test_product_plan.py checks that these sizes reach
every one of them."""
from __future__ import annotations

import pytest

from test_gpu_tokens_i8 import assert_product

pytestmark = pytest.mark.gpu

# K: 3 steps of 256 codes with a half one last, 1 step, 5 steps of 128
CASES = [(M, N, K) for N, K in ((7200, 520), (14400, 200), (25100, 620)) for M in (1, 16, 17, 32)]
CASES += [(M, N, K) for N, K in ((8225, 620), (14400, 520), (25100, 200)) for M in (33, 64)]
CASES += [(5, 70, 700), (20, 70, 700), (40, 300, 700), (200, 1500, 517),
          (4090, 4090, 328),  # 256 x 256 tiles
          (333, 11000, 328),  # 128 x 128 tiles
          (200, 9000, 328),   # 64 x 128 tiles, two stages
          (300, 5000, 700)]   # and four


@pytest.mark.parametrize("bits", range(2, 9))
def test_every_kernel(bits):
    for i, (M, N, K) in enumerate(CASES):
        kind = "gemv" if M <= 16 and i % 2 else "gemm"
        assert_product(kind, M, N, K, bits, (i + bits) % 2 == 1, "bf16" if (i // 2 + bits) % 2 else "f32",
                       9000 + 100 * bits + i)
