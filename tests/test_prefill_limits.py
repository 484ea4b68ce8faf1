"""The prefill refuses more CTAs than a grid has before any launch (no GPU needed)."""
import ctypes

import pytest

import mla_latent_decode_gb300 as mla
from mla_latent_decode_gb300 import build

ARG = -1


@pytest.mark.parametrize("num_work,H,ctas", [(1 << 28, 4, 2), (1 << 29, 4, 1), (0x7fffffff, 65535, 2)])
def test_more_ctas_than_a_grid(num_work, H, ctas):
    build.build()

    def P(x):
        return None if x is None else ctypes.c_void_p(x)

    assert mla.library().mla_prefill(
        P(16), 192 * H, 192, P(16), 192 * H, 192, 8, P(16), 256 * H, 256, P(16), 64, P(16), 256 * H, 256, 8, H, P(16),
        P(16), None, 1, 1, 0.07, P(16), num_work, ctas, 0, None, None, P(32), None, None, None) == ARG
    assert b"too large" in mla.library().mla_last_error_string()
