"""Dropout's rate is p to the nearest 2^-16, also where fp32 rounds p * 65536 + 1/2 up."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [0, 1, 2, 255, 32767, 65534])
def test_rate_next_to_a_border(t):
    """The fp32 values around t + 1/2 of 65536: t below, t + 1 above."""
    border = np.float32((t + 0.5) / 65536)
    assert float(border) * 65536 == t + 0.5
    x = torch.ones(1024, 4096, device="cuda")
    y = torch.empty_like(x)
    rng = torch.tensor([11, t], dtype=torch.int64, device="cuda")
    for p, want in ((np.nextafter(border, np.float32(0)), t), (np.nextafter(border, np.float32(1)), t + 1)):
        dg.dropout(x, y, float(p), rng)
        kept = y[y != 0]
        assert bool((kept == float(np.float32(65536.0 / (65536 - want)))).all())
        assert (kept.numel() == y.numel()) == (want == 0)
