"""The 64-bit reading of the paged cache against the dense oracle and by hand."""
import numpy as np
import pytest
import torch

from oracle import ref
from paged_ref import Cache, attend, quantise


@pytest.mark.parametrize("Nq,causal,window", [(1, True, -1), (3, True, -1), (3, True, 5), (2, False, 4), (4, False, -1)])
def test_paged_equals_the_dense_decode_oracle(Nq, causal, window):
    c = Cache([37], 2, 64, 8, "bf16", "nhd", seed=1).fill_random(2)
    q = torch.randn((1, 6, Nq, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    k = torch.from_numpy(c.rows("k", 0, torch.arange(37))).transpose(0, 1)[None]
    v = torch.from_numpy(c.rows("v", 0, torch.arange(37))).transpose(0, 1)[None]
    want_o, want_l = ref.forward(q, k, v, 0.125, causal, window)
    o, lse, _, _ = attend(c, q, causal, window)
    np.testing.assert_allclose(o, want_o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, want_l, rtol=1e-12, atol=1e-12)


def test_short_and_empty_sequences_leave_empty_rows():
    c = Cache([0, 1, 2], 1, 64, 4, "bf16", seed=4).fill_random(5)
    q = torch.ones((3, 1, 2, 64), dtype=torch.bfloat16)
    o, lse, _, _ = attend(c, q, True, -1)
    assert np.isinf(lse[0]).all() and np.isinf(lse[1, 0, 0]) and np.isfinite(lse[1, 0, 1]) and np.isfinite(lse[2]).all()
    assert (o[0] == 0).all() and (o[1, 0, 0] == 0).all()
    np.testing.assert_allclose(o[1, 0, 1], c.rows("v", 1, torch.tensor([0]))[0, 0])


def test_a_missing_page_hides_its_tokens():
    c = Cache([20], 1, 64, 4, "bf16", seed=6).fill_random(7)
    q = torch.randn((1, 1, 1, 64), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    full = attend(c, q, True, -1)[1]
    keep = c.table[0, 2].item()
    for bad in (-1, c.P, 2 ** 31 - 1):
        c.table[0, 2] = bad
        assert attend(c, q, True, -1)[1] < full
    c.table[0, 2] = keep


def test_quantised_rows_come_back_within_half_a_step():
    x = torch.randn((50, 3, 64), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    x[0, 0] = 0
    x[1, 1] *= 1e-30
    code, scale = quantise(x)
    y = code.double() * scale.double()[..., None]
    # half a step of e4m3 is 2^-4 of the value, or 2^-10 codes where they are subnormal; the two fp32
    # roundings of x * (448 / a) and of the scale add three times 2^-24
    tol = x.double().abs() * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10 * scale.double()[..., None]
    assert ((y - x.double()).abs() <= tol).all()
    assert (y[0, 0] == 0).all() and (scale > 0).all()
