"""Rows whose sum of squares fp32 cannot hold: what the header says of them, and that no other row
notices."""
import pytest
import torch

from test_qk_rope import make, run


@pytest.mark.gpu
@pytest.mark.parametrize("value,count,eps", [(2e19, 1, 1e-6), (1.7e18, 128, 1e-6), (3e38, 128, 1e-6), (1e-24, 128, 0.0)])
def test_rows_beyond_the_sum_of_squares(gcs_lib, value, count, eps):
    c = make(7, 4, 2, 128, 128, seed=26)
    (q0, k0), (dq0, dk0, _, _) = run(gcs_lib, c, eps)
    c["q"][3, 2, :count] = value
    c["k"][5, 1, :count] = -value
    (q, k), (dq, dk, _, _) = run(gcs_lib, c, eps)
    for got, was, t, h in ((q, q0, 3, 2), (k, k0, 5, 1), (dq, dq0, 3, 2), (dk, dk0, 5, 1)):
        rest = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
        rest[t, h] = False
        assert torch.equal(got[rest], was[rest])
        row = got[t, h]
        if value > 1:  # the sum is infinite
            assert bool(((row == 0) | torch.isnan(row)).all())
        else:  # the sum is 0
            assert not bool(torch.isfinite(row).any())
    # just inside, the rows are as ever
    c["q"][3, 2] = 1e15
    (q, _), _ = run(gcs_lib, c, eps)
    assert bool(torch.isfinite(q[3, 2]).all()) and bool((q[3, 2] != 0).any())
