"""Factors that are finite as doubles but not in the step's arithmetic (no GPU needed)."""
import pytest

from test_optim_api import F16, F32, F64, INVALID, OK, BF16, status, tensor


@pytest.mark.parametrize("name", ["lr_scale", "weight_decay"])
def test_factors_beyond_the_arithmetics_type_are_refused(name):
    for dtype in (F32, BF16, F16):
        assert status([tensor(dtype=dtype, **{name: 1e39})]) == INVALID
        assert status([tensor(dtype=dtype, **{name: 1e38})]) == OK
    assert status([tensor(dtype=F64, **{name: 1e39})]) == OK
