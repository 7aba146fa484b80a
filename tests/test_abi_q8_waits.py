"""Limits that the 8-bit kernels' waits may not have (no GPU)."""

import pytest

import fsdp_sharded_optimizer_flatparameter_gb300 as zs


@pytest.mark.parametrize("limit", [-1, 2 ** 32 + 1])
def test_limits_out_of_range_are_refused(limit):
    with pytest.raises(zs.ZsError, match="zs_set_q8_wait_limit: "):
        zs.zs_set_q8_wait_limit(limit)


@pytest.mark.parametrize("limit", [0, 1, 2 ** 32])
def test_limits_in_range_are_taken(limit):
    assert zs.zs_set_q8_wait_limit(limit) == zs.ZS_OK
    assert zs.zs_set_q8_wait_limit() == zs.ZS_OK
