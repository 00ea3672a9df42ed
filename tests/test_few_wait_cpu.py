"""The setting of how long the few-token layer's blocks wait, on the host."""
import pytest

import routing_expert_ffn_router_amd as moe


def test_the_number_is_set_and_returned():
    first = moe.few_wait_polls()
    assert first == 1 << 20
    try:
        assert moe.few_wait_polls(5) == first
        assert moe.few_wait_polls() == 5 and moe.few_wait_polls(-7) == 5
        assert moe.few_wait_polls(0) == 5 and moe.few_wait_polls((1 << 31) - 1) == 0
        with pytest.raises(ValueError):
            moe.few_wait_polls(1 << 31)
        assert moe.few_wait_polls() == (1 << 31) - 1
    finally:
        moe.few_wait_polls(first)
