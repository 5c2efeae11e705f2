"""CPU: what the entry points of the paged K/V cache operators refuse at the
ends of their arguments' ranges (before any device work)."""
import pytest

from test_paged import L, ODD, _attend  # noqa: F401


@pytest.mark.parametrize("cap", [1e31, 2.4e38, 3e38, 9e-21, 1e-38, 1e-45])
def test_attention_refuses_caps_that_float32_does_not_hold(L, cap):  # noqa: F811
    """cap log2(e) overflows from 2.36e38 on, the rows' factors over the cap lose bits from about 1e33 on, and
    1 / cap overflows for subnormal ones."""
    assert _attend(L, cap=cap, T=0, q=None) == -1
    assert b"softcap" in L.smla_last_error()


@pytest.mark.parametrize("cap", [0.0, 1e-20, 1.0, 1e30])
def test_attention_takes_other_caps(L, cap):  # noqa: F811
    assert _attend(L, cap=cap, T=0, q=None) == 0


def test_wait_check_refuses(L):  # noqa: F811
    assert L.smla_paged_wait_check(0, None, None) == -1
    assert L.smla_paged_wait_check(1, ODD, None) == -1
