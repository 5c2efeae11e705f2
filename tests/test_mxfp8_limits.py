"""CPU: refusals of sizes that the MXFP8 operators cannot count."""
import ctypes

import pytest

import sparse_mla_attention_fp8_gb300 as smla

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    smla.build()
    return smla.lib()


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 256])
@pytest.mark.parametrize("act", [0, 5])
def test_linear_refuses_tokens_beyond_32_bits(L, T, act):
    """A last tile behind them would not fit in 32 bits."""
    assert L.linear_mxfp8(FAKE, 32, FAKE, 4, FAKE, FAKE, 4, None, 0, act, None, 0, FAKE, None, None, 0, T, 8, 32, None) == -2
    assert b"T=" in L.smla_last_error()
