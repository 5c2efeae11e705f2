"""GPU: the paged 8-bit K/V cache operators at the ends of what their entry
points take, against the float64 reference (tests/paged_reference.py)."""
import numpy as np
import pytest

import paged_reference as ref
from helpers import torch_mod
from test_gpu_paged import attend, check, smla  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- caps

def capped(b):
    """The expected results of a batch with a cap, within what holds without it: the cap's own part
    in the reference's tolerance (2^-20 of the cap) is no limit where the cap is far above the logits."""
    want, want_lse, _, _ = b.expected()
    _, _, tol, ltol = ref.attention(b.q, *b.caches, *b.scales, b.table, b.lens, b.query_start, b.sm_scale, b.window,
                                    0.0, b.slopes, b.prefix, b.doc)
    return want, want_lse, tol, ltol


@pytest.mark.parametrize("cap", [300.0, 1e4, 1e6, 1e9, 1e30])
@pytest.mark.parametrize("G,D,new", [(4, 128, [1, 1]), (3, 64, [2, 5]), (6, 64, [30, 70]), (4, 128, [40, 20])])
def test_wide_caps(smla, G, D, new, cap):  # noqa: F811
    """Caps far above the logits leave them as they are, with few rows and with many."""
    b = ref.Batch(70, 2, G, D, [500, 90], new, softcap=cap)
    check(b, attend(smla, b), capped(b))


@pytest.mark.parametrize("cap", [1e4, 1e6])
@pytest.mark.parametrize("G,D,new", [(4, 128, [1, 1]), (3, 64, [2, 5]), (6, 64, [30, 70])])
def test_wide_caps_beside_rows_that_reach_them(smla, G, D, new, cap):  # noqa: F811
    """One head's logits go up to the cap; the other heads', a hundred thousandth of it, keep their own precision."""
    b = ref.Batch(71, 2, G, D, [500, 90], new, softcap=cap)
    b.q[:, 0] *= np.float32(cap / 4)
    b.q = ref.bf16_round(b.q)
    check(b, attend(smla, b), capped(b))


# ---------------------------------------------------------------- failed calls

@pytest.mark.parametrize("many_rows", [False, True])
def test_a_wait_that_runs_out_is_reported_whatever_the_workspace(smla, many_rows):  # noqa: F811
    """A device thread waits in vain, and reports it as the attention's kernels do, into a workspace that nothing
    has cleared (as the ones that calls allocate for themselves): the device's status says so once."""
    torch = torch_mod()
    workspace = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    smla.read_device_status()
    assert smla.read_device_status() == 0
    smla.paged_wait_check(workspace, many_rows=many_rows)
    assert smla.read_device_status(workspace) == 1
    assert smla.read_device_status(workspace) == 0
    del workspace
    assert smla.read_device_status() == 1
    assert smla.read_device_status() == 0
