"""Edges of the paged operators (GPU): ill-formed boundaries, waits that run
out, extreme sinks and scales, full sequences, and the sizes at which a
kernel's rule takes another form.  Tolerances are test_paged.py's unless a test
derives its own."""
import numpy as np
import pytest
import torch

from tests.paged_cases import Case
from tests.test_paged import append, attend, check_attend, fa  # noqa: F401

pytestmark = pytest.mark.gpu
INVALID = 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("mn", [2, 64])
def test_falling_boundaries_leave_the_others_right(fa, mn, fp8):  # noqa: F811
    """cu_new falls after runs of empty sequences, in a call with more tiles
    than CTAs: reported, and the well-formed sequences' rows are those of the
    call without the fall."""
    c = Case([30000, 0, 0, 20000, 0, 0], [2, 0, 0, 2, 0, 0], ps=64, fp8=fp8, seed=41)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    st, want, wl = attend(fa, c, t, max_new=mn)
    assert st == 0
    check_attend(c, t, want, wl, chunk=mn > 8)
    t["cu"] = torch.tensor([0, 2, 2, 2, 4, 2, 2], dtype=torch.int32, device="cuda")
    st, out, lse = attend(fa, c, t, max_new=mn)
    assert st == INVALID and torch.equal(out, want) and torch.equal(lse, wl)
    t["ctx"][5] = 5000000                                 # no new token: its length is not looked up
    st, out, lse = attend(fa, c, t, max_new=mn)
    assert st == INVALID and torch.equal(out, want) and torch.equal(lse, wl)
    assert append(fa, c, t) == INVALID
