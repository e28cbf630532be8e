"""Widths that take turns in one process: a kernel that has served a narrow
row still has the shared memory of the wide one it served before."""
import pytest
import torch

from test_gpu_gated_norm import Case, check_backward, check_forward

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# of a kernel's rings (bytes per block): forward 65536 / 49152 / 98304 / 73728, backward 65536 / 40960 / 98304 / 61440
# and 131072 / 98304 / 196608 / 147456, each wide one before and after its narrow one
WIDTHS = (8192, 6144, 8192, 4096, 2560, 4096, 2560, 8192)


@pytest.mark.parametrize("mod", [True, False])
@pytest.mark.parametrize("xt", [BF16, F32], ids=str)
def test_wide_narrow_wide(xt, mod):
    first = {}
    for D in WIDTHS:
        c = Case(3, D, mod=mod, weights=not mod, post=0 if mod else 1, xt=xt, seed=D)
        amax, amax_dy = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        r, h, stats = c.forward(amax_h=amax)
        out = c.backward(r, stats, amax_dy=amax_dy)
        check_forward(c, r, h, stats, amax)
        check_backward(c, r, stats, out, amax_dy)
        got = [r, h, stats, out.dx, out.dy]
        want = first.setdefault(D, got)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), D
