"""What the layer operators refuse for the size of their launches (no GPU
needed): a call is taken when the launches it makes have fewer than 2^24
workgroups of 256 threads, and refused with GDR2_ERR_UNSUPPORTED before any of
them otherwise.  Every pointer is NULL, so that a call whose sizes are taken
ends at the check of its workspace or its pointers and launches nothing."""
import ctypes

import pytest

from gated_delta_rule_86_amd import gdr2, layer
from tests.test_boundary_host import _gpu_visible, lib  # noqa: F401

pytestmark = pytest.mark.skipif(_gpu_visible(), reason="compute units of the machine without a GPU are assumed")

UNS = gdr2.ERR_UNSUPPORTED


def taken(lib, entry, args):  # noqa: F811
    status = getattr(lib, entry)(ctypes.byref(args), None)
    assert status in (gdr2.ERR_INVALID_ARG, gdr2.ERR_WORKSPACE, UNS), status
    if status == gdr2.ERR_INVALID_ARG:
        assert b"is NULL" in lib.gdr2_last_error(), lib.gdr2_last_error()
    return status != UNS


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("C,B,ok", [
    # one channel takes one lane of eight: 32 sequences of a token a workgroup
    (1, (1 << 29) - 64, True), (1, 1 << 29, False),
    # 65 channels, one by one: two blocks of 64 lanes, four sequences each; (B, T) beyond that is refused
    (65, (1 << 25) - 64, True), (65, 1 << 25, False),
    # 64: one block, in fours 16 lanes of 16 sequences
    (64, (1 << 26) - 64, True), (64, 1 << 26, False),
])
def test_conv_backward(lib, C, B, ok, packed):  # noqa: F811
    """Its grid rounds the channels up to blocks of 8 to 64 lanes."""
    a = layer.ConvBwdArgs(B=B, T=0 if packed else 1, C=C, x_stride=C, width=4, dtype=gdr2.F32)
    if packed:
        a.offsets = 1 << 40           # read on the device only
    assert taken(lib, "gdr2_conv_backward", a) == ok
    assert (lib.gdr2_conv_backward_workspace_size(ctypes.byref(a)) > 0) == ok
