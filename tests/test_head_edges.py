"""The vocabulary-head operators' refusals at the ends of their ranges, without a GPU."""
import ctypes

import pytest

import draft_verification_spec_amd as sv

torch = pytest.importorskip("torch")

FAKE, WS = 0x1000, 0x100000                           # never dereferenced: every call below is refused first


def test_logits_beyond_one_launch():
    """Logits that no launch of tiles covers (more than 500 GB) have no size and are
    refused before anything is enqueued."""
    lib = sv.load_library()
    for n, v in ((1 << 20, 1 << 24), (1 << 30, 1 << 9), ((1 << 31) - 1, 129)):
        s = sv.sv_logits_shape_t(n, 64, v, 2, 1, 0, 0, 0)
        assert lib.sv_head_logits_workspace_bytes(ctypes.byref(s)) == 0, (n, v)
        assert lib.sv_head_logits(ctypes.byref(s), FAKE, FAKE, FAKE, FAKE, FAKE, WS, 1 << 60, None) == sv.SV_ERR_SHAPE
    for n, v in ((1 << 20, 1 << 17), (1 << 30, 100), (32, 1 << 24)):
        s = sv.sv_logits_shape_t(n, 64, v, 2, 1, 0, 0, 0)
        assert lib.sv_head_logits_workspace_bytes(ctypes.byref(s)) > 0, (n, v)
