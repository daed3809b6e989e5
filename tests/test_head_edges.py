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


def test_two_terms_belong_to_a_gradient():
    """The flag alone asks for nothing; with a gradient it has a size of its own."""
    lib = sv.load_library()

    def need(grads, dt=1, n=300, kd=False):
        s = sv.sv_head_shape_t(n, 64, 5000, dt, dt, grads, 0, 0, 1.0, -1, 4, 2, float("inf"))
        return (lib.sv_head_kd_workspace_bytes if kd else lib.sv_head_ce_workspace_bytes)(ctypes.byref(s))
    assert sv.GRAD_TWO_TERMS == 4
    for kd in (False, True):
        assert need(4, kd=kd) == need(8, kd=kd) == need(15, kd=kd) == 0
        for g in (1, 2, 3):
            assert need(g | 4, kd=kd) > need(g, kd=kd) > 0
            assert need(g | 4, dt=0, kd=kd) == need(g, dt=0, kd=kd) and need(g | 4, n=32, kd=kd) == need(g, n=32, kd=kd)
