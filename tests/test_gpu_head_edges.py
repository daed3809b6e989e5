"""The vocabulary-head operators at the ends of their ranges: magnitudes next to the
smallest numbers, logits far from zero, launches of more than 2^32 work items,
indices beyond 32 bits, and the distillation's forms with several pieces of the
vocabulary or one gradient.  Tolerances as in test_gpu_head.py.
"""
import pytest

from test_gpu_head import BF, F, HALF, ce_case, check_ce, check_kd, gen, kd_case, log, plain_pack, sv, within  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ 8-bit rows
@pytest.mark.parametrize("h", [7, 300, 5000, 20001])
@pytest.mark.parametrize("dtype", [F, BF])
def test_act8_smallest_magnitudes(sv, h, dtype):  # noqa: F811
    """Scales that are subnormal, or next to the smallest normal number: the codes of
    the quotient rounded to even as if it were exact, in each of the row kernels."""
    log(f"act8 smallest magnitudes h={h} {dtype}")
    tops = [2.0 ** -149, 1e-44, 1e-43, 127 * 2.0 ** -149, 381 * 2.0 ** -149, 1e-42, 1e-41, 1e-40, 1e-38, 2.0 ** -126,
            1.5e-36, 2e-36, 1e-35, 1e-30, 1.28e-28]
    r = torch.rand(len(tops), h, generator=gen(h), device="cuda", dtype=torch.double) * 2 - 1
    x = (r * torch.tensor(tops, device="cuda", dtype=torch.double)[:, None]).float()
    x[:, 0] = torch.tensor(tops, device="cuda", dtype=torch.double).float()
    x = x.to(dtype)
    a = sv.act8_pack(x)
    codes, scale = plain_pack(x)
    assert torch.equal(a.scale, scale)
    assert torch.equal(a.codes, codes)
    # the same codes on the way into a product: a weight row of ones sums them
    ones = torch.ones(1, h, dtype=torch.int8, device="cuda")
    got = sv.head_logits(x, sv.Act8(ones, torch.ones(1, device="cuda")), out_dtype=F)
    s = codes.double().sum(1)
    within(got[:, 0], s * scale.double(), (s * scale.double()).abs() * 3 * HALF[F] + 2.0 ** -149, "row sums")
