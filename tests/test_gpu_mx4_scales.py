"""Products of 4-bit rows whose scales are anywhere in their range, at both ends of it
together and against each other."""
import math

import pytest

from test_gpu_mx4 import gen, join, plain_pack, sv, values  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F = torch.float32


@pytest.mark.parametrize("kind", ["mx4", "f32"])
@pytest.mark.parametrize("n,v", [(9, 255), (70, 255), (300, 255)])
def test_scales_of_all_sizes(sv, n, v, kind):  # noqa: F811
    """One block a row: row i's scale is 2^(i spread over -127 .. 127), column j's likewise."""
    h = 32
    g = gen(n)
    code = torch.randint(1, 8, (n, h), generator=g, device="cuda", dtype=torch.uint8)
    xe = torch.linspace(0, 254 if kind == "mx4" else 250, n, device="cuda").to(torch.uint8)[:, None]
    wc = torch.randint(0, 16, (v, h), generator=g, device="cuda", dtype=torch.uint8)
    we = torch.arange(v, device="cuda").to(torch.uint8)[:, None]
    code[:, 0] = 7                                        # (6: the scale that pack gives such a row is this one)
    a, b = values(code, xe), values(wc, we)
    hidden = sv.Mx4(join(code), xe, h) if kind == "mx4" else a.float()
    if kind != "mx4":
        assert torch.equal(hidden.double(), a)
        assert torch.equal(plain_pack(hidden)[1], xe)
    got = sv.head_logits(hidden, sv.Mx4(join(wc), we, h), out_dtype=F).double()
    want = a @ b.T
    size = a.abs() @ b.abs().T
    most = torch.finfo(F).max
    assert not torch.isnan(got).any()
    # sums that surely fit, whatever their order; subnormal ones may be taken for 0
    fits = size < most
    tol = size * h * 2.0 ** -24 + 2.0 ** -126
    assert ((got - want).abs() <= tol)[fits].all()
    beyond = want.abs() > most * 1.001
    assert torch.equal(got[beyond], want[beyond].sign() * math.inf)
