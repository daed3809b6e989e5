"""The logits' gradient at temperatures down to the smallest that are taken, where the
factors of the formula leave fp32 though its results, or most of them, do not."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import draft_verification_spec_amd as m
    m.load_library()
    return m


def want(z, t, g, h, T):
    """The formula in 64 bits on the CPU, and how far off fp32 may be before the last rounding."""
    z, g, h, T = z.double().cpu(), g.double().cpu(), h.double().cpu(), torch.tensor(T, dtype=F).double().item()
    y = (z - z.amax(1, keepdim=True)) / T
    lp = y - torch.logsumexp(y, 1, keepdim=True)
    p = lp.exp()
    entropy = torch.special.entr(p).sum(1, keepdim=True)
    one = torch.zeros_like(p).scatter_(1, t.long().cpu()[:, None], 1.0)
    d = (g[:, None] * (one - p) - h[:, None] * p * (lp.clamp(min=-1e4) + entropy)) / T
    # Probabilities here are 0, or equal shares of 1 / k, k a power of two: log2 of one is off by
    # the roundings of ln k, of two constants and products of magnitude log2 k, its exponential by
    # a step more; ln 2 and the entropy by half a step each.
    logs = math.log(z.shape[1]) + 1
    off = p * (g.abs() + 2 * h.abs() * logs)[:, None] * (8 * logs + 8) * U / T + one * g.abs()[:, None] * 3 * U / T
    return d, off


@pytest.mark.parametrize("dtype,out", [(F, F), (BF, BF), (F, BF)])
@pytest.mark.parametrize("T", [4.3e-39, 1e-38, 1e-36, 1e-33, 1e-20, 1.0])
def test_smallest_temperatures(sv, dtype, out, T):
    """Rows of 1, 2, 4 .. equal largest logits among others far below, in units of T; gradients of
    usual size, which 1 / T carries beyond fp32 at the largest entries of some."""
    n, v = 6, 300
    gen = torch.Generator(device="cuda").manual_seed(2)
    z = -1 - torch.rand(n, v, generator=gen, device="cuda") * 100
    t = torch.arange(n, device="cuda") * 40
    for i in range(n):
        z[i, torch.randperm(v, generator=gen, device="cuda")[:1 << i]] = 4096.0     # (T = 1: below them by e^-4097)
    z = z.to(dtype)
    for scale in (0.0, 1e-4, 1.0, 100.0):
        for both in (0.0, -0.01, 1.0):
            g, h = torch.randn(n, generator=gen, device="cuda") * scale, torch.full((n,), both, device="cuda")
            r = sv.logprobs(z, t, T)
            got = sv.logprobs_grad(z, t, r, g, h if both else None, T, out_dtype=out).cpu()
            d, off = want(z, t, g, h, T)
            assert not torch.isnan(got).any(), (T, scale, both)
            # beyond the type (surely, as near as it may round) infinite; else within the bound
            big = torch.finfo(out).max
            err = off + d.abs() * torch.finfo(out).eps / 2 + 1e-38
            assert (got[d.abs() - err > big * 1.01] == torch.sign(d[d.abs() - err > big * 1.01])
                    * math.inf).all(), (T, scale, both)
            fits = d.abs() + err < big
            assert ((got.double() - d).abs() <= err)[fits].all(), (T, scale, both)
            assert not got[(d == 0)].any(), (T, scale, both)
