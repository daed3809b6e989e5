"""A row's log-probabilities in batches of other sizes and orders, and with and without
alternatives: the same bits where the rows are shared out alike, and elsewhere the same
alternatives with all results within the bounds of the arithmetic."""
import pytest

from test_gpu_logprobs import BF, F, Want, check_top, gen, sv  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("top", [0, 9])
@pytest.mark.parametrize("n,few,v", [(40, 33, 100003), (600, 200, 40001), (1500, 1024, 3001)])
def test_other_rows_and_orders(sv, n, few, v, top, dtype):  # noqa: F811
    """Some of the rows, in another order, shared out alike (in parts; 16 waves a row; four)."""
    z = torch.randn(n, v, generator=gen(n), device="cuda").to(dtype)
    t = torch.randint(0, v, (n,), generator=gen(v), device="cuda")
    a = sv.logprobs(z, t, 0.7, top=top)
    some = torch.randperm(n, generator=gen(1), device="cuda")[:few]
    b = sv.logprobs(z[some], t[some], 0.7, top=top)
    for k in ("logp", "entropy", "lse", "status") + (("top_logp", "top_idx") if top else ()):
        assert torch.equal(getattr(a, k)[some], getattr(b, k)), k
    assert torch.equal(a.norm[:, some], b.norm)
    g = torch.randn(n, generator=gen(2), device="cuda")
    da = sv.logprobs_grad(z, t, a, g, -g, 0.7)
    assert torch.equal(da[some], sv.logprobs_grad(z[some], t[some], b, g[some], -g[some], 0.7))


@pytest.mark.parametrize("dtype", [BF, F])
def test_across_the_ways_of_sharing(sv, dtype):  # noqa: F811
    """The same 60 rows alone and among 127, 128, 1023 and 1024, each with and without alternatives."""
    v, kept = 70001, 60
    z = torch.randn(1024, v, generator=gen(3), device="cuda").to(dtype)
    z[7, 11:60000] = z[7, 11]                              # equal entries across every share of a row
    z[8, 1000:] = -float("inf")
    t = torch.randint(0, 1000, (1024,), generator=gen(4), device="cuda")
    w = Want(z[:kept], t[:kept], 0.7)
    for n in (kept, 127, 128, 1023, 1024):
        for top in (0, 1, 32):
            r = sv.logprobs(z[:n], t[:n], 0.7, top=top)
            first = sv.LogprobsResult(r.logp[:kept], r.entropy[:kept], r.lse[:kept], r.norm[:, :kept], r.status[:kept],
                                      r.top_logp[:kept] if top else None, r.top_idx[:kept] if top else None)
            w.check(first, f"{n} rows, {top}")
            if top:
                check_top(first, w, z[:kept], top, f"{n} rows, {top}")
