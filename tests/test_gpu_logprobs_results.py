"""What a caller may do with the tensors that logprobs returns: each is one of its own to
autograd, whatever the others are used for, and alternatives keep memory of their own."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import draft_verification_spec_amd as m
    m.load_library()
    return m


def rows(lead, v=1000):
    g = torch.Generator(device="cuda").manual_seed(len(lead) + v)
    return (torch.randn(*lead, v, generator=g, device="cuda"),
            torch.randint(0, v, lead, generator=g, device="cuda"))


@pytest.mark.parametrize("no_grad", [False, True])
@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("lead", [(), (1,), (7,), (2, 3)])
def test_in_place_under_autograd(sv, lead, top, no_grad):
    z, t = rows(lead)
    names = ["logp", "entropy", "lse", "norm"] + (["top_logp"] if top else [])
    for name in names:
        with torch.set_grad_enabled(not no_grad):
            r = sv.logprobs(z, t, top=top)
        before = {k: getattr(r, k).clone() for k in names}
        x = getattr(r, name)
        w = torch.full(x.shape, 0.5, device="cuda", requires_grad=True)
        x.add_(w)
        x.sum().backward()
        assert torch.equal(w.grad, torch.ones_like(w)), name
        assert torch.equal(x, before[name] + 0.5), name
        for other in set(names) - {name}:
            y = getattr(r, other)
            assert not y.requires_grad and y._version == 0 and torch.equal(y, before[other]), (name, other)


def test_changes_of_one_leave_what_another_saved(sv):
    z, t = rows((7,))
    r = sv.logprobs(z, t, top=3)
    w = torch.ones(7, device="cuda", requires_grad=True)
    loss = (w * r.logp).sum()
    r.entropy.neg_(), r.lse.zero_(), r.norm.zero_(), r.status.zero_(), r.top_logp.zero_(), r.top_idx.zero_()
    loss.backward()                                   # (a shared version would refuse it)
    assert torch.equal(w.grad, sv.logprobs(z, t).logp)


@pytest.mark.parametrize("lead", [(), (0,), (1,), (7,), (2, 3), (3, 0, 2)])
def test_shapes_and_memory(sv, lead):
    z, t = rows(lead) if 0 not in lead else (torch.zeros(*lead, 9, device="cuda"), torch.zeros(lead, dtype=torch.int64, device="cuda"))
    r = sv.logprobs(z, t, top=4)
    for x in (r.logp, r.entropy, r.lse, r.status):
        assert x.shape == lead and x.is_contiguous()
    assert r.norm.shape == (2, *lead) and r.top_logp.shape == r.top_idx.shape == (*lead, 4)
    assert r.status.dtype is r.top_idx.dtype is torch.int32
    # what a row's results keep alive is their own 24 bytes, not the alternatives
    assert r.logp.untyped_storage().nbytes() == 24 * t.numel()
    assert r.top_logp.untyped_storage().nbytes() == r.top_idx.untyped_storage().nbytes() == 16 * t.numel()
    assert not any(x._is_view() for x in r)
