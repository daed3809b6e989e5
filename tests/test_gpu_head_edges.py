"""The vocabulary-head operators at the ends of their ranges: magnitudes next to the
smallest numbers, logits far from zero, launches of more than 2^32 work items,
indices beyond 32 bits, and the distillation's forms with several pieces of the
vocabulary or one gradient.  Tolerances as in test_gpu_head.py.
"""
import pytest

from test_gpu_head import (BF, F, HALF, ce_case, check_ce, check_gradients, check_kd, gen, kd_case, log,  # noqa: F401
                           plain_pack, reference, rows_of, sv, within)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ 8-bit rows
@pytest.mark.parametrize("h", [7, 300, 5000, 20001])
@pytest.mark.parametrize("dtype", [F, BF])
def test_act8_smallest_magnitudes(sv, h, dtype):
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


# --------------------------------------------------------------- cross entropy
@pytest.mark.parametrize("n,h,v,dtype", [(9, 1001, 130000, F), (24, 1152, 262144, F), (20, 1001, 250000, BF), (9, 1000, 300000, BF)])
def test_ce_pieces_keep_the_bits(sv, n, h, v, dtype):
    """Few rows whose vocabulary is cut otherwise with gradients than without: the
    same bits of the loss and of each gradient whatever is asked for."""
    log(f"head_ce bits over pieces n={n} h={h} v={v} {dtype}")
    hidden, _, w, t, u = ce_case(sv, n, h, v, dtype, "same", 1.0, n + h)
    both = sv.head_ce(hidden, w, t, u)
    for grad in (False, "hidden", "weight"):
        r = sv.head_ce(hidden, w, t, u, grad=grad)
        for name in ("loss", "nll", "lse", "status"):
            assert torch.equal(getattr(r, name), getattr(both, name)), (grad, name)
        if grad == "hidden":
            assert torch.equal(r.grad_hidden, both.grad_hidden)
        if grad == "weight":
            assert torch.equal(r.grad_weight, both.grad_weight)


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("n", [4, 40, 300])
def test_sure_rows(sv, n, dtype):
    """Rows whose target stands far above the others: nll is what the exponentials'
    rounding leaves of 0, at any size of the logits, and never negative.  Logits are
    exact here (one product each, of powers of two and small numbers).  The largest
    exponential is 2 to the rounding of its own exponent: one rounding, one of the
    hardware's last place, 2^-23 each; the distillation's the same."""
    log(f"head_ce, head_kd sure rows n={n} {dtype}")
    z = torch.tensor([30.0, 100, 300, 1000, 1100, 9984, 28672], device="cuda")
    v = 700
    for sign in (1, -1):                              # 28672 above the others, which are at 0, or 0 above them
        w = torch.zeros(v, 64, device="cuda")
        w[7, 0] = 1
        x = torch.zeros(n, 64, device="cuda")
        x[:, 0] = z[torch.arange(n, device="cuda") % len(z)]
        if sign < 0:
            w[:, 0] -= 1
        x, w = x.to(dtype), w.to(dtype)
        t = torch.full((n,), 7, device="cuda")
        r = sv.head_ce(x, w, t)
        top = x[:, 0].double() if sign > 0 else torch.zeros(n, device="cuda").double()
        rest = (v - 1) * torch.exp(-x[:, 0].double())
        bound = rest + 2.0 ** -22
        assert not r.status.any() and (r.nll >= 0).all() and float(r.loss) >= 0
        within(r.nll, torch.zeros_like(top), bound, "nll")
        within(r.lse, top, bound + HALF[F] * top, "lse")
        val = torch.full((n, 32), -float("inf"), device="cuda")
        val[:, 3] = 1
        ids = torch.full((n, 32), -1, device="cuda")
        ids[:, 3] = 7
        k = sv.head_kd(x, w, val, ids, torch.arange(n, device="cuda") % 4, torch.ones(4, device="cuda"), 4)
        within(k.kl, torch.zeros_like(top), bound, "kl")


# ------------------------------------- launches of more than 2^32 work items
def test_act8_rows_beyond_one_launch(sv):
    """2^24 rows where a workgroup takes a row, 2^26 where it takes four: all rows, by
    the C entries at an odd distance and by the front end; then into a product."""
    import ctypes
    lib = sv.load_library()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    n, h = (1 << 24) + 5, 3
    log(f"act8 n={n} h={h}")
    x = torch.randn(n, h, generator=gen(5), device="cuda").to(BF)
    codes, scale = torch.full((n, h), 99, dtype=torch.int8, device="cuda"), torch.full((n,), -1.0, device="cuda")
    assert lib.sv_act8_pack(n, h, 1, p(x), 0, p(codes), 0, p(scale), st) == 0
    c, s = plain_pack(x)
    assert torch.equal(codes, c) and torch.equal(scale, s)
    del x, codes, scale, c, s
    n = (1 << 26) + 7
    log(f"act8 n={n} h=1")
    x = torch.randn(n, 1, generator=gen(6), device="cuda").to(BF)
    a = sv.act8_pack(x)
    c, s = plain_pack(x)
    assert torch.equal(a.codes, c) and torch.equal(a.scale, s)
    y = (c.float() * s[:, None]).to(BF)
    assert torch.equal(sv.act8_unpack(a), y)
    log("head_logits of as many rows")
    w = sv.Act8(torch.full((1, 1), 127, dtype=torch.int8, device="cuda"), torch.full((1,), 2.0 ** -7, device="cuda"))
    want = (c.double() * 127) * (s.double() * 2.0 ** -7)[:, None]
    for hidden in (a, x):
        got = sv.head_logits(hidden, w, out_dtype=F)
        assert bool(((got.double() - want).abs() <= want.abs() * 2 * HALF[F]).all())


@pytest.mark.parametrize("h", [32, 20])
def test_ce_forward_beyond_one_launch(sv, h):
    """2^20 rows of 65700 entries in fp32, a head read in place and one that is copied:
    the tiles of the forward product are more than a launch holds.  64 rows, each
    many times; targets in the last columns too."""
    n, v, k = 1 << 20, 65700, 64
    log(f"head_ce n={n} h={h} v={v}")
    g = gen(h)
    base = torch.randn(k, h, generator=g, device="cuda")
    w = torch.randn(v, h, generator=g, device="cuda") * 3 / h ** 0.5
    at = torch.cat([torch.arange(32, device="cuda") * 97, v - 1 - torch.arange(32, device="cuda") * 13])
    z = base.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    nll = lse - z.gather(1, at[:, None])[:, 0]
    # as in test_gpu_head.py: both logits' sums, and the exponents
    e = 2 * (h + 8) * 2.0 ** -24 * (base.double().abs() @ w.double().abs().T).amax(1) + 2.0 ** -18 * (1 + lse.abs() / 16) + 2.0 ** -22 * nll
    r = sv.head_ce(base.repeat(n // k, 1), w, at.repeat(n // k), grad=False)
    assert not r.status.any()
    for got, want in ((r.nll, nll), (r.lse, lse)):
        rows = got.view(-1, k)
        assert bool((rows == rows[:1]).all())
        within(rows[0], want, e, "rows")
    total = r.nll.double().sum()
    within(r.loss, total[None], total.abs()[None] * 2.0 ** -23, "loss")


def test_ce_hidden_gradient_beyond_one_launch(sv):
    """2^20 rows of 4096 in fp32: the sums of the hidden gradient take more than a launch."""
    n, h, v, k = 1 << 20, 4096, 60, 64
    log(f"head_ce grad_hidden n={n} h={h} v={v}")
    g = gen(3)
    base = torch.randn(k, h, generator=g, device="cuda")
    w = torch.randn(v, h, generator=g, device="cuda") * 3 / h ** 0.5
    at = torch.arange(k, device="cuda") % v
    x = base.repeat(n // k, 1)
    r = sv.head_ce(x, w, at.repeat(n // k), grad="hidden")
    del x
    assert not r.status.any()
    rows = r.grad_hidden.view(-1, k, h)
    for i in range(0, n // k, 2048):                  # each row's sums are its own
        assert bool((rows[i:i + 2048] == rows[:1]).all()), i
    pt = torch.nn.functional.one_hot(at, v).double()
    ones = torch.ones(k, device="cuda").double()
    ref = reference(base.double(), w.double(), pt, ones, 1.0)
    check_gradients(r._replace(grad_hidden=rows[0]), ref, base.double(), w.double(), F, ("hidden",))


def test_sizes_beyond_32_bits_are_refused(sv):
    """Counts of 2^32 and a few: refused, not taken for the few (broadcast rows, so that
    they need no memory)."""
    def many(shape, dtype, value=0):
        return torch.full((1,) * len(shape), value, dtype=dtype, device="cuda").expand(*shape)
    n = (1 << 32) + 5
    codes, scale = many((n, 1), torch.int8), many((n,), F)
    w = sv.Act8(torch.ones(3, 1, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"))
    x, t = torch.zeros(4, 1, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    log("sizes beyond 32 bits")
    calls = [lambda: sv.act8_pack(many((n, 1), BF)), lambda: sv.act8_pack(many((1 << 16, 1 << 16, 1), BF)),
             lambda: sv.act8_unpack(sv.Act8(codes, scale)),
             lambda: sv.head_logits(sv.Act8(codes, scale), w), lambda: sv.head_logits(many((n, 1), BF), w),
             lambda: sv.head_logits(x, sv.Act8(codes, scale)),
             lambda: sv.head_ce(many((n, 1), F), torch.ones(3, 1, device="cuda"), many((n,), torch.int32)),
             lambda: sv.head_ce(x, many((n, 1), F), t)]
    val, ids, rs = torch.zeros(4, 32, device="cuda"), torch.arange(32, device="cuda").expand(4, 32), t
    head, one = torch.zeros(40, 1, device="cuda"), torch.ones(4, device="cuda")
    calls += [lambda: sv.head_kd(x, head, val, ids, rs, one, (1 << 32) + 4),
              lambda: sv.head_kd(x, head, val, ids, rs, one, 4 - (1 << 32)),
              lambda: sv.head_kd(x, head, val, ids, rs, many((1 << 32,), F, 1), 4)]
    assert sv.head_kd(x, head, val, ids, rs, one, 4).status.tolist() == [0] * 4
    for i, call in enumerate(calls):
        with pytest.raises(sv.SpecVerifyError) as e:
            call()
        assert e.value.code == sv.SV_ERR_SHAPE, i


@pytest.mark.parametrize("ignore", [-(1 << 31), (1 << 31) - 1, -1, 3, -100])
def test_targets_beyond_32_bits_are_not_ignored(sv, ignore):
    """64-bit targets outside 32 bits are bad targets, whatever index is ignored; those
    that are that index are left out."""
    log(f"targets beyond 32 bits, ignore_index={ignore}")
    x = torch.randn(9, 64, generator=gen(1), device="cuda")
    w = torch.randn(50, 64, generator=gen(2), device="cuda")
    far = [-(1 << 40), 1 << 40, -(1 << 31) - 1, 1 << 31, (1 << 32) + 3, -(1 << 63), (1 << 63) - 1]
    t = torch.tensor([1, ignore, *far], device="cuda")
    r = sv.head_ce(x, w, t, ignore_index=ignore)
    assert r.status.tolist() == [0, 0] + [sv.HEAD_BAD_TARGET] * len(far)
    assert float(r.nll[0]) > 0 and float(r.nll[1]) == 0 and torch.isnan(r.nll[2:]).all()
    assert not r.grad_hidden[1:].any()


# ---------------------------------------------------------------- distillation
#: rows, width, vocabulary, type, kind of rows, and the pieces of the vocabulary that the
#: call takes with gradients (test_head_plans.py holds them against the host's plan)
KD_PIECES = [(2048, 128, 151936, BF, "same", 3, 50688), (1500, 128, 100000, F, "same", 3, 33536),
             (1100, 64, 151936, BF, "i8", 2, 76032), (1030, 64, 151936, F, "i8", 3, 50688),
             (20, 1001, 250000, BF, "same", 2, 125184), (9, 1001, 130000, F, "same", 2, 65024)]


def kd_piece_case(sv, n, h, v, dtype, kind, piece, seed):
    """Stored ids on both sides of every piece's border, the last entry and the first."""
    g = gen(seed)
    hidden, x = rows_of(kind, n, h, g, dtype, sv)
    w = (torch.randn(v, h, generator=g, device="cuda") * 3 / h ** 0.5).to(dtype)
    edge = sorted({0, v - 1} | {b + d for b in range(piece, v, piece) for d in (-1, 0, 1) if b + d < v})
    ids = torch.empty(n, 32, dtype=torch.int64, device="cuda")
    ids[:, :len(edge)] = torch.tensor(edge, device="cuda")
    # the others: steps of 40 from a place of the row's own, none of them an edge
    start = 4 + torch.randint(0, piece - 2000, (n, 1), generator=g, device="cuda") + torch.arange(n, device="cuda")[:, None] % 2 * piece
    ids[:, len(edge):] = start.clamp(max=v - 1400) + 40 * torch.arange(32 - len(edge), device="cuda")
    ids = ids.gather(1, torch.argsort(torch.rand(n, 32, generator=g, device="cuda"), 1))
    val = 10 + 2 * torch.randn(n, 32, generator=g, device="cuda")
    val[0, 3] = -float("inf")
    ids[n // 2, 5] = -1
    rewards = torch.rand(4 * -(-n // 12), generator=g, device="cuda")
    rewards[::5] = 0                                  # rows without a gradient, between the others
    return hidden, x, w, val, ids, torch.arange(n, device="cuda") // 3, rewards, 4


@pytest.mark.parametrize("n,h,v,dtype,kind,pieces,piece", KD_PIECES)
def test_kd_several_pieces(sv, n, h, v, dtype, kind, pieces, piece):
    """Distillation over several pieces, of more rows than find their own places (and of
    few): all results, and each gradient alone with the same bits."""
    log(f"head_kd pieces n={n} h={h} v={v} {dtype} {kind}")
    case = kd_piece_case(sv, n, h, v, dtype, kind, piece, n)
    check_kd(sv, *case, dtype, w_max=0.6)
    same_kd_bits(sv, case, w_max=0.6)


def same_kd_bits(sv, case, **kw):
    hidden, _, w, val, ids, rs, rewards, group = case
    call = lambda grad: sv.head_kd(hidden, w, val, ids, rs, rewards, group, grad=grad, **kw)  # noqa: E731
    both = call(True)
    assert both.grad_hidden.any() and both.grad_weight.any()
    for grad in (False, "hidden", "weight"):
        r = call(grad)
        for name in ("loss", "kl", "weight", "status"):
            assert torch.equal(getattr(r, name), getattr(both, name)), (grad, name)
        assert r.grad_hidden is None if grad != "hidden" else torch.equal(r.grad_hidden, both.grad_hidden)
        assert r.grad_weight is None if grad != "weight" else torch.equal(r.grad_weight, both.grad_weight)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("kind", ["same", "i8"])
@pytest.mark.parametrize("n,h,v", [(8, 200, 3000), (40, 200, 3000), (64, 72, 501), (150, 130, 2500), (1100, 64, 900),
                                   (300, 100, 22000)])
def test_kd_one_gradient_is_the_same(sv, n, h, v, dtype, kind):
    """The distillation's loss and each gradient alone: the bits of the call for both,
    which are checked against the formulas."""
    log(f"head_kd one gradient n={n} h={h} v={v} {dtype} {kind}")
    case = kd_case(sv, n, h, v, dtype, kind, n + v)
    check_kd(sv, *case, dtype)
    same_kd_bits(sv, case)


# ---------------------------------------------------- how near the gradients are
def near_case(sv, op, n, h, v, dtype, kind, seed):
    """Rows near a few entries of the head, as a trained drafter's are: the gradients
    hang on few entries of dz.  The call, and the exact dz, rows and head."""
    g = gen(seed)
    w = (torch.randn(v, h, generator=g, device="cuda") * 3 / h ** 0.5).to(dtype)
    ids = (torch.randint(0, v, (n, 1), generator=g, device="cuda") + 37 * torch.arange(32, device="cuda")) % v
    x = torch.randn(n, h, generator=g, device="cuda") + w[ids[:, :4 if op == "kd" else 1]].float().sum(1)
    if kind == "i8":
        hidden = sv.act8_pack(x)
        x = hidden.codes.double() * hidden.scale.double()[:, None]
    else:
        hidden = x.to(dtype)
        x = hidden.double()
    rows = torch.arange(n, device="cuda")
    pt = torch.zeros(n, v, dtype=torch.double, device="cuda")
    if op == "kd":
        val = 10 + 2 * torch.randn(n, 32, generator=g, device="cuda")
        rewards = 0.25 + torch.rand(4, generator=g, device="cuda")
        pt[rows[:, None], ids] = torch.softmax(val.double(), 1)
        u = (rewards.double() / rewards.double().sum())[rows % 4]
        call = lambda **kw: sv.head_kd(hidden, w, val, ids, rows % 4, rewards, 4, **kw)  # noqa: E731
    else:
        weight = torch.randn(n, generator=g, device="cuda") / n
        pt[rows, ids[:, 0]] = 1
        u = weight.double()
        call = lambda **kw: sv.head_ce(hidden, w, ids[:, 0], weight, **kw)  # noqa: E731
    return call, reference(x, w.double(), pt, u, 1.0), x, w.double(), u


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


#: a bf16 result's rounding alone: uniform within half a step, 2^-7 / sqrt(12) of the power of two below it, 0.0016 to
#: 0.0017 of the norm of results whose leading digits are spread; what two terms leave of dz is 2^-17
ROUNDED = 0.002


def check_two_terms(r, ref, x, w):
    dz, edz = ref["dz"], ref["edz"] + 2.0 ** -16 * ref["dz"].abs() + 1e-40
    for name, got, a, ea, b in (("hidden", r.grad_hidden, dz, edz, w), ("weight", r.grad_weight, dz.T, edz.T, x)):
        want = a @ b
        tol = ea @ b.abs() + (b.shape[0] + 8) * 2.0 ** -24 * (a.abs() @ b.abs())
        within(got, want, tol + HALF[BF] * (want.abs() + tol) + 1e-38, name)
        assert off(got, want) <= ROUNDED, name


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("kind", ["same", "i8"])
@pytest.mark.parametrize("n,h,v", [(24, 1024, 20000), (5, 520, 3001), (32, 200, 70000), (17, 1001, 9000)])
def test_few_rows_in_two_terms(sv, op, n, h, v, kind):
    """Up to 32 rows in bf16: the gradients are off by their own rounding, which dz in
    one term exceeds."""
    log(f"two terms {op} n={n} h={h} v={v} {kind}")
    call, ref, x, w, _ = near_case(sv, op, n, h, v, BF, kind, n + h)
    check_two_terms(call(), ref, x, w)
    if (n, kind) == (24, "same"):                     # what one term would give
        want = ref["dz"] @ w
        assert off((ref["dz"].to(BF).double() @ w).to(BF), want) > ROUNDED


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("kind", ["same", "i8"])
@pytest.mark.parametrize("n,h,v", [(24, 512, 20000), (9, 1001, 130000), (100, 512, 9000), (300, 256, 60000), (1100, 64, 30000)])
def test_float32_gradients_are_near(sv, op, n, h, v, kind):
    """fp32: dz is off by the rounding of its logits (below 32), of their sum and of its
    scaling, each uniform within half a step of 2^-20: 2^-20 sqrt(2 / 3) of u exp(z - lse)
    in the mean.  Roundings of different entries are independent, so the gradients' norms
    are off by no larger a share; 2^-20 leaves the exponentials a part."""
    log(f"float32 {op} n={n} h={h} v={v} {kind}")
    call, ref, x, w, u = near_case(sv, op, n, h, v, F, kind, n + h)
    assert float(ref["z"].abs().max()) < 32
    r = call()
    share = float((torch.exp(ref["z"] - ref["lse"][:, None]) * u[:, None]).norm() / ref["dz"].norm())
    for name, got, want in (("hidden", r.grad_hidden, ref["dz"] @ w), ("weight", r.grad_weight, ref["dz"].T @ x)):
        assert off(got, want) <= 2.0 ** -20 * max(share, 1.0), (name, off(got, want), share)


#: more than 32 rows: one step of rows, ragged ones, each tile, dW's tiles, several pieces
TWO_TERMS = [(33, 72, 501), (40, 1024, 20000), (64, 256, 3001), (65, 100, 1000), (150, 520, 9001), (300, 192, 21900),
             (1100, 64, 7300), (2048, 128, 151936), (50, 1001, 240000)]


@pytest.mark.parametrize("op", ["ce", "kd"])
@pytest.mark.parametrize("kind", ["same", "i8"])
@pytest.mark.parametrize("n,h,v", TWO_TERMS)
def test_two_terms(sv, op, n, h, v, kind):
    """dz in two terms at more rows: the gradients are off by their own rounding, the
    rest is the call's without; each gradient alone has the same bits."""
    log(f"two terms asked for {op} n={n} h={h} v={v} {kind}")
    call, ref, x, w, _ = near_case(sv, op, n, h, v, BF, kind, n + h)
    one, r = call(), call(two_terms=True)
    check_two_terms(r, ref, x, w)
    for name in r._fields[:4]:
        assert torch.equal(getattr(r, name), getattr(one, name)), name
    assert torch.equal(call(two_terms=True, grad="hidden").grad_hidden, r.grad_hidden)
    assert torch.equal(call(two_terms=True, grad="weight").grad_weight, r.grad_weight)
    assert torch.equal(call(two_terms=True, grad=False)[0], r[0])


@pytest.mark.parametrize("n", [150, 300, 1100])
def test_two_terms_with_rows_left_out(sv, n):
    """A front part of the rows that ends anywhere in a tile, and rows with data errors."""
    hidden, x, w, t, u = ce_case(sv, n, 136, 9001, BF, "same", 1.0, n)
    t[n // 7::3] = -1
    t[n // 3::2] = -1
    hidden[5, 3], t[5] = float("nan"), 4
    r = sv.head_ce(hidden, w, t, u, two_terms=True)
    assert int(r.status[5]) == sv.HEAD_NAN and int((r.status != 0).sum()) == 1
    used = (t >= 0) & (r.status == 0)
    ud = torch.where(used, u.double(), torch.zeros_like(u).double())
    x = torch.where(used[:, None], x, torch.zeros_like(x))
    pt = torch.zeros(n, 9001, dtype=torch.double, device="cuda")
    pt[used, t[used]] = 1
    check_two_terms(r, reference(x, w.double(), pt, ud, 1.0), x, w.double())
    assert not r.grad_hidden[~used].any()


@pytest.mark.parametrize("dtype,n", [(F, 100), (F, 20), (BF, 20)])
def test_two_terms_where_they_are_so_anyway(sv, dtype, n):
    """fp32, and up to 32 rows: the same bits with and without."""
    hidden, _, w, t, u = ce_case(sv, n, 128, 900, dtype, "same", 1.0, n)
    assert all(torch.equal(a, b) for a, b in zip(sv.head_ce(hidden, w, t, u), sv.head_ce(hidden, w, t, u, two_terms=True)))


def test_two_terms_guards_and_replays(sv):
    """A workspace of exactly the stated size, nothing behind it or the gradients
    written; a captured call replayed on other inputs."""
    import ctypes
    lib = sv.load_library()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for n, h, v in ((40, 100, 900), (300, 500, 70000)):
        log(f"two terms, guards n={n} h={h} v={v}")
        hidden, _, w, t, u = ce_case(sv, n, h, v, BF, "same", 1.0, n)
        want = sv.head_ce(hidden, w, t, u, two_terms=True)
        t = t.int()
        shape = sv.sv_head_shape_t(n, h, v, 1, 1, 7, 0, 0, 1.0, -1, 0, 0, float("inf"))
        need = lib.sv_head_ce_workspace_bytes(ctypes.byref(shape))
        ws = torch.full((need + 65536,), 0xff, dtype=torch.uint8, device="cuda")
        res, loss = torch.empty(n, device="cuda"), torch.empty(1, device="cuda")
        gh, gw = (torch.full((k * h + 16,), 5.0, dtype=BF, device="cuda") for k in (n, v))
        assert lib.sv_head_ce(ctypes.byref(shape), p(hidden), None, p(w), p(t), p(u), p(res), None, None, p(loss), p(gh), p(gw),
                              p(ws), need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        assert torch.equal(gh[:n * h].view(n, h), want.grad_hidden) and torch.equal(gw[:v * h].view(v, h), want.grad_weight)
        assert (gh[n * h:] == 5).all() and (gw[v * h:] == 5).all() and (ws[need:] == 0xff).all()
    held = ce_case(sv, 150, 128, 3000, BF, "same", 1.0, 1)
    call = lambda c: list(sv.head_ce(c[0], c[2], c[3], c[4], two_terms=True))  # noqa: E731
    call(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(held)
    for seed in (2, 3, 4):
        new = ce_case(sv, 150, 128, 3000, BF, "same", 1.0, seed)
        for a, b in zip(held, new):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call(new))), seed
