"""The vocabulary-head operators (8-bit rows, int8 head logits, cross entropy and
distillation from hidden rows) against their formulas in 64 bits.

Tolerances are bounds of the arithmetic, formed beside each check: half steps of
the roundings (2^-8 for bf16, 2^-24 for fp32), n 2^-24 times the sum of
magnitudes for an fp32 sum of n terms, and 2^-19 for what the hardware's exp2,
the fp32 logarithm of e and the row normaliser add to an exponent.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}
EXPO = 2.0 ** -19


def log(msg):
    print(f"[gpu-test] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import draft_verification_spec_amd as m
    m.load_library()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, want, tol, what):
    d = (got.double() - want).abs() - tol
    assert not torch.isnan(d).any(), what
    worst = int(d.argmax())
    assert float(d.max()) <= 0, (what, worst, float(got.reshape(-1)[worst]), float(want.reshape(-1)[worst]),
                                 float(tol.reshape(-1)[worst]) if torch.is_tensor(tol) else tol)


# ------------------------------------------------------------------ 8-bit rows
def plain_pack(x):
    # the nearest fp32 of the quotient (torch's fp32 tensor over a number multiplies by its reciprocal)
    scale = (x.abs().amax(-1).double() / 127).float()
    q = torch.where(scale[..., None] > 0, x.double() / scale[..., None].double(), torch.zeros_like(x, dtype=torch.double))
    return torch.round(q).clamp(-127, 127).to(torch.int8), scale


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,h", [(1, 1), (1, 1024), (3, 7), (5, 64), (130, 129), (4, 4096), (2, 20001), (1000, 96)])
def test_act8_round_trip(sv, n, h, dtype):
    log(f"act8 n={n} h={h} {dtype}")
    x = (torch.randn(n, h, generator=gen(n * h), device="cuda") * 3).to(dtype)
    x[0, h // 2] = 127.0                              # a scale of 1: halves are borders
    if h > 4:
        x[0, :4] = torch.tensor([0.5, 1.5, -2.5, -0.5], device="cuda")
        x[0] = x[0].clamp(-127, 127)
    a = sv.act8_pack(x)
    codes, scale = plain_pack(x)
    assert torch.equal(a.scale, scale)
    assert torch.equal(a.codes, codes)
    for out in (BF, F):
        assert torch.equal(sv.act8_unpack(a, out), (codes.float() * scale[:, None]).to(out))


def test_act8_borders_and_odd_rows(sv):
    """Quotients a hair from a border between two codes, rows of zeros, of the
    smallest magnitudes, with NaN and with infinities."""
    s = torch.tensor(0.0123, device="cuda")
    k = torch.arange(-126, 127, device="cuda").double()
    x = ((k + 0.5) * s.double()).float()
    up = torch.nextafter(x, torch.full_like(x, 1e9))
    down = torch.nextafter(x, torch.full_like(x, -1e9))
    row = torch.cat([x, up, down])
    top = s * 127
    while float(top / 127) < float(s):
        top = torch.nextafter(top, top * 2)
    row = torch.cat([row, top[None]])
    rows = torch.stack([row, torch.zeros_like(row), torch.full_like(row, 1e-45), torch.full_like(row, 3e38), row, row])
    rows[4, 5] = float("nan")
    rows[5, 9] = -float("inf")
    a = sv.act8_pack(rows)
    codes, scale = plain_pack(rows[:4])
    assert torch.equal(a.scale[:4], scale) and torch.equal(a.codes[:4], codes)
    assert torch.isnan(a.scale[4:]).all() and not a.codes[4:].any()
    assert torch.isnan(sv.act8_unpack(a, F)[4:]).all()


def test_act8_strides_and_shapes(sv):
    base = torch.randn(6, 5, 300, generator=gen(3), device="cuda")
    for x in (base[:, :, 3:200], base[:, 1], base.transpose(1, 2), base[2, 3], base[::2], base[:, :, ::3],
              base[0, :1].expand(4, 300)):
        a = sv.act8_pack(x)
        codes, scale = plain_pack(x)
        assert a.codes.shape == x.shape and a.scale.shape == x.shape[:-1]
        assert torch.equal(a.codes, codes) and torch.equal(a.scale, scale)
        assert torch.equal(sv.act8_unpack(a, F), codes.float() * scale[..., None])
    a = sv.act8_pack(torch.empty(0, 12, device="cuda"))
    assert a.codes.shape == (0, 12) and sv.act8_unpack(a).shape == (0, 12)


# ---------------------------------------------------------------- int8 logits
@pytest.mark.parametrize("kind,out", [(BF, BF), (F, F), ("i8", BF), ("i8", F)])
@pytest.mark.parametrize("n,h,v", [(1, 1, 1), (1, 1024, 1000), (3, 100, 77), (16, 128, 513), (31, 683, 3601), (33, 256, 130),
                                   (64, 64, 4099), (129, 200, 1021), (300, 384, 2048), (17, 4096, 999)])
def test_logits(sv, n, h, v, kind, out):
    log(f"head_logits n={n} h={h} v={v} {kind} {out}")
    g = gen(n + h + v)
    x = torch.randn(n, h, generator=g, device="cuda").to(F if kind == "i8" else kind)
    w = torch.randn(v, h, generator=g, device="cuda")
    wc, ws = plain_pack(w)
    xc, xs = plain_pack(x)
    hidden = sv.Act8(xc, xs) if kind == "i8" else x
    want = (xc.double() @ wc.double().T) * xs.double()[:, None] * ws.double()[None]
    got = sv.head_logits(hidden, sv.Act8(wc, ws), out_dtype=out)
    assert got.dtype == out and got.shape == (n, v)
    tol = want.abs() * ((HALF[BF] if out == BF else 0) + 4 * HALF[F])   # the sum, both scales' product, theirs, the output
    within(got, want, tol, "logits")
    # the head as act8_pack lays it out, and with rows at an odd distance: the same bits
    assert torch.equal(sv.head_logits(hidden, sv.act8_pack(w), out_dtype=out), got)
    wide = torch.zeros(v, h + 3, dtype=torch.int8, device="cuda")
    wide[:, 1:h + 1] = wc
    assert torch.equal(sv.head_logits(hidden, sv.Act8(wide[:, 1:h + 1], ws), out_dtype=out), got)


def test_logits_leading_axes_and_bad_rows(sv):
    """[B, k+1, H] in, [B, k+1, V] out; a NaN row gives NaN logits and no other
    row does; rows and columns outside the tensors stay as they were."""
    x = torch.randn(3, 4, 70, generator=gen(1), device="cuda")
    x[1, 2, 5] = float("nan")
    x[2, 0] = 0
    w = sv.act8_pack(torch.randn(90, 70, generator=gen(2), device="cuda"))
    y = sv.head_logits(x, w, out_dtype=F)
    assert y.shape == (3, 4, 90)
    bad = torch.isnan(y).all(-1)
    assert bad.sum() == 1 and bad[1, 2] and not torch.isnan(y[~bad]).any() and not y[2, 0].any()
    assert sv.head_logits(x[:0], w).shape == (0, 4, 90)


# -------------------------------------------------------------------- losses
def rows_of(kind, n, h, g, dtype, sv):
    """Hidden rows: (what the call takes, its values in 64 bits)."""
    x = torch.randn(n, h, generator=g, device="cuda")
    if kind == "i8":
        a = sv.act8_pack(x)
        return a, a.codes.double() * a.scale.double()[:, None]
    x = x.to(dtype)
    return x, x.double()


def reference(x, w, pt, u, tau):
    """From 64-bit rows, head, targets' probabilities [n, v] and row weights (NaN
    nowhere): z, lse, the gradients, and a bound of each one's error in fp32."""
    n, h = x.shape
    v = w.shape[0]
    z = x @ w.T / tau
    ez = (h + 8) * 2.0 ** -24 * (x.abs() @ w.abs().T) / tau + 2.0 ** -22 * z.abs()   # sum, 1 / T and log2 e
    lse = torch.logsumexp(z, 1)
    e = ez.amax(1, keepdim=True) * 2 + EXPO * (1 + lse.abs()[:, None] / 16)
    p = torch.exp(z - lse[:, None])
    dz = (p - pt) * u[:, None] / tau
    edz = (torch.expm1(e) * p + 2.0 ** -21 * (p + pt)) * u.abs()[:, None] / tau
    return dict(z=z, lse=lse, e=e, dz=dz, edz=edz)


def check_gradients(r, ref, x, w, dtype, which=("hidden", "weight"), rows=None):
    n, h = x.shape
    v = w.shape[0]
    dz, edz = ref["dz"], ref["edz"]
    half = HALF[dtype]
    edz = edz + (half * dz.abs() if dtype == BF else 0) + 1e-40
    for name, got, a, ea, b, terms in (("hidden", r.grad_hidden, dz, edz, w, v), ("weight", r.grad_weight, dz.T, edz.T, x, n)):
        if name not in which:
            assert got is None
            continue
        want = a @ b
        tol = ea @ b.abs() + (terms + 8) * 2.0 ** -24 * (a.abs() @ b.abs())
        tol = tol + half * (want.abs() + tol) + 1e-38
        assert got.dtype == dtype
        within(got, want, tol, "grad_" + name)
        # the roundings are independent: their norm is a fraction of the half steps' bound
        if float(want.norm()) > 0:
            bound = (2 * half if dtype == BF else float(tol.norm() / want.norm()))
            assert float((got.double() - want).norm() / want.norm()) <= bound, name


CE_SHAPES = [(1, 1, 1), (1, 64, 1000), (2, 7, 5), (31, 100, 333), (32, 128, 1024), (33, 192, 257), (100, 130, 1500),
             (192, 64, 700), (257, 512, 1023), (300, 96, 4099)]


def ce_case(sv, n, h, v, dtype, kind, tau, seed):
    g = gen(seed)
    hidden, x = rows_of(kind, n, h, g, dtype, sv)
    w = (torch.randn(v, h, generator=g, device="cuda") * 3 / h ** 0.5).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    u = torch.randn(n, generator=g, device="cuda")
    if n > 4:
        t[1] = -1
        t[n // 2] = -1
        u[2] = 0.0
    return hidden, x, w, t, u


def check_ce(sv, hidden, x, w, t, u, tau, dtype, grad=True):
    r = sv.head_ce(hidden, w, t, u, temperature=tau, grad=grad)
    n = x.shape[0]
    used = t >= 0
    ud = torch.ones(n, device="cuda").double() if u is None else u.double()
    ud = torch.where(used, ud, torch.zeros_like(ud))
    pt = torch.zeros(n, w.shape[0], dtype=torch.double, device="cuda")
    pt[used, t[used].long()] = 1
    ref = reference(x, w.double(), pt, ud, tau)
    nll = torch.where(used, ref["lse"] - (ref["z"] * pt).sum(1), torch.zeros_like(ud))
    e = torch.where(used, ref["e"][:, 0] + 2.0 ** -23 * (nll.abs() + ref["lse"].abs()), torch.zeros_like(ud))
    assert not r.status.any()
    within(r.nll, nll, e, "nll")
    within(r.lse, torch.where(used, ref["lse"], torch.zeros_like(ud)), e, "lse")
    within(r.loss, (ud * nll).sum()[None], ((ud.abs() * e).sum() + 2.0 ** -23 * (ud * nll).sum().abs())[None], "loss")
    which = {True: ("hidden", "weight"), False: (), "hidden": ("hidden",), "weight": ("weight",)}[grad]
    check_gradients(r, ref, x, w.double(), dtype, which)
    if r.grad_hidden is not None:
        assert not r.grad_hidden[~used].any()
    return r


@pytest.mark.parametrize("dtype,kind,tau", [(BF, "same", 1.0), (F, "same", 0.7), (BF, "i8", 0.7), (F, "i8", 1.0)])
@pytest.mark.parametrize("n,h,v", CE_SHAPES)
def test_ce(sv, n, h, v, dtype, kind, tau):
    log(f"head_ce n={n} h={h} v={v} {dtype} {kind} T={tau}")
    hidden, x, w, t, u = ce_case(sv, n, h, v, dtype, kind, tau, 7 * n + h + v)
    check_ce(sv, hidden, x, w, t, u, tau, dtype)


@pytest.mark.parametrize("kind,tau", [("same", 0.7), ("i8", 1.0)])
@pytest.mark.parametrize("n,h,v", [(129, 100, 33000), (257, 64, 22017), (300, 192, 21900), (600, 72, 13111), (1100, 128, 7300)])
def test_ce_large_tiles(sv, n, h, v, kind, tau):
    """Enough tiles of 128 for those of 256 to take their place, ragged both ways."""
    log(f"head_ce large n={n} h={h} v={v} {kind}")
    hidden, x, w, t, u = ce_case(sv, n, h, v, BF, kind, tau, n + h)
    t[n // 3::4] = -1
    check_ce(sv, hidden, x, w, t, u, tau, BF)


@pytest.mark.parametrize("n,h,v", [(2772, 192, 4343), (300, 1000, 4999), (1500, 72, 1300), (100, 2000, 3001), (700, 520, 9001)])
def test_ce_sizes_of_dw(sv, n, h, v):
    """Heads whose dW takes each of its tiles, beside each tile of the other products."""
    log(f"head_ce dw n={n} h={h} v={v}")
    hidden, x, w, t, u = ce_case(sv, n, h, v, BF, "same", 1.0, n + v)
    check_ce(sv, hidden, x, w, t, u, 1.0, BF)


@pytest.mark.parametrize("kind,out", [(BF, BF), (F, F), ("i8", BF), ("i8", F)])
@pytest.mark.parametrize("n,h,v", [(129, 200, 33001), (300, 384, 22000), (128, 100, 33000), (1000, 65, 8255)])
def test_logits_large_tiles(sv, n, h, v, kind, out):
    test_logits(sv, n, h, v, kind, out)


@pytest.mark.parametrize("grad", [False, "hidden", "weight"])
def test_ce_some_gradients(sv, grad):
    log(f"head_ce grad={grad}")
    hidden, x, w, t, u = ce_case(sv, 70, 128, 900, BF, "same", 1.0, 5)
    check_ce(sv, hidden, x, w, t, None, 1.0, BF, grad)


@pytest.mark.parametrize("n", [8, 40, 64, 150, 300])
@pytest.mark.parametrize("dtype", [BF, F])
def test_ce_one_gradient_is_the_same(sv, n, dtype):
    """The loss and each gradient alone: the bits of the call for both."""
    hidden, x, w, t, u = ce_case(sv, n, 200, 3000, dtype, "same", 1.0, n + 3)
    both = sv.head_ce(hidden, w, t, u)
    for grad in (False, "hidden", "weight"):
        r = sv.head_ce(hidden, w, t, u, grad=grad)
        for name in ("loss", "nll", "lse", "status"):
            assert torch.equal(getattr(r, name), getattr(both, name)), name
        assert r.grad_hidden is None if grad != "hidden" else torch.equal(r.grad_hidden, both.grad_hidden)
        assert r.grad_weight is None if grad != "weight" else torch.equal(r.grad_weight, both.grad_weight)


@pytest.mark.parametrize("n,h,v,dtype", [(2048, 256, 151936, BF), (40, 1024, 151936, BF), (1500, 128, 151936, F)])
def test_ce_several_pieces(sv, n, h, v, dtype):
    """Vocabularies that take several pieces, the last one ragged."""
    log(f"head_ce pieces n={n} h={h} v={v} {dtype}")
    hidden, x, w, t, u = ce_case(sv, n, h, v, dtype, "same", 1.0, 11)
    check_ce(sv, hidden, x, w, t, u, 1.0, dtype)


@pytest.mark.parametrize("n,v,dtype", [(9, 250000, BF), (50, 240000, BF), (9, 130000, F)])
def test_ce_few_rows_copied_pieces(sv, n, v, dtype):
    """Few rows against a head that no step divides: copied a piece at a time, and
    the last piece's launch joins the sums of all of them."""
    log(f"head_ce copied pieces n={n} v={v} {dtype}")
    hidden, x, w, t, u = ce_case(sv, n, 1001, v, dtype, "same", 1.0, 12)
    check_ce(sv, hidden, x, w, t, u, 1.0, dtype)
    check_ce(sv, hidden, x, w, t, u, 1.0, dtype, "hidden")


def test_ce_strides(sv):
    """Rows and head as parts of wider tensors, aligned or not, transposed, and
    32-bit targets: what the contiguous call gives."""
    g = gen(21)
    big = torch.randn(50, 3, 200, generator=g, device="cuda").to(BF)
    head = torch.randn(300, 260, generator=g, device="cuda").to(BF)
    t = torch.randint(0, 300, (50,), generator=g, device="cuda")
    for x, w in ((big[:, 1, :128], head[:, 4:132]), (big[:, 1, 1:129], head[:, 1:129]), (big[:, 2, 8:136], head[:, 8:136]),
                 (big[:, 0, :64], head[:, :64]), (big[::2, 0, :64], head[::3, 64:128])):
        tt = t[:x.shape[0]] % w.shape[0]
        a = sv.head_ce(x, w, tt)
        b = sv.head_ce(x.contiguous(), w.contiguous(), tt.int())
        for p, q in zip(a, b):
            assert torch.equal(p, q)
    x = torch.randn(64, 50, generator=g, device="cuda").to(BF).T
    a, b = sv.head_ce(x, head[:, :64], t), sv.head_ce(x.contiguous(), head[:, :64].contiguous(), t)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("n", [20, 100, 300])
@pytest.mark.parametrize("dtype", [BF, F])
def test_ce_data_errors(sv, n, dtype):
    """Bad rows: their status, NaN results, zero gradients, and nothing of them in
    the loss and the head's gradient; all rows left out; a large magnitude."""
    log(f"head_ce data errors n={n} {dtype}")
    h, v = 128, 600
    hidden, x, w, t, u = ce_case(sv, n, h, v, dtype, "same", 1.0, 31)
    t[:] = t.clamp(min=0)
    u = u.abs() + 0.5
    hidden[3, 4] = float("nan")
    hidden[5, 7] = float("inf")
    t[7] = v
    t[8] = -5
    u[9] = float("nan")
    u[10] = float("inf")
    r = sv.head_ce(hidden, w, t, u)
    st = r.status.tolist()
    assert st[3] == sv.HEAD_NAN and st[5] in (sv.HEAD_NAN, sv.HEAD_POSINF)
    assert st[7] == st[8] == sv.HEAD_BAD_TARGET and st[9] == st[10] == sv.HEAD_BAD_WEIGHT
    bad = r.status != 0
    assert int(bad.sum()) == 6
    assert torch.isnan(r.nll[bad]).all() and torch.isnan(r.lse[bad]).all()
    assert not r.grad_hidden[bad].any()
    good = sv.head_ce(hidden[~bad], w, t[~bad], u[~bad])
    assert torch.equal(good.nll, r.nll[~bad]) and not good.status.any()
    # the same products; rows sit at other places of the tiles' sums
    ref = good.grad_weight.double()
    scale = 8 * HALF[dtype] * ref.abs().amax()
    within(r.grad_weight, ref, scale, "grad_weight")
    within(r.grad_hidden[~bad], good.grad_hidden.double(), 8 * HALF[dtype] * good.grad_hidden.double().abs().amax(), "grad_hidden")
    none = sv.head_ce(hidden, w, torch.full_like(t, -1), u)
    assert float(none.loss) == 0 and not none.nll.any() and not none.grad_weight.any() and not none.grad_hidden.any()
    assert not none.status.any()
    far = sv.head_ce(torch.full_like(hidden[:2], 100), (w * 100).to(dtype), t[:2], u[:2])
    assert torch.isfinite(far.loss).all() and torch.isfinite(far.grad_weight).all()


def test_ce_ignore_index_and_empty(sv):
    g = gen(4)
    x = torch.randn(12, 64, generator=g, device="cuda")
    w = torch.randn(50, 64, generator=g, device="cuda")
    t = torch.randint(0, 50, (12,), generator=g, device="cuda")
    a = sv.head_ce(x, w, torch.where(t == 3, -100, t), ignore_index=-100)
    b = sv.head_ce(x, w, torch.where(t == 3, -1, t))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    t64 = t.clone()
    t64[0] = (1 << 32) + 1                            # does not wrap into the vocabulary
    assert int(sv.head_ce(x, w, t64).status[0]) == sv.HEAD_BAD_TARGET
    e = sv.head_ce(x[:0], w, t[:0])
    assert float(e.loss) == 0 and e.nll.shape == (0,) and not e.grad_weight.any() and e.grad_hidden.shape == (0, 64)


def test_ce_gradient_by_differences(sv):
    """The loss along random directions against its gradient (fp32): a central
    difference of step s is off by s^2 of the third derivative and 2^-22 / s of
    the loss's own rounding."""
    g = gen(9)
    x = torch.randn(37, 96, generator=g, device="cuda")
    w = torch.randn(210, 96, generator=g, device="cuda") * 0.3
    t = torch.randint(0, 210, (37,), generator=g, device="cuda")
    u = torch.rand(37, generator=g, device="cuda") / 37
    r = sv.head_ce(x, w, t, u, temperature=0.8)
    s = 2.0 ** -6
    for a, grad, other in ((x, r.grad_hidden, "w"), (w, r.grad_weight, "x")):
        d = torch.randn(a.shape, generator=g, device="cuda")
        d /= d.norm()
        up, down = ((a + k * d, w) if other == "w" else (x, a + k * d) for k in (s, -s))
        f = [float(sv.head_ce(*p, t, u, temperature=0.8, grad=False).loss) for p in (up, down)]
        want = float((grad.double() * d.double()).sum())
        # |third derivative| along a unit direction: at most (|w| / T)^3 resp. (|x| / T)^3 per unit of weight
        size = float((w if other == "w" else x).norm(dim=1).max()) / 0.8
        assert abs((f[0] - f[1]) / (2 * s) - want) <= s * s * size ** 3 / 6 * float(u.max()) + 2.0 ** -22 * abs(f[0]) / s


# ------------------------------------------------------------------ distillation
def kd_case(sv, n, h, v, dtype, kind, seed, group=4, per=3):
    g = gen(seed)
    hidden, x = rows_of(kind, n, h, g, dtype, sv)
    w = (torch.randn(v, h, generator=g, device="cuda") * 3 / h ** 0.5).to(dtype)
    k = min(32, v)
    ids = torch.full((n, 32), -1, device="cuda")
    val = torch.full((n, 32), -float("inf"), device="cuda")
    ids[:, :k] = torch.argsort(torch.rand(n, v, generator=g, device="cuda"), 1)[:, :k]
    val[:, :k] = 10 + 2 * torch.randn(n, k, generator=g, device="cuda")
    if k > 4:
        val[0, 3] = -float("inf")                     # padding that names a token
        ids[0, 1] = -1                                # padding with a value
    samples = group * -(-n // (per * group))
    rewards = torch.rand(samples, generator=g, device="cuda")
    rewards[0] = 0
    rs = torch.arange(n, device="cuda") // per
    return hidden, x, w, val, ids, rs, rewards, group


def check_kd(sv, hidden, x, w, val, ids, rs, rewards, group, dtype, w_max=float("inf")):
    r = sv.head_kd(hidden, w, val, ids, rs, rewards, group, w_max=w_max)
    n, v = x.shape[0], w.shape[0]
    pad = (ids < 0) | (val == -float("inf"))
    vals = torch.where(pad, torch.full_like(val, -float("inf")), val).double()
    pt = torch.softmax(vals, 1)
    total = rewards.double().view(-1, group).sum(1, keepdim=True)
    wt = torch.where(total > 0, rewards.double().view(-1, group) / total, torch.zeros_like(total)).view(-1).clamp(max=w_max)
    u = wt[rs.long()]
    dense = torch.zeros(n, v, dtype=torch.double, device="cuda")
    dense.scatter_add_(1, ids.clamp(min=0).long(), torch.where(pad, torch.zeros_like(pt), pt))
    ref = reference(x, w.double(), dense, u, 1.0)
    zt = ref["z"].gather(1, ids.clamp(min=0).long())
    kl = torch.where(pad, torch.zeros_like(pt), pt * (torch.log(pt.clamp(min=1e-300)) - zt + ref["lse"][:, None])).sum(1)
    e = ref["e"][:, 0] + 2.0 ** -23 * (kl.abs() + ref["lse"].abs())
    assert not r.status.any()
    within(r.kl, kl, e, "kl")
    within(r.weight, u, 2.0 ** -23 * u, "weight")
    within(r.loss, (u * kl).sum()[None], ((u * e).sum() + 2.0 ** -22 * (u * kl).sum().abs())[None], "loss")
    check_gradients(r, ref, x, w.double(), dtype)


@pytest.mark.parametrize("dtype,kind", [(BF, "same"), (F, "same"), (BF, "i8"), (F, "i8")])
@pytest.mark.parametrize("n,h,v", [(1, 64, 40), (3, 5, 20), (24, 100, 1000), (45, 256, 333), (200, 128, 2500), (1, 1, 1)])
def test_kd(sv, n, h, v, dtype, kind):
    log(f"head_kd n={n} h={h} v={v} {dtype} {kind}")
    check_kd(sv, *kd_case(sv, n, h, v, dtype, kind, n + h + v), dtype)


@pytest.mark.parametrize("kind", ["same", "i8"])
@pytest.mark.parametrize("n,h,v", [(140, 72, 33000), (520, 128, 13100)])
def test_kd_large_tiles(sv, n, h, v, kind):
    test_kd(sv, n, h, v, BF, kind)


def test_kd_clip_and_pieces(sv):
    log("head_kd clip, several pieces")
    check_kd(sv, *kd_case(sv, 40, 1024, 151936, BF, "same", 3), BF, w_max=0.3)


def test_kd_agrees_with_logits_form(sv):
    """kd on the logits and head_kd on the rows: the same status bits on every
    kind of bad input, and the same loss."""
    g = gen(17)
    n, h, v, group = 24, 64, 500, 4
    hidden, x, w, val, ids, rs, rewards, group = kd_case(sv, n, h, v, F, "same", 17, group, 2)
    val[2, 5] = float("nan")
    val[3, 5] = float("inf")
    ids[4, 7] = v
    ids[5, 9] = ids[5, 8]
    val[6] = -float("inf")
    rs[7] = 99
    hidden[8, 3] = float("nan")
    hidden[9] = 0
    rewards[4:8] = 0
    a = sv.kd((hidden @ w.T).contiguous(), val, ids.int(), rs.int(), rewards, group)
    b = sv.head_kd(hidden, w, val, ids, rs, rewards, group)
    assert torch.equal(a.status, b.status) and int((b.status != 0).sum()) == 7
    ok = b.status == 0
    assert torch.isnan(b.kl[~ok]).all() and not b.grad_hidden[~ok].any()
    # both within 1e-5 of the formula (kd's own bar); the weights are the same arithmetic
    within(b.kl[ok], a.kl[ok].double(), 2e-5, "kl")
    assert torch.equal(a.weight, b.weight)
    within(b.loss, a.loss.double(), 2e-5 * (1 + float(a.weight.sum())), "loss")
    want = a.grad.double() @ w.double()
    want[~ok] = 0
    within(b.grad_hidden, want, 1e-4, "grad_hidden")


def test_stored_row_that_was_not_finite(sv):
    """A row packed with a NaN in it has scale NaN: the losses report that row and
    leave it out of both gradients."""
    g = gen(71)
    x = torch.randn(40, 96, generator=g, device="cuda")
    x[7, 3] = float("nan")
    w = torch.randn(300, 96, generator=g, device="cuda").to(BF)
    t = torch.randint(0, 300, (40,), generator=g, device="cuda")
    r = sv.head_ce(sv.act8_pack(x), w, t)
    keep = torch.arange(40, device="cuda") != 7
    assert r.status.tolist() == [sv.HEAD_NAN if i == 7 else 0 for i in range(40)]
    assert torch.isnan(r.nll[7]) and torch.isfinite(r.loss).all()
    s = sv.head_ce(sv.act8_pack(x[keep]), w, t[keep])
    assert torch.equal(s.nll, r.nll[keep]) and not r.grad_hidden[7].any()
    within(r.grad_weight, s.grad_weight.double(), 4 * HALF[BF] * s.grad_weight.double().abs().amax(), "grad_weight")


def test_head_beyond_32_bits(sv):
    """A head of more than 2^32 bytes, and int8 codes of as many: offsets of its last
    rows, checked piece by piece."""
    h, v = 4096, 560000                               # 4.6 GB in bf16
    g = gen(81)
    w = torch.empty(v, h, dtype=BF, device="cuda")
    for i in range(0, v, 70000):
        w[i:i + 70000] = (torch.randn(70000, h, generator=g, device="cuda") * 0.04).to(BF)
    x = torch.randn(3, h, generator=g, device="cuda").to(BF)
    t = torch.tensor([v - 1, 5, v - 70000], device="cuda")
    log("head_ce over a 4.6 GB head")
    r = sv.head_ce(x, w, t)
    z = torch.cat([(x.float() @ w[i:i + 70000].float().T).double() for i in range(0, v, 70000)], 1)
    lse = torch.logsumexp(z, 1)
    at = z.gather(1, t[:, None])[:, 0]
    # fp32 sums of 4096 terms on both sides: 2 * 4096 * 2^-24 of their magnitudes (about 4096 * 0.8 * 0.032)
    e = 2 * h * 2.0 ** -24 * 4096 * 0.8 * 0.032 + 1e-5
    within(r.nll, lse - at, e, "nll")
    d = torch.exp(z - lse[:, None])
    d[torch.arange(3), t] -= 1
    for i in (0, v - 70000):
        want = d[:, i:i + 70000].T @ x.double()
        tol = (2 * e + 2 * HALF[BF]) * (d[:, i:i + 70000].abs().T @ x.double().abs()) + 1e-12
        within(r.grad_weight[i:i + 70000], want, tol, "grad_weight")
    want = sum(d[:, i:i + 70000] @ w[i:i + 70000].double() for i in range(0, v, 70000))
    size = sum(d[:, i:i + 70000].abs() @ w[i:i + 70000].double().abs() for i in range(0, v, 70000))
    within(r.grad_hidden, want, (2 * e + 2 * HALF[BF]) * size, "grad_hidden")
    del r, d, z, w
    v = 1100000                                       # 4.5 GB of codes
    codes = torch.randint(-127, 128, (v, h), generator=g, device="cuda", dtype=torch.int8)
    scale = torch.rand(v, generator=g, device="cuda")
    log("head_logits over 4.5 GB of codes")
    a = sv.act8_pack(x)
    y = sv.head_logits(a, sv.Act8(codes, scale), out_dtype=F)
    for i in (0, v - 50000):
        want = (a.codes.double() @ codes[i:i + 50000].double().T) * a.scale.double()[:, None] * scale[i:i + 50000].double()
        within(y[:, i:i + 50000], want, want.abs() * 4 * HALF[F], "logits")


@pytest.mark.parametrize("n", [32, 33, 64, 65, 191, 192, 256, 1024, 1025])
@pytest.mark.parametrize("dtype", [BF, F])
def test_ce_at_the_borders_of_the_rules(sv, n, dtype):
    """The row counts where tiles, the order of rows and dW change their form, with
    most rows left out: a front part that ends anywhere in a tile."""
    log(f"head_ce border n={n} {dtype}")
    hidden, x, w, t, u = ce_case(sv, n, 136, 777, dtype, "same", 1.0, n)
    t[n // 7::3] = -1
    t[n // 3::2] = -1
    check_ce(sv, hidden, x, w, t, u, 1.0, dtype)


# ------------------------------------------------- as a program uses them together
def test_deterministic_and_streams(sv):
    """The same bits again, on another stream, and beside another call that runs
    at the same time."""
    hidden, x, w, t, u = ce_case(sv, 300, 256, 3000, BF, "same", 1.0, 41)
    a = sv.head_ce(hidden, w, t, u)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        b = sv.head_ce(hidden, w, t, u)
    c = sv.head_ce(hidden, w, t, u, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    for p, q, z in zip(a, b, c):
        assert torch.equal(p, q) and torch.equal(p, z)


def test_own_workspace(sv):
    """A caller's workspace of exactly the stated size, with any contents; bytes
    behind it stay as they were."""
    import ctypes
    hidden, x, w, t, u = ce_case(sv, 40, 100, 700, BF, "same", 1.0, 43)
    shape = sv.sv_head_shape_t(40, 100, 700, sv.SV_BF16, sv.SV_BF16, 3, 0, 0, 1.0, -1, 0, 0, float("inf"))
    need = sv.load_library().sv_head_ce_workspace_bytes(ctypes.byref(shape))
    buf = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    a = sv.head_ce(hidden, w, t, u, workspace=buf[:need])
    b = sv.head_ce(hidden, w, t, u)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert (buf[need:] == 0xff).all()
    with pytest.raises(sv.SpecVerifyError):
        sv.head_ce(hidden, w, t, u, workspace=buf[:need - 256])
    with pytest.raises(ValueError):
        sv.head_ce(hidden, w, t, u, workspace=torch.empty(need, dtype=torch.uint8))


def ptr(t):
    import ctypes
    return ctypes.c_void_p(t.data_ptr())


def stream_now():
    import ctypes
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("off", [0, 1, 3])
@pytest.mark.parametrize("dtype,code", [(BF, 1), (F, 0)])
def test_c_strides_and_guards(sv, dtype, code, off):
    """The C entries with rows at odd distances from any element: what the front end
    gives, and what lies between the rows and around them stays as it was."""
    import ctypes
    lib = sv.load_library()
    g = gen(90 + off)
    for n, h, v in ((5, 37, 203), (40, 128, 1030), (300, 200, 515)):
        log(f"strides and guards n={n} h={h} v={v} {dtype} off={off}")
        x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
        w = sv.act8_pack(torch.randn(v, h, generator=g, device="cuda"))
        a = sv.act8_pack(x)
        codes = torch.full((16 + n * (h + off),), 77, dtype=torch.int8, device="cuda")
        scale = torch.empty(n, device="cuda")
        body = codes[off:off + n * (h + off)].view(n, h + off)
        assert lib.sv_act8_pack(n, h, code, ptr(x), 0, ptr(body), h + off, ptr(scale), stream_now()) == 0
        assert torch.equal(body[:, :h], a.codes) and torch.equal(scale, a.scale)
        assert (body[:, h:] == 77).all() and (codes[:off] == 77).all() and (codes[off + n * (h + off):] == 77).all()
        y = torch.full((n * h + 16,), 5.0, dtype=dtype, device="cuda")
        assert lib.sv_act8_unpack(n, h, ptr(body), h + off, ptr(scale), code, ptr(y[off:]), stream_now()) == 0
        assert torch.equal(y[off:off + n * h].view(n, h), sv.act8_unpack(a, dtype))
        assert (y[:off] == 5).all() and (y[off + n * h:] == 5).all()
        out = torch.full((off + n * (v + off) + 16,), 5.0, dtype=dtype, device="cuda")
        rows = out[off:off + n * (v + off)].view(n, v + off)
        shape = sv.sv_logits_shape_t(n, h, v, 2, code, h + off, w.codes.stride(0), v + off)
        ws = torch.empty(lib.sv_head_logits_workspace_bytes(ctypes.byref(shape)), dtype=torch.uint8, device="cuda")
        assert lib.sv_head_logits(ctypes.byref(shape), ptr(body), ptr(scale), ptr(w.codes), ptr(w.scale), ptr(rows), ptr(ws),
                                  ws.numel(), stream_now()) == 0
        assert torch.equal(rows[:, :v], sv.head_logits(a, w, out_dtype=dtype))
        assert (rows[:, v:] == 5).all() and (out[:off] == 5).all() and (out[off + n * (v + off):] == 5).all()


@pytest.mark.parametrize("n,h,v,dtype,code", [(24, 512, 3000, F, 0), (24, 77, 3001, BF, 1), (40, 100, 900, F, 0),
                                              (60, 1000, 4000, BF, 1), (150, 200, 5000, BF, 1), (260, 500, 70000, BF, 1)])
def test_ce_guards(sv, n, h, v, dtype, code):
    """A workspace of exactly the stated size and gradients that begin at any element:
    the front end's bits, and nothing around them is written."""
    import ctypes
    log(f"head_ce guards n={n} h={h} v={v} {dtype}")
    lib = sv.load_library()
    hidden, x, w, t, u = ce_case(sv, n, h, v, dtype, "same", 1.0, n + h)
    want = sv.head_ce(hidden, w, t, u)
    t = t.int()
    shape = sv.sv_head_shape_t(n, h, v, code, code, 3, 0, 0, 1.0, -1, 0, 0, float("inf"))
    need = lib.sv_head_ce_workspace_bytes(ctypes.byref(shape))
    ws = torch.full((need + 65536,), 0xff, dtype=torch.uint8, device="cuda")
    res = torch.full((n + 1 + 8,), 5.0, device="cuda")
    gh, gw = (torch.full((k * h + 16,), 5.0, dtype=dtype, device="cuda") for k in (n, v))
    assert lib.sv_head_ce(ctypes.byref(shape), ptr(hidden), None, ptr(w), ptr(t), ptr(u), ptr(res), None, None, ptr(res[n:]),
                          ptr(gh[3:]), ptr(gw[1:]), ptr(ws), need, stream_now()) == 0
    assert torch.equal(res[:n], want.nll) and torch.equal(res[n:n + 1], want.loss) and (res[n + 1:] == 5).all()
    assert torch.equal(gh[3:3 + n * h].view(n, h), want.grad_hidden)
    assert torch.equal(gw[1:1 + v * h].view(v, h), want.grad_weight)
    for b, lo, k in ((gh, 3, n * h), (gw, 1, v * h)):
        assert (b[:lo] == 5).all() and (b[lo + k:] == 5).all()
    assert (ws[need:] == 0xff).all()


def test_rollout_step_together(sv):
    """A rollout step and its distillation: hidden rows put away in 8 bits, the
    head's 8-bit logits verified, the stored top-32 distilled into the head from
    the stored rows.  The logits and stored targets agree with plain forms of the
    same codes, and the loss with the one from those logits."""
    g = gen(51)
    B, k, H, V = 4, 3, 256, 2000
    head = torch.randn(V, H, generator=g, device="cuda") * 3 / H ** 0.5
    hw = sv.act8_pack(head)
    rows = torch.randn(B, k + 1, H, generator=g, device="cuda").to(BF)
    store = sv.act8_pack(rows)
    target = sv.head_logits(store, hw, out_dtype=F)
    draft = (target[:, :k] + 0.3 * torch.randn(B, k, V, generator=g, device="cuda")).contiguous()
    tokens = draft.argmax(-1).int()
    u = torch.rand(B, k + 2, generator=g, device="cuda")
    r = sv.verify(target, draft, tokens, u, 1.0, aux=True)
    assert not r.status.any()
    want = torch.topk(target, 32, dim=-1)
    assert torch.equal(r.topk_val, want.values)
    n = B * (k + 1)
    flat = sv.Act8(store.codes.reshape(n, H), store.scale.reshape(n))
    rs = torch.arange(n, device="cuda") // (k + 1)
    rewards = torch.tensor([1.0, 0.0, 0.3, 0.8], device="cuda")
    w = head.to(BF)
    d = sv.head_kd(flat, w, r.topk_val.view(n, 32), r.topk_idx.view(n, 32), rs, rewards, 2)
    z = ((flat.codes.double() * flat.scale.double()[:, None]) @ w.double().T).float()
    e = sv.kd(z, r.topk_val.view(n, 32), r.topk_idx.view(n, 32), rs.int(), rewards, 2)
    within(d.loss, e.loss.double(), 1e-4, "loss")
    assert d.grad_weight.shape == (V, H) and torch.isfinite(d.grad_weight).all()
    dropped = rs == 1                                 # its reward is 0
    assert not d.grad_hidden[dropped].any() and d.grad_hidden[~dropped].abs().sum() > 0


@pytest.mark.parametrize("op", ["ce", "kd", "logits", "act8"])
def test_graph_replays(sv, op):
    """One captured call replayed on new inputs, with eager work between, against
    eager calls on the same inputs."""
    def inputs(seed):
        if op == "kd":
            hidden, x, w, val, ids, rs, rewards, group = kd_case(sv, 40, 128, 900, BF, "same", seed)
            return [hidden, w, val, ids.int(), rs.int(), rewards]
        hidden, x, w, t, u = ce_case(sv, 40, 128, 900, BF, "same", 1.0, seed)
        if op == "ce":
            return [hidden, w, t.int(), u]
        a = sv.act8_pack(w)
        return [hidden, a.codes.contiguous(), a.scale] if op == "logits" else [hidden]

    def call(a):
        if op == "kd":
            return list(sv.head_kd(*a, 4))
        if op == "ce":
            return list(sv.head_ce(*a))
        if op == "logits":
            return [sv.head_logits(a[0], sv.Act8(a[1], a[2]))]
        p = sv.act8_pack(a[0])
        return [p.codes, p.scale, sv.act8_unpack(p)]

    log(f"graph capture of {op}")
    held = inputs(60)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(held)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(held)
    for seed in (61, 62, 63):
        new = inputs(seed)
        for a, b in zip(held, new):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = call(new)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), (op, seed)


def test_two_graphs_take_turns(sv):
    """Two captured calls of different shapes, replayed in turn and with eager calls
    between: neither disturbs the other's scratch or results."""
    a, b = (ce_case(sv, n, 128, v, BF, "same", 1.0, n) for n, v in ((40, 900), (300, 1500)))
    call = lambda c: list(sv.head_ce(c[0], c[2], c[3], c[4]))  # noqa: E731
    want = [call(a), call(b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(c))
        graphs.append(graph)
    for turn in range(3):
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        call(b)
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(out, ref)), turn
