"""The log-probabilities of given tokens, their rows' entropies and alternatives, and the
logits' gradient, against their formulas in 64 bits.

Tolerances are bounds of the arithmetic.  With y the logits less the row's largest in
units of T: an entry's exponent is off by 3 half steps of |y| (the difference, the constant,
the product), its exponential by one step more, a sum of 32 terms by 32 half steps, and each
of at most 16 changes of the maximum by 2 half steps.  So the sum's relative error is below
(3 E|y| + 70) 2^-24, E over the row's probabilities, and ln of it is as far off absolutely.
"""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}
U = 2.0 ** -24
INF, NAN = math.inf, math.nan


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
    same = torch.isinf(want) & (got.double() == want)
    d = torch.where(same, torch.zeros_like(d), d)
    assert not torch.isnan(d).any(), what
    worst = int(d.argmax())
    assert float(d.max()) <= 0, (what, worst, float(got.reshape(-1)[worst]), float(want.reshape(-1)[worst]),
                                 float(tol.reshape(-1)[worst]) if torch.is_tensor(tol) else tol)


class Want:
    """The formulas in 64 bits, for rows without data errors."""

    def __init__(self, z, t, T):
        z = z.double()
        T = torch.tensor(T, dtype=F).double().item()              # as the call holds it
        self.T, self.m = T, z.amax(-1, keepdim=True)
        y = (z - self.m) / T
        self.lp = y - torch.logsumexp(y, -1, keepdim=True)
        self.p = self.lp.exp()
        size = torch.where(self.p > 0, y.abs(), torch.zeros_like(y))
        e1, e2 = (self.p * size).sum(-1), (self.p * size * size).sum(-1)
        self.sum_off = (3 * e1 + 70) * U
        self.logp = self.lp.gather(-1, t.long().clamp(0, z.shape[-1] - 1)[..., None])[..., 0]
        self.lse = torch.logsumexp(z / T, -1)
        self.log_total = torch.logsumexp(y, -1)
        self.entropy = torch.special.entr(self.p).sum(-1)
        self.entropy_off = 2 * self.sum_off * (1 + e1) + 3 * e2 * U + self.entropy * U

    def check(self, r, what, keep=None):
        keep = torch.ones_like(self.logp, dtype=torch.bool) if keep is None else keep
        k = lambda v: v[keep]  # noqa: E731
        within(k(r.logp), k(self.logp), k(self.sum_off + self.logp.abs() * U).nan_to_num(posinf=0), what + " logp")
        within(k(r.lse), k(self.lse), k(self.sum_off + self.lse.abs() * U), what + " lse")
        within(k(r.entropy), k(self.entropy), k(self.entropy_off), what + " entropy")
        assert torch.equal(k(r.norm[0]).double(), k(self.m[..., 0])), what
        within(k(r.norm[1]), k(self.log_total), k(self.sum_off + self.log_total * U), what + " norm")
        assert not k(r.status).any(), what
        assert (r.logp <= 0).all() and (r.entropy >= 0).all()

    def grad(self, t, g, h, dtype):
        """(gradient, how far off it may be)."""
        g, h = g.double()[..., None], torch.zeros_like(g.double())[..., None] if h is None else h.double()[..., None]
        lp = self.lp.clamp(min=-1e4)
        one = torch.zeros_like(self.p).scatter_(-1, t.long()[..., None], 1.0)
        d = (g * (one - self.p) - h * self.p * (lp + self.entropy[..., None])) / self.T
        # log2 p: the difference, the constant and the product, the normaliser's own error and roundings
        off = (3 * (lp.abs() + self.log_total[..., None]) + 4 * self.log_total[..., None] + 2) * U + self.sum_off[..., None]
        size = g.abs() + h.abs() * (lp.abs() + self.entropy[..., None])
        tol = self.p * (size * (off + 8 * U) + h.abs() * (off + self.entropy_off[..., None])) / self.T + (one * g.abs() / self.T) * 3 * U
        return d, tol + HALF[dtype] * d.abs() + 1e-38


def best_of(z, top):
    """Indices of the largest entries by (value, lower index), -1 past those above -inf."""
    order = torch.sort(z.float() + 0.0, dim=-1, descending=True, stable=True)
    n = min(top, z.shape[-1])
    idx = torch.full((*z.shape[:-1], top), -1, dtype=torch.int64, device=z.device)
    idx[..., :n] = torch.where(order.values[..., :n] > -INF, order.indices[..., :n], -1)
    return idx


def check_top(r, w, z, top, what):
    idx = best_of(z, top)
    assert torch.equal(r.top_idx.long(), idx), what
    want = torch.where(idx >= 0, w.lp.gather(-1, idx.clamp(min=0)), -INF)
    tol = w.sum_off[..., None] + want.abs().nan_to_num(posinf=0) * U
    within(r.top_logp, want, tol, what + " top")


SIZES = [(1, 1), (1, 5), (3, 31), (2, 1000), (5, 8191), (4, 8193), (7, 32003), (1, 32768), (1, 32769), (1, 151936), (3, 262145),
         (130, 4099), (1030, 777), (1024, 20011)]


@pytest.mark.parametrize("top", [0, 1, 5, 32])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,v", SIZES)
def test_rows(sv, n, v, dtype, top):
    log(f"logprobs n={n} v={v} {dtype} top={top}")
    g = gen(n * 7 + v + top)
    z = (torch.randn(n, v, generator=g, device="cuda") * 3).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    t[0] = int(z[0].argmax())
    T = [1.0, 0.7, 2.5][(n + v) % 3]
    r = sv.logprobs(z, t, T, top=top)
    w = Want(z, t, T)
    w.check(r, "rows")
    if top:
        check_top(r, w, z, top, "rows")
    else:
        assert r.top_logp is None and r.top_idx is None


def hard_rows(v, dtype):
    """Rows whose order or masks are the difficulty."""
    low = torch.finfo(dtype).min
    up = torch.arange(v, device="cuda").float()
    rows = dict(
        constant=torch.zeros(v, device="cuda"),
        signs=torch.where(up % 3 == 0, -0.0, 0.0),
        ascending=up / v * 20,
        descending=-up / v * 20,
        steps=torch.floor(up / 50) % 7,
        lowest=torch.full((v,), low, device="cuda"),
        mostly_lowest=torch.where(up % 997 == 5, up / v, torch.tensor(low, device="cuda")),
        masked=torch.where(up % 3 == 1, -INF, torch.sin(up)),
        one_left=torch.where(up == v - 1, 2.0, -INF),
        three_left=torch.where(up % (v // 3 + 1) == v // 4, up / v, -INF),
        late=torch.where(up < v - 40, -INF, up / v),
        huge=torch.sin(up) * 1e30,
        large=1e6 + torch.sin(up),
        tiny=torch.sin(up) * 1e-38,
        last=torch.where(up == v - 1, 50.0, 0.0),
        sure=torch.where(up == v // 2, 200.0, torch.sin(up)))
    return list(rows), torch.stack(list(rows.values())).to(dtype)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("v", [40, 5003, 70001])
def test_hard_rows(sv, v, dtype, many):
    """Ties, masks, orders and magnitudes, in few rows (rows in parts) and in many."""
    names, z = hard_rows(v, dtype)
    if many:
        z = z.repeat(70, 1)
    t = z.float().argmax(-1).int()
    log(f"logprobs hard rows v={v} {dtype} many={many}")
    r = sv.logprobs(z, t, 1.0, top=32)
    w = Want(z, t, 1.0)
    for i, name in enumerate(names):
        s = slice(i, None, len(names)) if many else slice(i, i + 1)
        sub = Want(z[s], t[s], 1.0)
        part = sv.LogprobsResult(r.logp[s], r.entropy[s], r.lse[s], r.norm[:, s], r.status[s], r.top_logp[s], r.top_idx[s])
        sub.check(part, name)
        check_top(part, sub, z[s], 32, name)
    g = torch.linspace(-1, 1, z.shape[0], device="cuda")
    h = torch.linspace(0.5, -0.3, z.shape[0], device="cuda")
    for e in (None, h):
        got = sv.logprobs_grad(z, t, r, g, e)
        want, tol = w.grad(t, g, e, dtype)
        within(got, want, tol, "gradient of hard rows")


def test_data_errors(sv):
    """A row's own NaN, +inf, emptiness or bad token is its own."""
    v = 9001
    for dtype in (BF, F):
        z = torch.randn(9, v, generator=gen(4), device="cuda").to(dtype)
        t = torch.arange(9, device="cuda", dtype=torch.int32) * 10
        z[1, v - 1] = NAN
        z[2, 77] = INF
        z[3] = -INF
        t[4], t[5] = v, -2
        t[6] = -1
        z[6, 3] = NAN                                  # left out: not read
        z[7, 9], z[7, 10] = NAN, INF
        r = sv.logprobs(z, t, top=4)
        B = sv
        assert r.status.tolist() == [0, B.HEAD_NAN, B.HEAD_POSINF, B.HEAD_EMPTY, B.HEAD_BAD_TARGET, B.HEAD_BAD_TARGET, 0,
                                     B.HEAD_NAN, 0]
        bad = r.status != 0
        for f in (r.logp, r.entropy, r.lse, r.norm[0], r.norm[1], r.top_logp[:, 0]):
            assert torch.isnan(f[bad]).all() and not torch.isnan(f[~bad]).any()
        assert (r.top_idx[bad] == -1).all()
        assert r.logp[6] == r.entropy[6] == r.lse[6] == 0 and (r.top_idx[6] == -1).all() and (r.top_logp[6] == -INF).all()
        keep = torch.tensor([0, 8], device="cuda")
        w = Want(z[keep], t[keep], 1.0)
        w.check(sv.LogprobsResult(r.logp[keep], r.entropy[keep], r.lse[keep], r.norm[:, keep], r.status[keep], None, None), "others")
        ones = torch.ones(9, device="cuda")
        grad = sv.logprobs_grad(z, t, r, ones, ones)
        assert not grad[1:8].any() and grad[0].any() and grad[8].any()
        z[0, 3] = -INF                                 # the given token itself ruled out
        t[0] = 3
        r = sv.logprobs(z, t)
        assert r.logp[0] == -INF and r.status[0] == 0
        assert torch.isfinite(sv.logprobs_grad(z, t, r, ones, ones)[0]).all()


def test_tokens_types_and_shapes(sv):
    """Leading shapes, 64-bit tokens (some beyond 32 bits), another ignore_index, rows apart."""
    z = torch.randn(4, 3, 1000, generator=gen(8), device="cuda")
    t = torch.randint(0, 1000, (4, 3), generator=gen(9), device="cuda")
    r = sv.logprobs(z, t, top=3)
    assert r.logp.shape == r.status.shape == (4, 3) and r.norm.shape == (2, 4, 3) and r.top_idx.shape == (4, 3, 3)
    Want(z, t, 1.0).check(r, "3-d")
    one = sv.logprobs(z[1, 2], t[1, 2], top=3)
    assert one.logp.shape == () and torch.equal(one.top_idx, r.top_idx[1, 2]) and one.logp == r.logp[1, 2]
    big = t.clone()
    big[0, 0], big[0, 1], big[0, 2] = (1 << 32) + 5, -(1 << 40), 1 << 31
    b = sv.logprobs(z, big, ignore_index=7)
    assert (b.status[0] == sv.HEAD_BAD_TARGET).all()
    t[2, 1] = 7
    b = sv.logprobs(z, t, ignore_index=7)
    assert b.logp[2, 1] == 0 and b.lse[2, 1] == 0
    empty = sv.logprobs(z[:0], t[:0], top=2)
    assert empty.logp.shape == (0, 3) and empty.top_idx.shape == (0, 3, 2)
    assert sv.logprobs_grad(z[:0], t[:0], empty, torch.zeros(0, 3, device="cuda")).shape == (0, 3, 1000)


@pytest.mark.parametrize("dtype", [BF, F])
def test_strides(sv, dtype):
    """Rows at odd distances and addresses, transposed and repeated ones."""
    base = torch.randn(6, 5, 2003, generator=gen(3), device="cuda").to(dtype)
    for z in (base[:, :, 3:1800], base[:, 1], base.transpose(0, 1), base[2, 3], base[::2], base[:, :, ::3],
              base[0, :1].expand(4, 2003), base[:, :, 1:2]):
        t = torch.randint(0, z.shape[-1], z.shape[:-1], generator=gen(1), device="cuda")
        r = sv.logprobs(z, t, 0.9, top=5)
        w = Want(z, t, 0.9)
        w.check(r, "strides")
        check_top(r, w, z, 5, "strides")
        g, h = (torch.randn(z.shape[:-1], generator=gen(s), device="cuda") for s in (5, 6))
        for out in (dtype, F):
            got = sv.logprobs_grad(z, t, r, g, h, 0.9, out_dtype=out)
            assert got.dtype is out and got.is_contiguous()
            want, tol = w.grad(t, g, h, out)
            within(got, want, tol, "strided gradient")


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F), (F, F), (F, BF)])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 31), (5, 8191), (2, 8200), (24, 20000), (9, 40001)])
def test_gradient(sv, n, v, dtype, out):
    log(f"logprobs_grad n={n} v={v} {dtype} {out}")
    g = gen(n + v)
    z = (torch.randn(n, v, generator=g, device="cuda") * 3).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    T = [1.0, 0.7, 2.5][(n + v) % 3]
    r = sv.logprobs(z, t, T)
    w = Want(z, t, T)
    gl, gh = (torch.randn(n, generator=g, device="cuda") for _ in range(2))
    for h in (None, gh):
        got = sv.logprobs_grad(z, t, r, gl, h, T, out_dtype=out)
        want, tol = w.grad(t, gl, h, out)
        within(got, want, tol, "gradient")


def test_gradient_against_differences(sv):
    """sum g logp + h entropy, stepped along each of some logits: the forward operator's own
    differences in float32 say the gradient to about 1e-3."""
    v, T = 50, 0.8
    z = torch.randn(1, v, generator=gen(2), device="cuda")
    t = torch.tensor([11], device="cuda")
    g, h = torch.tensor([0.7], device="cuda"), torch.tensor([-0.4], device="cuda")
    got = sv.logprobs_grad(z, t, sv.logprobs(z, t, T), g, h, T)[0]
    step = 2.0 ** -6
    eye = torch.eye(v, device="cuda") * step
    f = []
    for sign in (1, -1):
        r = sv.logprobs(z + sign * eye, t.expand(v), T)
        f.append(0.7 * r.logp.double() - 0.4 * r.entropy.double())
    d = (f[0] - f[1]) / (2 * step)
    # third derivatives of both are below 10 / T^3, so the differences are off by 10 / T^3 step^2 / 6; the values by 1e-5 / step
    assert float((d - got.double()).abs().max()) < 10 / T ** 3 * step ** 2 / 6 + 1e-5 / step


def test_gradient_memory(sv):
    """Into given memory, strided memory and the logits' own; what lies between rows stays."""
    for dtype in (BF, F):
        z = torch.randn(6, 5001, generator=gen(3), device="cuda").to(dtype)
        t = torch.arange(6, device="cuda")
        t[4] = -1
        r = sv.logprobs(z, t)
        g = torch.linspace(-1, 1, 6, device="cuda")
        want = sv.logprobs_grad(z, t, r, g, g)
        assert not want[4].any()
        wide = torch.full((6, 5010), 7.0, dtype=dtype, device="cuda")
        got = sv.logprobs_grad(z, t, r, g, g, out=wide[:, 3:5004])
        assert got.data_ptr() == wide[:, 3:].data_ptr() and torch.equal(got, want)
        assert (wide[:, :3] == 7).all() and (wide[:, 5004:] == 7).all()
        with pytest.raises(ValueError):
            sv.logprobs_grad(z, t, r, g, out=wide[:, ::2][:, :2501])
        with pytest.raises(ValueError):
            sv.logprobs_grad(z, t, r, g, out=torch.empty(5001, 6, dtype=dtype, device="cuda").t())
        same = sv.logprobs_grad(z, t, r, g, g, out=z)
        assert same.data_ptr() == z.data_ptr() and torch.equal(z, want)


def test_guarded_outputs(sv):
    """The C entries write their results and nothing beside them."""
    import ctypes
    lib = sv.load_library()
    n, v, top = 5, 3001, 7
    z = torch.randn(n, v, generator=gen(1), device="cuda")
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    s = sv.sv_logprobs_shape_t(n, v, 0, top, 0, 1.0, -1)
    pad = 64
    outs = [torch.full((k + 2 * pad,), 7.0, device="cuda") for k in (n, n, n, 2 * n, n, n * top, n * top)]
    ptr = [o.data_ptr() + 4 * pad for o in outs]
    need = lib.sv_logprobs_workspace_bytes(ctypes.byref(s))
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    base = (ws.data_ptr() + 255) // 256 * 256
    assert lib.sv_logprobs(ctypes.byref(s), z.data_ptr(), t.data_ptr(), *ptr[:4], ptr[4], ptr[5], ptr[6], base, need, None) == 0
    torch.cuda.synchronize()
    for o in outs:
        assert (o[:pad] == 7).all() and (o[-pad:] == 7).all()
    r = sv.logprobs(z, t, top=top)
    assert torch.equal(outs[0][pad:-pad], r.logp) and torch.equal(outs[5][pad:-pad].view(n, top), r.top_logp)
    assert torch.equal(outs[3][pad:-pad].view(2, n), r.norm)
    alone = torch.empty(n, device="cuda")
    s0 = sv.sv_logprobs_shape_t(n, v, 0, 0, 0, 1.0, -1)
    assert lib.sv_logprobs(ctypes.byref(s0), z.data_ptr(), t.data_ptr(), alone.data_ptr(), None, None, None, None, None, None,
                           base, need, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(alone, r.logp)


def test_same_bits_again_and_in_any_batch(sv):
    """Results do not depend on the run, the stream, the alternatives asked for, or (in one
    way of taking rows) the other rows."""
    z = torch.randn(40, 100003, generator=gen(3), device="cuda")
    t = torch.arange(40, device="cuda")
    a = sv.logprobs(z, t, 0.7, top=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = sv.logprobs(z, t, 0.7, top=9, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    c = sv.logprobs(z, t, 0.7, top=32)
    for x, y, w in zip(a[:5], b[:5], c[:5]):
        assert torch.equal(x, y) and torch.equal(x, w)
    assert torch.equal(a.top_idx, b.top_idx) and torch.equal(a.top_idx, c.top_idx[:, :9])
    assert torch.equal(a.top_logp, c.top_logp[:, :9])


def test_offsets_past_32_bits(sv):
    """Logits of more than 2^31 elements and 2^32 bytes."""
    n, v = 17000, 131077
    z = torch.randn(40, v, generator=gen(1), device="cuda").to(BF)
    big = torch.empty(n, v, dtype=BF, device="cuda")
    big[:-40] = 0
    big[-40:] = z
    t = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    t[-40:] = torch.arange(40, device="cuda", dtype=torch.int32)
    r = sv.logprobs(big, t, top=3)
    few = sv.logprobs(z, t[-40:], top=3)
    assert torch.equal(r.top_idx[-40:], few.top_idx)
    Want(z, t[-40:], 1.0).check(sv.LogprobsResult(*[x[-40:] for x in r[:3]], r.norm[:, -40:], r.status[-40:], None, None), "far")
    assert not r.logp[:-40].any()
    g = torch.ones(n, device="cuda")
    w, tol = Want(z, t[-40:], 1.0).grad(t[-40:], g[-40:], None, BF)
    got = sv.logprobs_grad(big, t, r, g, out=big)
    within(got[-40:], w, tol, "far gradient")
    assert not got[:-40].any()


@pytest.mark.parametrize("dtype", [BF, F])
def test_longest_rows(sv, dtype):
    v = 1 << 24
    z = torch.randn(2, v, generator=gen(1), device="cuda").to(dtype)
    t = torch.tensor([v - 1, 0], device="cuda")
    r = sv.logprobs(z, t, 0.9, top=32)
    w = Want(z, t, 0.9)
    w.check(r, "longest rows")
    check_top(r, w, z, 32, "longest rows")
    none = sv.logprobs(z, t, 0.9)
    w.check(none, "longest rows without alternatives")
    g, h = torch.tensor([1.0, -2.0], device="cuda"), torch.tensor([0.5, 0.0], device="cuda")
    within(sv.logprobs_grad(z, t, r, g, h, 0.9), *w.grad(t, g, h, dtype), "longest rows")


def test_many_short_rows(sv):
    n = 1 << 20
    z = torch.randn(n, 3, generator=gen(1), device="cuda")
    t = torch.randint(0, 3, (n,), generator=gen(2), device="cuda")
    r = sv.logprobs(z, t, top=2)
    w = Want(z, t, 1.0)
    w.check(r, "short rows")
    check_top(r, w, z, 2, "short rows")
    got = sv.logprobs_grad(z, t, r, torch.ones(n, device="cuda"))
    within(got, *w.grad(t, torch.ones(n, device="cuda"), None, F), "short rows")


def test_graphs(sv):
    """Two captured graphs and eager calls between their replays; each replay of new inputs."""
    v, n = 60000, 5
    z = [torch.empty(n, v, device="cuda") for _ in range(2)]
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    g = torch.linspace(-1, 1, n, device="cuda")
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for k in range(2):
        z[k].normal_(generator=gen(k))
        with torch.cuda.stream(side):
            sv.logprobs(z[k], t, top=4)
        side.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            r = sv.logprobs(z[k], t, top=4)
            d = sv.logprobs_grad(z[k], t, r, g, g)
        graphs.append(gr)
        outs.append((r, d))
    for turn in range(4):
        for k in range(2):
            z[k].normal_(generator=gen(10 + 2 * turn + k))
            graphs[k].replay()
            r = sv.logprobs(z[k], t, top=4)
            d = sv.logprobs_grad(z[k], t, r, g, g)
            torch.cuda.synchronize()
            for x, y in zip(r, outs[k][0]):
                assert torch.equal(x, y)
            assert torch.equal(d, outs[k][1])


def test_with_verification(sv):
    """A rollout step: the bonus row's and the drafts' log-probabilities from the logits that
    verify read agree with its own normaliser and stored alternatives."""
    B, k, v = 3, 2, 9000
    g = gen(5)
    target = torch.randn(B, k + 1, v, generator=g, device="cuda") * 3
    draft = target[:, :k] + torch.randn(B, k, v, generator=g, device="cuda")
    x = torch.randint(0, v, (B, k), generator=g, device="cuda", dtype=torch.int32)
    o = sv.verify(target, draft, x, torch.rand(B, k + 2, generator=g, device="cuda"), 0.7, aux=True)
    full = torch.cat([x, torch.zeros(B, 1, dtype=torch.int32, device="cuda")], 1)
    r = sv.logprobs(target, full, 0.7, top=32)
    assert torch.equal(r.top_idx, o.topk_idx)
    torch.testing.assert_close(r.lse, o.lse_target, rtol=1e-6, atol=1e-6)
    torch.testing.assert_close(r.logp[:, :k].exp(), o.p_tok, rtol=1e-5, atol=0)
    # the tokens that came out, scored for the policy step; what follows them is left out
    s = sv.logprobs(target, o.out_tokens, 0.7)
    assert torch.equal(s.logp == 0, o.out_tokens == -1)
    assert not sv.logprobs_grad(target, o.out_tokens, s, torch.ones(B, k + 1, device="cuda"), None, 0.7)[o.out_tokens == -1].any()
