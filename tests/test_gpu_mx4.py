"""Microscaled 4-bit rows and the head logits formed from them, against their formulas in
64 bits.

Rows are exact: codes and scales are compared bit for bit.  Logits: products of two codes and
scales are exact, their sum of H terms in fp32 is off by at most H 2^-24 of the sum of
magnitudes, and the result is rounded once.
"""
import ctypes
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


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


def two(k):
    """2 ** k in 64 bits, from its bits (a library's power need not be exact)."""
    return (k.long() + 1023 << 52).view(torch.float64)


def plain_pack(x):
    """(codes a byte each [..., H], exponent bytes [..., blocks]): the nearest of the grid by
    distance in 64 bits, the even code at a tie."""
    H = x.shape[-1]
    b = torch.nn.functional.pad(x.double(), (0, -H % 32)).unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(top)
    k = torch.frexp(torch.where(bad | (top == 0), torch.ones_like(top), top)).exponent - 1
    e = torch.where(top == 0, 0, (k - 2 + 127).clamp(min=0))
    e = torch.where(bad, 255, e)
    y = b * two(127 - e)[..., None]
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    d = (y.abs()[..., None] - grid).abs()
    d = d + torch.tensor([0, 1] * 4, device=x.device) * 1e-13      # ties to the even code
    code = d.argmin(-1) + 8 * torch.signbit(b).long()
    code = torch.where(bad[..., None], 0, code)
    return code.flatten(-2)[..., :H].to(torch.uint8), e.to(torch.uint8)


def join(code):
    """Two codes a byte."""
    code = torch.nn.functional.pad(code, (0, code.shape[-1] % 2))
    return code[..., 0::2] | code[..., 1::2] << 4


def values(code, e):
    """What codes [..., H] and exponent bytes stand for, in 64 bits."""
    H = code.shape[-1]
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64, device=code.device)
    p = two(e.long() - 127)
    p = torch.where(e == 255, torch.full_like(p, float("nan")), p)
    return grid[code.long()] * p.repeat_interleave(32, -1)[..., :H]


def hard(n, h, dtype, seed):
    """Rows whose blocks hold borders between codes, their neighbours, and magnitudes from the
    smallest to the largest."""
    g = gen(seed)
    x = torch.randn(n, h, generator=g, device="cuda") * torch.exp2(torch.randint(-30, 30, (n, 1), generator=g, device="cuda").float())
    if h >= 32:
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, 0.0, 0.5, 1.0, 2.0, 4.0, 6.5], device="cuda")
        for i in range(min(n, 6)):
            p = 2.0 ** [0, -126, -140, 100, 125, 3][i]
            b = torch.cat([mids * p, -mids * p])
            b[20] = 7.75 * p
            up = torch.nextafter(b, torch.full_like(b, 3e38)) if i % 2 else torch.nextafter(b, torch.zeros_like(b))
            x[i, :32] = b
            if h >= 64:
                x[i, 32:64] = up
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,h", [(1, 1), (1, 2), (3, 7), (2, 31), (2, 32), (5, 33), (6, 64), (7, 129), (6, 1000), (1, 1024),
                                 (9, 4096), (2, 20001), (1000, 96), (5000, 65), (300, 1111), (1, 131072)])
def test_round_trip(sv, n, h, dtype):
    log(f"mx4 n={n} h={h} {dtype}")
    x = hard(n, h, dtype, n * 3 + h)
    a = sv.mx4_pack(x)
    code, e = plain_pack(x)
    assert a.width == h and a.codes.shape == (n, (h + 1) // 2) and a.scale.shape == (n, (h + 31) // 32)
    assert torch.equal(a.scale, e)
    assert torch.equal(a.codes, join(code))
    want = values(code, e)
    for out in (BF, F):
        got = sv.mx4_unpack(a, out)
        assert got.dtype is out and torch.equal(got.double(), want)


def test_blocks_of_their_own(sv):
    """Zeros, the smallest and largest magnitudes, NaN and infinities: a block each."""
    tops = [0.0, -0.0, 1e-45, 1.2e-38, 2.0 ** -125, 3.4028234e38, float("nan"), float("inf"), -float("inf"), 1.0]
    x = torch.zeros(3, 32 * len(tops), device="cuda")
    for i, t in enumerate(tops):
        x[:, 32 * i + 7] = t
        x[1, 32 * i + 8] = t / 2
        x[2, 32 * i + 31] = -t / 3
    for dtype in (F, BF):
        y = x.to(dtype)
        a = sv.mx4_pack(y)
        code, e = plain_pack(y)
        assert torch.equal(a.scale, e) and torch.equal(a.codes, join(code))
        got = sv.mx4_unpack(a, F).double()
        want = values(code, e)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
        assert torch.isnan(got[:, 32 * 6:32 * 9]).all()


def test_every_code_and_scale(sv):
    """Unpacking what pack does not make too: all 256 scales, all codes."""
    e = torch.arange(256, device="cuda").to(torch.uint8)[:, None]
    code = (torch.arange(32, device="cuda") % 16).to(torch.uint8).expand(256, 32)
    a = sv.Mx4(join(code).contiguous(), e, 32)
    want = values(code, e)
    for dtype in (F, BF):
        got = sv.mx4_unpack(a, dtype).double()
        w = torch.where(want.abs() >= 2.0 ** 128, torch.sign(want) * float("inf"), want)
        assert torch.equal(torch.isnan(got), torch.isnan(w)), dtype
        assert torch.equal(got.nan_to_num(), w.nan_to_num()), dtype


def test_strides_and_shapes(sv):
    base = torch.randn(6, 5, 300, generator=gen(3), device="cuda")
    for x in (base[:, :, 3:200], base[:, 1], base.transpose(1, 2), base[2, 3], base[::2], base[:, :, ::3],
              base[0, :1].expand(4, 300), base.bfloat16()[:, :, 1:]):
        a = sv.mx4_pack(x)
        code, e = plain_pack(x)
        assert torch.equal(a.codes, join(code)) and torch.equal(a.scale, e)
        want = values(code, e)
        assert torch.equal(sv.mx4_unpack(a, F).double(), want)
        # rows at odd distances
        wide = torch.full((*a.codes.shape[:-1], a.codes.shape[-1] + 3), 255, dtype=torch.uint8, device="cuda")
        wide[..., 1:-2] = a.codes
        ws = torch.full((*a.scale.shape[:-1], a.scale.shape[-1] + 1), 255, dtype=torch.uint8, device="cuda")
        ws[..., 1:] = a.scale
        b = sv.Mx4(wide[..., 1:-2], ws[..., 1:], a.width)
        assert torch.equal(sv.mx4_unpack(b, F).double(), want)
    a = sv.mx4_pack(torch.empty(0, 12, device="cuda"))
    assert a.codes.shape == (0, 6) and sv.mx4_unpack(a).shape == (0, 12)


def test_guarded_rows(sv):
    """The C entries write rows and nothing between or behind them."""
    lib = sv.load_library()
    for n, h, dt in ((5, 77, F), (3, 64, BF), (1, 1, F), (4, 4097, BF)):
        x = torch.randn(n, h, generator=gen(h), device="cuda").to(dt)
        cb, sb = (h + 1) // 2, (h + 31) // 32
        codes = torch.full((n + 2, cb + 5), 170, dtype=torch.uint8, device="cuda")
        scale = torch.full((n + 2, sb + 3), 170, dtype=torch.uint8, device="cuda")
        assert lib.sv_mx4_pack(n, h, 1 if dt is BF else 0, x.data_ptr(), 0, codes[1].data_ptr(), cb + 5,
                               scale[1].data_ptr(), sb + 3, None) == 0
        torch.cuda.synchronize()
        code, e = plain_pack(x)
        assert torch.equal(codes[1:-1, :cb], join(code)) and torch.equal(scale[1:-1, :sb], e)
        assert (codes[0] == 170).all() and (codes[-1] == 170).all() and (codes[:, cb:] == 170).all()
        assert (scale[0] == 170).all() and (scale[-1] == 170).all() and (scale[:, sb:] == 170).all()
        y = torch.full((n * h + 16,), 7.0, dtype=dt, device="cuda")
        assert lib.sv_mx4_unpack(n, h, codes[1].data_ptr(), cb + 5, scale[1].data_ptr(), sb + 3, 1 if dt is BF else 0,
                                 y[8:].data_ptr(), None) == 0
        torch.cuda.synchronize()
        assert torch.equal(y[8:-8].view(n, h).double(), values(code, e)) and (y[:8] == 7).all() and (y[-8:] == 7).all()


def test_rows_past_32_bits(sv):
    """More than 2^32 elements."""
    n, h = 1 << 17, 32800
    x = torch.empty(n, h, dtype=BF, device="cuda")
    x.fill_(0.75)
    last = torch.randn(3, h, generator=gen(1), device="cuda").to(BF)
    x[-3:] = last
    a = sv.mx4_pack(x)
    code, e = plain_pack(last)
    assert torch.equal(a.codes[-3:], join(code)) and torch.equal(a.scale[-3:], e)
    del x
    assert (a.scale[:-3] == 124).all()
    y = sv.mx4_unpack(a)
    assert torch.equal(y[-3:].double(), values(code, e)) and (y[:-3] == 0.75).all()


# -------------------------------------------------------------------- head logits
LOGITS = [(1, 1, 1), (1, 1024, 1000), (3, 100, 77), (16, 128, 513), (17, 4096, 999), (31, 683, 3601), (32, 96, 260),
          (33, 256, 130), (64, 64, 4099), (64, 4096, 300), (65, 512, 2049), (65, 1000, 517), (70, 7, 131), (129, 200, 1021),
          (300, 384, 2048), (200, 1056, 70001), (257, 512, 66001), (5, 20001, 50), (90, 480, 70000), (90, 512, 70000), (128, 2048, 33), (40, 12000, 333), (1, 131072, 18),
          (2, 131071, 130), (150, 97, 511)]


@pytest.mark.parametrize("kind,out", [(BF, BF), (F, F), ("mx4", BF), ("mx4", F)])
@pytest.mark.parametrize("n,h,v", LOGITS)
def test_logits(sv, n, h, v, kind, out):
    log(f"head_logits4 n={n} h={h} v={v} {kind} {out}")
    g = gen(n + h + v)
    x = torch.randn(n, h, generator=g, device="cuda").to(F if kind == "mx4" else kind)
    w = torch.randn(v, h, generator=g, device="cuda")
    wc, we = plain_pack(w)
    xc, xe = plain_pack(x)
    head = sv.Mx4(join(wc), we, h)
    hidden = sv.Mx4(join(xc), xe, h) if kind == "mx4" else x
    a, b = values(xc, xe), values(wc, we)
    want = a @ b.T
    size = a.abs() @ b.abs().T
    got = sv.head_logits(hidden, head, out_dtype=out)
    assert got.dtype is out and got.shape == (n, v)
    within(got, want, size * h * 2.0 ** -24 + HALF[out] * want.abs(), "logits")
    # and of the head as pack lays it
    assert torch.equal(sv.head_logits(hidden, sv.mx4_pack(w), out_dtype=out), got)


@pytest.mark.parametrize("n", [3, 40, 100, 300])
def test_logits_strides(sv, n):
    """Weights and hidden rows at any address and distance, several leading axes; what lies
    between rows has no part."""
    h, v = 415, 700
    g = gen(n)
    x, w = torch.randn(n, h, generator=g, device="cuda"), torch.randn(v, h, generator=g, device="cuda")
    (wc, we), (xc, xe) = plain_pack(w), plain_pack(x)
    want = sv.head_logits(x, sv.Mx4(join(wc), we, h), out_dtype=F)
    for pad, off in ((1, 0), (5, 3), (48, 16), (64, 8)):
        c = torch.full((v, (h + 1) // 2 + pad), 255, dtype=torch.uint8, device="cuda")
        s = torch.full((v, (h + 31) // 32 + pad), 255, dtype=torch.uint8, device="cuda")
        off = min(off, pad)
        c[:, off:off + (h + 1) // 2], s[:, off:off + (h + 31) // 32] = join(wc), we
        c[:, off + (h + 1) // 2 - 1] |= 0xf0               # the half byte behind an odd row
        head = sv.Mx4(c[:, off:off + (h + 1) // 2], s[:, off:off + (h + 31) // 32], h)
        assert torch.equal(sv.head_logits(x, head, out_dtype=F), want), (pad, off)
        xx = torch.full((n, (h + 1) // 2 + pad), 255, dtype=torch.uint8, device="cuda")
        xx[:, off:off + (h + 1) // 2] = join(xc)
        xx[:, off + (h + 1) // 2 - 1] |= 0xf0
        assert torch.equal(sv.head_logits(sv.Mx4(xx[:, off:off + (h + 1) // 2], xe, h), head, out_dtype=F), want)
    wide = torch.full((n, h + 9), float("nan"), device="cuda")
    wide[:, 4:h + 4] = x
    head = sv.mx4_pack(w)
    assert torch.equal(sv.head_logits(wide[:, 4:h + 4], head, out_dtype=F), want)
    x3 = x.view(1, n, h).transpose(0, 1)
    got = sv.head_logits(x3, head, out_dtype=F)
    assert got.shape == (n, 1, v) and torch.equal(got[:, 0], want)
    assert sv.head_logits(x[:0], head).shape == (0, v)


@pytest.mark.parametrize("n", [2, 50, 100, 300])
def test_logits_nan_blocks(sv, n):
    """A NaN block makes its own row's, or its own column's, logits NaN and no others."""
    h, v = 600, 66000 if n == 300 else 400
    x, w = torch.randn(n, h, generator=gen(1), device="cuda"), torch.randn(v, h, generator=gen(2), device="cuda")
    clean = sv.head_logits(x, sv.mx4_pack(w), out_dtype=F)
    x[1, 599], w[7, 0] = float("nan"), float("inf")
    got = sv.head_logits(x, sv.mx4_pack(w), out_dtype=F)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[1], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], clean[~nan])


def test_logits_guards(sv):
    """The C entry at an odd output stride writes logits and nothing between them."""
    lib = sv.load_library()
    for n, h, v in ((3, 64, 333), (90, 130, 333), (300, 64, 66001)):
        x, w = torch.randn(n, h, generator=gen(1), device="cuda"), torch.randn(v, h, generator=gen(2), device="cuda")
        a = sv.mx4_pack(w)
        for dt, oc in ((F, 0), (BF, 1)):
            want = sv.head_logits(x, a, out_dtype=dt)
            out = torch.full((n + 1, v + 5), 7.0, dtype=dt, device="cuda")
            s = sv.sv_logits4_shape_t(n, h, v, 0, oc, 0, 0, a.codes.stride(0), a.scale.stride(0), v + 5)
            need = lib.sv_head_logits4_workspace_bytes(ctypes.byref(s))
            ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
            assert lib.sv_head_logits4(ctypes.byref(s), x.data_ptr(), None, a.codes.data_ptr(), a.scale.data_ptr(),
                                       out.data_ptr(), ws.data_ptr(), need, None) == 0
            torch.cuda.synchronize()
            assert (ws[need:] == 255).all()
            assert torch.equal(out[:n, :v], want) and (out[:, v:] == 7).all() and (out[n] == 7).all()


@pytest.mark.parametrize("n,h,v,step", [(3, 131072, 65900, 65536), (70, 20001, 13100, 13056), (130, 20000, 13100, None)])
def test_logits_in_pieces(sv, n, h, v, step):
    """Vocabularies that are taken in pieces: of staged scales (a weight read in place), and of
    copied rows (one at no 16-byte distance); and one that is not.  The columns about the pieces'
    borders against 64 bits."""
    log(f"head_logits4 in pieces n={n} h={h} v={v}")
    g = gen(v)
    codes = torch.randint(0, 256, (v, (h + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(120, 128, (v, (h + 31) // 32), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(n, h, generator=g, device="cuda")
    got = sv.head_logits(x, sv.Mx4(codes, scale, h), out_dtype=F)
    cols = {0, 1, v // 2, *range(v - 60, v)}
    cols |= set(range(step - 3, step + 40)) if step else set()
    cols = torch.tensor(sorted(cols), device="cuda")
    code = torch.stack((codes[cols] & 15, codes[cols] >> 4), -1).flatten(1)[:, :h]
    a, b = values(*plain_pack(x)), values(code, scale[cols])
    want = a @ b.T
    tol = (a.abs() @ b.abs().T) * h * 2.0 ** -24 + HALF[F] * want.abs()
    within(got[:, cols], want, tol, "columns about the borders")


def test_logits_do_not_depend_on_the_stream(sv):
    x, w = torch.randn(20, 640, generator=gen(1), device="cuda"), torch.randn(5000, 640, generator=gen(2), device="cuda")
    a = sv.mx4_pack(w)
    want = sv.head_logits(x, a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = sv.mx4_pack(w, stream=s.cuda_stream)
    got = sv.head_logits(x, b, stream=s.cuda_stream)
    back = sv.mx4_unpack(b, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(back, sv.mx4_unpack(a))


def test_graphs(sv):
    """Captured calls of few and of many rows, replayed on new inputs beside eager ones."""
    w = torch.randn(3000, 320, generator=gen(2), device="cuda")
    a = sv.mx4_pack(w)
    graphs = []
    side = torch.cuda.Stream()
    for n in (2, 30, 100):
        x = torch.randn(n, 320, generator=gen(n), device="cuda")
        with torch.cuda.stream(side):
            sv.head_logits(x, a)
        side.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            r = sv.head_logits(x, a)
            p = sv.mx4_unpack(sv.mx4_pack(x))
        graphs.append((gr, x, r, p))
    for turn in range(4):
        for gr, x, r, p in graphs:
            x.normal_(generator=gen(50 + turn))
            gr.replay()
            want, back = sv.head_logits(x, a), sv.mx4_unpack(sv.mx4_pack(x))
            torch.cuda.synchronize()
            assert torch.equal(r, want) and torch.equal(p, back)


def test_first_call_captured(sv):
    """A call that asks for more than 64 KB of LDS, captured before any like it was made."""
    x, w = torch.randn(90, 2048, generator=gen(1), device="cuda"), torch.randn(700, 2048, generator=gen(2), device="cuda")
    a, b = sv.mx4_pack(w), sv.mx4_pack(x)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        r = sv.head_logits(b, a, out_dtype=F)
    for turn in range(3):
        r.zero_()
        gr.replay()
        want = sv.head_logits(x, a, out_dtype=F)
        torch.cuda.synchronize()
        assert torch.equal(r, want)


def test_largest_vocabulary(sv):
    v, h = 1 << 24, 33
    w = torch.randn(v, h, generator=gen(1), device="cuda")
    a = sv.mx4_pack(w)
    del w
    for n in (2, 66):
        x = torch.randn(n, h, generator=gen(n), device="cuda")
        got = sv.head_logits(x, a, out_dtype=BF)
        cols = torch.cat([torch.arange(50, device="cuda"), torch.arange(v - 50, v, device="cuda")])
        wf = sv.mx4_unpack(sv.Mx4(a.codes[cols], a.scale[cols], h), F).double()
        xf = values(*plain_pack(x))
        want = xf @ wf.T
        within(got[:, cols], want, (xf.abs() @ wf.abs().T) * h * 2.0 ** -24 + HALF[BF] * want.abs(), "ends of the vocabulary")


def test_draft_step(sv):
    """A rollout step with a drafter's head in 4 bits and the target's in 8: drafted tokens
    verified against the target, then scored, and the policy gradient of what came out."""
    B, k, H, V = 4, 3, 256, 5000
    g = gen(11)
    head = torch.randn(V, H, generator=g, device="cuda") * 0.2
    h = torch.randn(B, k + 1, H, generator=g, device="cuda")
    target = sv.head_logits(h, sv.act8_pack(head))
    draft = sv.head_logits(h[:, :k], sv.mx4_pack(head))
    # the coarse head is near the other: 4-bit elements are off by 2^-2 of themselves at most
    corr = torch.corrcoef(torch.stack([draft.float().flatten(), target[:, :k].float().flatten()]))[0, 1]
    assert float(corr) > 0.9
    x = draft.float().argmax(-1).int()
    o = sv.verify(target, draft, x, torch.rand(B, k + 2, generator=g, device="cuda"), 1.0, aux=True)
    assert not o.status.any()
    r = sv.logprobs(target, o.out_tokens, top=32)
    used = o.out_tokens >= 0
    assert torch.equal(r.top_idx[used].long(), o.topk_idx[used].long())
    d = sv.logprobs(draft, x)
    torch.testing.assert_close(d.logp.exp(), o.q_tok, rtol=1e-5, atol=1e-7)
    grad = sv.logprobs_grad(target, o.out_tokens, r, torch.ones(B, k + 1, device="cuda"), torch.full((B, k + 1), 0.01, device="cuda"))
    assert torch.isfinite(grad.float()).all() and grad[used].any() and not grad[~used].any()
