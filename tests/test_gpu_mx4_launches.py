"""Head logits of more hidden rows in 4 bits than one launch stages, about the border."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values(codes, scale, h):
    """What codes [..., H / 2] and exponent bytes stand for, in 64 bits."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)[..., :h].long()
    v = torch.tensor(GRID + tuple(-s for s in GRID), dtype=torch.float64, device=codes.device)[code]
    return v * ((scale.long() + 896) << 52).view(torch.float64).repeat_interleave(32, -1)[..., :h]


def test_rows_of_a_second_launch():
    """64 elements a row: a launch stages 268435392 rows.  The logits before, at and behind that
    border, and of the first rows, which a misplaced scale would meet as well."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import draft_verification_spec_amd as sv
    border, h, v = 268435392, 64, 3
    n = border + 200
    if torch.cuda.mem_get_info()[0] < (140 << 30):
        pytest.skip("needs 140 GB of memory")
    print(f"[gpu-test] head_logits4 n={n} h={h} v={v} mx4 f32", file=sys.stderr, flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.empty(n, h // 2, dtype=torch.uint8, device="cuda")
    scale = torch.full((n, h // 32), 127, dtype=torch.uint8, device="cuda")
    looked = torch.cat([torch.arange(300), torch.arange(border // 2, border // 2 + 70), torch.arange(border - 300, n)]).cuda()
    codes.zero_()
    codes[looked] = torch.randint(0, 256, (len(looked), h // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale[looked] = torch.randint(100, 150, (len(looked), h // 32), generator=g, device="cuda", dtype=torch.uint8)
    wc = torch.randint(0, 256, (v, h // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(120, 135, (v, h // 32), generator=g, device="cuda", dtype=torch.uint8)
    got = sv.head_logits(sv.Mx4(codes, scale, h), sv.Mx4(wc, ws, h), out_dtype=torch.float32)
    a, b = values(codes[looked], scale[looked], h).cpu(), values(wc, ws, h).cpu()
    want, size = a @ b.T, a.abs() @ b.abs().T
    # fp32 sums of 64 exact products, rounded once
    off = (got[looked].cpu().double() - want).abs()
    assert (off <= size * h * 2.0 ** -24 + want.abs() * 2.0 ** -24).all(), int((off - size * 1e-5).max(1).values.argmax())
    del codes, scale, got
    torch.cuda.empty_cache()
