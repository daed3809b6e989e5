"""The gradient's memory: what may overlap the logits' and what is refused."""
import pytest

torch = pytest.importorskip("torch")

from draft_verification_spec_amd.score import _shared  # noqa: E402

BF, F = torch.bfloat16, torch.float32


def bytes_of(t, ld):
    """Bytes of rows of a tensor, each with the element that holds it."""
    e, at = t.element_size(), t.data_ptr()
    return {at + (i * ld + j) * e + k: (i, j, k) for i in range(t.shape[0]) for j in range(t.shape[1]) for k in range(e)}


@pytest.mark.parametrize("n", [0, 1, 2, 5])
@pytest.mark.parametrize("dt,gt", [(F, F), (BF, BF), (F, BF), (BF, F)])
def test_against_bytes(n, dt, gt):
    """Every distance in bytes, of rows at equal and at other distances."""
    V, seen = 3, [0, 0]
    memory = torch.zeros(4096, dtype=torch.uint8)

    def rows(at, ld, dtype):
        e = torch.empty(0, dtype=dtype).element_size()
        return memory[at:at + 1600].view(dtype)[:1600 // e].as_strided((n, V), (ld, 1))
    for lda in (3, 4, 7, 12):
        for ldb in (3, 4, 6, 7, 8, 12, 14, 24):
            ea, eb = torch.empty(0, dtype=dt).element_size(), torch.empty(0, dtype=gt).element_size()
            for d in range(-400, 400, 2 if eb == 2 else 4):
                a, b = rows(1024, lda, dt), rows(1024 + d, ldb, gt)
                x, y = bytes_of(a, lda), bytes_of(b, ldb)
                both = x.keys() & y.keys()
                real = any(x[k] != y[k] for k in both) or bool(both) and dt is not gt
                got = _shared(a, lda if n > 1 else V, b, ldb if n > 1 else V)
                # nothing that overlaps passes; rows at one distance, or one row, are told apart exactly
                assert got or not real, (lda, ldb, d)
                if lda * ea == ldb * eb or n < 2:
                    assert got == real, (lda, ldb, d)
                elif not both:
                    ends = [(min(s), max(s)) for s in (x, y)]
                    assert not got or ends[0][0] <= ends[1][1] and ends[1][0] <= ends[0][1], (lda, ldb, d)
                seen[got] += 1
    assert seen[0] and (seen[1] or not n)


@pytest.mark.gpu
def test_refused_and_taken():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import draft_verification_spec_amd as sv
    n, v = 6, 500
    t, g = torch.arange(n, device="cuda"), torch.ones(n, device="cuda")
    wide = torch.randn(n, 3 * v, device="cuda")
    z = wide[:, :v]
    r = sv.logprobs(z, t)
    want = sv.logprobs_grad(z, t, r, g)
    kept = wide.clone()
    rows_later = wide.view(-1)[v // 2:].as_strided((n, v), (3 * v, 1), v // 2)
    for out in (wide[:, 1:v + 1], wide[:, v - 1:2 * v - 1], rows_later):
        with pytest.raises(ValueError, match="apart"):
            sv.logprobs_grad(z, t, r, g, out=out)
    with pytest.raises(ValueError, match="apart"):
        sv.logprobs_grad(z, t, r, g, out=wide.view(BF)[:, :v])           # the same rows as another type
    assert torch.equal(wide, kept)
    assert torch.equal(sv.logprobs_grad(z, t, r, g, out=wide[:, v:2 * v]), want)   # between the rows
    assert torch.equal(wide[:, :v], kept[:, :v]) and torch.equal(wide[:, 2 * v:], kept[:, 2 * v:])
    assert torch.equal(sv.logprobs_grad(z, t, r, g, out=z), want)
    assert torch.equal(wide[:, :v], want)
