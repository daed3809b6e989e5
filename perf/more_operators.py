"""Operators around sampled tokens and a small head as measured work.

  mx4       rows (a head's, or hidden ones) in microscaled 4-bit floating point, blocks
            of 32 with a power-of-two scale, and read back
  logits    hidden rows times a vocabulary head held in that format: a drafter's
            logits at a quarter of the bytes of a bfloat16 head
  score     log-probabilities of given tokens from logits, with the entropy and the
            largest alternatives of each row
  train     log-probabilities and entropies of a batch, and the gradient of the
            logits from theirs: a policy step with an entropy term

listed() and draw() give cases, prepare() their inputs, run() one pass (the
plain torch form, or the framework's calls where `own` is true), work() what a
pass cannot do without and exact() its result in 64 bits.
"""
import math

import torch

own = False

IGNORE = -1
BLOCK = 32                             # elements that share a scale
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
STEPS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # the magnitudes of the 4-bit numbers
BORDER = 1e-9                          # a drawn size is spread over the logarithm of its range


def listed():
    return [
        # one drafted position's hidden row: a launch-bound call
        dict(name="mx4 one row", op="mx4", n=1, h=1024, type="bf16"),
        # a whole head put into 4 bits after a weight update, and read back
        dict(name="mx4 head", op="mx4", n=151936, h=4096, type="bf16"),
        # rows of an odd width in float32, as a probe or a small drafter keeps them
        dict(name="mx4 odd f32", op="mx4", n=4999, h=1111, type="f32"),
        # one drafted token of one sequence, a small vocabulary: latency
        dict(name="logits one token", op="logits", n=1, h=1024, v=32000, type="bf16", out="bf16"),
        # the drafter's step at the steady batch: 32 sequences, one token each
        dict(name="logits draft", op="logits", n=32, h=4096, v=151936, type="bf16", out="bf16"),
        # a small float32 drafter at a ragged batch and an odd vocabulary
        dict(name="logits odd f32", op="logits", n=77, h=1000, v=50001, type="f32", out="f32"),
        # drafted logits of a whole rollout step formed again: 256 sequences of 4 positions
        dict(name="logits rollout", op="logits", n=1024, h=4096, v=151936, type="bf16", out="bf16"),
        # a server's reply for one sampled token: its log-probability and five alternatives
        dict(name="score one token", op="score", n=1, v=32000, type="bf16", top=5, temperature=1.0, masked=False),
        # a serving batch under token masks, twenty alternatives each
        dict(name="score serving", op="score", n=256, v=151936, type="bf16", top=20, temperature=0.7, masked=True),
        # log-probabilities of a rollout's tokens from float32 logits, no alternatives
        dict(name="score rollout f32", op="score", n=2000, v=100001, type="f32", top=0, temperature=1.0, masked=False),
        # a policy step over a few tokens of a small vocabulary
        dict(name="train few f32", op="train", n=24, v=20000, type="f32", temperature=1.0),
        # a policy step with an entropy term over a rollout batch: the largest
        dict(name="train rollout", op="train", n=4096, v=151936, type="bf16", temperature=1.0),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low) - BORDER, math.log(high) + BORDER))))


def draw(rng):
    op = rng.choice(["mx4", "logits", "logits", "score", "score", "train"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op in ("mx4", "logits"):
        h = _spread(rng, 64, 4096)
        if rng.random() < 0.75:
            h = max(64, h // 64 * 64)                  # heads are mostly whole multiples of 64; the others stay odd
        if op == "mx4":
            return dict(op=op, n=_spread(rng, 1, 75968 if kind == "f32" else 151936), h=h, type=kind)
        return dict(op=op, n=_spread(rng, 1, 1024), h=h, v=_spread(rng, 1000, 151936), type=kind,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    v, temperature = _spread(rng, 1000, 151936), rng.choice([1.0, 0.7])
    if op == "train":
        return dict(op=op, n=_spread(rng, 1, 2048 if kind == "f32" else 4096), v=v, type=kind, temperature=temperature)
    top = rng.choice([0, 1, 5, 20, 32])
    return dict(op=op, n=_spread(rng, 1, 256 if top else 2048), v=v, type=kind, top=top, temperature=temperature,
                masked=rng.random() < 0.25)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, n, kind = case["op"], case["n"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if op == "mx4":
        # rows near unit size, some larger
        x = normal(n, case["h"]).mul_(0.5 + 2 * uniform(n, 1))
        return dict(op=op, x=x.to(kind))
    v = case["v"]
    if op == "logits":
        # the head was put into 4 bits once, when it was loaded
        h = case["h"]
        codes, scale = _mx4(normal(v, h).mul_(3.0 / math.sqrt(h)))
        codes = torch.nn.functional.pad(codes[:, :h], (0, h % 2))
        return dict(op=op, x=normal(n, h).to(kind), codes=codes[:, 0::2] | codes[:, 1::2] << 4, scale=scale,
                    out=TYPES[case["out"]])
    # logits of a trained model: a bell with a few tokens well above it, and the given
    # token drawn near the top
    z = normal(n, v).mul_(2.5)
    row = torch.arange(n, device="cuda")[:, None]
    peaks = torch.randint(0, v, (n, 8), generator=g, device="cuda")
    z[row, peaks] += 4 + 8 * uniform(n, 8)
    tokens = peaks[:, 0].to(torch.int32)
    s = dict(op=op, temperature=case["temperature"], tokens=tokens)
    if op == "score":
        s["top"] = case["top"]
        if case["masked"]:                             # tokens that a grammar rules out
            away = uniform(n, v) < 0.3
            away[row, peaks[:, :1]] = False
            z.masked_fill_(away, -math.inf)
    else:
        # a quarter of the positions is prompt or padding
        away = torch.randperm(n, generator=g, device="cuda")[:n // 4]
        tokens[away] = IGNORE
        s["grad_logp"] = normal(n) / n
        s["grad_entropy"] = -0.01 * uniform(n) / n
    s["logits"] = z.to(kind)
    return s


# ------------------------------------------------------------------ plain forms
def _power(e):
    """2 ** (e - 127) in float32 for whole e of 0 .. 254."""
    return torch.where(e > 0, e << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _mx4(x):
    """Rows as 4-bit codes (one a byte) in whole blocks, and the blocks' exponents."""
    n, h = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -h % BLOCK)).view(n, -1, BLOCK)
    e = ((b.abs().amax(2).view(torch.int32) >> 23) - 2).clamp_(min=0)
    y = b.abs() * _power(254 - e)[:, :, None]
    code = (y > 0.25).to(torch.uint8)
    code += y >= 0.75
    code += y > 1.25
    code += y >= 1.75
    code += y > 2.5
    code += y >= 3.5
    code += y > 5
    code += (b < 0).to(torch.uint8) * 8
    return code.view(n, -1), e.to(torch.uint8)


def _values(code, e):
    table = torch.tensor(STEPS + tuple(-s for s in STEPS), device="cuda")
    n = code.shape[0]
    return (table[code.view(n, -1, BLOCK).int()] * _power(e.int())[:, :, None]).view(n, -1)


def _plain_mx4(s):
    h = s["x"].shape[1]
    return dict(x=_values(*_mx4(s["x"]))[:, :h].to(s["x"].dtype))


def _plain_logits(s):
    x = _values(*_mx4(s["x"]))
    v, nb = s["scale"].shape
    code = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).view(v, -1)
    w = _values(torch.nn.functional.pad(code, (0, nb * BLOCK - code.shape[1])), s["scale"])
    return dict(logits=torch.matmul(x, w.t()).to(s["out"]))


def _rows(s):
    """Scaled logits less their maximum, their exponentials and sums."""
    z = s["logits"].float() / s["temperature"]
    m = z.amax(1, keepdim=True)
    z -= m
    e = torch.exp(z)
    return z, m[:, 0], e, e.sum(1)


def _results(s, z, m, e, total):
    used = s["tokens"] != IGNORE
    zero = torch.zeros_like(m)
    log_total = torch.log(total)
    mean = (e * z.clamp(min=-1e30)).sum(1) / total    # (an entry of -inf has no part in it)
    logp = z.gather(1, s["tokens"].long().clamp(min=0)[:, None])[:, 0] - log_total
    return dict(logp=torch.where(used, logp, zero), entropy=torch.where(used, log_total - mean, zero),
                lse=torch.where(used, m + log_total, zero))


def _plain_score(s):
    z, m, e, total = _rows(s)
    out = _results(s, z, m, e, total)
    if s["top"]:
        v = z.shape[1]
        bits = (s["logits"].float() + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, bits ^ 0x7fffffff, bits) << 32
        key |= torch.arange(v - 1, -1, -1, device="cuda")     # equal logits: the lowest token first
        best = v - 1 - (torch.topk(key, s["top"], dim=1).values & 0xffffffff)
        out["top_logp"] = z.gather(1, best) - torch.log(total)[:, None]
        out["top_idx"] = best.to(torch.int32)
    return out


def _plain_train(s):
    z, m, e, total = _rows(s)
    out = _results(s, z, m, e, total)
    used = s["tokens"] != IGNORE
    g = torch.where(used, s["grad_logp"], torch.zeros_like(m))[:, None]
    h = torch.where(used, s["grad_entropy"], torch.zeros_like(m))[:, None]
    p = e.div_(total[:, None])
    z -= torch.log(total)[:, None]                    # every token's log-probability
    d = p * (z.add_(out["entropy"][:, None]).mul_(-h) - g)
    d.scatter_add_(1, s["tokens"].long().clamp(min=0)[:, None], g)
    out["grad"] = (d / s["temperature"]).to(s["logits"].dtype)
    return out


# ---------------------------------------------------------- the framework's calls
def _own(s):
    import draft_verification_spec_amd as sv
    op = s["op"]
    if op == "mx4":
        return dict(x=sv.mx4_unpack(sv.mx4_pack(s["x"]), s["x"].dtype))
    if op == "logits":
        return dict(logits=sv.head_logits(s["x"], sv.Mx4(s["codes"], s["scale"], s["x"].shape[1]), out_dtype=s["out"]))
    r = sv.logprobs(s["logits"], s["tokens"], s["temperature"], top=s.get("top", 0), ignore_index=IGNORE)
    out = dict(logp=r.logp, entropy=r.entropy, lse=r.lse)
    if op == "train":
        out["grad"] = sv.logprobs_grad(s["logits"], s["tokens"], r, s["grad_logp"], s["grad_entropy"], s["temperature"],
                                       ignore_index=IGNORE)
    elif s["top"]:
        out["top_logp"], out["top_idx"] = r.top_logp, r.top_idx
    return out


def run(state):
    if own:
        return _own(state)
    return {"mx4": _plain_mx4, "logits": _plain_logits, "score": _plain_score, "train": _plain_train}[state["op"]](state)


def _packed(n, h):
    return n * (-(-h // 2) + -(-h // BLOCK))


def work(case):
    op, n, e = case["op"], case["n"], SIZES[case["type"]]
    if op == "mx4":                                    # rows in, codes and scales out; codes and scales in, rows out
        return dict(bytes=2 * n * case["h"] * e + 2 * _packed(n, case["h"]), flops=4 * n * case["h"])
    v = case["v"]
    if op == "logits":
        h = case["h"]
        return dict(bytes=n * h * e + _packed(v, h) + n * v * SIZES[case["out"]], flops=2 * n * h * v)
    if op == "score":
        return dict(bytes=n * v * e + n * (16 + 8 * case["top"]), flops=6 * n * v)
    used = n - n // 4                                  # rows left out are not read; their gradients are written
    return dict(bytes=used * v * e + n * v * e + n * 24, flops=12 * used * v)


# -------------------------------------------------------------- results in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]

    def two(k):
        """2 ** k in 64 bits, from its bits."""
        return (k.long() + 1023 << 52).view(torch.float64)

    def nearest(x):
        """x in 64 bits, each block of 32 on the grid of its largest magnitude's binade."""
        x = x.double()
        blocks = torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))
        unit = torch.frexp(blocks.abs().amax(2, keepdim=True)).exponent - 3    # top = m 2^k, m of 1/2 .. 1: floor(log2) = k - 1
        y = blocks * two(-unit)
        size = y.abs()
        step = 0.5 + 0.5 * (size >= 2) + (size >= 4)
        q = torch.round(size / step).mul(step).clamp(max=6.0) * y.sign()
        return (q * two(unit)).flatten(1)[:, :x.shape[1]]

    if op == "mx4":
        return dict(x=nearest(s["x"]))
    if op == "logits":
        h = case["h"]
        c = torch.empty(case["v"], 2 * s["codes"].shape[1], dtype=torch.uint8, device="cuda")
        c[:, ::2], c[:, 1::2] = s["codes"] % 16, s["codes"] // 16
        c = c[:, :h].long()
        power, odd = (c >> 1) % 4, c % 2              # two bits of exponent, one of mantissa
        w = torch.where(power > 0, (1 + 0.5 * odd) * two(power - 1), 0.5 * odd.double())
        w = torch.where(c > 7, -w, w)
        unit = s["scale"].int().sub(127).repeat_interleave(BLOCK, 1)[:, :h]
        return dict(logits=nearest(s["x"]) @ (w * two(unit)).T)
    z = s["logits"].double().div_(s["temperature"])
    n, v = z.shape
    t = s["tokens"].long()
    keep = (t >= 0).double()
    row = torch.arange(n, device="cuda")
    lse = torch.logsumexp(z, 1)
    z.sub_(lse[:, None])
    p = z.exp()
    entropy = torch.special.entr(p).sum(1)
    out = dict(logp=z[row, t.clamp(min=0)] * keep, entropy=entropy * keep, lse=lse * keep)
    if op == "score":
        if s["top"]:
            out["top_logp"], out["top_idx"] = torch.sort(z, dim=1, descending=True, stable=True).values[:, :s["top"]], None
        return out
    g, h = (s["grad_logp"].double() * keep)[:, None], (s["grad_entropy"].double() * keep)[:, None]
    d = -p * g - h * (p * z + p * entropy[:, None])
    d[row, t.clamp(min=0)] += g[:, 0]
    out["grad"] = d.div_(s["temperature"])
    return out
