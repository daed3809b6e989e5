"""The vocabulary-head operators as measured work: what a drafter or a policy
does around spec_verify and sv_kd when its logits do not exist yet.

  act8    hidden rows stored in 8 bits with a scale per row, and read back
  logits  hidden rows times a vocabulary head held in 8-bit integers (a scale
          per token and per vocabulary entry): the logits spec_verify takes
  ce      softmax cross entropy of hidden rows under the head, from pieces of
          the vocabulary, with the gradients of hidden rows and head
  kd      the reward-weighted distillation over the stored top-32, the same way

listed() and draw() give cases, prepare() their inputs, run() one pass (the
plain torch form, or the framework's calls where `own` is true), work() what a
pass cannot do without and exact() its result in 64 bits.
"""
import math

import torch

own = False

GROUP, LEN, TOP = 8, 16, 32            # rollouts a prompt, stored positions a rollout, stored targets a position
IGNORE = -1
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BORDER = 1e-9                          # a drawn size is spread over the logarithm of its range


def listed():
    return [
        # one decoded position's hidden row put away: a launch-bound call
        dict(name="act8 one row", op="act8", n=1, h=1024, type="bf16"),
        # the hidden rows of a rollout batch (2048 sequences of 16 positions) for the replay buffer
        dict(name="act8 rollout", op="act8", n=32768, h=4096, type="bf16"),
        # rows of an odd width in float32, as a probe or a small drafter keeps them
        dict(name="act8 odd f32", op="act8", n=4999, h=1111, type="f32"),
        # one drafted token of one sequence, a small vocabulary: latency
        dict(name="logits one token", op="logits", n=1, h=1024, v=32000, type="bf16", out="bf16"),
        # the drafter's step at the steady batch: 32 sequences, one token each
        dict(name="logits draft", op="logits", n=32, h=4096, v=151936, type="bf16", out="bf16"),
        # the verification step of a GRPO batch: 256 sequences, 3 drafts and a bonus position each
        dict(name="logits verify", op="logits", n=1024, h=4096, v=128256, type="bf16", out="bf16"),
        # online fine-tuning of a small drafter on a few accepted tokens, float32 weights
        dict(name="ce few rows f32", op="ce", n=24, h=512, v=20000, type="f32", stored=False, grad=True, temperature=1.0),
        # log-probabilities of rolled-out tokens under the policy, no gradient
        dict(name="ce log-probs", op="ce", n=2048, h=4096, v=128256, type="bf16", stored=False, grad=False, temperature=0.7),
        # drafter fine-tuning from hidden rows that the replay buffer holds in 8 bits, a ragged batch
        dict(name="ce stored rows", op="ce", n=1000, h=2048, v=151936, type="bf16", stored=True, grad=True, temperature=1.0),
        # a policy step over a rollout batch: the largest
        dict(name="ce rollout", op="ce", n=4096, h=4096, v=151936, type="bf16", stored=False, grad=True, temperature=1.0),
        # distillation over three prompts' first positions
        dict(name="kd few rows", op="kd", n=24, h=1024, v=20000, type="bf16", stored=False, grad=True),
        # the distillation batch of one GRPO step: 32 prompts, 8 rollouts, 16 positions
        dict(name="kd rollout", op="kd", n=4096, h=2048, v=151936, type="bf16", stored=False, grad=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low) - BORDER, math.log(high) + BORDER))))


def draw(rng):
    op = rng.choice(["act8", "logits", "ce", "ce", "kd"])
    h = _spread(rng, 64, 4096)
    if rng.random() < 0.75:
        h = max(64, h // 64 * 64)                      # heads are mostly whole multiples of 64; the others stay odd
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "act8":
        return dict(op=op, n=_spread(rng, 1, 32768), h=h, type=kind)
    v = _spread(rng, 1000, 151936)
    if op == "logits":
        return dict(op=op, n=_spread(rng, 1, 1024), h=h, v=v, type=kind, out=rng.choice(["bf16", "bf16", "f32"]))
    c = dict(op=op, n=_spread(rng, 1, 4096), h=h, v=v, type=kind, stored=rng.random() < 0.25, grad=rng.random() < 0.75)
    if op == "ce":
        c["temperature"] = rng.choice([1.0, 0.7])
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, n, h = case["op"], case["n"], case["h"]
    kind = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "act8":
        # hidden rows behind a norm: near unit size, some rows larger
        x = normal(n, h) * (0.5 + 2 * torch.rand(n, 1, generator=g, device="cuda"))
        return dict(op=op, x=x.to(kind))
    v = case["v"]
    if op == "logits":
        # the head was put into 8 bits once, when it was loaded
        w = normal(v, h) * (3.0 / math.sqrt(h))
        scale = w.abs().amax(1) / 127
        codes = torch.round(w / scale[:, None]).to(torch.int8)
        return dict(op=op, x=normal(n, h).to(kind), codes=codes, scale=scale, out=TYPES[case["out"]])
    w = (normal(v, h) * (3.0 / math.sqrt(h))).to(kind)
    s = dict(op=op, w=w, grad=case["grad"])
    if op == "ce":
        # a model in training: the target's logit stands above the others; a quarter of the positions is prompt or padding
        t = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
        x = normal(n, h) + w[t.long()].float()
        away = torch.rand(n, generator=g, device="cuda") < 0.25
        away[0] = False
        s["targets"] = torch.where(away, torch.full_like(t, IGNORE), t)
        s["row_weight"] = (0.25 + torch.rand(n, generator=g, device="cuda")) / n
        s["temperature"] = case["temperature"]
    else:
        # 32 tokens a position as the verification stores them, the drafter near the target on the first four
        base = torch.randint(0, v, (n, 1), generator=g, device="cuda")
        step = torch.randint(1, v // TOP, (n, 1), generator=g, device="cuda")
        ids = (base + step * torch.arange(TOP, device="cuda")) % v
        x = normal(n, h) + w[ids[:, 0]].float() + w[ids[:, 1]].float() + w[ids[:, 2]].float() + w[ids[:, 3]].float()
        val = (10 + 2 * normal(n, TOP)).to(torch.bfloat16).float()
        samples = GROUP * -(-n // (LEN * GROUP))
        levels = torch.tensor([0.0, 0.3, 0.8, 1.0], device="cuda")
        rewards = levels[torch.randint(0, 4, (samples,), generator=g, device="cuda")]
        rewards[0] = 1.0                               # one answer at least was right
        s.update(topk_val=val, topk_idx=ids.to(torch.int32), rewards=rewards,
                 row_sample=(torch.arange(n, device="cuda") // LEN).to(torch.int32))
    if case["stored"]:                                 # as the replay buffer holds them
        scale = x.abs().amax(1) / 127
        s["codes"], s["scale"] = torch.round(x / scale[:, None]).to(torch.int8), scale
    else:
        s["x"] = x.to(kind)
    return s


# ------------------------------------------------------------------ plain forms
def _codes(x):
    """Rows as whole numbers of -127..127 and their scales; the border between two codes is told in 64 bits."""
    scale = (x.abs().amax(1).double() / 127).float()   # (a tensor over a number in 32 bits is not rounded right)
    return torch.round(x.double() / scale[:, None].double()), scale


def _hidden(s):
    return s["codes"].float() * s["scale"][:, None] if "codes" in s else s["x"].float()


def _plain_act8(s):
    c, scale = _codes(s["x"])
    return dict(x=(c.float() * scale[:, None]).to(s["x"].dtype), scale=scale)


def _plain_logits(s):
    c, scale = _codes(s["x"])
    z = torch.matmul(c.float(), s["codes"].float().t())
    return dict(logits=(z * (scale[:, None] * s["scale"])).to(s["out"]))


def _normaliser(z):
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    return (m + torch.log(total))[:, 0], e.div_(total)


def _gradients(s, x, w, dz):
    kind = s["w"].dtype
    return torch.matmul(dz, w).to(kind), torch.matmul(dz.t(), x).to(kind)


def _plain_ce(s):
    x, w, t = _hidden(s), s["w"].float(), s["targets"].long()
    used = t != IGNORE
    at = t.clamp(min=0)[:, None]
    z = torch.matmul(x, w.t()) / s["temperature"]
    lse, p = _normaliser(z)
    zero = torch.zeros_like(lse)
    nll = torch.where(used, lse - z.gather(1, at)[:, 0], zero)
    weight = torch.where(used, s["row_weight"], zero)
    out = dict(loss=(weight.double() * nll.double()).sum().float(), nll=nll, lse=torch.where(used, lse, zero))
    if s["grad"]:
        dz = p.mul_((weight / s["temperature"])[:, None])
        dz.scatter_add_(1, at, (-weight / s["temperature"])[:, None])
        out["grad_hidden"], out["grad_weight"] = _gradients(s, x, w, dz)
    return out


def _plain_kd(s):
    x, w, ids = _hidden(s), s["w"].float(), s["topk_idx"].long()
    z = torch.matmul(x, w.t())
    lse, q = _normaliser(z)
    stored, pt = _normaliser(s["topk_val"])
    kl = (pt * (s["topk_val"] - stored[:, None] - z.gather(1, ids) + lse[:, None])).sum(1)
    total = s["rewards"].view(-1, GROUP).sum(1, keepdim=True)
    share = torch.where(total > 0, s["rewards"].view(-1, GROUP) / total, torch.zeros_like(total)).view(-1)
    weight = share[s["row_sample"].long()]
    out = dict(loss=(weight.double() * kl.double()).sum().float(), kl=kl, weight=weight)
    if s["grad"]:
        dz = q.mul_(weight[:, None])
        dz.scatter_add_(1, ids, -weight[:, None] * pt)
        out["grad_hidden"], out["grad_weight"] = _gradients(s, x, w, dz)
    return out


# ---------------------------------------------------------- the framework's calls
def _own(s):
    import draft_verification_spec_amd as sv
    op = s["op"]
    if op == "act8":
        a = sv.act8_pack(s["x"])
        return dict(x=sv.act8_unpack(a, s["x"].dtype), scale=a.scale)
    if op == "logits":
        return dict(logits=sv.head_logits(s["x"], sv.Act8(s["codes"], s["scale"]), out_dtype=s["out"]))
    x = sv.Act8(s["codes"], s["scale"]) if "codes" in s else s["x"]
    if op == "ce":
        r = sv.head_ce(x, s["w"], s["targets"], s["row_weight"], temperature=s["temperature"], ignore_index=IGNORE,
                       grad=s["grad"])
        out = dict(loss=r.loss[0], nll=r.nll, lse=r.lse)
    else:
        r = sv.head_kd(x, s["w"], s["topk_val"], s["topk_idx"], s["row_sample"], s["rewards"], GROUP, grad=s["grad"])
        out = dict(loss=r.loss[0], kl=r.kl, weight=r.weight)
    if s["grad"]:
        out["grad_hidden"], out["grad_weight"] = r.grad_hidden, r.grad_weight
    return out


def run(state):
    if own:
        return _own(state)
    return {"act8": _plain_act8, "logits": _plain_logits, "ce": _plain_ce, "kd": _plain_kd}[state["op"]](state)


def work(case):
    op, n, h = case["op"], case["n"], case["h"]
    e = 2 if case["type"] == "bf16" else 4
    if op == "act8":                                   # rows in, codes and scales out; codes and scales in, rows out
        return dict(bytes=2 * n * h * e + 2 * n * (h + 4), flops=4 * n * h)
    v = case["v"]
    if op == "logits":
        return dict(bytes=n * h * e + v * (h + 4) + n * v * (2 if case["out"] == "bf16" else 4), flops=2 * n * h * v)
    rows = n * (h + 4) if case["stored"] else n * h * e
    few = n * (4 + 4 + 4 + 4) if op == "ce" else n * (TOP * 8 + 4 + 4 + 4)
    if not case["grad"]:
        return dict(bytes=rows + v * h * e + few, flops=2 * n * h * v)
    return dict(bytes=rows + n * h * e + 2 * v * h * e + few, flops=6 * n * h * v)


# -------------------------------------------------------------- results in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]

    def eight(x):
        scale = (x.double().abs().max(dim=1).values / 127).float().double().unsqueeze(1)
        return (x.double() / scale).round(), scale

    if op == "act8":
        c, scale = eight(s["x"])
        return dict(x=c * scale, scale=scale.squeeze(1))
    if op == "logits":
        c, scale = eight(s["x"])
        return dict(logits=(c @ s["codes"].double().T) * scale * s["scale"].double().unsqueeze(0))
    x = s["codes"].double() * s["scale"].double().unsqueeze(1) if case["stored"] else s["x"].double()
    w = s["w"].double()
    tau = case.get("temperature", 1.0)
    z = (x @ w.T).div_(tau)
    lse = torch.logsumexp(z, 1)
    row = torch.arange(case["n"], device="cuda")
    if op == "ce":
        t = s["targets"].long()
        keep = (t >= 0).double()
        nll = (lse - z[row, t.clamp(min=0)]) * keep
        weight = s["row_weight"].double() * keep
        out = dict(nll=nll, lse=lse * keep)
    else:
        ids, val = s["topk_idx"].long(), s["topk_val"].double()
        pt = torch.softmax(val, 1)
        at = z[row.unsqueeze(1), ids]
        nll = (pt * (pt.log() - (at - lse.unsqueeze(1)))).sum(1)
        r = s["rewards"].double().reshape(-1, GROUP)
        total = r.sum(1, keepdim=True)
        weight = (r / total.where(total > 0, torch.ones_like(total))).reshape(-1)[s["row_sample"].long()]
        out = dict(kl=nll, weight=weight)
    out["loss"] = (weight * nll).sum()
    if case["grad"]:
        d = torch.exp(z - lse.unsqueeze(1))
        if op == "ce":
            d[row, t.clamp(min=0)] -= 1
        else:
            d[row.unsqueeze(1), ids] -= pt
        d *= weight.unsqueeze(1) / tau
        out["grad_hidden"], out["grad_weight"] = d @ w, d.T @ x
    return out
