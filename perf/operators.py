"""The operators next to the output head that are measured: log probabilities of given tokens
(with entropy, logsumexp and top alternatives) from logits and from hidden states, their
gradients, and the global gradient norm with clipping.

``own`` false computes them from elementary torch operations in float32; ``own`` true calls
the package.  ``exact`` gives the same outputs from the definitions in float64.

Definitions, for a row of logits z and its token t (negative: no token):
  lse = log sum exp z,  logp = z[t] - lse (0 without a token),  p = exp(z - lse),
  entropy = -sum p log p,  top alternatives by falling z, equal ones by rising index;
  a row with no finite logit: lse = logp = -inf, entropy = 0, gradient 0;
  dz = p * (g_lse - g_logp - g_entropy * (log p + entropy)) + g_logp * [v = t];
  head: z = h W^T, dh = dz W, dW = dz^T h, gradients in the type of h and W;
  clipping: norm = sqrt(sum g^2) over all tensors, out = g * max_norm / norm where
  norm > max_norm, else g.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence's decoding step with its 20 best alternatives
        dict(name="logprobs_one_row", op="logits", n=1, v=128256, dtype="bf16", top=20, pad=0, masked=False, grad=False),
        # a decoding batch with constrained vocabularies (masked entries) and 5 alternatives
        dict(name="logprobs_batch", op="logits", n=48, v=201088, dtype="bf16", top=5, pad=0, masked=True, grad=False),
        # scoring of stored text: every position, its 8 best alternatives
        dict(name="logprobs_score", op="logits", n=4096, v=128256, dtype="bf16", top=8, pad=0, masked=False, grad=False),
        # float32 logits of an odd vocabulary inside padded rows, masked entries and an empty row
        dict(name="logprobs_f32_odd", op="logits", n=1037, v=32003, dtype="f32", top=0, pad=61, masked=True, grad=False),
        # training on given tokens with an entropy term: forward and gradient of the logits
        dict(name="logprobs_train", op="logits", n=4095, v=128256, dtype="bf16", top=0, pad=0, masked=False, grad=True),
        # one sequence's log probability straight from its hidden state
        dict(name="head_one_row", op="head", n=1, d=4096, v=128256, dtype="bf16", grad=False),
        # a decoding batch from hidden states
        dict(name="head_batch", op="head", n=48, d=2880, v=201088, dtype="bf16", grad=False),
        # scoring of stored text without logits in memory
        dict(name="head_score", op="head", n=4096, d=2048, v=128256, dtype="bf16", grad=False),
        # a training step of the head: log probabilities, entropy, dh and dW
        dict(name="head_train", op="head", n=4096, d=2880, v=201088, dtype="bf16", grad=True),
        # the float32 head of the small workload, forward and backward
        dict(name="head_train_f32", op="head", n=512, d=256, v=8192, dtype="f32", grad=True),
        # the gradients of a small model: many tensors of mixed sizes and types
        dict(name="clip_many", op="clip", tensors=48, elements=3000017, dtype="mixed", clip=True),
        # the output head's dW with the gradients beside it
        dict(name="clip_head", op="clip", tensors=6, elements=420000003, dtype="f32", clip=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["logits", "logits", "logits", "head", "head", "clip"])
    if op == "logits":
        v = _log_int(rng, 1000, 262144)
        n = _log_int(rng, 1, max(1, min(8192, 525000000 // v)))
        grad = rng.random() < 0.4
        return dict(op=op, n=n, v=v, dtype=rng.choice(["bf16", "bf16", "f32"]), top=0 if grad else rng.choice([0, 1, 5, 20, 50]),
                    pad=rng.choice([0, 0, 3, 64]), masked=rng.random() < 0.5, grad=grad)
    if op == "head":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = 8 * _log_int(rng, 8, 512)
        v = _log_int(rng, 1000, 201088)
        most = 2.3e12 if dtype == "bf16" else 1.5e11
        n = _log_int(rng, 1, max(1, min(4096, int(most / (d * v)))))
        return dict(op=op, n=n, d=d, v=v, dtype=dtype, grad=rng.random() < 0.5)
    return dict(op=op, tensors=rng.randint(1, 60), elements=_log_int(rng, 1000, 400000000), dtype=rng.choice(["f32", "bf16", "mixed"]), clip=rng.random() < 0.7)


def _sizes(case):
    """The tensors' lengths: one large, the others of all sizes down to a few elements."""
    rng = random.Random(case["elements"] * 131 + case["tensors"])
    shares = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    shares[0] += sum(shares)
    left = case["elements"]
    whole = sum(shares)
    sizes = [max(1, int(left * s / whole)) for s in shares]
    return sizes


def _types(case):
    kinds = ["f32", "bf16"] if case["dtype"] == "mixed" else [case["dtype"]]
    return [DTYPES[kinds[i % len(kinds)]] for i in range(case["tensors"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    if case["op"] == "clip":
        grads = [(0.01 * randn(k)).to(t) for k, t in zip(_sizes(case), _types(case))]
        expected = 0.01 * math.sqrt(sum(g.numel() for g in grads))
        return dict(case=case, grads=grads, outs=[torch.empty_like(g) for g in grads], max_norm=expected * (0.3 if case["clip"] else 3.0))
    n, v, dtype = case["n"], case["v"], DTYPES[case["dtype"]]
    # frequent tokens are drawn more often, as in text
    tokens = (torch.rand(n, generator=gen, device="cuda", dtype=torch.float64).pow(3) * v).long().clamp_(0, v - 1)
    skip = torch.rand(n, generator=gen, device="cuda") < 0.05  # padded positions have no token
    if n > 1:
        tokens = tokens.masked_fill(skip, -1)
    state = dict(case=case, tokens=tokens)
    if case["grad"]:
        state["g_logp"] = randn(n) / n
        state["g_entropy"] = 0.1 * randn(n) / n
    if case["op"] == "head":
        d = case["d"]
        state["h"] = randn(n, d).to(dtype)
        state["w"] = randn(v, d).mul_(2.0 / math.sqrt(d)).to(dtype)
        return state
    wide = torch.empty((n, v + case["pad"]), device="cuda", dtype=dtype)
    logits = wide[:, :v]
    for at in range(0, n, 1024):
        part = randn(min(1024, n - at), v).mul_(2.5)
        # the given token is likely in most rows, as in text that a model has learnt
        own_tokens = tokens[at:at + 1024].clamp(min=0)
        part.scatter_add_(1, own_tokens[:, None], 12.0 * torch.rand((part.shape[0], 1), generator=gen, device="cuda"))
        if case["masked"]:
            part.masked_fill_(torch.rand(part.shape, generator=gen, device="cuda") < 0.3, -math.inf)
        logits[at:at + 1024] = part
    if case["masked"] and n > 2:
        logits[n // 2] = -math.inf  # a row whose mask leaves nothing
    state["logits"] = logits
    return state


def _plain_rows(z, tokens):
    """(shifted logits, exp of them, their sum, logp, entropy, lse, empty rows), z in float32."""
    top = z.max(1).values
    empty = top == -math.inf
    shifted = z - top.masked_fill(empty, 0.0)[:, None]
    e = shifted.exp()
    total = e.sum(1)
    log_total = total.log()
    moment = (e * shifted.masked_fill(e == 0, 0.0)).sum(1)
    entropy = torch.where(empty, 0.0, log_total - moment / total)
    own_z = shifted.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    logp = torch.where(empty, -math.inf, own_z - log_total).masked_fill(tokens < 0, 0.0)
    return shifted, e, total, logp, entropy, top + log_total.masked_fill(empty, 0.0), empty


def _plain_grad(shifted, e, total, entropy, empty, tokens, g_logp, g_entropy):
    """The gradient of the logits, in float32."""
    g_tok = g_logp.masked_fill(tokens < 0, 0.0)
    p = e / total[:, None]
    log_p = (shifted - total.log()[:, None]).masked_fill(p == 0, 0.0)
    dz = p * (-g_tok[:, None] - g_entropy[:, None] * (log_p + entropy[:, None]))
    dz.scatter_add_(1, tokens.clamp(min=0)[:, None], g_tok[:, None])
    return dz.masked_fill_(empty[:, None], 0.0)


def _plain_top(logits, logp_of, top):
    """The largest logits' places and log probabilities, equal ones by rising index: one
    whole number orders both, so no two are equal."""
    z = logits.float() + 0.0  # -0 is 0
    bits = z.view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = (order << 32) | (0x7FFFFFFF - torch.arange(z.shape[1], device=z.device))
    best = key.topk(top, dim=1).values
    at = 0x7FFFFFFF - (best & 0x7FFFFFFF)
    return at.int(), logp_of.gather(1, at)


def _plain(state):
    case = state["case"]
    if case["op"] == "clip":
        squares = torch.stack([g.double().square().sum() for g in state["grads"]])
        norm = squares.sum().sqrt()
        scale = torch.where(norm > state["max_norm"], state["max_norm"] / norm, 1.0).float()
        return [norm.float().reshape(1)] + [(g.float() * scale).to(g.dtype) for g in state["grads"]]
    tokens = state["tokens"]
    if case["op"] == "head":
        h, w = state["h"].float(), state["w"].float()
        shifted, e, total, logp, entropy, lse, empty = _plain_rows(h @ w.t(), tokens)
        if not case["grad"]:
            return [logp, entropy, lse]
        dz = _plain_grad(shifted, e, total, entropy, empty, tokens, state["g_logp"], state["g_entropy"])
        return [logp, entropy, lse, (dz @ w).to(state["h"].dtype), (dz.t() @ h).to(state["w"].dtype)]
    shifted, e, total, logp, entropy, lse, empty = _plain_rows(state["logits"].float(), tokens)
    if case["grad"]:
        dz = _plain_grad(shifted, e, total, entropy, empty, tokens, state["g_logp"], state["g_entropy"])
        return [logp, entropy, lse, dz.to(state["logits"].dtype)]
    if not case["top"]:
        return [logp, entropy, lse]
    every = torch.where(empty[:, None], -math.inf, shifted - total.log()[:, None])
    return [logp, entropy, lse, *_plain_top(state["logits"], every, case["top"])]


def run(state):
    if not own:
        return _plain(state)
    import output_head_kl_amd as kd
    case = state["case"]
    if case["op"] == "clip":
        norm = kd.clip_grads(state["grads"], state["max_norm"], out=state["outs"])
        return [norm] + state["outs"]
    if not case["grad"]:
        if case["op"] == "head":
            return list(kd.head_logprobs(state["h"], state["w"], state["tokens"]))
        return list(kd.token_logprobs(state["logits"], state["tokens"], top=case["top"]))
    upstream = (state["g_logp"], state["g_entropy"])
    if case["op"] == "head":
        h, w = state["h"].detach().requires_grad_(), state["w"].detach().requires_grad_()
        logp, entropy, lse = kd.head_logprobs(h, w, state["tokens"])
        dh, dw = torch.autograd.grad((logp, entropy), (h, w), upstream)
        return [logp, entropy, lse, dh, dw]
    logits = state["logits"].detach().requires_grad_()
    logp, entropy, lse = kd.token_logprobs(logits, state["tokens"])
    dz, = torch.autograd.grad((logp, entropy), logits, upstream)
    return [logp, entropy, lse, dz]


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "clip":
        # every gradient read once and written once; its square and its product with the scale
        return dict(bytes=2 * sum(k * t.itemsize for k, t in zip(_sizes(case), _types(case))) + 4, flops=3 * sum(_sizes(case)))
    n, v, es = case["n"], case["v"], size[case["dtype"]]
    if case["op"] == "logits":
        # logits read once (and their gradient written once); tokens, three numbers a row,
        # the alternatives; an exponential, three sums and a shift for each logit
        return dict(bytes=n * v * es * (2 if case["grad"] else 1) + n * (20 + 8 * case["top"] + (8 if case["grad"] else 0)), flops=n * v * (10 if case["grad"] else 5))
    d = case["d"]
    # h and W read once (dh and dW written once); the product h W^T, and with gradients dz W
    # and dz^T h
    return dict(bytes=(n + v) * d * es * (2 if case["grad"] else 1) + n * (20 + (8 if case["grad"] else 0)), flops=2 * n * v * d * (3 if case["grad"] else 1))


def _exact_rows(z, tokens):
    """Definitions in float64: (log p of every entry, logp, entropy, lse)."""
    lse = torch.logsumexp(z, 1)
    none = torch.isinf(lse) & (lse < 0)
    log_p = z - torch.where(none, torch.zeros_like(lse), lse)[:, None]
    p = torch.exp(log_p)
    entropy = -torch.special.xlogy(p, p).sum(1)
    rows = torch.arange(z.shape[0], device=z.device)
    logp = torch.where(tokens < 0, torch.zeros_like(lse), log_p[rows, tokens.clamp(min=0)])
    return log_p, p, logp, entropy, lse


def _exact_grad(log_p, p, tokens, entropy, g_logp, g_entropy):
    g = torch.where(tokens < 0, torch.zeros_like(g_logp), g_logp).double()
    hot = torch.zeros_like(p)
    hot[torch.arange(p.shape[0], device=p.device), tokens.clamp(min=0)] = 1.0
    dz = g[:, None] * (hot - p)
    spread = torch.special.xlogy(p, p) + p * entropy[:, None]
    dz -= g_entropy.double()[:, None] * spread
    dz[p.sum(1) == 0] = 0.0
    return dz


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "clip":
        total = math.fsum(float(torch.dot(g.double(), g.double())) for g in state["grads"])
        norm = math.sqrt(total)
        factor = state["max_norm"] / norm if norm > state["max_norm"] else 1.0
        return [torch.tensor([norm], dtype=torch.float64)] + [g.double() * factor for g in state["grads"]]
    tokens, rows, parts = state["tokens"], 512, []
    w = state["w"].double() if case["op"] == "head" else None
    dw = torch.zeros_like(w) if case["grad"] and w is not None else None
    for at in range(0, case["n"], rows):
        here = slice(at, at + rows)
        h = state["h"][here].double() if w is not None else None
        z = state["logits"][here].double() if w is None else h @ w.t()
        log_p, p, logp, entropy, lse = _exact_rows(z, tokens[here])
        got = [logp, entropy, lse]
        if case["grad"]:
            dz = _exact_grad(log_p, p, tokens[here], entropy, state["g_logp"][here], state["g_entropy"][here])
            if w is not None:
                dw += dz.t() @ h
                dz = dz @ w
            got.append(dz)
        elif case["op"] == "logits" and case["top"]:
            got.append(torch.topk(log_p, case["top"], dim=1).values)
        parts.append(got)
    out = [torch.cat(x) for x in zip(*parts)]
    if dw is not None:
        out.append(dw)
    if case["op"] == "logits" and case["top"]:
        out.insert(3, None)
    return out
