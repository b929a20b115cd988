"""Cases of a training step's matrix products: the gated feed-forward block, token log probabilities from the hidden
state without logits, and the orthogonalised update, each with the gradients it has.

``run`` computes an operator from elementary torch operations in 32 bits, or,
with ``own`` set, through the package's plans; ``exact`` says in 64 bits what
either should give.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


def listed():
    return [
        # one decoding step of a small batch: three matrices are read for eight rows
        {"name": "ffn_decode", "op": "ffn", "n": 8, "d": 4096, "f": 11008, "t": "bf16", "act": "silu"},
        # a prompt, or the forward pass of a validation batch
        {"name": "ffn_prompt", "op": "ffn", "n": 2048, "d": 4096, "f": 11008, "t": "bf16", "act": "silu"},
        # forward and backward pass of a training batch
        {"name": "ffn_train", "op": "ffn_grad", "n": 8192, "d": 4096, "f": 11008, "t": "bf16", "act": "silu"},
        # the same in fp32 for a small model whose sizes fill no vector and no tile
        {"name": "ffn_train_odd", "op": "ffn_grad", "n": 1000, "d": 1023, "f": 2731, "t": "f32", "act": "gelu_tanh"},
        # scoring one decoding step's tokens: the output matrix is read for eight rows
        {"name": "head_decode", "op": "head", "n": 8, "v": 131072, "d": 4096, "t": "bf16"},
        # log probabilities of a prompt's tokens (perplexity, a reference policy), an odd vocabulary
        {"name": "head_score", "op": "head", "n": 2048, "v": 100003, "d": 2048, "t": "bf16"},
        # loss of a training batch with its gradients
        {"name": "head_train", "op": "head_grad", "n": 4096, "v": 131072, "d": 4096, "t": "bf16"},
        # loss and gradients in fp16, ragged sizes
        {"name": "head_train_f16", "op": "head_grad", "n": 1531, "v": 50257, "d": 1000, "t": "f16"},
        # updates of a small model's layers, a stack of equal ones: latency of short launches
        {"name": "ortho_small", "op": "ortho", "b": 4, "n": 256, "m": 1024, "t": "f32"},
        # a square weight of a middling model in fp32, odd sizes
        {"name": "ortho_odd", "op": "ortho", "b": 1, "n": 1777, "m": 1301, "t": "f32"},
        # a block's four square weights
        {"name": "ortho_square", "op": "ortho", "b": 4, "n": 2048, "m": 2048, "t": "bf16"},
        # a feed-forward weight, taller than wide
        {"name": "ortho_tall", "op": "ortho", "b": 1, "n": 11008, "m": 4096, "t": "bf16"},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi], a multiple of 64 about half the time."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 128 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["ffn", "ffn_grad", "head", "head_grad", "ortho"])
    t = rng.choice(["bf16", "bf16", "f32", "f16"])
    if op.startswith("ffn"):
        d = _size(rng, 16, 8192)
        f = _size(rng, 16, min(28672, (1 << 27) // d))
        n = _size(rng, 1, min(8192, int(3e11 / d / f)))
        return {"op": op, "n": n, "d": d, "f": f, "t": t, "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])}
    if op.startswith("head"):
        d = _size(rng, 16, 8192)
        v = _size(rng, 64, min(262144, (1 << 29) // d))
        n = _size(rng, 1, min(4096, (1 << 29) // v, max(1, int(2e12 / d / v))))
        return {"op": op, "n": n, "v": v, "d": d, "t": t}
    n, m = _size(rng, 1, 4096), _size(rng, 1, 8192)
    if rng.random() < 0.5:
        n, m = m, n
    return {"op": op, "b": rng.choice([1, 1, 2, 5]) if n * m <= 1 << 22 else 1, "n": n, "m": m, "t": t}


def work(case):
    """Bytes: every input once, every output once.  Flops: the products' additions and multiplications, of a symmetric
    product one half; a gradient needs its forward pass's products once."""
    op, s = case["op"], SIZE[case["t"]]
    if op in ("ffn", "ffn_grad"):
        n, d, f = case["n"], case["d"], case["f"]
        one = {"bytes": (2 * n * d + 3 * d * f) * s, "flops": 6 * n * d * f}
        return one if op == "ffn" else {"bytes": (4 * n * d + 6 * d * f) * s, "flops": 18 * n * d * f}
    if op in ("head", "head_grad"):
        n, v, d = case["n"], case["v"], case["d"]
        if op == "head":
            return {"bytes": (n * d + v * d) * s + 20 * n, "flops": 2 * n * v * d}
        return {"bytes": 2 * (n * d + v * d) * s + 24 * n, "flops": 6 * n * v * d}
    b, n, m = case["b"], min(case["n"], case["m"]), max(case["n"], case["m"])
    return {"bytes": 2 * b * n * m * s, "flops": b * STEPS * (3 * n * n * m + n * n * n)}


def _tokens(n, v, g):
    """Token ids with the frequencies of text (the k-th most frequent about 1/k), spread over the table; a few are padding."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1)
    tok = (rank * 48271 + 11) % v
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.01, torch.full_like(tok, -1), tok)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op, t = case["op"], TYPES[case["t"]]
    s = {"op": op}
    if op in ("ffn", "ffn_grad"):
        n, d, f = case["n"], case["d"], case["f"]
        s["act"] = case["act"]
        s["x"] = (rand(n, d) * torch.exp(rand(d) * 0.3)).to(t)  # a norm's output: channels of unlike spread
        s["w_gate"], s["w_up"] = ((rand(f, d) / math.sqrt(d)).to(t) for _ in range(2))
        s["w_down"] = (rand(d, f) / math.sqrt(f)).to(t)
        if op == "ffn_grad":
            s["dout"] = (rand(n, d) * 0.01).to(t)
        return s
    if op in ("head", "head_grad"):
        n, v, d = case["n"], case["v"], case["d"]
        s["tokens"] = _tokens(n, v, g)
        weight = rand(v, d) / math.sqrt(d)
        # the hidden state leans to its token, as a trained model's does: some targets likely, others far down
        s["hidden"] = (rand(n, d) + weight[s["tokens"].clamp(min=0)] * (rand(n, 1).abs() * 4)).to(t)
        s["weight"] = (weight * 1.5).to(t)
        if op == "head_grad":
            s["dlogprob"] = -(0.5 + torch.rand(n, generator=g, device="cuda")) / n  # a weighted mean's
        return s
    b, n, m = case["b"], case["n"], case["m"]
    k = min(16, n, m)
    # a momentum: a few strong directions over noise, rows and columns of unlike size
    strong = torch.bmm(rand(b, n, k), rand(b, k, m))
    s["update"] = ((strong + rand(b, n, m)) * torch.exp(rand(b, n, 1) * 0.3) * torch.exp(rand(b, 1, m) * 0.3) * 1e-3).to(t)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # The package's plans hold tensors' addresses, output buffers and workspaces; a program makes them once for
        # its buffers.  No input is read here.
        import collective_reduction_ring_amd as rsx
        op = s["op"]
        if op in ("ffn", "ffn_grad"):
            w = s["w_gate"], s["w_up"], s["w_down"]
            fwd = rsx.FeedForward(s["x"], *w, activation=s["act"], keep=op == "ffn_grad")
            s["plans"] = [fwd]
            if op == "ffn_grad":
                s["plans"].append(rsx.FeedForwardGrad(s["dout"], s["x"], *w, fwd.gate, fwd.up, activation=s["act"]))
        elif op in ("head", "head_grad"):
            fwd = rsx.LinearLogprobs(s["hidden"], s["weight"], s["tokens"])
            s["plans"] = [fwd]
            if op == "head_grad":
                s["plans"].append(rsx.LinearLogprobsGrad(s["hidden"], s["weight"], s["tokens"], fwd.lse, s["dlogprob"],
                                                         lse_rest=fwd.lse_rest))
        else:
            s["plans"] = [rsx.NewtonSchulz(s["update"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)]
    return s


def _run_own(s):
    op, plans = s["op"], s["plans"]
    for p in plans:
        p()
    if op == "ffn":
        return plans[0].out
    if op == "ffn_grad":
        d = plans[1]
        return {"y": plans[0].out, "dx": d.dx, "dw_gate": d.dw_gate, "dw_up": d.dw_up, "dw_down": d.dw_down}
    if op == "ortho":
        return plans[0].out
    out = {"logprob": plans[0].logprob, "entropy": plans[0].entropy, "lse": plans[0].lse}
    if op == "head_grad":
        out["dhidden"], out["dweight"] = plans[1].dhidden, plans[1].dweight
    return out


def _activation(name, x):
    """The activation and its derivative."""
    if name == "relu":
        on = (x > 0).float()
        return x * on, on
    if name == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + th), 0.5 * (1 + th) + 0.5 * x * (1 - th * th) * c * (1 + 3 * 0.044715 * x * x)


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op in ("ffn", "ffn_grad"):
        t = s["x"].dtype
        x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
        gate, up = x @ wg.t(), x @ wu.t()
        act, slope = _activation(s["act"], gate)
        y = ((act * up) @ wd.t()).to(t)
        if op == "ffn":
            return y
        dy = s["dout"].float()
        dh = dy @ wd
        dgate, dup = dh * up * slope, dh * act
        return {"y": y, "dx": (dgate @ wg + dup @ wu).to(t), "dw_gate": (dgate.t() @ x).to(t), "dw_up": (dup.t() @ x).to(t),
                "dw_down": (dy.t() @ (act * up)).to(t)}
    if op in ("head", "head_grad"):
        tok, t = s["tokens"], s["hidden"].dtype
        h, w = s["hidden"].float(), s["weight"].float()
        z = h @ w.t()
        c = z - z.amax(1, keepdim=True)
        p = torch.exp(c)
        total = p.sum(1, keepdim=True)
        p /= total
        logp = c - torch.log(total)
        at = tok.clamp(min=0)[:, None]
        mine = logp.gather(1, at)[:, 0]
        out = {"logprob": torch.where(tok >= 0, mine, 0.0), "entropy": -(p * logp).sum(1), "lse": z.gather(1, at)[:, 0] - mine}
        if op == "head_grad":
            g = torch.where(tok >= 0, s["dlogprob"], 0.0)[:, None]
            dz = (p * -g).scatter_add_(1, at, g)
            out["dhidden"], out["dweight"] = (dz @ w).to(t), (dz.t() @ h).to(t)
        return out
    x = s["update"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = torch.stack([m @ m.t() for m in x])
        poly = b * gram + c * torch.bmm(gram, gram)
        x = a * x + torch.bmm(poly, x.contiguous())
    return (x.transpose(1, 2) if tall else x).to(s["update"].dtype).contiguous()


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("ffn", "ffn_grad"):
        fn = torch.nn.functional
        act = {"silu": fn.silu, "relu": fn.relu, "gelu": fn.gelu, "gelu_tanh": lambda v: fn.gelu(v, approximate="tanh")}[s["act"]]
        x, wg, wu, wd = (s[k].double().requires_grad_(op == "ffn_grad") for k in ("x", "w_gate", "w_up", "w_down"))
        y = fn.linear(act(fn.linear(x, wg)) * fn.linear(x, wu), wd)
        if op == "ffn":
            return y
        grads = torch.autograd.grad(y, (x, wg, wu, wd), s["dout"].double())
        return dict(zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y.detach(), *grads)))
    if op in ("head", "head_grad"):
        n, v = case["n"], case["v"]
        h, w, tok = s["hidden"].double(), s["weight"].double(), s["tokens"]
        lp, ent, lse, dh, dw = [], [], [], [], torch.zeros_like(w) if op == "head_grad" else None
        step = max(1, (1 << 27) // v)
        for i in range(0, n, step):
            z = torch.nn.functional.linear(h[i:i + step], w)
            lse.append(torch.logsumexp(z, 1))
            p = torch.softmax(z, 1)
            ent.append(lse[-1] - (p * z).sum(1))
            real = tok[i:i + step] >= 0
            to = tok[i:i + step].clamp(min=0)
            rows = torch.arange(len(to), device="cuda")
            lp.append(torch.where(real, z[rows, to] - lse[-1], 0.0))
            if op == "head_grad":
                p[rows, to] -= 1
                p *= torch.where(real, -s["dlogprob"][i:i + step].double(), 0.0)[:, None]
                dh.append(p @ w)
                dw += p.t() @ h[i:i + step]
        out = {"logprob": torch.cat(lp), "entropy": torch.cat(ent), "lse": torch.cat(lse)}
        return dict(out, dhidden=torch.cat(dh), dweight=dw) if op == "head_grad" else out
    # the polynomials of the Gram matrix alone, and their product with the matrix at the end
    out = torch.empty(s["update"].shape, dtype=torch.float64, device="cuda")
    a, b, c = COEFFICIENTS
    for one, x in zip(out, s["update"].double()):
        x = x / (torch.linalg.vector_norm(x) + EPS)
        wide = x.shape[0] <= x.shape[1]
        gram = x @ x.t() if wide else x.t() @ x
        eye = torch.eye(len(gram), dtype=torch.float64, device="cuda")
        total = eye
        for _ in range(STEPS):
            q = a * eye + gram @ (b * eye + c * gram)
            total = q @ total
            gram = q @ gram @ q
        one.copy_(total @ x if wide else x @ total)
    return out
