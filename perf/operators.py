"""The cases on which the INT8 product with scales and the linear cross entropy are measured.

Five operators, written for T tokens:

  i8gemm     C[t, n] = (sum_k A[t, k] B[n, k]) * a_scale[t] * b_scale[n] (+ bias[n]), A and B int8
  i8linear   the same from 16-bit activations, quantised row by row first: s = max|x| / 127, q = rint(x * (127 / max|x|))
  xent       loss[t] = logsumexp_v(X[t] . W[v]) - X[t] . W[y[t]], 0 where y[t] is the ignored index
  xent_grad  the loss with its gradients for a given d/d loss[t]: dX and dW
  i8xent     xent for logits that are i8gemm's products

`own` selects between the plain form (elementary torch operations in 32 bits, rounded once at the end) and the calls of this
package. exact() gives the definitions in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # -- products of operands that are int8 already
        # the smallest call: a 64 x 64 x 64 product, all latency
        {"name": "i8gemm 64", "op": "i8gemm", "t": 64, "n": 64, "k": 64, "type": "bf16", "bias": False},
        # a batch of ragged prompts into an odd width, with a bias, binary32 output
        {"name": "i8gemm ragged", "op": "i8gemm", "t": 997, "n": 2051, "k": 1040, "type": "fp32", "bias": True},
        # a square layer over a full batch (the size of this repository's headline product)
        {"name": "i8gemm 4096", "op": "i8gemm", "t": 4096, "n": 4096, "k": 4096, "type": "bf16", "bias": False},
        # -- layers that quantise their own input
        # one token through a square layer: the step of decoding one sequence
        {"name": "i8linear token", "op": "i8linear", "t": 1, "n": 4096, "k": 4096, "type": "bf16", "bias": False},
        # a decoding batch of odd size through a widening layer with a bias
        {"name": "i8linear batch", "op": "i8linear", "t": 37, "n": 11008, "k": 4096, "type": "fp16", "bias": True},
        # a long prefill through a widening layer
        {"name": "i8linear prefill", "op": "i8linear", "t": 8192, "n": 14336, "k": 4096, "type": "bf16", "bias": False},
        # -- the loss of an output layer
        # the log-likelihood of one token
        {"name": "xent token", "op": "xent", "t": 1, "v": 32000, "d": 4096, "type": "bf16"},
        # the log-likelihood of a long text under a large vocabulary
        {"name": "xent text", "op": "xent", "t": 4096, "v": 128000, "d": 4096, "type": "bf16"},
        # a training step of a small model: an odd vocabulary, fp16
        {"name": "xent_grad small", "op": "xent_grad", "t": 509, "v": 32003, "d": 768, "type": "fp16"},
        # a training step of a large one
        {"name": "xent_grad large", "op": "xent_grad", "t": 8192, "v": 128000, "d": 4096, "type": "bf16"},
        # -- the loss of a quantised output layer
        # a few positions scored at once (the candidates of a search)
        {"name": "i8xent few", "op": "i8xent", "t": 12, "v": 50001, "d": 2048, "type": "fp32"},
        # a text scored for the quality of the quantised model
        {"name": "i8xent text", "op": "i8xent", "t": 4096, "v": 65537, "d": 4096, "type": "fp32"},
    ]


def draw(rng):
    def size(lo, hi, even):
        x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, x // even * even)

    op = rng.choice(["i8gemm", "i8linear", "xent", "xent_grad", "i8xent"])
    inner = rng.choice([128, 64, 16, 1])  # what inner sizes are multiples of
    if op in ("i8gemm", "i8linear"):
        return {"op": op, "t": size(1, 8192, 1), "n": size(16, 14336, rng.choice([128, 16, 1])), "k": size(128, 4096, inner),
                "type": rng.choice(["bf16", "fp16", "fp32"]), "bias": rng.random() < 0.5}
    return {"op": op, "t": size(1, 4096, 1), "v": size(1000, 128000, rng.choice([128, 1])), "d": size(128, 4096, inner),
            "type": "fp32" if op == "i8xent" else rng.choice(["bf16", "fp16"])}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    op, t, out = case["op"], case["t"], DTYPES[case["type"]]
    if op in ("i8gemm", "i8linear"):
        n, k = case["n"], case["k"]
        # a layer's weights, quantised once per output channel; a few channels much larger than the others
        w = normal(n, k) / math.sqrt(k) * torch.exp(0.5 * normal(n, 1))
        B, b_scale = quantised(w)
        # activations with a few outlying features, as after a normalisation
        x = normal(t, k) * torch.exp(0.3 * normal(t, 1)) * (1 + 8 * (torch.rand(k, generator=g, device="cuda") < 0.01))
        state = {"case": case, "B": B, "b_scale": b_scale, "bias": normal(n) if case["bias"] else None}
        if op == "i8linear":
            state["X"] = x.to(out)
        else:
            state["A"], state["a_scale"] = quantised(x)
        return state
    v, d = case["v"], case["d"]
    # logits with a standard deviation of 1.5 and, for most tokens, a target that stands out by up to 12
    w = normal(v, d) * (1.5 / math.sqrt(d))
    y = torch.randint(v, (t,), generator=g, device="cuda")
    x = normal(t, d) + w[y] * torch.rand(t, 1, generator=g, device="cuda") * (12 / 1.5 ** 2)
    # about a tenth of the positions (padding, prompts) have no target; the first one always has
    skipped = torch.rand(t, generator=g, device="cuda") < 0.1
    skipped[0] = False
    state = {"case": case, "y": torch.where(skipped, torch.full_like(y, IGNORE), y)}
    if op == "i8xent":
        state["A"], state["a_scale"] = quantised(x)
        state["B"], state["b_scale"] = quantised(w)
    else:
        state["X"], state["W"] = x.to(out), w.to(out)
        # the gradient that reaches each token's loss: a mean over the tokens, weighted
        state["g"] = (0.5 + torch.rand(t, generator=g, device="cuda")) / t
    return state


def quantised(x):
    """Rows as int8 with a scale each, in 32 bits: s = max|x| / 127, q = rint(x * (127 / max|x|))."""
    x = x.float()
    top = x.abs().amax(1)
    up = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    return torch.round(x * up[:, None]).to(torch.int8), top / 127.0


def run(state):
    if own:
        return run_own(state)
    op, out = state["case"]["op"], DTYPES[state["case"]["type"]]
    if op == "i8gemm":
        return product(state["A"], state["a_scale"], state).to(out)
    if op == "i8linear":
        q, s = quantised(state["X"])
        return product(q, s, state).to(out)
    if op == "i8xent":
        z = (state["A"].float() @ state["B"].float().t()) * state["a_scale"][:, None] * state["b_scale"]
        loss, lse, _ = loss_of(z, state["y"])
        return {"loss": loss, "lse": lse}
    x, w = state["X"].float(), state["W"].float()
    loss, lse, z = loss_of(x @ w.t(), state["y"])
    if op == "xent":
        return {"loss": loss, "lse": lse}
    p = torch.exp(z - lse[:, None])
    rows = torch.arange(len(lse), device=p.device)
    kept = state["y"] != IGNORE
    p[rows, torch.where(kept, state["y"], 0)] -= 1.0
    p *= torch.where(kept, state["g"], torch.zeros_like(state["g"]))[:, None]
    return {"loss": loss, "dx": (p @ w).to(out), "dw": (p.t() @ x).to(out)}


def product(q, s, state):
    c = (q.float() @ state["B"].float().t()) * s[:, None] * state["b_scale"]
    return c if state["bias"] is None else c + state["bias"]


def loss_of(z, y):
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    kept = y != IGNORE
    at = z.gather(1, torch.where(kept, y, torch.zeros_like(y))[:, None])[:, 0]
    return torch.where(kept, lse - at, torch.zeros_like(lse)), lse, z


def run_own(state):
    import rns_emulated_fp64_amd as oz

    op, out = state["case"]["op"], DTYPES[state["case"]["type"]]
    if op == "i8gemm":
        return oz.i8gemm(state["A"], state["B"], state["a_scale"], state["b_scale"], bias=state["bias"], out_dtype=out)
    if op == "i8linear":
        return oz.i8linear(state["X"], state["B"], state["b_scale"], bias=state["bias"])
    if op == "i8xent":
        loss, lse = oz.i8xent(state["A"], state["B"], state["a_scale"], state["b_scale"], state["y"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    loss, lse = oz.xent(state["X"], state["W"], state["y"], ignore_index=IGNORE)
    if op == "xent":
        return {"loss": loss, "lse": lse}
    dx, dw = oz.xent_grad(state["X"], state["W"], state["y"], lse, state["g"], ignore_index=IGNORE)
    return {"loss": loss, "dx": dx, "dw": dw}


def work(case):
    op, t = case["op"], case["t"]
    size = 4 if case["type"] == "fp32" else 2
    if op in ("i8gemm", "i8linear"):
        n, k = case["n"], case["k"]
        read = n * k + 4 * n + (4 * n if case["bias"] else 0) + (t * k + 4 * t if op == "i8gemm" else size * t * k)
        return {"bytes": read + size * t * n, "flops": 2 * t * n * k}
    v, d = case["v"], case["d"]
    if op == "i8xent":
        return {"bytes": (t + v) * (d + 4) + 8 * t + 8 * t, "flops": 2 * t * v * d}
    read = size * (t + v) * d + 8 * t
    if op == "xent":
        return {"bytes": read + 8 * t, "flops": 2 * t * v * d}
    # the logits once, and a product for each gradient
    return {"bytes": read + 4 * t + 4 * t + size * (t + v) * d, "flops": 6 * t * v * d}


def exact(case, seed):
    """The definitions in 64 bits. An activation's int8 value is defined by its binary32 formula, so it is taken as it is."""
    state = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op in ("i8gemm", "i8linear"):
        if op == "i8linear":
            x32 = state["X"].to(torch.float32)
            amax = torch.linalg.vector_norm(x32, ord=math.inf, dim=1, keepdim=True)
            a = (x32 * torch.where(amax == 0, amax, 127.0 / amax)).round().to(f64)
            sa = (amax / 127.0).to(f64)
        else:
            a, sa = state["A"].to(f64), state["a_scale"].to(f64).unsqueeze(1)
        b = state["B"].to(f64) * state["b_scale"].to(f64).unsqueeze(1)
        c = torch.mm(a * sa, b.t().contiguous())
        return c if state["bias"] is None else c + state["bias"].to(f64)
    if op == "i8xent":
        x = state["A"].to(f64) * state["a_scale"].to(f64).unsqueeze(1)
        w = state["B"].to(f64) * state["b_scale"].to(f64).unsqueeze(1)
    else:
        x, w = state["X"].to(f64), state["W"].to(f64)
    y = state["y"]
    has = (y != IGNORE).to(f64)
    at = y.clamp(min=0)
    logits = torch.mm(x, w.t().contiguous())
    lse = torch.logsumexp(logits, 1)
    loss = (lse - (x * w[at]).sum(1)) * has
    if op != "xent_grad":
        return {"loss": loss, "lse": lse}
    weight = state["g"].to(f64) * has
    prob = logits.sub_(lse.unsqueeze(1)).exp_().mul_(weight.unsqueeze(1))
    # softmax part as products, the targets' part as a subtraction of rows
    dx = torch.mm(prob, w) - weight.unsqueeze(1) * w[at]
    dw = torch.mm(prob.t().contiguous(), x)
    dw.index_add_(0, at, x * weight.unsqueeze(1), alpha=-1.0)
    return {"loss": loss, "dx": dx, "dw": dw}
