"""The cases on which the norm, the layers with an epilogue and the sampler are measured.

Six operators, written for T tokens:

  norm         h = X + residual, y = h / sqrt(mean(h^2) + eps) * weight, and y as int8 with a scale per token
  linear       Z = X W^T + bias, Y = act(Z) + residual, X and W in 16 bits; Z too, where a gradient will need it
  linear_grad  for d/dY: G = dY act'(Z), dX = G W, dW = G^T X, dbias = sum over tokens of G
  i8gemm       act((sum_k A[t, k] B[n, k]) a_scale[t] b_scale[n] + bias[n]) + residual[t, n], A and B int8
  i8linear     the same from 16- or 32-bit activations, quantised row by row first
  sample       a token per row of logits: temperature, top-k, top-p, min-p, then the inverse of the distribution function in the
               order of indexes at a given u in [0, 1); and the logarithm of that token's probability

`own` selects between the plain form (elementary torch operations in 32 bits, in 64 where a value next to a border decides, rounded
once at the end) and the calls of this package. exact() gives the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def listed():
    return [
        # -- the norm in front of a quantised layer
        # one token of a decoding step, added to the residual stream
        {"name": "norm token", "op": "norm", "t": 1, "k": 4096, "type": "fp16", "residual": True},
        # a long prompt
        {"name": "norm prompt", "op": "norm", "t": 4096, "k": 4096, "type": "bf16", "residual": True},
        # -- 16-bit layers
        # one token through a square layer with an activation: the step of decoding one sequence
        {"name": "linear token", "op": "linear", "t": 1, "n": 4096, "k": 4096, "type": "bf16", "act": "silu", "bias": True,
         "residual": False, "pre": False},
        # a batch of ragged sequences in training: odd sizes, Z kept for the gradient
        {"name": "linear ragged", "op": "linear", "t": 997, "n": 2051, "k": 1001, "type": "fp16", "act": "gelu", "bias": True,
         "residual": False, "pre": True},
        # a long prompt through a widening layer
        {"name": "linear prompt", "op": "linear", "t": 8192, "n": 14336, "k": 4096, "type": "bf16", "act": "gelu_tanh", "bias": True,
         "residual": False, "pre": False},
        # -- their gradients
        # a training step of a small model
        {"name": "linear_grad small", "op": "linear_grad", "t": 509, "n": 2051, "k": 768, "type": "fp16", "act": "gelu"},
        # a training step of a large one
        {"name": "linear_grad large", "op": "linear_grad", "t": 8192, "n": 14336, "k": 4096, "type": "bf16", "act": "silu"},
        # -- quantised layers
        # a decoding batch through a narrowing layer, added to the residual stream
        {"name": "i8linear batch", "op": "i8linear", "t": 37, "n": 4096, "k": 11008, "type": "bf16", "act": "none", "bias": False,
         "residual": True},
        # a prompt whose norm is quantised already, through a widening layer
        {"name": "i8gemm prompt", "op": "i8gemm", "t": 4096, "n": 14336, "k": 4096, "type": "bf16", "act": "silu", "bias": True,
         "residual": False},
        # -- the next token
        # one sequence: the few most probable tokens
        {"name": "sample one", "op": "sample", "t": 1, "v": 32000, "type": "fp32", "top_k": True, "top_p": True, "min_p": False},
        # a batch of odd size over an odd vocabulary, nucleus alone
        {"name": "sample nucleus", "op": "sample", "t": 37, "v": 50001, "type": "fp16", "top_k": False, "top_p": True, "min_p": False},
        # a large serving batch over a large vocabulary: every request with settings of its own
        {"name": "sample requests", "op": "sample", "t": 256, "v": 128000, "type": "bf16", "top_k": True, "top_p": True, "min_p": True},
    ]


def draw(rng):
    def size(lo, hi, even=1):
        x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, x // even * even)

    op = rng.choice(["norm", "linear", "linear_grad", "i8gemm", "i8linear", "sample"])
    if op == "norm":
        return {"op": op, "t": size(1, 4096), "k": size(64, 8192, rng.choice([128, 8, 1])),
                "type": rng.choice(["bf16", "fp16", "fp32"]), "residual": rng.random() < 0.7}
    if op == "sample":
        return {"op": op, "t": size(1, 256), "v": size(1000, 128000, rng.choice([128, 1])),
                "type": rng.choice(["bf16", "fp16", "fp32"]), "top_k": rng.random() < 0.5, "top_p": rng.random() < 0.5,
                "min_p": rng.random() < 0.3}
    case = {"op": op, "t": size(1, 8192), "n": size(16, 14336, rng.choice([128, 16, 1])),
            "k": size(128, 4096, rng.choice([128, 64, 16, 1])), "type": rng.choice(["bf16", "fp16"]),
            "act": rng.choice(ACTIVATIONS)}
    if op != "linear_grad":
        case["bias"], case["residual"] = rng.random() < 0.5, rng.random() < 0.5
    if op == "linear":
        case["pre"] = rng.random() < 0.3
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    op, t, out = case["op"], case["t"], DTYPES[case["type"]]
    state = {"case": case}
    if op == "sample":
        v = case["v"]
        # logits with a standard deviation of 2, some entries that stand out, and a few that are banned
        z = normal(t, v) * 2 + 6 * (uniform(t, v) < 2e-4)
        z[uniform(t, v) < 0.01] = -math.inf
        state["logits"] = z.to(out)
        state["u"] = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
        if t == 1:  # one request's settings are plain numbers
            state["settings"] = {"temperature": 0.8, "top_k": 50 if case["top_k"] else 0, "top_p": 0.9 if case["top_p"] else 1.0,
                                 "min_p": 0.02 if case["min_p"] else 0.0}
            return state
        # a batch has those of each request, in vectors; one in ten asks for the most probable token, and half leave a filter off
        temperature = 0.5 + uniform(t)
        temperature[uniform(t) < 0.1] = 0.0
        top_k = torch.randint(10, 200, (t,), generator=g, device="cuda", dtype=torch.int32)
        top_k[uniform(t) < 0.5] = 0
        top_p = 0.7 + 0.28 * uniform(t)
        top_p[uniform(t) < (0.5 if case["top_k"] else 0.0)] = 1.0
        min_p = 0.1 * uniform(t)
        min_p[uniform(t) < 0.5] = 0.0
        state["settings"] = {"temperature": temperature, "top_k": top_k if case["top_k"] else 0,
                             "top_p": top_p if case["top_p"] else 1.0, "min_p": min_p if case["min_p"] else 0.0}
        return state
    k = case["k"]
    # activations with a few outlying features, of tokens of different sizes
    x = normal(t, k) * torch.exp(0.3 * normal(t, 1)) * (1 + 8 * (uniform(k) < 0.01))
    if op == "norm":
        state["X"] = x.to(out)
        state["weight"] = 1 + 0.2 * normal(k)
        state["residual"] = (3 * normal(t, k)).to(out) if case["residual"] else None
        return state
    n = case["n"]
    w = normal(n, k) / math.sqrt(k) * torch.exp(0.3 * normal(n, 1))
    if op == "linear_grad":
        state["X"], state["W"] = x.to(out), w.to(out)
        state["Z"] = (1.5 * normal(t, n)).to(out) if case["act"] != "none" else None
        state["dY"] = (0.05 * normal(t, n)).to(out)
        return state
    state["bias"] = normal(n) if case["bias"] else None
    state["residual"] = (2 * normal(t, n)).to(out) if case["residual"] else None
    if op == "linear":
        state["X"], state["W"] = x.to(out), w.to(out)
        return state
    state["B"], state["b_scale"] = quantised(w)
    if op == "i8linear":
        state["X"] = x.to(out)
    else:
        state["A"], state["a_scale"] = quantised(x)
    return state


def quantised(x):
    """Rows as int8 with a scale each, in 32 bits as quantize_rows documents it: s = max|x| * (1 / 127), q = rint(x * ((1 / max|x|) * 127))."""
    x = x.float()
    top = x.abs().amax(1)
    up = torch.where(top > 0, (1.0 / top) * 127.0, torch.zeros_like(top))
    return torch.round(x * up[:, None]).to(torch.int8), top * (1.0 / 127.0)


# ---- plain forms -------------------------------------------------------------
def run(state):
    if own:
        return run_own(state)
    case = state["case"]
    op, out = case["op"], DTYPES[case["type"]]
    if op == "norm":
        h = state["X"].float()
        if state["residual"] is not None:
            h = h + state["residual"].float()
        # in 64 bits: a value next to the border of two codes decides
        h64 = h.double()
        r = 1.0 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + EPS)
        q, scale = quantised((h64 * r * state["weight"].double()).float())
        res = {"y": q * scale[:, None], "scale": scale}
        if state["residual"] is not None:
            res["sum"] = h.to(out)
        return res
    if op == "sample":
        return sampled(state["logits"], state["u"], **state["settings"])
    if op == "linear":
        z = state["X"].float() @ state["W"].float().t()
        if state["bias"] is not None:
            z = z + state["bias"]
        y = finished(z, case["act"], state["residual"]).to(out)
        return {"y": y, "z": z.to(out)} if case["pre"] else {"y": y}
    if op == "linear_grad":
        grad = state["dY"].float()
        if state["Z"] is not None:
            grad = grad * slope(state["Z"].float(), case["act"])
        return {"dx": (grad @ state["W"].float()).to(out), "dw": (grad.t() @ state["X"].float()).to(out), "dbias": grad.sum(0)}
    A, a_scale = quantised(state["X"]) if op == "i8linear" else (state["A"], state["a_scale"])
    z = (A.float() @ state["B"].float().t()) * a_scale[:, None] * state["b_scale"]
    if state["bias"] is not None:
        z = z + state["bias"]
    return finished(z, case["act"], state["residual"]).to(out)


def finished(z, act, residual):
    if act == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif act == "gelu":
        z = 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        z = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    elif act == "silu":
        z = z / (1 + torch.exp(-z))
    return z if residual is None else z + residual.float()


def slope(z, act):
    """d act / dz."""
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        th = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def sampled(logits, u, temperature, top_k, top_p, min_p):
    t, v = logits.shape

    def column(x, dtype):
        return x.to(dtype)[:, None] if isinstance(x, torch.Tensor) else torch.full((t, 1), x, dtype=dtype, device=logits.device)

    temperature, top_p, min_p = (column(x, torch.float64) for x in (temperature, top_p, min_p))
    top_k = column(top_k, torch.int64)
    z, order = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    greedy = temperature == 0
    z = (z - z[:, :1]) / torch.where(greedy, torch.ones_like(temperature), temperature)
    w = torch.exp(z)
    rank = torch.arange(v, device=z.device)
    kept = (top_k <= 0) | (rank < top_k)
    kept &= ~greedy | (rank < 1)
    first = torch.where(kept, w, torch.zeros_like(w))
    before = torch.cumsum(first, 1) - first
    kept &= (top_p >= 1) | (before < top_p * first.sum(1, keepdim=True)) | (rank < 1)
    kept &= w >= min_p
    w = torch.where(kept, w, torch.zeros_like(w))
    # back in the order of the indexes
    w = torch.zeros_like(w).scatter_(1, order, w)
    running = torch.cumsum(w, 1)
    token = (running <= u[:, None] * running[:, -1:]).sum(1)
    return {"token": token, "logprob": torch.log(w.gather(1, token[:, None])[:, 0] / running[:, -1]).float()}


# ---- the calls of this package ---------------------------------------------------
def run_own(state):
    import rns_emulated_fp64_amd as oz

    case = state["case"]
    op = case["op"]
    if op == "norm":
        q, scale, total = oz.rmsnorm_quantize(state["X"], state["weight"], state["residual"], eps=EPS)
        res = {"y": q * scale[:, None], "scale": scale}
        if total is not None:
            res["sum"] = total
        return res
    if op == "sample":
        token, logprob = oz.sample(state["logits"], state["u"], **state["settings"])
        return {"token": token, "logprob": logprob}
    if op == "linear":
        y, z = oz.linear(state["X"], state["W"], bias=state["bias"], activation=case["act"], residual=state["residual"],
                         want_pre=case["pre"])
        return {"y": y, "z": z} if case["pre"] else {"y": y}
    if op == "linear_grad":
        dx, dw, dbias = oz.linear_grad(state["dY"], state["X"], state["W"], Z=state["Z"], activation=case["act"])
        return {"dx": dx, "dw": dw, "dbias": dbias}
    if op == "i8linear":
        return oz.i8linear(state["X"], state["B"], state["b_scale"], bias=state["bias"], activation=case["act"],
                           residual=state["residual"])
    return oz.i8gemm(state["A"], state["B"], state["a_scale"], state["b_scale"], bias=state["bias"],
                     out_dtype=DTYPES[case["type"]], activation=case["act"], residual=state["residual"])


# ---- work and definitions ----------------------------------------------------------
def work(case):
    op, t = case["op"], case["t"]
    size = 4 if case["type"] == "fp32" else 2
    if op == "norm":
        moved = 3 if case["residual"] else 1
        return {"bytes": t * case["k"] * (size * moved + 1) + 4 * case["k"] + 4 * t, "flops": 6 * t * case["k"]}
    if op == "sample":
        return {"bytes": size * t * case["v"] + 20 * t, "flops": 2 * t * case["v"]}
    n, k = case["n"], case["k"]
    if op == "linear_grad":
        read = size * ((t + n) * k + t * n * (1 if case["act"] == "none" else 2))
        return {"bytes": read + size * (t + n) * k + 4 * n, "flops": 4 * t * n * k}
    planes = 1 + (1 if case["residual"] else 0) + (1 if op == "linear" and case["pre"] else 0)
    outer = size * t * n * planes + (4 * n if case["bias"] else 0)
    if op == "linear":
        return {"bytes": size * (t + n) * k + outer, "flops": 2 * t * n * k}
    rows = size * t * k if op == "i8linear" else t * k + 4 * t
    return {"bytes": rows + n * k + 4 * n + outer, "flops": 2 * t * n * k}


def exact(case, seed):
    """The definitions in 64 bits. An int8 value is defined by the binary32 formula of the value that it codes, so it is taken as it is."""
    state = prepare(case, seed)
    op, f64 = case["op"], torch.float64

    def codes(x32):
        amax = torch.linalg.vector_norm(x32, ord=math.inf, dim=1, keepdim=True)
        up = torch.reciprocal(amax) * 127.0
        return (x32 * torch.where(amax == 0, amax, up)).round().to(f64), amax.to(f64) / 127

    def curve(z):
        return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
                "gelu": lambda: z * torch.special.ndtr(z),
                "gelu_tanh": lambda: z * torch.sigmoid(math.sqrt(8 / math.pi) * z * (1 + 0.044715 * z ** 2))}[case["act"]]()

    if op == "norm":
        h = state["X"].to(f64)
        if case["residual"]:
            h = (h + state["residual"].to(f64)).to(torch.float32).to(f64)  # the sum is a binary32 value
        rms = torch.linalg.vector_norm(h, dim=1, keepdim=True) / math.sqrt(case["k"])
        y = state["weight"].to(f64) * h * torch.rsqrt(rms ** 2 + EPS)
        q, scale = codes(y.to(torch.float32))
        res = {"y": q * scale, "scale": scale[:, 0]}
        if case["residual"]:
            res["sum"] = h
        return res
    if op == "sample":
        return drawn(state)
    if op == "linear_grad":
        grad = state["dY"].to(f64)
        if state["Z"] is not None:
            z = state["Z"].to(f64)
            if case["act"] == "relu":
                grad = grad.masked_fill(z <= 0, 0.0)
            elif case["act"] == "gelu":
                grad = grad * (torch.special.ndtr(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi))
            else:
                # x sigmoid(f(x)): sigmoid + x f' sigmoid (1 - sigmoid)
                c = math.sqrt(8 / math.pi)
                f, df = (z, 1.0) if case["act"] == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z ** 2))
                s = torch.sigmoid(f)
                grad = grad * (s + z * df * s * torch.sigmoid(-f))
        return {"dx": torch.mm(grad, state["W"].to(f64)), "dw": torch.mm(grad.t().contiguous(), state["X"].to(f64)),
                "dbias": torch.mv(grad.t().contiguous(), torch.ones(case["t"], dtype=f64, device=grad.device))}
    if op == "linear":
        z = torch.mm(state["X"].to(f64), state["W"].to(f64).t().contiguous())
    else:
        a, sa = codes(state["X"].to(torch.float32)) if op == "i8linear" else (state["A"].to(f64), state["a_scale"].to(f64)[:, None])
        z = torch.mm(a * sa, (state["B"].to(f64) * state["b_scale"].to(f64)[:, None]).t().contiguous())
    if state["bias"] is not None:
        z = z.add_(state["bias"].to(f64))
    y = curve(z)
    if state["residual"] is not None:
        y = y + state["residual"].to(f64)
    if op != "linear":
        return y
    return {"y": y, "z": z} if case["pre"] else {"y": y}


def drawn(state):
    """The sampler row by row: the kept entries alone, never the whole row sorted where a filter leaves few."""
    tokens, logs = [], []
    settings = {name: value.tolist() if isinstance(value, torch.Tensor) else [value] * state["case"]["t"]
                for name, value in state["settings"].items()}
    for i, row in enumerate(state["logits"]):
        x = row.to(torch.float64)
        temperature, k, p, m = (settings[name][i] for name in ("temperature", "top_k", "top_p", "min_p"))
        top = x.max()
        if temperature == 0:
            tokens.append(int((x == top).nonzero()[0, 0]))
            logs.append(0.0)
            continue
        w = torch.exp((x - top) / temperature)
        index = torch.arange(len(x), device=x.device)
        if 0 < k < len(x):
            border = torch.topk(x, k).values[-1]
            above, at = index[x > border], index[x == border]
            index = torch.cat([above, at[:k - len(above)]]).sort().values
        if p < 1:
            some = index[torch.argsort(-w[index], stable=True)]
            sums = torch.cumsum(w[some], 0)
            needed = int((sums < p * sums[-1]).sum()) + 1
            index = some[:needed].sort().values
        index = index[w[index] >= m]
        sums = torch.cumsum(w[index], 0)
        at = int(torch.searchsorted(sums, state["u"][i] * sums[-1], right=True))
        tokens.append(int(index[at]))
        logs.append(float(torch.log(w[index[at]] / sums[-1])))
    device = state["logits"].device
    return {"token": torch.tensor(tokens, device=device), "logprob": torch.tensor(logs, dtype=torch.float64, device=device)}
