"""Cases of the codebook-training operators: table lookup and its gradient,
the linear layer with its epilogue and its gradients, and clipping by the
global gradient norm.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` is one pass as a program calls it (the framework's operators
where ``own`` is true, elementary torch operations in 32 bits otherwise),
``exact`` the same outputs from the definitions in 64 bits and ``work`` the
bytes and operations that a pass cannot do without.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")

# Most elements of a drawn case's rows, table and gradients, and most
# multiply-adds: those of the largest listed ones.
MOST_ROWS = 16384 * 4096
MOST_TABLE = 32768 * 4096
MOST_LINEAR = 16384 * 4096 * 4096
MOST_LINEAR_GRAD = 8192 * 4096 * 4096
MOST_CLIP = 1 << 28


def listed():
    return [
        # Rows of the next tokens of 16 sequences being generated: latency.
        dict(name="lookup_step", op="lookup", N=16, K=32768, D=4096, type="bf16", index="int64",
             labels="zipf", scale=1.0),
        # Decoding the assigned points of the repository's headline codebook.
        dict(name="lookup_codebook", op="lookup", N=262144, K=4096, D=128, type="bf16",
             index="int32", labels="uniform", scale=1.0),
        # Wide fp32 rows with an odd count and width, scaled.
        dict(name="lookup_ragged_fp32", op="lookup", N=50021, K=5003, D=321, type="fp32",
             index="int64", labels="uniform", scale=17.916472867168917),
        # Gradient of the headline codebook from all its points.
        dict(name="lookup_grad_codebook", op="lookup_grad", N=262144, K=4096, D=128, type="bf16",
             index="int32", labels="uniform", scale=1.0),
        # Gradient of a token embedding: few frequent tokens, many rare, some
        # never seen, one in a hundred positions padding (no token).
        dict(name="lookup_grad_tokens", op="lookup_grad", N=16384, K=32768, D=4096, type="bf16",
             index="int64", labels="zipf", scale=1.0),
        # One generated token through a square projection: streams the weights.
        dict(name="linear_step", op="linear", N=1, D=4096, F=4096, type="bf16",
             activation="silu", bias=True, residual=True, pre=False),
        # A ragged batch through widths that are no multiple of anything.
        dict(name="linear_ragged_fp16", op="linear", N=4133, D=515, F=1001, type="fp16",
             activation="gelu", bias=True, residual=True, pre=True),
        # A training batch: the forward pass keeps the pre-activations.
        dict(name="linear_batch", op="linear", N=16384, D=4096, F=4096, type="bf16",
             activation="gelu_tanh", bias=True, residual=True, pre=True),
        # Projection of the headline points into the codebook's space, backward.
        dict(name="linear_grad_points", op="linear_grad", N=65536, D=512, F=128, type="bf16",
             activation="none", bias=True),
        # Backward pass of a training batch.
        dict(name="linear_grad_batch", op="linear_grad", N=8192, D=4096, F=4096, type="bf16",
             activation="silu", bias=True),
        # A small model: a dozen gradients of mixed and odd sizes, latency.
        dict(name="clip_small", op="clip", count=12, total=100003, type="mixed", max_norm=1.0),
        # All gradients of a larger one, far beyond the caches.
        dict(name="clip_large", op="clip", count=48, total=1 << 28, type="bf16", max_norm=1.0),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]: half of the sizes as they fall (odd ones among
    them), half rounded down to a multiple of 64 or 16 where that leaves them
    in range.  Never 3 * 1024, a size that stands for nothing here."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    if rng.random() < 0.5:
        for m in (64, 16):
            if n // m * m >= lo:
                n = n // m * m
                break
    return n + 1 if n == 3 << 10 else n


def draw(rng):
    op = rng.choice(("lookup", "lookup_grad", "linear", "linear_grad", "clip"))
    if op in ("lookup", "lookup_grad"):
        D = _size(rng, 16, 4096)
        N = _size(rng, 1, min(262144, MOST_ROWS // D))
        K = _size(rng, 16, min(65536, MOST_TABLE // D))
        return dict(op=op, N=N, K=K, D=D, type=rng.choice(("bf16", "fp16", "fp32")),
                    index=rng.choice(("int32", "int64")), labels=rng.choice(("uniform", "zipf")),
                    scale=rng.choice((1.0, math.sqrt(D))))
    if op in ("linear", "linear_grad"):
        D = _size(rng, 16, 8192)
        F = _size(rng, 16, 8192)
        most = MOST_LINEAR if op == "linear" else MOST_LINEAR_GRAD
        N = _size(rng, 1, min(65536, most // (D * F), MOST_ROWS // max(D, F)))
        case = dict(op=op, N=N, D=D, F=F, type=rng.choice(("bf16", "fp16")),
                    activation=rng.choice(ACTIVATIONS), bias=rng.random() < 0.7)
        if op == "linear":
            case.update(residual=rng.random() < 0.5, pre=rng.random() < 0.5)
        return case
    return dict(op="clip", count=rng.randint(1, 48), total=_size(rng, 1 << 10, MOST_CLIP),
                type=rng.choice(("bf16", "fp16", "fp32", "mixed")),
                max_norm=rng.choice((0.1, 1.0, 1e6)))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _labels(case, gen):
    """Labels of N positions: uniform over the table (a balanced codebook), or
    by Zipf's law over a shuffled table (token frequencies).  One position in
    a hundred carries -1, which stands for no row."""
    N, K = case["N"], case["K"]
    dev = gen.device
    if case["labels"] == "zipf":
        p = 1.0 / torch.arange(1, K + 1, dtype=torch.float64, device=dev)
        cdf = torch.cumsum(p, 0)
        u = torch.rand(N, generator=gen, device=dev, dtype=torch.float64) * cdf[-1]
        rank = torch.searchsorted(cdf, u).clamp_(max=K - 1)
        lab = torch.randperm(K, generator=gen, device=dev)[rank]
    else:
        lab = torch.randint(0, K, (N,), generator=gen, device=dev)
    lab[torch.rand(N, generator=gen, device=dev) < 0.01] = -1
    return lab.to(torch.int32 if case["index"] == "int32" else torch.int64)


def _randn(shape, dtype, gen, scale=1.0):
    x = torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)
    return x.mul_(scale).to(dtype)


def _clip_sizes(case):
    """Sizes of the gradients: a few matrices hold most of the elements, the
    rest are vectors, as in a model's parameter list."""
    count, total = case["count"], case["total"]
    weights = [2.0 ** ((i * 7 + 3) % 12) for i in range(count)]
    s = sum(weights)
    sizes = [max(1, int(total * w / s)) for w in weights]
    sizes[-1] = max(1, sizes[-1] + total - sum(sizes))
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    state = dict(case)
    if op == "lookup":
        state["C"] = _randn((case["K"], case["D"]), TYPES[case["type"]], gen)
        state["labels"] = _labels(case, gen)
    elif op == "lookup_grad":
        state["dY"] = _randn((case["N"], case["D"]), TYPES[case["type"]], gen)
        state["labels"] = _labels(case, gen)
    elif op == "linear":
        t, N, D, F = TYPES[case["type"]], case["N"], case["D"], case["F"]
        state["X"] = _randn((N, D), t, gen)
        state["W"] = _randn((F, D), t, gen, D ** -0.5)
        state["b"] = _randn((F,), t, gen, 0.5) if case["bias"] else None
        state["R"] = _randn((N, F), t, gen) if case["residual"] else None
    elif op == "linear_grad":
        t, N, D, F = TYPES[case["type"]], case["N"], case["D"], case["F"]
        state["X"] = _randn((N, D), t, gen)
        state["W"] = _randn((F, D), t, gen, D ** -0.5)
        state["dY"] = _randn((N, F), t, gen, 1e-2)
        state["Z"] = _randn((N, F), t, gen) if case["activation"] != "none" else None
    else:
        kinds = (["bf16", "fp32", "fp16"] if case["type"] == "mixed" else [case["type"]])
        state["grads"] = [_randn((n,), TYPES[kinds[i % len(kinds)]], gen, 10.0 ** -(i % 3))
                          for i, n in enumerate(_clip_sizes(case))]
        state["out"] = [torch.empty_like(g) for g in state["grads"]]
    return state


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _act(z, activation):
    if activation == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if activation == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if activation == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if activation == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, activation):
    if activation == "relu":
        return (z > 0).to(z.dtype)
    if activation == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if activation == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if activation == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _plain(state):
    op = state["op"]
    if op == "lookup":
        C, lab = state["C"], state["labels"].long()
        seen = (lab >= 0) & (lab < state["K"])
        rows = C[torch.where(seen, lab, torch.zeros_like(lab))].float() * state["scale"]
        return torch.where(seen[:, None], rows, torch.zeros_like(rows)).to(C.dtype)
    if op == "lookup_grad":
        dY, lab, K = state["dY"], state["labels"].long(), state["K"]
        seen = (lab >= 0) & (lab < K)
        sums = torch.zeros((K + 1, state["D"]), dtype=torch.float32, device=dY.device)
        sums.index_add_(0, torch.where(seen, lab, torch.full_like(lab, K)), dY.float())
        return (sums[:K] * state["scale"]).to(dY.dtype)
    if op == "linear":
        X, W = state["X"], state["W"]
        z = X.float() @ W.float().t()
        if state["b"] is not None:
            z = z + state["b"].float()
        y = _act(z, state["activation"])
        if state["R"] is not None:
            y = y + state["R"].float()
        out = {"Y": y.to(X.dtype)}
        if state["pre"]:
            out["Z"] = z.to(X.dtype)
        return out
    if op == "linear_grad":
        X, W, dZ = state["X"], state["W"], state["dY"].float()
        if state["Z"] is not None:
            dZ = dZ * _act_slope(state["Z"].float(), state["activation"])
        out = {"dX": (dZ @ W.float()).to(X.dtype), "dW": (dZ.t() @ X.float()).to(X.dtype)}
        if state["bias"]:
            out["db"] = dZ.sum(0).to(X.dtype)
        return out
    grads = state["grads"]
    norm = torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()
    coef = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.reshape(1), "grads": [(g.float() * coef).to(g.dtype) for g in grads]}


def _kernels(state):
    import means_nearest_centroid_amd as km
    op = state["op"]
    if op == "lookup":
        return km.kmeans_lookup(state["C"], state["labels"], scale=state["scale"])
    if op == "lookup_grad":
        return km.kmeans_lookup_grad(state["dY"], state["labels"], state["K"],
                                     scale=state["scale"])
    if op == "linear":
        got = km.kmeans_linear(state["X"], state["W"], bias=state["b"], residual=state["R"],
                               activation=state["activation"], save_pre=state["pre"])
        return {"Y": got[0], "Z": got[1]} if state["pre"] else {"Y": got}
    if op == "linear_grad":
        dX, dW, db = km.kmeans_linear_grad(state["dY"], state["X"], state["W"], Z=state["Z"],
                                           activation=state["activation"], bias=state["bias"])
        out = {"dX": dX, "dW": dW}
        if state["bias"]:
            out["db"] = db
        return out
    norm, clipped = km.kmeans_clip_gradients(state["grads"], state["max_norm"], out=state["out"])
    return {"norm": norm, "grads": clipped}


def run(state):
    return _kernels(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_act(z, activation):
    """(act(z), act'(z)) in fp64: through the normal distribution's and the
    logistic function's own forms."""
    if activation == "none":
        return z, torch.ones_like(z)
    if activation == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if activation == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
    if activation == "silu":
        s = torch.special.expit(z)
        return z * s, s + z * s * torch.special.expit(-z)
    # 0.5 (1 + tanh(u)) = logistic(2 u)
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s, s1 = torch.special.expit(u2), torch.special.expit(-u2)
    return z * s, s + z * s * s1 * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        table = torch.cat([state["C"].double() * case["scale"],
                           torch.zeros((1, case["D"]), dtype=torch.float64, device="cuda")])
        lab = state["labels"].long()
        lab[(lab < 0) | (lab >= case["K"])] = case["K"]
        return table.index_select(0, lab)
    if op == "lookup_grad":
        # Sorted by label, the sum of a label is a difference of running sums.
        lab, order = torch.sort(state["labels"].long(), stable=True)
        run_sum = torch.cumsum(state["dY"][order].double(), 0)
        run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])
        ks = torch.arange(case["K"], device="cuda")
        lo = torch.searchsorted(lab, ks)
        hi = torch.searchsorted(lab, ks, right=True)
        return (run_sum[hi] - run_sum[lo]) * case["scale"]
    if op == "linear":
        z = torch.mm(state["X"].double(), state["W"].double().t().contiguous())
        if case["bias"]:
            z += state["b"].double()
        y = _exact_act(z, case["activation"])[0]
        if case["residual"]:
            y = y + state["R"].double()
        return {"Y": y, "Z": z} if case["pre"] else {"Y": y}
    if op == "linear_grad":
        dZ = state["dY"].double()
        if state["Z"] is not None:
            dZ = dZ * _exact_act(state["Z"].double(), case["activation"])[1]
        out = {"dX": torch.mm(dZ, state["W"].double()),
               "dW": torch.mm(dZ.t().contiguous(), state["X"].double())}
        if case["bias"]:
            out["db"] = torch.mv(dZ.t().contiguous(),
                                 torch.ones(case["N"], dtype=torch.float64, device="cuda"))
        return out
    squares = [float(torch.dot(g.double(), g.double())) for g in state["grads"]]
    norm = math.sqrt(math.fsum(squares))
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64),
            "grads": [g.double() * coef for g in state["grads"]]}


def work(case):
    op = case["op"]
    e = 4 if case["type"] == "fp32" else 2
    if op == "lookup":
        N, K, D = case["N"], case["K"], case["D"]
        i = 4 if case["index"] == "int32" else 8
        return {"bytes": N * i + (min(N, K) + N) * D * e, "flops": N * D}
    if op == "lookup_grad":
        N, K, D = case["N"], case["K"], case["D"]
        i = 4 if case["index"] == "int32" else 8
        return {"bytes": N * i + (N + K) * D * e, "flops": N * D}
    if op == "linear":
        N, D, F = case["N"], case["D"], case["F"]
        n = N * D + F * D + (F if case["bias"] else 0)
        n += N * F * (1 + case["residual"] + case["pre"])
        return {"bytes": n * e, "flops": 2 * N * D * F}
    if op == "linear_grad":
        N, D, F = case["N"], case["D"], case["F"]
        n = 2 * (N * D + F * D) + N * F * (2 if case["activation"] != "none" else 1)
        return {"bytes": (n + (F if case["bias"] else 0)) * e, "flops": 4 * N * D * F}
    sizes = _clip_sizes(case)
    e = (2, 4, 2) if case["type"] == "mixed" else (e,)
    return {"bytes": 2 * sum(n * e[i % len(e)] for i, n in enumerate(sizes)),
            "flops": 3 * sum(sizes)}
