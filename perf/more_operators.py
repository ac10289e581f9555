"""Cases of the operators around a model that predicts codebook labels: the
root-mean-square norm with the residual's addition (its output in the inputs'
type or in 8 bits with scales) and its gradient, quantisation by blocks of 128,
the linear layer on 8-bit operands, and the draw of a label from each row of
logits.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` is one pass as a program calls it (the framework's operators
where ``own`` is true, elementary torch operations otherwise: in 32 bits, the
draw's weights and the sums over all rows in 64), ``exact`` the same outputs
from the definitions in 64 bits and ``work`` the bytes and operations that a
pass cannot do without.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
BLOCK = 128
EPS = 1e-6

# Most elements of a drawn case's rows, multiply-adds and logits: those of the
# largest listed ones.
MOST_ROWS = 16384 * 4096
MOST_LINEAR = 16384 * 4096 * 4096
MOST_LOGITS = 512 * 65536


def listed():
    return [
        # One generated token before its projection: latency.
        dict(name="norm_step", op="norm", N=1, D=4096, type="bf16", residual=True, weight=True,
             quantize=True),
        # A prompt's tokens before an 8-bit projection.
        dict(name="norm_batch", op="norm", N=16384, D=4096, type="bf16", residual=True,
             weight=True, quantize=True),
        # A ragged batch through a width that is no multiple of anything.
        dict(name="norm_ragged_fp16", op="norm", N=4133, D=1001, type="fp16", residual=True,
             weight=True, quantize=False),
        # Backward pass of a training batch; the residual path brings a gradient too.
        dict(name="norm_grad_batch", op="norm_grad", N=16384, D=4096, type="bf16", weight=True,
             skip=True),
        # Narrow fp32 rows with an odd count and width.
        dict(name="norm_grad_ragged_fp32", op="norm_grad", N=50021, D=321, type="fp32",
             weight=True, skip=False),
        # The headline points in 8 bits, a scale for each.
        dict(name="quantize_points", op="quantize", N=262144, D=128, type="bf16", rows=1),
        # A square projection's weights in 8 bits, 128 x 128 blocks.
        dict(name="quantize_weights", op="quantize", N=4096, D=4096, type="bf16", rows=128),
        # One token's scores of every row of a table: streams the weights.
        dict(name="linear_fp8_step", op="linear_fp8", N=1, D=4096, F=32768, type="fp32",
             activation="none", bias=False, residual=False),
        # A ragged batch through widths that are no multiple of anything.
        dict(name="linear_fp8_ragged", op="linear_fp8", N=4133, D=515, F=1001, type="fp16",
             activation="gelu", bias=True, residual=True),
        # A prompt's tokens through a square projection.
        dict(name="linear_fp8_batch", op="linear_fp8", N=16384, D=4096, F=4096, type="bf16",
             activation="gelu_tanh", bias=True, residual=True),
        # The next tokens of 16 sequences, each with settings of its own: latency.
        dict(name="sample_step", op="sample", N=16, K=32768, type="fp32", per_row=True,
             temperature=0.8, top_k=50, top_p=0.95, min_p=0.05),
        # Many sequences at once, the nucleus alone.
        dict(name="sample_batch", op="sample", N=512, K=65536, type="fp32", per_row=False,
             temperature=1.0, top_k=0, top_p=0.9, min_p=0.0),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]: half of the sizes as they fall (odd ones among
    them), half rounded down to a multiple of 64 or 16 where that leaves them
    in range."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    if rng.random() < 0.5:
        for m in (64, 16):
            if n // m * m >= lo:
                return n // m * m
    return n


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "quantize", "linear_fp8", "linear_fp8", "sample",
                     "sample"))
    if op in ("norm", "norm_grad", "quantize"):
        D = _size(rng, 16, 16384)
        case = dict(op=op, N=_size(rng, 1, min(262144, MOST_ROWS // 2 // D)), D=D,
                    type=rng.choice(("bf16", "fp16", "fp32")))
        if op == "quantize":
            case.update(rows=rng.choice((1, BLOCK)))
        else:
            case.update(weight=rng.random() < 0.8)
        if op == "norm":
            case.update(residual=rng.random() < 0.6, quantize=rng.random() < 0.5)
        if op == "norm_grad":
            case.update(skip=rng.random() < 0.5)
        return case
    if op == "linear_fp8":
        D = _size(rng, 16, 8192)
        F = _size(rng, 16, 32768)
        N = _size(rng, 1, min(65536, MOST_LINEAR // (D * F), MOST_ROWS // max(D, F)))
        return dict(op=op, N=N, D=D, F=F, type=rng.choice(("bf16", "fp16", "fp32")),
                    activation=rng.choice(ACTIVATIONS), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    K = _size(rng, 16, 131072)
    return dict(op=op, N=_size(rng, 1, min(4096, MOST_LOGITS // K)), K=K,
                type=rng.choice(("bf16", "fp16", "fp32")), per_row=rng.random() < 0.5,
                temperature=rng.choice((0.5, 0.7, 1.0, 1.3)), top_k=rng.choice((0, 0, 20, 50, 1000)),
                top_p=rng.choice((0.5, 0.9, 0.95, 1.0)), min_p=rng.choice((0.0, 0.0, 0.02, 0.1)))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _randn(shape, dtype, gen, scale=1.0):
    x = torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)
    return x.mul_(scale).to(dtype)


def _hidden(N, D, dtype, gen):
    """Rows of a residual stream: sizes differ from row to row, and one column
    in 64 is far larger than the rest."""
    x = torch.randn((N, D), generator=gen, device=gen.device, dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((N, 1), generator=gen, device=gen.device))
    x *= torch.where(torch.rand(D, generator=gen, device=gen.device) < 1 / 64, 20.0, 1.0)
    return x.to(dtype)


def _quantized(x, rows):
    """e4m3 values and scales of the blocks of ``rows`` x 128, in fp32."""
    N, D = x.shape
    n, b = -(-N // rows), -(-D // BLOCK)
    x = torch.nn.functional.pad(x, (0, b * BLOCK - D, 0, n * rows - N))
    x = x.view(n, rows, b, BLOCK)
    most = x.abs().amax((1, 3))
    scales = torch.where(most > 0, (most / FP8_MAX).clamp(min=2.0 ** -126), torch.ones_like(most))
    q = (x / scales[:, None, :, None]).view(n * rows, b * BLOCK)[:N, :D]
    return q.to(FP8).contiguous(), scales


def _sampling(case, gen):
    """The settings as the call takes them: numbers, or a tensor of one value
    for each row (mixed requests, some of them greedy or unfiltered)."""
    names = ("temperature", "top_k", "top_p", "min_p")
    if not case["per_row"]:
        return {n: case[n] for n in names}
    N = case["N"]
    r = torch.rand((4, N), generator=gen, device="cuda")
    pick = lambda x, y: torch.where(x < 0.7, case[y[0]], y[1]).to(y[2])  # noqa: E731
    return {"temperature": torch.where(r[0] < 0.1, 0.0, case["temperature"] * (0.5 + r[0])),
            "top_k": pick(r[1], ("top_k", 0, torch.int32)),
            "top_p": pick(r[2], ("top_p", 1.0, torch.float32)),
            "min_p": pick(r[3], ("min_p", 0.0, torch.float32))}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, N = case["op"], case["N"]
    state = dict(case)
    if op in ("norm", "norm_grad"):
        t, D = TYPES[case["type"]], case["D"]
        state["w"] = None
        if case["weight"]:
            state["w"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(t)
        if op == "norm":
            state["X"] = _hidden(N, D, t, gen)
            state["R"] = _hidden(N, D, t, gen) if case["residual"] else None
        else:
            state["H"] = _hidden(N, D, t, gen)
            state["dY"] = _randn((N, D), t, gen, 1e-2)
            state["dH"] = _randn((N, D), t, gen, 1e-2) if case["skip"] else None
    elif op == "quantize":
        state["X"] = _hidden(N, case["D"], TYPES[case["type"]], gen)
    elif op == "linear_fp8":
        t, D, F = TYPES[case["type"]], case["D"], case["F"]
        state["X"], state["sx"] = _quantized(_hidden(N, D, torch.float32, gen), 1)
        state["W"], state["sw"] = _quantized(_randn((F, D), torch.float32, gen, D ** -0.5), BLOCK)
        state["b"] = _randn((F,), t, gen, 0.5) if case["bias"] else None
        state["R"] = _randn((N, F), t, gen) if case["residual"] else None
    else:
        K = case["K"]
        z = torch.randn((N, K), generator=gen, device="cuda") * 2.5
        likely = torch.randint(0, K, (N, 16), generator=gen, device="cuda")
        z.scatter_add_(1, likely, 8.0 * torch.rand((N, 16), generator=gen, device="cuda"))
        state["logits"] = z.to(TYPES[case["type"]])
        state["u"] = torch.rand(N, generator=gen, device="cuda")
        state["settings"] = _sampling(case, gen)
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


def _dequantized(q, scales, rows):
    s = scales.repeat_interleave(rows, 0)[:q.shape[0]]
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _setting(value, N, dtype):
    if isinstance(value, torch.Tensor):
        return value[:, None]
    return torch.full((N, 1), value, dtype=dtype, device="cuda")


def _draw(logits, u, settings):
    N, K = logits.shape
    t = _setting(settings["temperature"], N, torch.float32).double()
    k = _setting(settings["top_k"], N, torch.int32).long()
    p = _setting(settings["top_p"], N, torch.float32).double()
    least = _setting(settings["min_p"], N, torch.float32).double()
    z = logits.float()
    z = torch.where(torch.isnan(z), -math.inf, z)
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    d = torch.where(z == z[:, :1], 0.0, z.double() - z[:, :1].double())
    w = torch.exp(d / torch.where(t > 0, t, torch.ones_like(t)))
    w = torch.where(z > -math.inf, w, 0.0)
    rank = torch.arange(K, device=z.device)
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    sums = torch.cumsum(w, 1)
    before = torch.cat([torch.zeros_like(sums[:, :1]), sums[:, :-1]], 1)
    kept = ((p >= 1) | (before < p * sums[:, -1:]) | (rank == 0)) & (w >= least)
    kept &= (t > 0) | (rank == 0)
    sums = torch.cumsum(torch.where(kept, w, 0.0), 1)
    at = (sums <= u.double()[:, None] * sums[:, -1:]).sum(1, keepdim=True)
    label = order.gather(1, at.clamp(max=K - 1))[:, 0]
    return torch.where(sums[:, -1] > 0, label, -1).to(torch.int32)


def _plain(state):
    op = state["op"]
    if op == "norm":
        t = state["X"].dtype
        h = state["X"].float()
        out = {}
        if state["R"] is not None:
            h = h + state["R"].float()
            out["H"] = h.to(t)
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        if state["w"] is not None:
            y = y * state["w"].float()
        if state["quantize"]:
            out["Q"], out["scales"] = _quantized(y, 1)
        else:
            out["Y"] = y.to(t)
        return out
    if op == "norm_grad":
        t = state["H"].dtype
        h, dy = state["H"].float(), state["dY"].float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        g = dy * state["w"].float() if state["w"] is not None else dy
        dx = r * g - h * (r * r * r * (g * h).mean(1, keepdim=True))
        if state["dH"] is not None:
            dx = dx + state["dH"].float()
        out = {"dX": dx.to(t)}
        if state["w"] is not None:
            out["dw"] = (dy * h * r).double().sum(0).to(t)
        return out
    if op == "quantize":
        q, scales = _quantized(state["X"].float(), state["rows"])
        return {"Q": q, "scales": scales}
    if op == "linear_fp8":
        z = (_dequantized(state["X"], state["sx"], 1)
             @ _dequantized(state["W"], state["sw"], BLOCK).t())
        if state["b"] is not None:
            z = z + state["b"].float()
        y = _act(z, state["activation"])
        if state["R"] is not None:
            y = y + state["R"].float()
        return y.to(TYPES[state["type"]])
    return _draw(state["logits"], state["u"], state["settings"])


def _kernels(state):
    import means_nearest_centroid_amd as km
    op = state["op"]
    if op == "norm":
        got = km.kmeans_rms_norm(state["X"], state["w"], residual=state["R"], eps=EPS,
                                 quantize=state["quantize"])
        got = got if isinstance(got, tuple) else (got,)
        names = (("Q", "scales") if state["quantize"] else ("Y",)) + ("H",)
        return dict(zip(names, got))
    if op == "norm_grad":
        dX, dw = km.kmeans_rms_norm_grad(state["dY"], state["H"], state["w"], eps=EPS,
                                         dH=state["dH"])
        return {"dX": dX} if state["w"] is None else {"dX": dX, "dw": dw}
    if op == "quantize":
        q, scales = km.kmeans_quantize(state["X"], rows=state["rows"])
        return {"Q": q, "scales": scales}
    if op == "linear_fp8":
        return km.kmeans_linear_fp8(state["X"], state["sx"], state["W"], state["sw"],
                                    bias=state["b"], residual=state["R"],
                                    activation=state["activation"], dtype=TYPES[state["type"]])
    return km.kmeans_sample(state["logits"], state["u"], **state["settings"])


def run(state):
    return _kernels(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_act(z, activation):
    """Through the normal distribution's and the logistic function's own forms."""
    if activation == "relu":
        return z.clamp(min=0)
    if activation == "gelu":
        return z * torch.special.ndtr(z)
    if activation == "silu":
        return z * torch.special.expit(z)
    if activation == "gelu_tanh":     # (1 + tanh(v)) / 2 = logistic(2 v)
        return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _exact_blocks(y, rows):
    """Scale of every value, and of every block: block by block."""
    n, b = -(-y.shape[0] // rows), -(-y.shape[1] // BLOCK)
    cols = torch.stack([y[:, c * BLOCK:(c + 1) * BLOCK].abs().amax(1) for c in range(b)], 1)
    at = torch.arange(y.shape[0], device=y.device) // rows
    most = torch.zeros((n, b), dtype=y.dtype, device=y.device)
    most.scatter_reduce_(0, at[:, None].expand(-1, b), cols, "amax")
    scales = torch.where(most == 0, 1.0, most / FP8_MAX)
    return y / scales[at][:, torch.arange(y.shape[1], device=y.device) // BLOCK], scales


def _exact_draw(logits, u, settings):
    """Row by row on the host."""
    z_all, u = logits.double().cpu().numpy(), u.double().cpu().numpy()
    N, K = z_all.shape
    column = {n: np.broadcast_to(np.asarray(v.cpu() if isinstance(v, torch.Tensor)
                                            else np.float32(v)), (N,))
              for n, v in settings.items()}
    labels = np.empty(N, np.int32)
    for i in range(N):
        z = np.where(np.isnan(z_all[i]), -np.inf, z_all[i])
        t, k = float(column["temperature"][i]), int(column["top_k"][i])
        p, least = float(column["top_p"][i]), float(column["min_p"][i])
        top = int(np.argmax(z))
        if not t > 0 or z[top] == -np.inf:
            labels[i] = top if z[top] > -np.inf else -1
            continue
        w = np.where(z == z[top], 1.0, np.exp((z - z[top]) / t))
        ranked = np.lexsort((np.arange(K), -z))
        if k > 0:
            ranked = ranked[:k]
        if p < 1:
            run_sum = np.cumsum(w[ranked])
            ranked = ranked[:int(np.searchsorted(run_sum, p * run_sum[-1])) + 1]
        ranked = ranked[w[ranked] >= least]
        run_sum = np.cumsum(w[ranked])
        labels[i] = ranked[min(int(np.searchsorted(run_sum, u[i] * run_sum[-1], side="right")),
                               len(ranked) - 1)]
    return torch.from_numpy(labels)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = state["X"].double()
        out = {}
        if case["residual"]:
            h = h + state["R"].double()
            out["H"] = h
        y = h / torch.sqrt(torch.linalg.vecdot(h, h)[:, None] / case["D"] + EPS)
        if case["weight"]:
            y = y * state["w"].double()
        if case["quantize"]:
            out["Q"], out["scales"] = _exact_blocks(y, 1)
        else:
            out["Y"] = y
        return out
    if op == "norm_grad":
        h = state["H"].double().requires_grad_()
        w = state["w"].double() if case["weight"] else torch.ones(
            case["D"], dtype=torch.float64, device="cuda")
        w.requires_grad_()
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w
        dx, dw = torch.autograd.grad(y, (h, w), state["dY"].double())
        if case["skip"]:
            dx = dx + state["dH"].double()
        return {"dX": dx, "dw": dw} if case["weight"] else {"dX": dx}
    if op == "quantize":
        q, scales = _exact_blocks(state["X"].double(), case["rows"])
        return {"Q": q, "scales": scales}
    if op == "linear_fp8":
        N, D, F = case["N"], case["D"], case["F"]
        z = torch.zeros((N, F), dtype=torch.float64, device="cuda")
        rows = torch.arange(F, device="cuda") // BLOCK
        for b in range(-(-D // BLOCK)):
            k = slice(b * BLOCK, (b + 1) * BLOCK)
            part = torch.mm(state["X"][:, k].double(), state["W"][:, k].double().t().contiguous())
            z += part * state["sx"][:, b].double()[:, None] * state["sw"][rows, b].double()
        if case["bias"]:
            z += state["b"].double()
        y = _exact_act(z, case["activation"])
        return y + state["R"].double() if case["residual"] else y
    return _exact_draw(state["logits"], state["u"], state["settings"])


def work(case):
    op, N = case["op"], case["N"]
    e = 4 if case["type"] == "fp32" else 2
    if op == "sample":
        return {"bytes": N * case["K"] * e + 8 * N + (16 * N if case["per_row"] else 0),
                "flops": 4 * N * case["K"]}
    D = case["D"]
    eight = N * D + 4 * N * -(-D // BLOCK)       # rows in 8 bits and their scales
    if op == "norm":
        bytes_ = N * D * e * (3 if case["residual"] else 1) + (D * e if case["weight"] else 0)
        bytes_ += eight if case["quantize"] else N * D * e
        return {"bytes": bytes_, "flops": 6 * N * D}
    if op == "norm_grad":
        return {"bytes": (N * D * (4 if case["skip"] else 3) + (2 * D if case["weight"] else 0)) * e,
                "flops": 12 * N * D}
    if op == "quantize":
        return {"bytes": N * D * (e + 1) + 4 * -(-N // case["rows"]) * -(-D // BLOCK),
                "flops": 2 * N * D}
    F = case["F"]
    n = N * F * (1 + case["residual"]) + (F if case["bias"] else 0)
    return {"bytes": n * e + eight + F * D + 4 * -(-F // BLOCK) * -(-D // BLOCK),
            "flops": 2 * N * D * F}
