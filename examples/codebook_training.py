"""A codebook trained by gradients between two linear layers: features are
encoded, each is replaced by its nearest centroid, and decoded again.

    H = gelu(X W1^T + b1)              kmeans_linear
    l = nearest centroid of each H[i]  kmeans_centroid_norms, kmeans_assign
    Q = C[l]                           kmeans_lookup
    Y = Q W2^T + b2                    kmeans_linear

The loss is the mean over points of |Y - X|^2 / 2 + |Q - H|^2 / 2.  The
nearest-centroid step has no gradient of its own: the decoder's gradient of Q
goes to the codebook and, unchanged, to H.

    dQ = dY W2,  dW2, db2              kmeans_linear_grad
    dC[k] = sum over l[i] == k of dQ[i] + (Q[i] - H[i]) / N    kmeans_lookup_grad
    dH = dQ + (H - Q) / N
    dW1, db1                           kmeans_linear_grad
    clip by the global norm            kmeans_clip_gradients

    python examples/codebook_training.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import means_nearest_centroid_amd as km  # noqa: E402


def parameters(width, code, K, seed=0, device="cuda"):
    """fp32 parameters: encoder, codebook, decoder."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale: (torch.randn(*s, generator=g) * scale).to(device)  # noqa: E731
    return {"W1": r(code, width, scale=width ** -0.5), "b1": r(code, scale=0.1),
            "C": r(K, code, scale=0.5),
            "W2": r(width, code, scale=code ** -0.5), "b2": r(width, scale=0.1)}


def synthetic(N, width, kinds, seed=0, device="cuda"):
    """bf16 points around `kinds` centres."""
    g = torch.Generator().manual_seed(seed)
    centres = torch.randn(kinds, width, generator=g)
    X = centres[torch.randint(0, kinds, (N,), generator=g)]
    return (X + 0.1 * torch.randn(N, width, generator=g)).to(torch.bfloat16).to(device)


def gradients(p, X):
    """Loss (fp32 scalar tensor) and gradients by parameter name, for bf16
    parameters ``p`` and points ``X``."""
    N = X.shape[0]
    H, Z = km.kmeans_linear(X, p["W1"], p["b1"], activation="gelu", save_pre=True)
    labels, _ = km.kmeans_assign(H, p["C"], km.kmeans_centroid_norms(p["C"]))
    Q = km.kmeans_lookup(p["C"], labels)
    Y = km.kmeans_linear(Q, p["W2"], p["b2"])

    miss = Y.float() - X.float()
    gap = Q.float() - H.float()
    loss = (miss.square().sum() + gap.square().sum()) / (2 * N)

    dY = (miss / N).to(X.dtype)
    dQ, dW2, db2 = km.kmeans_linear_grad(dY, Q, p["W2"])
    dC = km.kmeans_lookup_grad((dQ + gap / N).to(X.dtype), labels, p["C"].shape[0])
    dH = (dQ - gap / N).to(X.dtype)
    _, dW1, db1 = km.kmeans_linear_grad(dH, X, p["W1"], Z, activation="gelu", need_dx=False)
    return loss, {"W1": dW1, "b1": db1, "C": dC, "W2": dW2, "b2": db2}


def train(X, master, steps, rate=1.0, max_norm=1.0, say=None):
    """Plain gradient descent on the fp32 ``master`` parameters (in place);
    returns the loss of each step."""
    losses = []
    for step in range(steps):
        loss, grads = gradients({n: t.to(X.dtype) for n, t in master.items()}, X)
        norm, clipped = km.kmeans_clip_gradients([grads[n] for n in master], max_norm)
        for t, g in zip(master.values(), clipped):
            t.sub_(g, alpha=rate)
        losses.append(loss)
        if say is not None and step % 10 == 0:
            say(f"step {step}: loss {loss.item():.4f}, gradient norm {norm.item():.4f}")
    return [x.item() for x in losses]


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 100
    X = synthetic(65536, 512, 256)
    losses = train(X, parameters(512, 128, 1024), steps, say=lambda s: print(s, flush=True))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")


if __name__ == "__main__":
    main()
