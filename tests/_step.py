"""Plain 64-bit forms of the operators around a speculative step, written from
their formulas (include/kivi.h), for the tests."""
import numpy as np
import torch

ONE = 2.0 ** 42


def norm_rope64(x, weight, eps, inv_freq, pos, axis, interleaved, turn=True):
    """x [B, N, heads, D] -> float64 [B, heads, N, D]; pos int64 [n_axes, B, N]."""
    y = x.double().cpu()
    D = y.shape[-1]
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + float(np.float32(eps))) * weight.double().cpu()
    half = 0 if inv_freq is None else inv_freq.numel()
    if turn and half:
        z = y.clone()
        for j in range(half):
            a, c = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            n_axes = pos.shape[0]
            p = pos[0 if axis is None else min(max(int(axis[j]), 0), n_axes - 1)]
            t = (p.double() * float(inv_freq[j])).unsqueeze(-1)
            z[..., a] = y[..., a] * torch.cos(t) - y[..., c] * torch.sin(t)
            z[..., c] = y[..., c] * torch.cos(t) + y[..., a] * torch.sin(t)
        y = z
    return y.permute(0, 2, 1, 3)


def probs64(logits, temperature=1.0):
    """One row: float64 numpy of the documented probabilities."""
    l = logits.double().cpu().numpy()
    out = np.zeros(l.shape)
    if np.isnan(l).any() or np.isnan(temperature) or np.isposinf(l).any():
        return np.full(l.shape, np.nan)
    if np.isneginf(l).all():
        return out
    if temperature <= 0:
        out[int(np.argmax(l))] = 1.0        # the first of the largest
        return out
    with np.errstate(over="ignore"):
        x = (l - l.max()) / temperature if np.isfinite(temperature) else np.where(np.isneginf(l), -np.inf, 0.0)
    e = np.exp(x)
    return e / e.sum()


def clamp01(row):
    row = np.asarray(row, dtype=np.float32)
    return np.clip(np.where(np.isnan(row), np.float32(0), row), np.float32(0), np.float32(1))


def whole(r):
    return np.rint(r.astype(np.float64) * ONE).astype(np.int64)


def verify(tokens, parent, u, target, draft, n=None):
    """One sequence (numpy, fp32 and int32): (path, next), node by node down the
    tree with whole numbers for the sums."""
    f = np.float32
    N, V = target.shape
    n = N if n is None else min(max(n, 0), N)
    if n == 0:
        return [], -1
    path = [0]
    while True:
        c = path[-1]
        rho, s = clamp01(target[c]), f(1)
        q = None if draft is None else clamp01(draft[c])
        new = None
        for i in range(1, n):
            if parent[i] != c or not c < i or not 0 <= tokens[i] < V:
                continue
            x = tokens[i]
            if f(u[i]) * (f(1) if q is None else q[x]) < rho[x] * s:
                new = i
                break
            if q is None:
                rho = rho.copy()
                rho[x] = 0
            else:
                rho = np.maximum(rho * s - q, f(0))
            z = int(whole(rho).sum())
            s = f(ONE / float(z)) if z else f(0)
        if new is None:
            break
        path.append(new)
    w = whole(rho)
    if not w.any():
        w = whole(clamp01(target[c]))
    z = sum(int(x) for x in w)
    if z == 0:
        return path, -1
    u0 = float(u[0])
    d = 0 if not u0 > 0 else min(int(u0 * 2.0 ** 32), 2 ** 32 - 1)
    t = z * d >> 32
    cum = np.cumsum(w)
    return path, int(np.nonzero(cum > t)[0][0])
