"""Plain references of the operators around the layer, in 64 bits (numpy, CPU)."""
import numpy as np
import torch

EPS = {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10, torch.float32: 2.0 ** -23}


def f64(t):
    return t.detach().double().cpu().numpy()


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True,
          scale=1.0):
    """ids [T, k], weights [T, k] in binary64, token by token from the rule."""
    l = np.array(f64(logits) if isinstance(logits, torch.Tensor) else logits, np.float64)
    top = float(np.finfo(np.float32).max)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, top))
    T, E = l.shape
    b = None
    if bias is not None:
        b = np.array(f64(bias) if isinstance(bias, torch.Tensor) else bias, np.float64)
        b = np.where(np.isnan(b), -np.inf, np.minimum(b, top))
    ids = np.zeros((T, k), np.int64)
    out = np.zeros((T, k))
    for t in range(T):
        ok = l[t] > -np.inf
        s = np.zeros(E)
        if score == "softmax":
            if ok.any():
                s[ok] = np.exp(l[t, ok] - l[t, ok].max())
                s /= s.sum()
        else:
            with np.errstate(over="ignore"):
                s[ok] = 1.0 / (1.0 + np.exp(-l[t, ok]))
        if b is not None:
            ok = ok & (b > -np.inf)
        v = s + (0.0 if b is None else np.where(b > -np.inf, b, 0.0))
        rank = l[t] if b is None else v
        if groups > 1:
            size = E // groups
            tot = np.full(groups, -np.inf)
            for g in range(groups):
                at = np.arange(g * size, (g + 1) * size)
                at = at[ok[at]]
                if at.size:
                    # (by one value without a bias: the largest logit, which has the largest score)
                    tot[g] = l[t, at].max() if b is None and group_best == 1 else np.sort(v[at])[::-1][:group_best].sum()
            kept = sorted(range(groups), key=lambda g: (-tot[g], g))[:top_groups]
            ok = ok & np.isin(np.arange(E) // size, kept)
        order = sorted(range(E), key=lambda e: (not ok[e], -rank[e] if ok[e] else 0.0, e))[:k]
        ids[t] = order
        w = s[order] * ok[order]
        if renormalize:
            on = ok[order]
            if score == "softmax" and on.any():  # the same ratio where the k lie far below the largest
                lk = l[t, order]
                w = np.where(on, np.exp(np.where(on, lk - lk[on].max(), -np.inf)), 0.0)
            elif on.any():  # e^-c / (1 + e^-l) = 1 / (e^c + e^(c - l)): the same ratios for scores far below 1
                lk = np.where(on, l[t, order], 0.0)
                c = min(lk[on].max(), 0.0)
                w = np.where(on, 1.0 / (np.exp(c) + np.exp(np.minimum(c - lk, 709.0))), 0.0)
            w = w / w.sum() if w.sum() > 0 else w
        out[t] = scale * w
    return ids, out


def _norm(v, size, weight, bias, kind, eps, offset):
    """N(v) and how large the terms are that its binary32 errors are relative to."""
    mean = v.mean(1, keepdims=True) if kind == "layer" else 0.0
    d = v - mean
    inv = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    w = 1.0 if weight is None else np.abs(weight + offset)
    spread = (size + np.sqrt((size * size).mean(1, keepdims=True))) * inv * w
    n = d * inv * (1.0 if weight is None else weight + offset)
    return (n, spread) if bias is None else (n + bias, spread + np.abs(bias))


def block_norm(r, y, before=None, after=None, gate=None, gate_sigmoid=False, res_scale=1.0, out_scale=1.0):
    """r', h and the magnitudes of their terms; before / after: (weight, bias, kind, eps, offset) in binary64."""
    r = f64(r)
    out, size = res_scale * r, np.abs(res_scale * r)
    if y is not None:
        d = f64(y)
        ds = np.abs(d)
        if after is not None:
            d, ds = _norm(d, ds, *after)
        g = np.ones(1) if gate is None else f64(gate)
        if gate is not None and gate_sigmoid:
            g = 1.0 / (1.0 + np.exp(-g))
        out, size = out + out_scale * g * d, size + np.abs(out_scale * g) * ds
    h, hs = (None, None) if before is None else _norm(out, size, *before)
    return out, size, h, hs


def check_norm(got, ref, size):
    """A value's own rounding (half a step of its type) and the binary32 steps.

    Of the binary32 steps, the sums are the longest chain: a thread adds at
    most 64 products, then 6 + 16 sums over lanes and waves, so a mean is off by
    at most 90 * 2^-24 of its terms' size, the root of the mean square by half
    of that; the second norm takes the first one's error as its input's.  Some
    20 single steps (products, the exponential, the root, the quotient) come
    beside it: 2 * (90 + 45) + 20 < 300 steps of 2^-24 of the terms' size."""
    got64 = f64(got)
    eps = EPS[got.dtype]
    tiny = float(torch.finfo(got.dtype).tiny)
    tol = eps / 2 * np.maximum(np.abs(ref), tiny) * (1 + eps) + 300 * 2.0 ** -24 * size
    assert np.isfinite(got64).all()
    worst = (np.abs(got64 - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the tolerance"


def int8_rows(x):
    """codes and scale of each row, step by step in binary32."""
    x = x.detach().float().cpu().numpy()
    am = np.abs(x).max(1)
    some = am >= np.float32(2.0 ** -119)
    safe = np.where(some, am, np.float32(127.0)).astype(np.float32)
    inv = np.where(some, np.float32(127.0) / safe, np.float32(0.0)).astype(np.float32)
    q = np.rint(x * inv[:, None]).astype(np.int8)
    return q, np.where(some, am / np.float32(127.0), np.float32(1.0)).astype(np.float32)


def int8_product(a, sa, b, sb, bias=None):
    """The product in binary64 and the size of its terms."""
    acc = a.astype(np.float64) @ b.astype(np.float64).T  # whole numbers below 2^53: exact
    out = acc * sa.astype(np.float64)[:, None] * sb.astype(np.float64)
    return (out, np.abs(out)) if bias is None else (out + bias.astype(np.float64), np.abs(out) + np.abs(bias))


def check_product(got, ref, size):
    """Half a step of the result's type, and four binary32 roundings (the sum's
    conversion, the product of the scales, their product, the bias's sum)."""
    got64 = f64(got)
    eps = EPS[got.dtype]
    tol = eps / 2 * np.maximum(np.abs(ref), float(torch.finfo(got.dtype).tiny)) * (1 + eps) + 5 * 2.0 ** -24 * size
    assert np.isfinite(got64).all()
    worst = (np.abs(got64 - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the tolerance"
