"""MX4 (MXFP4) and the router's training losses in 64 bits, written from their definitions: what the
MX4 and balance-loss tests compare with.  numpy only; shares no code with the library or the inputs."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def decode(q, scale):
    """uint8 codes [..., K/2] and E8M0 scales [..., K/32] -> float64 [..., K]."""
    q, scale = np.asarray(q), np.asarray(scale)
    v = np.empty((*q.shape[:-1], q.shape[-1] * 2))
    v[..., 0::2] = E2M1[q & 15]
    v[..., 1::2] = E2M1[q >> 4]
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def quantize(v):
    """float64 [..., K] (fp32 or bf16 values) -> (codes [..., K/2], scales [..., K/32]), by comparing
    each value with the eight magnitudes."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(-1, 32)
    codes = np.zeros(b.shape, np.uint8)
    scales = np.zeros(len(b), np.uint8)
    for i, row in enumerate(b):
        if not np.isfinite(row).all():
            scales[i] = 255
            continue
        a = np.abs(row).max()
        e = -127
        if a > 0:
            e = max(-127, int(np.frexp(a)[1]) - 1 - 2)
        scales[i] = e + 127
        x = np.abs(np.ldexp(row, -e))
        d = np.abs(x[:, None] - E2M1[None, :8])
        c = d.argmin(1)                                   # the lower of two equally near ones
        tie = (c < 7) & (d[np.arange(32), np.minimum(c + 1, 7)] == d[np.arange(32), c])
        c = np.where(tie & (c % 2 == 1), c + 1, c)        # ties to the even code
        codes[i] = c + 8 * np.signbit(row)
    codes = codes.reshape(*v.shape[:-1], v.shape[-1])
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scales.reshape(*v.shape[:-1], v.shape[-1] // 32)


def activate(y, act):
    if act == "swiglu":
        f = y.shape[-1] // 2
        g, u = y[..., :f], y[..., f:]
        with np.errstate(over="ignore"):
            return g / (1 + np.exp(-g)) * u
    return np.where(np.isnan(y), y, np.maximum(y, 0) ** 2) if act == "relu2" else y


def product(x, w, offsets, src):
    """Rows x[src[r]] times w[g].T for the groups' rows; NaN-filled where no group has the row.
    Returns (y, sum of the magnitudes of the products)."""
    out = np.full((len(src), w.shape[1]), np.nan)
    mag = np.zeros_like(out)
    for g in range(len(w)):
        r = slice(int(offsets[g]), int(offsets[g + 1]))
        out[r] = x[src[r]] @ w[g].T
        mag[r] = np.abs(x[src[r]]) @ np.abs(w[g]).T
    return out, mag


def balance(logits, idx, mask=None):
    """(loss [2], counts [E], mean_prob [E]) in float64."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    k = idx.shape[1]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool).copy()
    keep &= ~np.all(l == -np.inf, axis=1)
    n = int(keep.sum())
    counts = np.bincount(np.clip(idx[keep], 0, E - 1).reshape(-1), minlength=E)
    if n == 0:
        return np.zeros(2), counts, np.zeros(E)
    p, lse = softmax(l[keep])
    P = p.mean(0)
    return np.array([E * np.sum(counts / (n * k) * P), np.mean(lse ** 2)]), counts, P


def softmax(l):
    m = l.max(1, keepdims=True)
    e = np.exp(l - m)
    s = e.sum(1, keepdims=True)
    return e / s, (m + np.log(s))[:, 0]


def balance_grad(logits, idx, counts, d_loss, w=None, dw=None, mask=None):
    """(d_logits, magnitude) in float64; magnitude is the sum of the absolute values of the terms
    each element adds up, for error bounds."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    k = idx.shape[1]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool).copy()
    keep &= ~np.all(l == -np.inf, axis=1)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    total = counts.sum()
    f = counts / total if total else np.zeros(E)
    n = total / k
    for t in np.flatnonzero(keep):
        p, lse = softmax(l[t:t + 1])
        p, lse = p[0], lse[0]
        if n:
            d[t] = p * (d_loss[0] * E / n * (f - f @ p) + d_loss[1] * 2 / n * lse)
            mag[t] = p * (abs(d_loss[0]) * E / n * (f + f @ p) + abs(d_loss[1]) * 2 / n * abs(lse))
        if w is not None:
            wd = w[t].astype(np.float64) @ dw[t].astype(np.float64)
            wm = np.abs(w[t].astype(np.float64)) @ np.abs(dw[t].astype(np.float64))
            for j in range(k):
                e = min(max(int(idx[t, j]), 0), E - 1)
                d[t, e] += float(w[t, j]) * (float(dw[t, j]) - wd)
                mag[t, e] += abs(float(w[t, j])) * (abs(float(dw[t, j])) + wm)
    return d, mag
