"""Plain 64-bit implementations of the tree-verify operators (NumPy, no code shared with the library)."""
import numpy as np


def parents(rs, B, shape="tree"):
    if shape == "chain":
        return np.arange(-1, B - 1, dtype=np.int32)
    if shape == "star":
        return np.where(np.arange(B) == 0, -1, 0).astype(np.int32)
    p = np.array([-1] + [rs.randint(max(0, b - 6), b) for b in range(1, B)], dtype=np.int32)
    if shape == "forest" and B > 2:
        p[B // 2] = -1
    return p


def ancestors(parent):
    seen = np.zeros((len(parent), len(parent)), dtype=bool)
    for b in range(len(parent)):
        c = b
        while c >= 0:
            seen[b, c] = True
            c = parent[c] if parent[c] < c else -1
    return seen


def pack(bits, words=None):
    """Truth values as int32 words, lowest bit first."""
    rows, n = bits.shape
    words = words or (n + 31) // 32
    full = np.zeros((rows, words * 32), dtype=np.uint8)
    full[:, :n] = bits
    return np.packbits(full, axis=1, bitorder="little").view(np.int32).copy()


def rotate(x, gamma, eps, inv_freq, layout, amplitude, pos):
    """x [B][H][D] (float64) normed and rotated."""
    x = x.astype(np.float64)
    if gamma is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * gamma.astype(np.float64)
    h = len(inv_freq)
    first, second = (np.arange(h), np.arange(h) + h) if layout == 0 else (2 * np.arange(h), 2 * np.arange(h) + 1)
    ang = pos.astype(np.float64)[:, None] * inv_freq[None]
    c, s = amplitude * np.cos(ang)[:, None], amplitude * np.sin(ang)[:, None]
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def attend(q, k, v, prefix, row0, sees):
    """q [B][Hq][D], k and v [Hkv][ts][D]; sees [B][B]; a node that sees nothing gets 0."""
    B, Hq, D = q.shape
    Hkv = k.shape[0]
    out = np.zeros((B, Hq, D))
    for b in range(B):
        at = np.concatenate([np.arange(prefix), row0 + np.flatnonzero(sees[b])])
        if not len(at):
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = k[g, at].astype(np.float64) @ q[b, h].astype(np.float64) / np.sqrt(D)
            w = np.exp(s - s.max())
            out[b, h] = w @ v[g, at].astype(np.float64) / w.sum()
    return out


def adjust(x, counts, rep, freq, pres, bias, allowed, t=np.float64):
    """Adjusted logits in type t, step by step."""
    x = x.astype(t)
    used = counts > 0
    y = np.where(x > 0, x / t(rep), x * t(rep))
    y = (y - t(freq) * counts.astype(t)) - t(pres)
    y = np.where(used, y, x)
    if bias is not None:
        y = y + bias.astype(t)
    if allowed is not None:
        y = np.where(allowed, y, t(-np.inf))
    return y


def choice(y):
    """Lowest index of the largest value above -inf, NaN left out; -1 if there is none."""
    z = np.where(np.isnan(y), -np.inf, y)
    return np.where(z.max(-1) > -np.inf, z.argmax(-1), -1).astype(np.int32)


def accept(parent, token, argmax):
    path = [0]
    while True:
        cur = path[-1]
        kids = [c for c in range(cur + 1, len(parent)) if parent[c] == cur and token[c] == argmax[cur]]
        if not kids:
            return path, [int(argmax[n]) for n in path]
        path.append(kids[0])
