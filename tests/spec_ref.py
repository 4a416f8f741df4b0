"""Plain implementations of the operators of a speculative decoding step, for the
tests (CPU only).  Appending is fixed to the bit: every step below is one rounding
to fp32 of a 64-bit operation on fp32 values, which is the correctly rounded fp32
operation (53 bits are more than twice 24 and two).  Verification is token by
token in 64 bits."""
import math

import numpy as np
import torch


def places(starts, T, lens):
    """Of every token: sequence, node, cached token (or None outside every sequence)."""
    out = [None] * T
    for b in range(len(starts) - 1):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            out[starts[b] + i] = (b, i, lens[b] - n + i)
    return out


def cache_row(table, page, S, b, token):
    if token < 0 or token // page >= table.shape[1]:
        return -1
    pg = int(table[b][token // page])
    return pg * page + token % page if 0 <= pg < S // page else -1


def _r(x):
    return x.float().double()


def turned(x, cos, sin, pos, inter, norm, w, eps):
    """x [T][H][D] of a 16-bit type, turned by its tokens' positions, in that type."""
    D, rot = x.shape[2], 2 * cos.shape[1]
    y = x.double()
    if norm:
        ms = _r((y * y).sum(-1, keepdim=True) / D)
        r = _r(1.0 / _r(torch.sqrt(_r(ms + float(np.float32(eps))))))
        y = _r(y * r)
        if w is not None:
            y = _r(y * w.double())
    c, s = (t.double()[pos.long().clamp(0, cos.shape[0] - 1)][:, None, :] for t in (cos, sin))
    ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    out = y.clone()
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = _r(_r(a * c) - _r(b * s)), _r(_r(b * c) + _r(a * s))
    return out.float().to(x.dtype)


def probabilities(row, t):
    """(likeliest token, probabilities in float64) of a row of logits, or None."""
    x = np.asarray(row, np.float64)
    if np.isnan(x).any() or not np.isfinite(x.max()):
        return None
    top = int(np.argmax(x))
    if not t > 0:
        return top, None
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(np.isneginf(x), 0.0, np.exp(np.where(np.isneginf(x), 0.0, x - x.max()) / np.float64(np.float32(t))))
    return top, w


def take(w, u):
    """The first token whose cumulated weight is above u of the whole."""
    cdf = np.cumsum(w)
    at = int(np.searchsorted(cdf, np.float64(np.float32(u)) * cdf[-1], side="right"))
    return min(at, int(np.nonzero(w > 0)[0][-1]))


def verify(logits, tokens, uniform, starts, width, parents=None, draft=None, temperature=None):
    """(out_tokens, path, counts) as lists of rows; logits float64 arrays [T][V]."""
    outs, paths, counts = [], [], []
    V = logits.shape[1]
    for b in range(len(starts) - 1):
        q0, n = starts[b], min(starts[b + 1] - starts[b], width)
        t = 1.0 if temperature is None else float(temperature[b])
        out, path, node = [], [], 0
        while n > 0:
            path.append(node)
            row = q0 + node
            d = probabilities(logits[row], t)
            if draft is not None:
                if d is None:
                    out.append(-1)
                    break
                top, w = d
                if node == n - 1:
                    out.append(top if w is None else take(w, uniform[q0]))
                    break
                x = int(tokens[row + 1])
                if w is None:
                    if x == top:
                        out.append(x)
                        node += 1
                        continue
                    out.append(top)
                    break
                e = probabilities(draft[row], t)
                if e is None:
                    out.append(-1)
                    break
                p, q = w / w.sum(), e[1] / e[1].sum()
                if 0 <= x < V and np.float64(np.float32(uniform[row + 1])) * q[x] < p[x]:
                    out.append(x)
                    node += 1
                    continue
                left = np.maximum(p - q, 0)
                out.append(take(left if left.sum() > 0 else p, uniform[q0]))
                break
            x = -1 if d is None else d[0] if d[1] is None else take(d[1], uniform[row])
            out.append(x)
            if x < 0:
                break
            nxt = [i for i in range(node + 1, n) if (i - 1 if parents is None else int(parents[q0 + i])) == node and int(tokens[q0 + i]) == x]
            if not nxt:
                break
            node = nxt[0]
        outs.append(out + [-1] * (width - len(out)))
        paths.append(path + [-1] * (width - len(path)))
        counts.append(len(path))
    return outs, paths, counts


def random_tree(rng, n, width=4):
    """Parents of n nodes (the root's: -1) and, per node, its ancestors and itself."""
    parents, sees = [-1], [{0}]
    for i in range(1, n):
        p = int(rng.integers(max(0, i - width), i))
        parents.append(p)
        sees.append(sees[p] | {i})
    return parents, sees


def mask_words(sees, words):
    """Rows of sets of nodes as int64 mask words."""
    out = np.zeros((len(sees), words), np.uint64)
    for i, s in enumerate(sees):
        for j in s:
            out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64))


def depth_of(parents):
    out = []
    for p in parents:
        out.append(0 if p < 0 else out[p] + 1)
    return out


assert math.isclose(probabilities([0.0, 0.0], 1.0)[1].sum(), 2.0)
