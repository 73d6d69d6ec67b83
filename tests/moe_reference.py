"""Plain 64-bit statements of the mixture-of-experts operators, for the tests
(NumPy on the host; no code shared with the kernels)."""

import numpy as np

BLOCK = 128


def scores(x, softmax):
    """Scores of float64 logits; closed experts (not finite) score 0."""
    x = np.where(np.isfinite(x), x, -np.inf)
    if not softmax:
        with np.errstate(over="ignore"):
            return np.where(np.isfinite(x), 1.0 / (1.0 + np.exp(-x)), 0.0)
    top = x.max(1, keepdims=True)
    e = np.where(np.isfinite(x), np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
    s = e.sum(1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def choice_values(x, softmax, bias, group_top, by_logit):
    s = scores(x, softmax)
    c = np.array(x) if by_logit else s.copy()
    if bias is not None:
        c = c + bias
    return np.where(np.isfinite(x), c, -np.inf)


def route(x, k, *, softmax, bias=None, mask=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """(ids, weights, choice values after the groups' choice)."""
    x = np.asarray(x, dtype=np.float64)
    t, e = x.shape
    by_logit = softmax and bias is None and (group_top == 1 or groups == 1)
    c = choice_values(x, softmax, bias, group_top, by_logit)
    if groups > 1:
        by = c.reshape(t, groups, -1)
        best = -np.sort(-by, axis=2)[:, :, :group_top]
        value = np.where(np.isfinite(best), best, 0.0).sum(2)
        value = np.where(np.isfinite(best[:, :, 0]), value, -np.inf)
        order = np.argsort(-value, axis=1, kind="stable")[:, top_groups:]
        by = by.copy()
        np.put_along_axis(by, order[:, :, None], -np.inf, 1)
        c = by.reshape(t, e)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    ids = np.where(np.isfinite(np.take_along_axis(c, ids, 1)), ids, -1)
    if mask is not None:
        ids = np.where(mask[:, None] != 0, ids, -1)
    return ids, weights_of(x, ids, softmax=softmax, renorm=renorm, scale=scale), c


def weights_of(x, ids, *, softmax, renorm, scale):
    s = scores(np.asarray(x, dtype=np.float64), softmax)
    picked = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renorm:
        total = picked.sum(1, keepdims=True)
        picked = np.divide(picked, total, out=np.zeros_like(picked), where=total > 0)
    return picked * scale


def route_backward(x, ids, grad, *, softmax, renorm, scale):
    """Gradient of sum(weights * grad) by the logits, the choice held fixed."""
    x = np.asarray(x, dtype=np.float64)
    s = scores(x, softmax)
    live = ids >= 0
    at = np.maximum(ids, 0)
    p = np.where(live, np.take_along_axis(s, at, 1), 0.0)
    g = np.where(live, np.asarray(grad, dtype=np.float64) * scale, 0.0)
    if renorm:
        total = p.sum(1, keepdims=True)
        total = np.where(total > 0, total, np.inf)
        g = np.where(live, (g - (g * p).sum(1, keepdims=True) / total) / total, 0.0)
    full = np.zeros_like(x)
    for j in range(ids.shape[1]):
        rows = np.nonzero(live[:, j])[0]
        full[rows, ids[rows, j]] += g[rows, j]
    if softmax:
        return s * (full - (full * s).sum(1, keepdims=True))
    return full * s * (1.0 - s)


def plan(ids, experts):
    """(offsets, slots, pos) of flat ids."""
    ids = np.asarray(ids).reshape(-1)
    live = np.nonzero(ids >= 0)[0]
    order = live[np.argsort(ids[live], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[live], minlength=experts))])
    slots = np.full(ids.size, -1, dtype=np.int64)
    slots[:order.size] = order
    pos = np.full(ids.size, -1, dtype=np.int64)
    pos[order] = np.arange(order.size)
    return offsets, slots, pos


def exponent(amax):
    """Exponent of the least power of two 2^e with amax / 2^e <= 448."""
    m, e = np.frexp(np.asarray(amax, dtype=np.float64))
    out = np.where(amax > 0, e - 9 + (m > 0.875), 0)
    return np.clip(out, -127, 127).astype(np.int64)


def e4m3(v):
    """Values rounded to e4m3 (to nearest even), as float64; |v| <= 448."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.where(v == 0, 1.0, v))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(v / step) * step


def quantize(x, axis_blocks):
    """x split as (..., blocks, values of a block): (q values, exponents)."""
    e = exponent(np.abs(axis_blocks).max(-1))
    return e4m3(np.ldexp(axis_blocks, -e[..., None])), e


def pad_to(x, n, axis):
    width = [(0, 0)] * x.ndim
    width[axis] = (0, -x.shape[axis] % n)
    return np.pad(x, width)


def quantize_rows(x):
    r, d = x.shape
    q, e = quantize(x, pad_to(x, BLOCK, 1).reshape(r, -1, BLOCK))
    return q.reshape(r, -1)[:, :d], e + 127


def quantize_blocks(w):
    e, n, k = w.shape
    p = pad_to(pad_to(w, BLOCK, 1), BLOCK, 2)
    nb, kb = p.shape[1] // BLOCK, p.shape[2] // BLOCK
    b = p.reshape(e, nb, BLOCK, kb, BLOCK).transpose(0, 1, 3, 2, 4).reshape(e, nb, kb, -1)
    q, ex = quantize(w, b)
    q = q.reshape(e, nb, kb, BLOCK, BLOCK).transpose(0, 1, 3, 2, 4).reshape(e, nb * BLOCK, kb * BLOCK)
    return q[:, :n, :k], ex + 127


def quantize_cols(rows, offsets):
    """rows: [R, d] in row order; (q [d, used], scale bytes [used / 128, d])."""
    d = rows.shape[1]
    qs, ss = [np.zeros((0, d))], [np.zeros((0, d), dtype=np.int64)]
    for e in range(len(offsets) - 1):
        part = pad_to(rows[offsets[e]:offsets[e + 1]], BLOCK, 0)
        if part.shape[0]:
            b = part.reshape(-1, BLOCK, d).transpose(0, 2, 1)
            q, ex = quantize(part, b)
            qs.append(q.transpose(0, 2, 1).reshape(-1, d))
            ss.append(ex + 127)
    return np.concatenate(qs).T, np.concatenate(ss)


def rows_values(q, s):
    """FP8 values [r, d] with scale bytes [r, ceil(d / 128)] as float64."""
    return q * np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), BLOCK, axis=1)[:, :q.shape[1]]


def cols_values(q, s):
    """FP8 values [d, cap] with scale bytes [cap / 128, d] as float64."""
    return q * np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), BLOCK, axis=0).T


def padded_starts(offsets):
    return np.concatenate([[0], np.cumsum(-(-np.diff(offsets) // BLOCK))]) * BLOCK


def written_columns(offsets):
    """Which columns up to the last expert's end the column quantiser writes:
    each expert's rows, and on to the next multiple of 32."""
    starts = padded_starts(offsets)
    out = np.zeros(starts[-1], dtype=bool)
    for e in range(len(offsets) - 1):
        out[starts[e]:starts[e] + -(-(offsets[e + 1] - offsets[e]) // 32) * 32] = True
    return out
