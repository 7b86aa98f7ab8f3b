"""Float64 forms of the operators around a chunk of new tokens
(include/mla_chunk.h), with bounds on the 32-bit arithmetic of the kernels.

U is half a step of f32 and BF16 of bf16, relative to the value.  A score is a
sum of 576 exact products whose additions may each round, or truncate, to 32
bits (2 U of the sum of magnitudes so far, at most 576 of them)."""
import numpy as np

U, BF16 = 2.0 ** -24, 2.0 ** -8


def seen(length: int, count: int, causal: bool = True) -> np.ndarray:
    """Rows that each of a request's `count` new tokens sees."""
    j = np.arange(count)
    return np.clip(length - count + j + 1, 0, length) if causal else np.full(count, length)


def scores(q, rows, scale):
    """(s, t): q [n, H, 576] against rows [T, 576], and the bound on an error
    of s: the additions, and the product with the scale in the exponent's base
    (three roundings of it)."""
    s = scale * np.einsum("jhd,td->jht", q, rows)
    size = scale * np.einsum("jhd,td->jht", np.abs(q), np.abs(rows))
    return s, 576 * 2 * U * size + 4 * U * np.abs(s)


def attend(q, rows, scale, causal=True):
    """(o, t_o, lse, t_lse) of one request: q [n, H, 576], rows [T, 576]."""
    n, heads = q.shape[:2]
    o, t_o = np.zeros((n, heads, 512)), np.zeros((n, heads, 512))
    lse, t_lse = np.full((n, heads), -np.inf), np.zeros((n, heads))
    for j, m in enumerate(seen(len(rows), n, causal)):
        if m == 0:
            continue
        s, t = scores(q[j:j + 1], rows[:m], scale)
        s, t = s[0], t[0]
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        total = p.sum(-1, keepdims=True)
        lse[j] = top[:, 0] + np.log(total[:, 0])
        p /= total
        c = rows[:m, :512]
        # each weight is off by its score's error, the exponential's (4 U) and,
        # in the product with the rows and in the sum that divides it, bf16's
        # rounding; both sums round once a row or part (2 U) and once for each
        # rescaling, of which there are fewer than rows
        off = t + 4 * U
        e = (p * off).sum(-1)
        o[j] = p @ c
        grow = 2 * BF16 + 2 * e[:, None] + (4 * m + 64) * U
        t_o[j] = (p * off) @ np.abs(c) + grow * (p @ np.abs(c))
        t_lse[j] = e + (m + 64) * U + 4 * U * np.abs(lse[j])
    return o, t_o, lse, t_lse


def weights(q, lse, rows, scale, causal=True):
    """(w, t) [T]: the weight that each row gets from the request's queries."""
    n, heads = q.shape[:2]
    w, t_w = np.zeros(len(rows)), np.zeros(len(rows))
    for j, m in enumerate(seen(len(rows), n, causal)):
        s, t = scores(q[j:j + 1], rows[:m], scale)
        z = lse[j][:, None]
        with np.errstate(invalid="ignore"):
            p = np.where(np.isneginf(z), 0.0, np.exp(s[0] - z))
            off = np.where(np.isneginf(z), 0.0, t[0] + 4 * U * np.abs(z) + 4 * U)
        w[:m] += p.sum(0)
        t_w[:m] += (p * off).sum(0)
    return w, t_w + (n * heads + 64) * U * w


def evict(w, positions, budget, sinks=0, recent=0):
    """(kept, origin): how many rows stay of a request's len(w), and the slot
    that each of their slots is filled from."""
    n = len(w)
    kept = min(n, budget)
    origin = np.arange(kept)
    if n <= budget:
        return kept, origin
    newest = int(positions.max())
    key = []
    for t in range(n):
        safe = positions[t] < sinks or int(positions[t]) > newest - recent
        value = float(w[t])
        key.append((0, 0.0, t) if safe else (2, 0.0, t) if np.isnan(value) else (1, -value, t))
    best = [k[2] for k in sorted(key)[:budget]]
    stay = set(best)
    movers = sorted(t for t in best if t >= budget)
    holes = [t for t in range(budget) if t not in stay]
    origin[holes] = movers
    return kept, origin
