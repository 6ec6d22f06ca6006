"""Plain 64-bit numpy implementations of the paged-cache operators, and the
tolerances of their outputs, for the tests."""
from __future__ import annotations

import numpy as np


def rotate(x, pos, theta):
    """Rows x [..., n, d] turned to positions pos [n] (half-split pairs)."""
    d = x.shape[-1]
    h = d // 2
    ang = np.asarray(pos, np.float64)[:, None] * theta ** (-2.0 * np.arange(h) / d)
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * c - b * s, a * s + b * c], -1)


def tree(parents):
    """(depth [T], attends [T, T]) of nodes with the given parents (-1: the last committed row)."""
    T = len(parents)
    up = np.zeros((T, T), bool)
    for t, p in enumerate(parents):
        up[t, t] = True
        if p >= 0:
            up[t] |= up[p]
    return up.sum(1) - 1, up


def gather(cache, pages, n):
    """Rows [0, n) of one request as [Hkv, n, d]."""
    ps = cache.shape[2]
    r = np.arange(n)
    return cache[np.asarray(pages)[r // ps], :, r % ps].transpose(1, 0, 2)


def attend(q, kcache, vcache, pages, L, parents, *, w0, w_pre, theta, scale, dtype):
    """One request: q [T, Hq, d] (float64), the fp64 caches.  Returns (out, tol),
    both [T, Hq, d].

    tol is an elementwise bound of the rounding a kernel of this dtype may do.
    A logit is off by at most e (natural units), a weight by a factor 1 +- 2 e (to
    first order, its own and the normaliser's), so the output by (2 e + w) sum_j
    p_j |v_j| + r |out|, where w covers the rounding of the weights and of the sums
    over keys, and r the final rounding.
      bf16: operands of the logits rounded to 11 bits (2^-11 each, relative to
        |q| |k| by Cauchy-Schwarz), the angles to 2^-20 (each of the two rotations),
        weights to bf16 (2^-8), result to bf16 (2^-8); fp32 sums add (n + d) 2^-24.
      fp32: products and sums of d terms (d + 8) 2^-24, angles 2^-21 each, weights
        and sums over n keys (n + 64) 2^-24, result 2^-24.
    """
    T, Hq, d = q.shape
    Hkv = kcache.shape[1]
    group = Hq // Hkv
    n = L + T
    depth, up = tree(parents)
    k, v = gather(kcache, pages, n), gather(vcache, pages, n)
    qpos = L + depth
    kpos = np.concatenate([np.arange(L), qpos])
    seen = np.concatenate([np.ones((T, L), bool), up], 1)
    out = np.empty((T, Hq, d))
    tol = np.empty((T, Hq, d))
    ke = rotate(k, kpos, theta)
    for t in range(T):
        i = qpos[t]
        G = max(1, -(-(i + 1) // w_pre))
        kr = rotate(k, kpos // G, theta)
        js = np.nonzero(seen[t])[0]
        near = i - kpos[js] < w0
        for h in range(Hq):
            g = h // group
            qe, qr = rotate(q[t, h][None], [i], theta)[0], rotate(q[t, h][None], [i // G], theta)[0]
            s = scale * np.where(near, ke[g][js] @ qe, kr[g][js] @ qr)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h] = p @ v[g][js]
            mass = p @ np.abs(v[g][js])
            big = scale * np.linalg.norm(q[t, h]) * np.linalg.norm(k[g][js], axis=1).max()
            if dtype == "bf16":
                e = big * (2 * 2.0 ** -11 + 2 * 2.0 ** -20 + d * 2.0 ** -24)
                tol[t, h] = (2 * e + 2.0 ** -8 + (n + d) * 2.0 ** -24) * mass + 2.0 ** -8 * np.abs(out[t, h])
            else:
                e = big * ((d + 8) * 2.0 ** -24 + 2 * 2.0 ** -21)
                tol[t, h] = (2 * e + (n + 64) * 2.0 ** -24) * mass + 2.0 ** -24 * np.abs(out[t, h])
    return out, tol


class Tables:
    """block_tables on Python lists: state of a page pool, stepped in place."""

    def __init__(self, table, lens, held, free, page_size):
        self.table = [list(r) for r in table]
        self.lens, self.held, self.free, self.ps = list(lens), list(held), list(free), page_size

    def step(self, grow, release, n_rows):
        B, wide, ps = len(self.lens), len(self.table[0]), self.ps
        for b in reversed(range(B)):
            if release[b]:
                for c in reversed(range(self.held[b])):
                    self.free.append(self.table[b][c])
                self.held[b] = self.lens[b] = 0
        avail, need_sum = len(self.free), 0
        status, slots, starts = [0] * B, [], [0]
        for b in range(B):
            pages = -(-(self.lens[b] + grow[b]) // ps)
            if pages > wide:
                status[b] = 2
            else:
                need = max(0, pages - self.held[b])
                need_sum += need
                if need and need_sum > avail:
                    status[b] = 1
                else:
                    for _ in range(need):
                        self.table[b][self.held[b]] = self.free.pop()
                        self.held[b] += 1
            for o in range(grow[b]):
                r = self.lens[b] + o
                slots.append(-1 if status[b] else self.table[b][r // ps] * ps + r % ps)
            starts.append(starts[-1] + grow[b])
        return slots + [-1] * (n_rows - len(slots)), starts, status
