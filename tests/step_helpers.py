"""Plain 64-bit forms of the operators around the attention (page plan, norm + rotation and its
gradient, packed queries over a paged cache), for the tests of a serving or training step."""
from __future__ import annotations

import numpy as np

import oracle


# ------------------------------------------------------------------------------------------
# page plan
# ------------------------------------------------------------------------------------------

def page_plan(cached, fresh, table, free, head, P, num_pages, T):
    """(cu, used, positions, slots, head_out, table, bad) token by token, as the header states it."""
    B, width = table.shape
    cap = width * P
    table, bad = table.copy(), False
    cu, used, positions, slots = [0], [], [], []
    take = head

    def usable(pg):
        return pg if 0 <= pg < num_pages else -1

    for b in range(B):
        c, n = int(cached[b]), int(fresh[b])
        bad |= c < 0 or n < 0 or c + n > cap
        c, n = min(max(c, 0), cap), max(n, 0)
        old, total = -(-c // P), -(-min(c + n, cap) // P)
        for j in range(old, total):
            pg = usable(int(free[take])) if 0 <= take < len(free) else -1
            bad |= pg < 0
            table[b, j] = pg
            take += 1
        for pos in range(c, c + n):
            if pos >= cap:
                positions.append(-1)
                slots.append(-1)
                continue
            pg = usable(int(table[b, pos // P]))
            bad |= pg < 0 and len(slots) < T
            positions.append(pos)
            slots.append(-1 if pg < 0 else pg * P + pos % P)
        bad |= len(slots) > T
        cu.append(min(len(slots), T))
        used.append(min(c + n, cap))
    positions, slots = (x[:T] + [-1] * (T - len(x)) for x in (positions, slots))
    i32 = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return i32(cu), i32(used), i32(positions), i32(slots), take, table, bad


# ------------------------------------------------------------------------------------------
# norm + rotation
# ------------------------------------------------------------------------------------------

def angles(n, rot, base=10000.0):
    """cos, sin fp32 [n, rot / 2] from 64-bit angles."""
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def rotate(x, cos, sin, adjacent, back=False):
    """x [T, h, d] turned by each token's angles cos, sin [T, rot / 2]."""
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    c, s = cos[:, None].astype(np.float64), sin[:, None].astype(np.float64) * (-1 if back else 1)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, cos, sin, eps, adjacent):
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
    return rotate(y, cos, sin, adjacent)


def norm_rope_bwd(x, w, cos, sin, eps, adjacent, dy):
    """(dx, dw, sum |terms| of dw)."""
    g = rotate(dy, cos, sin, adjacent, back=True)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh = x * r
    dx = r * (g * w - xh * np.mean(g * w * xh, -1, keepdims=True))
    return dx, (g * xh).sum((0, 1)), np.abs(g * xh).sum((0, 1))


# ------------------------------------------------------------------------------------------
# packed queries over a paged cache
# ------------------------------------------------------------------------------------------

def gather(pool, table, used):
    """The keys (or values) [sum used, h_kv, d] that the sequences' tables stand for."""
    P = pool.shape[1]
    rows = [pool[table[b, np.arange(n) // P], np.arange(n) % P] for b, n in enumerate(used)]
    return np.concatenate(rows) if rows else pool.reshape(-1, *pool.shape[2:])[:0]


def attention(q, k_pool, v_pool, cu_q, used, table, *, scale, causal, window=(-1, -1), sinks=None):
    """O [T, h_q, d], LSE [h_q, T] and, for error bounds, sum_j p_ij |v_j|."""
    cu_k = np.concatenate([[0], np.cumsum(used)]).astype(np.int32)
    k, v = gather(k_pool, table, used), gather(v_pool, table, used)
    kw = dict(scale=scale, causal=causal, window=window, sinks=sinks, cu_q=np.asarray(cu_q, np.int32), cu_k=cu_k)
    o, lse, _ = oracle.fwd(q, k, v, **kw)
    spread, _, _ = oracle.fwd(q, k, np.abs(v), **kw)
    return o, lse, spread
