"""fp64 NumPy oracle of the paged softmax-attention calls: per-head norm and rotation,
appending to a paged cache, and attention of the new tokens over it.  Written from the
formulas in include/gdn.h, token by token; shares no code with the kernels.
"""

import numpy as np


def norm_rope_row(x, w, eps, cos_sin_row, interleaved):
    """One head vector x [D]; w [D] or None; cos_sin_row [r] (cosines, then sines) or None."""
    u = np.array(x, dtype=np.float64)
    if w is not None:
        u = u / np.sqrt(np.mean(u * u) + eps) * w
    if cos_sin_row is None:
        return u
    r = len(cos_sin_row)
    y = u.copy()
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c, s = cos_sin_row[i], cos_sin_row[i + r // 2]
        y[a] = u[a] * c - u[b] * s
        y[b] = u[b] * c + u[a] * s
    return y


def norm_rope(x, w, eps, cos_sin, positions, interleaved):
    """x [T, H, D]; cos_sin [P, r] or None; positions [T]."""
    x = np.asarray(x, dtype=np.float64)
    y = np.empty_like(x)
    for t in range(x.shape[0]):
        row = None if cos_sin is None else cos_sin[positions[t]]
        for h in range(x.shape[1]):
            y[t, h] = norm_rope_row(x[t, h], w, eps, row, interleaved)
    return y


def new_token_indices(cu, kv_lens):
    """(sequence, cache index) of each new token; (s, None) in an inactive sequence."""
    out = []
    for s in range(len(kv_lens)):
        n = int(cu[s + 1] - cu[s])
        for i in range(n):
            out.append((s, None if kv_lens[s] == 0 else int(kv_lens[s]) - n + i))
    return out


def append(cache_k, cache_v, k, v, block_table, cu, kv_lens):
    """Writes rows k, v [T, H, D] into caches [pages, H, P, D] (fp64 arrays, in place)."""
    P = cache_k.shape[2]
    for t, (s, p) in enumerate(new_token_indices(cu, kv_lens)):
        if p is None:
            continue
        page = block_table[s][p // P]
        cache_k[page, :, p % P] = k[t]
        cache_v[page, :, p % P] = v[t]


def attention(q, cache_k, cache_v, block_table, cu, kv_lens, scale, gate=None):
    """q [T, Nq, D] over caches [pages, H, P, D].  Returns (y, mass, smax): y [T, Nq, D]; for error
    bounds, mass = sum_j p_j |v_j| (times the gate) and smax [T, Nq] = max_j scale sum_i |q_i k_ji|."""
    q = np.asarray(q, dtype=np.float64)
    T, Nq, D = q.shape
    H, P = cache_k.shape[1], cache_k.shape[2]
    G = Nq // H
    y, mass, smax = np.zeros((T, Nq, D)), np.zeros((T, Nq, D)), np.zeros((T, Nq))
    rows = new_token_indices(cu, kv_lens)
    for t, (s, p) in enumerate(rows):
        if p is None:
            continue
        j = np.arange(p + 1)
        pages = np.asarray(block_table[s])[j // P]
        for h in range(H):
            K, V = cache_k[pages, h, j % P], cache_v[pages, h, j % P]
            for g in range(h * G, (h + 1) * G):
                x = scale * (K @ q[t, g])
                w = np.exp(x - x.max())
                w /= w.sum()
                y[t, g] = w @ V
                mass[t, g] = w @ np.abs(V)
                smax[t, g] = scale * (np.abs(K) @ np.abs(q[t, g])).max()
    if gate is not None:
        sg = 1.0 / (1.0 + np.exp(-np.asarray(gate, dtype=np.float64)))
        y, mass = y * sg, mass * sg
    return y, mass, smax
