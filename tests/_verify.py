"""Plain float64 reference of verify_tree, sequence by sequence."""
import numpy as np


def clean(row):
    x = np.asarray(row, np.float64).copy()
    with np.errstate(invalid="ignore"):
        x[~(np.isfinite(x) & (x > 0))] = 0.0
    return x


def walk(tokens, parents, nodes, p, q, r, u, most):
    """One sequence: (accepted nodes, next token)."""
    if nodes == 0:
        return [], -1
    path, at, start = [0], 0, 1
    P, Q, Z, Y = clean(p[0]), None if q is None else clean(q[0]), 1.0, 1.0
    while len(path) < most:
        c = next((t for t in range(start, nodes) if parents[t] == at), None)
        if c is None:
            break
        start, x = c + 1, int(tokens[c])
        if float(r[c]) * (1.0 if q is None else Q[x]) * Z < P[x] * Y:
            path.append(c)
            at = c
            P, Q, Z, Y = clean(p[c]), None if q is None else clean(q[c]), 1.0, 1.0
            continue
        if q is None:
            P[x] = 0.0
        else:
            P = np.maximum(P - (Z / Y if Y > 0 else 0.0) * Q, 0.0)
            Q[x] = 0.0
            Y = Q.sum()
        Z = P.sum()
    if not P.sum() > 0:
        P = clean(p[at])
    if not P.sum() > 0:
        return path, -1
    sums = np.cumsum(P)
    over = np.flatnonzero(sums > float(u) * sums[-1])
    return path, int(over[0]) if len(over) else int(np.flatnonzero(P > 0)[-1])


def verify(tokens, parents, nodes, p, q, r, u, most):
    B = len(tokens)
    idx, count, nxt = np.full((B, most), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        path, nxt[b] = walk(tokens[b], parents[b], int(nodes[b]), p[b], None if q is None else q[b], r[b], u[b], most)
        idx[b, :len(path)] = path
        count[b] = len(path)
    return idx, count, nxt
