"""Plain forms of the speculative-decoding and state-pool operators, for the tests: whole numbers
for the verification of drafted tokens, fp64 for the decode step over drafted tokens, Python lists
for the slots of a pool. Written from the definitions in include/sala_gla.h."""
from fractions import Fraction

import numpy as np
import torch

UNIT = 2.0 ** 43   # probabilities count as whole numbers of 2^-43


def _probability(p):
    """p taken into [0, 1]; NaN, which compares false, counts as 0."""
    return np.where(p > 0, np.minimum(p, 1.0), 0.0)


def _units(p):
    """fp64 array of probabilities -> whole numbers of 2^-43, at most 2^43 each: 2^20 of them sum to 2^63,
    which takes unsigned 64-bit sums."""
    return np.rint(_probability(p) * UNIT).astype(np.uint64)


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def verify_drafts(p, q, x, u, s, num_drafts=None):
    """(tokens [N, K + 1], accepted [N]) of torch tensors p [N, K + 1, V], q [N, K, V] or None,
    x [N, K], u [N, K], s [N]."""
    N, K1, V = p.shape
    K = K1 - 1
    tokens = np.full((N, K1), -1, np.int64)
    accepted = np.zeros(N, np.int64)
    for n in range(N):
        count = K if num_drafts is None else min(K, max(0, int(num_drafts[n])))
        a, rejected = 0, False
        while a < count:
            t = int(x[n, a])
            if t < 0 or t >= V:
                break
            qx = 1.0 if q is None else _probability(float(q[n, a, t]))
            if not float(u[n, a]) * qx < _probability(float(p[n, a, t])):
                rejected = True
                break
            tokens[n, a] = t
            a += 1
        accepted[n] = a
        target = _units(_f64(p[n, a]))
        w = target
        if rejected:
            if q is None:
                less = np.zeros(V, np.uint64)
                less[int(x[n, a])] = int(UNIT)
            else:
                less = _units(_f64(q[n, a]))
            w = np.maximum(target, less) - less
            if w.sum() == 0:
                w = target
        total = int(w.sum())
        if total:
            at = float(s[n])
            at = min(at, float(np.nextafter(np.float32(1), np.float32(0)))) if at >= 0 else 0.0
            bound = Fraction(at) * total
            cum = np.cumsum(w)
            # the first sum above the bound: sums are whole, so compare with its whole part
            tokens[n, a] = int(np.searchsorted(cum, np.uint64(bound.numerator // bound.denominator), side="right"))
    return tokens, accepted


def draft_step(q, k, v, g, scale, S, pending=None, commits=0, tokens=None):
    """One (sequence, head): q, k, v [T, 128], g [T], S [128, 128], pending (k, v, g) of which
    `commits` are added. Returns o [T, 128] (zeros past `tokens`), the committed state, both fp64."""
    S = np.asarray(S, np.float64).copy()
    for j in range(commits):
        with np.errstate(over="ignore"):
            S = np.exp(float(pending[2][j])) * S + np.outer(pending[0][j], pending[1][j])
    kept = S.copy()
    T = 0 if q is None else len(q)
    o = np.zeros((T, 128))
    for t in range(T if tokens is None else tokens):
        S = np.exp(float(g[t])) * S + np.outer(k[t], v[t])
        o[t] = scale * (q[t] @ S)
    return o, kept


def fork(used, parents):
    """(children, the mask after it) of a mask and the requests' parents."""
    used = [int(x != 0) for x in used]
    before, children = list(used), []
    for p in parents:
        ok = p == -1 or (0 <= p < len(used) and before[p])
        child = -1
        if ok and 0 in used:
            child = used.index(0)
            used[child] = 1
        children.append(child)
    return children, used


def compact(used):
    """(moves [(from, to)], mapping, live count) of a mask."""
    m = sum(1 for x in used if x)
    holes = [s for s in range(m) if not used[s]]
    movers = [s for s in range(m, len(used)) if used[s]]
    moves = list(zip(movers, holes))
    mapping = [s if x else -1 for s, x in enumerate(used)]
    for a, b in moves:
        mapping[a] = b
    return moves, mapping, m
