"""Plain fp64 forms of the parts of a layer over packed sequences: causal conv, selective
scan, gated RMSNorm, dense projection (numpy, one row at a time, no chunks).

Besides each result y the functions return A, the same sum with every term replaced by
its magnitude: an fp32 evaluation in any order is off by at most a small count of
roundings times 2^-24 A, which the tests' tolerances are made of."""
import numpy as np

EPS = 1e-5


def f64(v):
    return np.asarray(v, dtype=np.float64)


def live_sequences(n_seqs, n_rows, start, slot, n_slots):
    """(s, first row, end row, slot) of every sequence that takes part, by the rules of the
    calls: slots outside the pool, slots named before and bad starts are left out."""
    seen, out = set(), []
    for s in range(n_seqs):
        sl = s if slot is None else int(slot[s])
        b, e = (s, s + 1) if start is None else (int(start[s]), int(start[s + 1]))
        twice = sl in seen
        if slot is not None:
            seen.add(sl)
        if n_slots is not None and (sl < 0 or sl >= n_slots or twice):
            continue
        if not 0 <= b <= e <= n_rows or b == e:
            continue
        out.append((s, b, e, sl))
    return out


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def softplus(v):
    with np.errstate(over="ignore"):
        return np.where(v > 20.0, v, np.log1p(np.exp(v)))


def conv(x, w, b, start, slot, fresh, state, act=True):
    """x [rows, C], w [C, W], state [slots, W-1, C] or None -> y (NaN where nothing is
    written), A, state after."""
    x, w = f64(x), f64(w)
    n_rows, C = x.shape
    W = w.shape[1]
    y, A = np.full((n_rows, C), np.nan), np.zeros((n_rows, C))
    new = None if state is None else np.array(state, dtype=np.float64)
    n_seqs = n_rows if start is None else len(start) - 1
    for s, lo, hi, sl in live_sequences(n_seqs, n_rows, start, slot if state is not None else None,
                                        None if state is None else len(state)):
        old = np.zeros((W - 1, C))
        if state is not None and not (fresh is not None and fresh[s]):
            old = f64(state[sl])
        line = np.concatenate([old, x[lo:hi]])
        for t in range(hi - lo):
            win = line[t:t + W]
            v = (win * w.T).sum(0) + (0.0 if b is None else f64(b))
            A[lo + t] = np.abs(win * w.T).sum(0) + (0.0 if b is None else np.abs(f64(b)))
            y[lo + t] = silu(v) if act else v
        if new is not None:
            new[sl] = line[hi - lo:]
    return y, A, new


def scan(x, dt, B, C, dt_bias, A_log, D, start, slot, fresh, state, shape=None):
    """x [rows, H*P], dt [rows, H], B, C [rows, G*N], state [slots, H, P, N] or None (then
    shape = (H, P, N, G)) -> y (NaN where nothing is written), A, state after, its A."""
    x, dt, B, C = f64(x), f64(dt), f64(B), f64(C)
    n_rows = x.shape[0]
    H, P, N = shape[:3] if state is None else state.shape[1:]
    G = B.shape[1] // N
    y, A = np.full((n_rows, H * P), np.nan), np.zeros((n_rows, H * P))
    new = None if state is None else np.array(state, dtype=np.float64)
    newA = None if state is None else np.abs(new)
    rate = -np.exp(f64(A_log))
    n_seqs = n_rows if start is None else len(start) - 1
    for s, lo, hi, sl in live_sequences(n_seqs, n_rows, start, slot if state is not None else None,
                                        None if state is None else len(state)):
        h = np.zeros((H, P, N))
        if state is not None and not (fresh is not None and fresh[s]):
            h = f64(state[sl]).copy()
        ha = np.abs(h)
        for t in range(lo, hi):
            step = softplus(dt[t] + f64(dt_bias))
            xt = x[t].reshape(H, P)
            Bt = np.repeat(B[t].reshape(G, N), H // G, axis=0)
            Ct = np.repeat(C[t].reshape(G, N), H // G, axis=0)
            keep = np.exp(step * rate)[:, None, None]
            add = (step[:, None] * xt)[:, :, None] * Bt[:, None, :]
            h = keep * h + add
            ha = keep * ha + np.abs(add)
            yt = (h * Ct[:, None, :]).sum(-1)
            ya = (ha * np.abs(Ct)[:, None, :]).sum(-1)
            if D is not None:
                yt = yt + f64(D)[:, None] * xt
                ya = ya + np.abs(f64(D)[:, None] * xt)
            y[t], A[t] = yt.ravel(), ya.ravel()
        if new is not None:
            new[sl], newA[sl] = h, ha
    return y, A, new, newA


def gated_norm(y, z, w, groups=1):
    g = f64(y)
    if z is not None:
        g = g * silu(f64(z))
    rows, cols = g.shape
    p = g.reshape(rows, groups, -1)
    return (p / np.sqrt((p * p).mean(-1, keepdims=True) + EPS)).reshape(rows, cols) * f64(w)


def dense(x, w, b, residual, act):
    """y and the magnitudes A of the product's own sum."""
    x, w = f64(x), f64(w)
    v = x @ w.T + (0.0 if b is None else f64(b))
    A = np.abs(x) @ np.abs(w).T + (0.0 if b is None else np.abs(f64(b)))
    if act:
        v = silu(v)
    if residual is not None:
        v = v + f64(residual)
    return v, A
