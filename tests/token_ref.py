"""float64 references of the operators on rows of logits and of the block norm seam, from their formulas (plain NumPy),
with the error bounds the GPU tests hold float32 arithmetic to.

Rounding steps are counted in u = 2^-24 (half a float32 step). A row sum of exponentials relative to the row's maximum
carries, relative to itself: the argument (two roundings of s d, so 2 u |s d| on each term, on average at most
2 u log V), the exponential (2 u), and the additions (at most 128 in sequence before the partial sums are joined in
pairs, 140 u). With log V <= 17 that is DZ = 176 u on Z, hence absolutely on log Z."""
import numpy as np

U = 2.0 ** -24
DZ = 176 * U
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step of the output's type, relative


def logprobs(z, s=1.0):
    """log p, p, H of each row (rows of -inf only: -inf, 0, 0)."""
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        m = z.max(1, keepdims=True)
        none = ~np.isnan(z).any(1, keepdims=True) & (m == -np.inf)
        d = np.where(none, -np.inf, (z - np.where(np.isnan(m), np.nan, m)) * s)
        e = np.exp(d)
        Z = e.sum(1, keepdims=True)
        lp = np.where(none, -np.inf, d - np.log(Z))
        p = np.where(none, 0.0, e / Z)
        H = -np.where(p == 0, 0.0, p * lp).sum(1)
    return lp, p, H


def top(z, K):
    """Places of the K largest of each row, equal ones by the lower place, NaN last."""
    z = np.asarray(z, np.float64)
    key = np.where(np.isnan(z), np.inf, -z)
    nan = np.isnan(z)
    return np.stack([np.lexsort((np.arange(z.shape[1]), k, n))[:K] for k, n in zip(key, nan)])


def logprobs_grad(z, s, ids, gl, gh):
    """dz and its float32 error bound (before the output's rounding)."""
    lp, p, H = logprobs(z, s)
    T, V = lp.shape
    gl = np.zeros(T) if gl is None else np.where((ids >= 0) & (ids < V), gl, 0.0).astype(np.float64)
    gh = np.zeros(T) if gh is None else np.asarray(gh, np.float64)
    lpc = np.where(p == 0, 0.0, lp)
    dz = -p * (gl[:, None] + gh[:, None] * (lpc + H[:, None]))
    for t in range(T):
        if gl[t] != 0:
            dz[t, ids[t]] += gl[t]
    dz[(gl == 0) & (gh == 0)] = 0.0
    dz[(lp == -np.inf).all(1)] = 0.0  # a row that holds nothing
    rel = DZ + 6 * U * (1 + np.abs(lpc))  # of p: the argument's roundings and the sum's
    dH = entropy_bound(z, s)[:, None]
    err = p * ((np.abs(gl)[:, None] + np.abs(gh)[:, None] * (np.abs(lpc) + H[:, None])) * (rel + 4 * U)
               + np.abs(gh)[:, None] * (DZ + 4 * U * np.abs(lpc) + dH))
    for t in range(T):
        if gl[t] != 0:
            err[t, ids[t]] += 2 * U * abs(gl[t])
    return dz * s, (err + U * np.abs(dz)) * s


def entropy_bound(z, s=1.0):
    """Absolute float32 error of log Z - S / Z: log Z's (DZ), and the sum S = sum e d, whose terms carry 2 u |d| + 3 u
    and whose additions carry 140 u, over Z's own error."""
    lp, p, H = logprobs(z, s)
    with np.errstate(all="ignore"):
        d = np.abs(np.where(p == 0, 0.0, lp - lp.max(1, keepdims=True)))
    m1, m2 = (p * d).sum(1), (p * d * d).sum(1)
    return DZ + U * (2 * m2 + 143 * m1) + DZ * m1 + 2 * U * (m1 + np.abs(H))


def distill(z, s, t_ids, t_z, ts, tail=False, t_lse=None, w=None):
    """loss, its bound, dz (or None), its bound."""
    lp, p, _ = logprobs(z, s)
    T, V = lp.shape
    K = t_ids.shape[1]
    loss, lerr = np.zeros(T), np.zeros(T)
    dz, derr = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        ok = [k for k in range(K) if 0 <= t_ids[t, k] < V]
        if not ok:
            continue
        a = np.array([float(t_z[t, k]) for k in ok]) * ts
        ids = np.array([t_ids[t, k] for k in ok])
        with np.errstate(all="ignore"):
            if tail:
                lq = a - (0.0 if t_lse is None else float(t_lse[t]))
            else:
                lq = a - a.max() - np.log(np.exp(a - a.max()).sum())
            q = np.exp(lq)
            live = q > 0
            loss[t] = (q[live] * (lq[live] - lp[t, ids][live])).sum()
            ab = np.where(live, np.abs(lq), 0) + np.where(live, np.abs(np.where(np.isfinite(lp[t, ids]), lp[t, ids], 0)), 0)
            lerr[t] = (q * (DZ + 8 * U * (1 + ab))).sum()
            g, e = p[t].copy(), p[t] * (DZ + 6 * U * (1 + np.abs(np.where(p[t] == 0, 0, lp[t]))))
            unl = np.ones(V, bool)
            unl[ids] = False
            if tail:
                qt = max(0.0, 1.0 - q.sum())
                pt = p[t][unl]
                lz = np.where(unl, lp[t], -np.inf)
                mt = lz.max() if unl.any() else -np.inf
                lpt = mt + np.log(np.exp(lz - mt).sum()) if mt > -np.inf else -np.inf
                if qt > 0:
                    loss[t] += qt * (np.log(qt) - lpt)
                # q_t is a float32 number of a sum of probabilities: 4 u absolutely
                lerr[t] += qt * (2 * DZ + 8 * U * (1 + abs(np.log(max(qt, 1e-300))) + (abs(lpt) if np.isfinite(lpt) else 0)))
                lerr[t] += 4 * U * (2 + abs(np.log(max(qt, U))) + (abs(lpt) if np.isfinite(lpt) else 0))
                if mt > -np.inf:
                    r = np.where(unl, np.exp(lz - lpt), 0.0)
                    g -= qt * r
                    e += r * (qt * (DZ + 8 * U * (1 + np.abs(np.where(unl & np.isfinite(lz), lz - lpt, 0)))) + 4 * U)
            np.add.at(g, ids, -q)
            np.add.at(e, ids, 6 * U * q)
        if w is not None and w[t] != 0 and np.isfinite(lp[t].max()):
            dz[t] = g * float(w[t]) * s
            derr[t] = (e + 4 * U * np.abs(g)) * abs(float(w[t])) * s
    return loss, lerr, dz, derr


def norm_fwd(h, y, gate, w_post, w_pre, res_scale, eps, gate_tokens, round_h):
    """h', x, (r_y, r_h) and the float32 bounds of h' and x. round_h rounds h' to the residual stream's type."""
    T, d = h.shape
    S = (3 * U + U * (np.log2(d) + d / 64 + 8)) / 2  # relative error of a root of a mean square: half its sum's
    ry = np.ones((T, 1))
    if y is None:
        ho, eh = h, np.zeros_like(h)
    else:
        b = y
        if w_post is not None:
            ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
            b = y * ry * w_post
        if gate is not None:
            b = b * gate[np.arange(T) // gate_tokens]
        ho = res_scale * h + b
        eh = np.abs(b) * (S + 5 * U) + np.abs(res_scale * h) * U + 2 * U * np.abs(ho)
    hr = round_h(ho)
    rh = 1 / np.sqrt((hr * hr).mean(1, keepdims=True) + eps)
    x = None if w_pre is None else hr * rh * w_pre
    ex = None if x is None else np.abs(x) * (S + 5 * U)
    return ho, eh, x, ex, ry, rh


def norm_bwd(h, y, gate, w_post, w_pre, ry, rh, dh_out, dx, res_scale, gate_tokens, tokens_in_seq):
    """{name: (value, float32 bound)} of the backward. tokens_in_seq: additions in sequence of a sum over tokens."""
    d = (h if h is not None else dh_out).shape[1]
    T = (h if h is not None else dh_out).shape[0]
    A = U * (np.log2(d) + d / 64 + 8)  # a row sum's additions, relative to the sum of the absolute terms
    out = {}
    t, et = (np.zeros((T, d)), np.zeros((T, d))) if dh_out is None else (dh_out.copy(), np.zeros((T, d)))
    if dx is not None:
        n, u = h * rh, dx * w_pre
        c, ec = (u * n).mean(1, keepdims=True), np.abs(u * n).mean(1, keepdims=True) * (A + 4 * U)
        t = t + rh * (u - n * c)
        et = et + rh * (3 * U * np.abs(u) + np.abs(n) * (ec + 4 * U * np.abs(c))) + 4 * U * (np.abs(rh * u) + np.abs(rh * n * c) + np.abs(t))
        q = dx * n
        out["dw_pre"] = (q.sum(0), np.abs(q).sum(0) * (tokens_in_seq + 4) * U)
    out["dh"] = (res_scale * t, abs(res_scale) * (et + U * np.abs(t)))
    G = 1.0 if gate is None else gate[np.arange(T) // gate_tokens]
    b = y * ry if w_post is not None else y
    W = 1.0 if w_post is None else w_post
    if gate is not None:
        rows = gate.shape[0]
        q, e = t * W * b, et * np.abs(W * b) + 4 * U * np.abs(t * W * b)
        at = np.arange(T) // gate_tokens
        v, ev = np.zeros((rows, d)), np.zeros((rows, d))
        np.add.at(v, at, q)
        np.add.at(ev, at, e + np.abs(q) * min(gate_tokens, tokens_in_seq) * U)
        out["dgate"] = (v, ev)
    v = t * G * W
    ev = et * np.abs(G * W) + 3 * U * np.abs(v)
    if w_post is not None:
        q = t * G * b
        out["dw_post"] = (q.sum(0), (et * np.abs(G * b)).sum(0) + np.abs(q).sum(0) * (tokens_in_seq + 5) * U)
        c = (v * b).mean(1, keepdims=True)
        ec = (ev * np.abs(b)).mean(1, keepdims=True) + np.abs(v * b).mean(1, keepdims=True) * (A + 4 * U)
        dy = ry * (v - b * c)
        edy = ry * (ev + np.abs(b) * (ec + 3 * U * np.abs(c))) + 4 * U * (np.abs(ry * v) + np.abs(ry * b * c))
    else:
        dy, edy = v, ev
    out["dy"] = (dy, edy)
    return out
