"""The losses on logits and the clipping in 64 bits (numpy), written from their
definitions row by row, with the error bounds the GPU tests allow.

Bounds (e = 2^-24, the fp32 rounding):
  y = (z - m) k takes a subtraction, a product and the rounding of k, so it is
  off by at most 3 e |y|; 2^y by 4 e more; the sum s of positive terms by the
  terms' weighted error and by e for each addition on a thread's chain (at most
  64 here, the rest is a tree): log-probabilities are off by at most
  e (8 |logp| + 8 |z_t - m| / tau + 128).
  A gradient term p (a + b y) takes the same errors in p, a and b.
"""
import numpy as np

E = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": E}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-37}


def rows_of(z, target, tau, live):
    """Per row: logp, lse, H, p and ln p (0 where p = 0); zeros where not live.
    A row of -inf alone: logp = lse = -inf, H = 0, p = 0."""
    R, V = z.shape
    out = dict(logp=np.zeros(R), lse=np.zeros(R), h=np.zeros(R), p=np.zeros((R, V)), lnp=np.zeros((R, V)),
               tol=np.zeros(R), hol=np.zeros(R), ymax=np.zeros(R), none=np.zeros(R, bool))
    for i in range(R):
        if not live[i]:
            continue
        x = z[i] / tau
        m = x.max()
        if m == -np.inf:
            out["logp"][i] = out["lse"][i] = -np.inf
            out["none"][i] = True
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            e = np.exp(x - m)
        s = e.sum()
        lse = m + np.log(s)
        p = e / s
        lnp = np.where(p > 0, (x - m) - np.log(s), 0.0)
        y = np.where(p > 0, x - m, 0.0)
        out["p"][i], out["lnp"][i] = p, lnp
        with np.errstate(over="ignore"):  # past fp32's range: infinite
            out["lse"][i] = lse if abs(lse) < 3.4028235e38 else np.float32(lse)
            lp = (x[target[i]] - m) - np.log(s)
            out["logp"][i] = lp if abs(lp) < 3.4028235e38 else np.float32(lp)
        out["h"][i] = -(p * lnp).sum()
        yt = abs(x[target[i]] - m)
        out["tol"][i] = E * (8 * min(abs(out["logp"][i]), 1e30) + 8 * min(yt, 1e30) + 128)
        out["hol"][i] = E * (8 * out["h"][i] + (p * (16 * np.abs(y) + 8 * y * y)).sum() + 256)
        out["ymax"][i] = np.abs(y).max()
    return out


def dlogits(r, target, live, g, gh, scale, tau, dg=None):
    """scale d(g logp + gh H)/dz and its bound (without the last rounding)."""
    R, V = r["p"].shape
    d, tol = np.zeros((R, V)), np.zeros((R, V))
    for i in range(R):
        if not live[i] or r["none"][i] or (g[i] == 0 and (gh is None or gh[i] == 0)):
            continue
        p, lnp, h = r["p"][i], r["lnp"][i], r["h"][i]
        one = np.zeros(V)
        one[target[i]] = 1
        a = gh[i] if gh is not None else 0.0
        d[i] = scale / tau * (g[i] * (one - p) - a * p * (lnp + h))
        rel = E * (16 * r["ymax"][i] + 512)
        tol[i] = abs(scale / tau) * (rel * p * (abs(g[i]) + abs(a) * (np.abs(lnp) + h + 1)) + 8 * E * abs(g[i]) * one)
        tol[i] += abs(scale / tau) * abs(a) * p * r["hol"][i]
        if dg is not None:
            tol[i] += abs(scale / tau) * dg[i] * (p + one)
    return d, tol


def policy(z, target, live, adv, old, ref, w, lo, hi, kl_coef, ent_coef, scale, tau):
    """adv, old, ref, w per row (w = 0 where not live)."""
    r = rows_of(z, target, tau, live)
    R = len(w)
    st, kl, g, gh, dg = np.zeros(5), np.zeros(R), np.zeros(R), np.zeros(R), np.zeros(R)
    stol = np.zeros(5)
    for i in range(R):
        if not live[i] or r["none"][i]:
            continue
        lp, a = r["logp"][i], adv[i]
        q = np.exp(lp - old[i])
        u, v = q * a, np.clip(q, 1 - lo, 1 + hi) * a
        pg = -min(u, v)
        dlp = -u if u <= v else 0.0
        tol = r["tol"][i] + 16 * E
        dg[i] = abs(u) * tol
        if ref is not None:
            d = ref[i] - lp
            kl[i] = np.exp(d) - d - 1
            dlp += kl_coef * (1 - np.exp(d))
            dg[i] += abs(kl_coef) * (np.exp(d) + 1) * tol
        h = r["h"][i]
        st += w[i] * np.array([pg + kl_coef * kl[i] - ent_coef * h, pg, kl[i], h, float(u > v)])
        ekl = (np.exp(ref[i] - lp) + 1 + abs(ref[i] - lp)) * tol if ref is not None else 0.0
        stol += abs(w[i]) * np.array([abs(pg) * tol + abs(kl_coef) * ekl + abs(ent_coef) * r["hol"][i] +
                                      4 * E * (abs(pg) + abs(kl_coef * kl[i]) + abs(ent_coef) * h),
                                      abs(pg) * tol, ekl, r["hol"][i], 4 * E])
        g[i], gh[i] = w[i] * dlp, -w[i] * ent_coef
        dg[i] = abs(w[i]) * dg[i] + 8 * E * abs(g[i])
    d, tol = dlogits(r, target, live, g, gh if ent_coef else None, scale, tau, dg)
    return dict(r=r, stats=st, stol=stol + 2 * E * np.abs(st), kl=kl, d=d, tol=tol)


def preference(z, target, live, off, ref, pw, kind, beta, smooth, average, scale, tau):
    r = rows_of(z, target, tau, live)
    pairs = (len(off) - 1) // 2
    l, n, lt = np.zeros(2 * pairs), np.zeros(2 * pairs), np.zeros(2 * pairs)
    for k in range(2 * pairs):
        for i in range(off[k], off[k + 1]):
            if live[i]:
                n[k] += 1
                if not r["none"][i]:
                    l[k] += r["logp"][i]
                    lt[k] += r["tol"][i]
        if average and n[k]:
            l[k] /= n[k]
            lt[k] /= n[k]
    h = (l[0::2] - ref[0::2]) - (l[1::2] - ref[1::2])
    ht = lt[0::2] + lt[1::2]
    x = beta * h
    if kind == "sigmoid":
        f = (1 - smooth) * np.logaddexp(0, -x) + smooth * np.logaddexp(0, x)
        df = beta * (smooth / (1 + np.exp(-x)) - (1 - smooth) / (1 + np.exp(x)))
        d2 = np.full(pairs, beta * beta / 4)
    elif kind == "hinge":
        f, df, d2 = np.maximum(0, 1 - x), np.where(x < 1, -beta, 0.0), np.zeros(pairs)
    else:
        f, df, d2 = (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta), np.full(pairs, 2.0)
    ft = (np.abs(df) + d2 * ht) * ht + 4 * E * np.abs(f)
    g, dg = np.zeros(len(z)), np.zeros(len(z))
    for k in range(2 * pairs):
        b = k // 2
        for i in range(off[k], off[k + 1]):
            share = (n[k] if average and n[k] else 1)
            g[i] = pw[b] * df[b] * (1 if k % 2 == 0 else -1) / share
            dg[i] = abs(pw[b]) * d2[b] * ht[b] / share + 8 * E * abs(g[i])
    d, tol = dlogits(r, target, live, g, None, scale, tau, dg)
    return dict(r=r, l=l, ltol=lt + 2 * E * np.abs(l), f=f, ftol=ft, loss=float((pw * f).sum()),
                losstol=float((np.abs(pw) * ft).sum() + 4 * E * (np.abs(pw) * np.abs(f)).sum()), d=d, tol=tol)


def close(got, want, tol, what=""):
    """|got - want| <= tol, the same NaN and infinities."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = np.broadcast_to(np.asarray(tol, np.float64), want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), f"{what}: other infinities"
    off = np.abs(got[fin] - want[fin])
    bad = off > tol[fin]
    assert not bad.any(), f"{what}: {bad.sum()} values off, worst {off[bad].max()} where {tol[fin][bad][off[bad].argmax()]} is allowed"
