"""The verification of drafted tokens in 64 bits (numpy), row by row from its rules.

Bound of a log-probability: as in loss_ref, e (8 |logp| + 8 |z_t - m| / tau + 128), e = 2^-24.
"""
import numpy as np

E = 2.0 ** -24


def log_softmax(z, tau):
    """ln p of a row, or None where it has no distribution."""
    if np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        return None
    x = (z - z.max()) / tau
    with np.errstate(divide="ignore"):
        return x - np.log(np.exp(x).sum())


def draw(r, noise):
    """argmax r / E, the lowest index of equal ones; -1 where r is nothing."""
    e = np.where(noise > 2.0 ** -126, noise, 2.0 ** -126)  # (NaN and what is not positive, too)
    if not (r > 0).any():
        return -1
    return int(np.argmax(r / e))


def verify(z, tokens, off, u=None, noise=None, zd=None, greedy=False, tau=1.0, tau_d=1.0):
    """accepted [seqs], tokens [rows] (None: left as it was), logp, its bound, the error
    word's bits (16: no distribution, 32: a token past the vocabulary)."""
    rows, vocab = z.shape
    accepted, out, logp, tol, bits = [], [None] * rows, [None] * rows, np.zeros(rows), 0
    for b, (lo, hi) in enumerate(zip(off, off[1:])):
        lo, hi = (min(max(int(v), 0), rows) for v in (lo, hi))
        n = 0
        if hi <= lo:
            accepted.append(0)
            continue
        for i in range(lo, hi):
            lp = log_softmax(z[i], tau)
            if lp is None:
                bits |= 16
                new = -1
                break
            if i == hi - 1:
                new = int(np.argmax(z[i])) if greedy else draw(np.exp(lp), noise[b])
                break
            x = int(tokens[i])
            if x >= vocab:
                bits |= 32
            if greedy:
                if x == int(np.argmax(z[i])):
                    ok = True
                else:
                    new = int(np.argmax(z[i]))
                    break
            elif not 0 <= x < vocab:
                new = draw(np.exp(lp), noise[b])
                break
            else:
                q = np.zeros(vocab)
                q[x] = 1
                if zd is not None:
                    lq = log_softmax(zd[i], tau_d)
                    if lq is None:
                        bits |= 16
                        new = draw(np.exp(lp), noise[b])
                        break
                    q = np.exp(lq)
                ok = u[i] * q[x] < np.exp(lp[x])
                if not ok:
                    new = draw(np.maximum(np.exp(lp) - q, 0), noise[b])
                    if new < 0:
                        new = draw(np.exp(lp), noise[b])
                    break
            out[i], logp[i] = x, lp[x]
            tol[i] = E * (8 * abs(lp[x]) + 8 * abs(z[i, x] - z[i].max()) / tau + 128)
            n += 1
        i = lo + n
        out[i], logp[i] = new, np.nan if new < 0 else lp[new]
        if new >= 0:
            tol[i] = E * (8 * abs(lp[new]) + 8 * abs(z[i, new] - z[i].max()) / tau + 128)
        for k in range(i + 1, hi):
            out[k], logp[k] = -1, 0.0
        accepted.append(n)
    return accepted, out, logp, tol, bits
