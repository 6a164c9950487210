"""The operators around the sequential head in 64 bits -- TEST INFRASTRUCTURE ONLY.

Plain numpy definitions of the scaled lookup, the gated recurrence, the 4-bit
vocabulary product and the verification from probabilities, and of the first
two's gradients.  Inputs are float64 arrays that hold the operands' values.
Where a result is a sum or a recurrence, the function also returns a magnitude:
the same sum or recurrence over absolute values, from which the tests derive
how far a 32-bit evaluation may be off.
"""
from __future__ import annotations

import numpy as np


# ---- scaled lookup ------------------------------------------------------------
def embed(table, ids, scale):
    out = np.zeros((len(ids), table.shape[1]))
    for i, t in enumerate(ids):
        if 0 <= t < len(table):
            out[i] = scale * table[t]
    return out


def embed_grad(ids, drows, scale, dtable):
    """dtable + scale * sums; its magnitude; tokens summed per table row."""
    out, mag = dtable.copy(), np.abs(dtable)
    count = np.zeros(len(dtable), np.int64)
    for i, t in enumerate(ids):
        if 0 <= t < len(dtable):
            out[t] += scale * drows[i]
            mag[t] += np.abs(scale * drows[i])
            count[t] += 1
    return out, mag, count


# ---- gated recurrence ------------------------------------------------------------
def sigmoid(g):
    return 1.0 / (1.0 + np.exp(-g))


def gated_scan(gate, x, h0, lens):
    """(h, h_last, states before each step, magnitude recurrence before each
    step).  h is NaN past the end of a sequence."""
    B, T, D = gate.shape
    h = np.full((B, T, D), np.nan)
    before, mag = np.zeros((B, T, D)), np.zeros((B, T + 1, D))
    s = h0.copy()
    m = np.abs(h0)
    for t in range(T):
        before[:, t], mag[:, t] = s, m
        f, i = sigmoid(gate[:, t]), sigmoid(-gate[:, t])
        live = (lens > t)[:, None]
        with np.errstate(invalid="ignore"):
            s = np.where(live, f * s + i * x[:, t], s)
            m = np.where(live, f * m + i * np.abs(x[:, t]), m)
        h[:, t] = np.where(live, s, np.nan)
    mag[:, T] = m
    return h, s, before, mag


def gated_scan_error(gate, x, h0, lens, unit):
    """[B, T+1, D]: a bound for the error of the state before each step (and
    after the last) when every step is evaluated with relative error `unit` of
    its two terms: E_t = f E_{t-1} + unit (f M_{t-1} + i |x|), M the magnitude."""
    B, T, D = gate.shape
    _, _, _, mag = gated_scan(gate, x, h0, lens)
    e = np.zeros((B, T + 1, D))
    for t in range(T):
        f, i = sigmoid(gate[:, t]), sigmoid(-gate[:, t])
        live = (lens > t)[:, None]
        step = f * e[:, t] + unit * (f * mag[:, t] + i * np.abs(x[:, t]))
        e[:, t + 1] = np.where(live, step, e[:, t])
    return e


def gated_scan_grad(gate, x, h0, lens, dh, dh_last, unit=0.0):
    """(dgate, dx, dh0) and, for relative step errors `unit`, bounds of their
    errors laid out the same."""
    B, T, D = gate.shape
    _, _, before, mag = gated_scan(gate, x, h0, lens)
    eh = gated_scan_error(gate, x, h0, lens, unit)
    dg, dx = np.zeros((B, T, D)), np.zeros((B, T, D))
    eg, ex = np.zeros((B, T, D)), np.zeros((B, T, D))
    carry, cmag, cerr = dh_last.copy(), np.abs(dh_last), np.zeros((B, D))
    for t in reversed(range(T)):
        f, i = sigmoid(gate[:, t]), sigmoid(-gate[:, t])
        live = (lens > t)[:, None]
        d = np.where(live, dh[:, t], 0.0)  # padded steps may hold anything
        delta, dmag = carry + d, cmag + np.abs(d)
        derr = cerr + unit * dmag
        u, umag = before[:, t] - x[:, t], mag[:, t] + np.abs(x[:, t])
        dx[:, t] = np.where(live, delta * i, 0.0)
        dg[:, t] = np.where(live, delta * u * f * i, 0.0)
        ex[:, t] = np.where(live, i * (derr + unit * dmag), 0.0)
        eg[:, t] = np.where(live, f * i * (derr * umag + dmag * eh[:, t] + 3 * unit * dmag * umag), 0.0)
        carry = np.where(live, delta * f, carry)
        cmag = np.where(live, dmag * f, cmag)
        cerr = np.where(live, f * (derr + unit * dmag), cerr)
    return (dg, dx, carry), (eg, ex, cerr)


# ---- 4-bit vocabulary product -------------------------------------------------------
def w4_unpack(wq, r):
    """Codes [V, r] of the packed bytes, one by one from the layout's words."""
    V = wq.shape[0]
    codes = np.empty((V, r), np.int64)
    for k in range(r):
        w = (k % 128) // 8                         # word of eight features
        place = 4 * (w % 4) + w // 4               # where that word stands
        byte = wq[:, (k // 128) * 64 + 4 * place + (k % 8) // 2].astype(np.int64)
        codes[:, k] = byte % 16 if k % 2 == 0 else byte // 16
    return codes


def w4_pack(codes):
    V, r = codes.shape
    R = -(-r // 128) * 128
    wq = np.full((V, R // 2), 0x88, np.uint8)
    for k in range(r):
        w = (k % 128) // 8
        at = (k // 128) * 64 + 4 * (4 * (w % 4) + w // 4) + (k % 8) // 2
        c = codes[:, k].astype(np.uint8)
        wq[:, at] = (wq[:, at] & 0xF0) | c if k % 2 == 0 else (wq[:, at] & 0x0F) | (c << 4)
    return wq


def bias_w4(X, codes, wscale, group, base):
    """base + X . W and the sum of absolute terms."""
    W = (codes - 8) * np.repeat(wscale, group, axis=1)
    return base + X @ W.T, np.abs(base) + np.abs(X) @ np.abs(W).T


# ---- verification from probabilities --------------------------------------------------
def mass(p):
    p = np.asarray(p, np.float64)
    with np.errstate(invalid="ignore"):
        return np.where((p > 0) & (p < np.inf), p, 0.0)


def verify_probs(target, draft_probs, draft, u_accept, u_draw, verify_len=None):
    """(out, tau, p_draft, q_draft); rows with a negative length hold -9 / NaN."""
    B, K, V = draft_probs.shape
    out = np.full((B, K + 1), -1, np.int32)
    tau = np.zeros(B, np.int32)
    pd, qd = np.full((B, K), np.nan), np.full((B, K), np.nan)
    for b in range(B):
        kb = K if verify_len is None else min(int(verify_len[b]), K)
        if kb < 0:
            out[b], tau[b] = -9, -9
            continue
        j = 0
        while j < kb:
            d = draft[b, j]
            if not 0 <= d < V:
                break
            p, q = float(target[b, j, d]), float(draft_probs[b, j, d])
            pd[b, j], qd[b, j] = p, q
            if not float(u_accept[b, j]) * q < p:
                break
            out[b, j] = d
            j += 1
        m = mass(target[b, j])
        if j < kb:
            with np.errstate(invalid="ignore"):
                q = np.asarray(draft_probs[b, j], np.float64)
                res = np.maximum(m - np.where(q > 0, q, 0.0), 0.0)
            if res.sum() > 0:
                m = res
        cum = np.cumsum(m)
        if cum[-1] > 0:
            past = np.nonzero((cum > float(u_draw[b]) * cum[-1]) & (m > 0))[0]
            out[b, j] = past[0] if len(past) else np.nonzero(m)[0][-1]
            tau[b] = j + 1
        else:
            tau[b] = j
    return out, tau, pd, qd
