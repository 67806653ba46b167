"""Reference of the packed gated delta rule's tests, in plain Python and
float64: the plan as its header describes it, and the rule by blocks with a
bound on what the kernels' roundings can add up to.

Bounds. A rounding is off by at most half a step, relative to the value: bf16
2^-8, fp32 2^-24 (H, F below). Errors E of a state pass on through the exact
recurrence X -> X prod g (I - b k k^T), which stretches nothing when b |k|^2
<= 2, so the errors that the tokens (blocks) add are summed as Frobenius norms.
"""
from __future__ import annotations

import numpy as np

H, F = 2.0 ** -8, 2.0 ** -24
FAULT_ROWS, FAULT_FREE, FAULT_SLOT, FAULT_OWNER, FAULT_STATE, FAULT_OVERFLOW = 1, 2, 4, 8, 16, 32


def plan(lengths, seen, slots, free, free_count, pool, rows):
    """The plan of a step, request by request. Returns a dict of lists; slots,
    free stack and count as they are afterwards."""
    R = len(lengths)
    free, slots = list(free), list(slots)
    count = min(max(free_count, 0), pool)
    offsets = [0]
    for n in lengths:
        offsets.append(min(offsets[-1] + max(n, 0), rows + 1))
    fits = [offsets[r + 1] <= rows for r in range(R)]
    faults, owner, mine = 0, {}, [False] * R
    for r, s in enumerate(slots):
        if 0 <= s < pool:
            mine[r] = s not in owner
            owner.setdefault(s, r)
            if not mine[r]:
                faults |= FAULT_OWNER
        elif s != -1:
            faults |= FAULT_SLOT
    now = list(slots)
    for r in range(R):
        if lengths[r] > 0 and not fits[r]:
            faults |= FAULT_ROWS
        if lengths[r] > 0 and slots[r] == -1 and seen[r] != 0:
            faults |= FAULT_STATE
        if lengths[r] < 0 and mine[r]:
            if count < pool:
                free[count] = slots[r]
                count += 1
            else:
                faults |= FAULT_OVERFLOW
            del owner[slots[r]]
            now[r] = -1
    use = [-1] * R
    for r in range(R):
        if lengths[r] > 0 and slots[r] == -1 and seen[r] == 0 and fits[r]:
            if count == 0:
                faults |= FAULT_FREE
                continue
            count -= 1
            s = free[count]
            if not 0 <= s < pool:
                faults |= FAULT_SLOT
            elif s in owner:
                faults |= FAULT_OWNER
            else:
                owner[s] = r
                now[r] = use[r] = s
        elif lengths[r] > 0 and mine[r] and fits[r]:
            use[r] = slots[r]
    key = [((lengths[r] + 31) // 32).bit_length() if use[r] >= 0 else 0 for r in range(R)]
    treq, tpos = [-1] * rows, [-1] * rows
    for r in range(R):
        if lengths[r] > 0 and fits[r]:
            for i in range(lengths[r]):
                treq[offsets[r] + i] = r
                tpos[offsets[r] + i] = seen[r] + i
    return dict(counts=[min(offsets[R], rows), sum(u >= 0 for u in use), count, faults], offsets=offsets, state_slots=use,
                order=sorted(range(R), key=lambda r: -key[r]), token_request=treq, token_position=tpos,
                slots=now, free_slots=free, free_count=[count])


def rule_by_blocks(q, k, v, g, b, X, C=32):
    """One request's head in blocks of C tokens: q, k [T, dk], v [T, dv], g, b
    [T], X [dv, dk]. Returns (o, X, bound on |o - its bf16 result| per value,
    bound on the Frobenius norm of the state's error) for the blockwise
    kernel: X, R, T and U in two bf16 parts (each split off by H^2), the lower
    parts' product dropped (H^2), X of the output and P in one (H), sums of
    fp32 products (64 F covers the longest, 128 terms by eight accumulations
    of 16, with the decay products and the inverse's 32 or 64
    steps)."""
    T = len(g)
    o, bo, E = np.zeros((T, v.shape[1])), np.zeros((T, v.shape[1])), 0.0
    e = H * H + 64 * F
    X = X.copy()
    for t0 in range(0, T, C):
        s = slice(t0, min(t0 + C, T))
        n = s.stop - s.start
        qq, kk, vv, gg, bb = q[s], k[s], v[s], g[s], b[s]
        D = np.zeros((n, n))
        for j in range(n):
            D[j:, j] = np.cumprod(np.concatenate([[1.0], gg[j + 1:]]))
        G = np.cumprod(gg)
        A = np.tril(bb[:, None] * D * (kk @ kk.T), -1)
        Ti = np.linalg.inv(np.eye(n) + A)
        P = np.tril(D * (qq @ kk.T))
        Z = kk @ X.T
        R = bb[:, None] * (vv - G[:, None] * Z)
        U = Ti @ R
        o[s] = G[:, None] * (qq @ X.T) + P @ U
        # what the block's roundings add
        aX, aK, aQ = np.abs(X), np.abs(kk), np.abs(qq)
        dR = np.abs(bb * G)[:, None] * e * (aK @ aX.T) + 4 * F * np.abs(bb)[:, None] * (np.abs(vv) + np.abs(G)[:, None] * (aK @ aX.T))
        aT = np.abs(Ti)
        dT = 64 * F * aT @ (np.tril(np.abs(bb)[:, None] * np.abs(D) * (aK @ aK.T), -1) + np.eye(n)) @ aT
        dU = aT @ dR + (2 * H * H + e) * aT @ np.abs(R) + dT @ np.abs(R)
        DC = D[n - 1]
        loc = (dU * np.abs(DC)[:, None]).T @ aK + e * (np.abs(U) * np.abs(DC)[:, None]).T @ aK + 4 * F * np.abs(G[-1]) * aX
        aP = np.abs(P) + 64 * F * np.tril(np.abs(D) * (aQ @ aK.T))
        carried = np.abs(G)[:, None] * E * np.linalg.norm(qq, axis=1)[:, None] \
            + (aP.sum(1) * np.abs(aT).sum(1).max() * E * np.abs(bb).max() * np.linalg.norm(kk, axis=1).max())[:, None]
        raw = (H + e) * (np.abs(G)[:, None] * (aQ @ aX.T) + aP @ np.abs(U)) + aP @ dU + carried
        bo[s] = raw + H * (np.abs(o[s]) + raw)
        X = G[-1] * X + (U * DC[:, None]).T @ kk
        E = abs(G[-1]) * E + np.linalg.norm(loc)
    return o, X, bo, E


def rule_by_tokens(q, k, v, g, b, X, half):
    """The same token by token, for the recurrent kernel: fp32 throughout, a
    product S k of d terms in a tree of at most 12 roundings; `half`: half a
    step of the output type."""
    T = len(g)
    o, bo, E = np.zeros((T, v.shape[1])), np.zeros((T, v.shape[1])), 0.0
    X = X.copy()
    for t in range(T):
        aX = np.abs(X)
        sk, ask = X @ k[t], aX @ np.abs(k[t])
        u = b[t] * (v[t] - g[t] * sk)
        du = 14 * F * abs(b[t]) * (np.abs(v[t]) + abs(g[t]) * ask)
        sq, asq, akq = X @ q[t], aX @ np.abs(q[t]), np.abs(k[t]) @ np.abs(q[t])
        o[t] = g[t] * sq + u * (k[t] @ q[t])
        raw = 14 * F * (abs(g[t]) * asq + np.abs(u) * akq) + du * akq + E * np.linalg.norm(q[t]) * (1 + abs(b[t]) * np.dot(k[t], k[t]))
        bo[t] = raw + half * (np.abs(o[t]) + raw)
        loc = np.outer(du, np.abs(k[t])) + 3 * F * (abs(g[t]) * aX + np.abs(np.outer(u, k[t])))
        X = g[t] * X + np.outer(u, k[t])
        E = abs(g[t]) * E + np.linalg.norm(loc)
    return o, X, bo, E
