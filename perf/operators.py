"""The packed gated delta rule's operators as a serving program calls them, for
measurement: the step plan built on the GPU from request lengths, the chunkwise
prefill of packed sequences, and the recurrent step through a pool of states.

Requests of different lengths lie one behind the other in packed tensors
(q, k [tokens, H_k, d_k], v [tokens, H_v, d_v], slices of one projection's
rows, so that a row is longer than a tensor's own part of it). Every request
owns a slot in a pool of fp32 states [slots, H_v, d_v, d_k], updated in place.
Per value head (its key head is h * H_k // H_v), for each token of a request:

    S = g S (I - beta k k^T) + beta v k^T,    o = S q

A request that has seen no token yet starts from a zero state, whatever its
slot holds.

``own`` false: elementary torch operations. ``own`` true: the library.
"""
import math
import random

import torch

own = False

BLOCK = 64            # tokens per block of the plain chunkwise form
FEW = 8               # up to so many tokens per request the plain form walks token by token


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The plan of a small decode step: what a lightly loaded server waits for.
        dict(name="plan_r8", op="plan", R=8, N=24, pattern="decode", rows=32),
        # A busy server's mixed step: prompts and decodes, some requests ending.
        dict(name="plan_r512", op="plan", R=512, N=16000, pattern="mixed", rows=16384),
        # Offline batch: thousands of requests, a quarter of a million rows.
        dict(name="plan_r8192", op="plan", R=8192, N=260000, pattern="ragged", rows=262144),
        # One whole serving step: the plan, then prompts and decodes in one call.
        dict(name="step_mixed_r64", op="step", R=64, N=4001, pattern="mixed", Hk=8, Hv=16, dk=128, dv=128, io="bf16"),
        # One short prompt on small heads: the time to a first token.
        dict(name="prefill_one_t130", op="prefill", R=1, N=130, pattern="even", Hk=8, Hv=16, dk=64, dv=64, io="bf16"),
        # A batch of prompts of very different lengths, four value heads a key head.
        dict(name="prefill_ragged_r16", op="prefill", R=16, N=8191, pattern="ragged", Hk=8, Hv=32, dk=128, dv=128, io="bf16"),
        # Two long prompts: the library's own prefill workload (B2 H16 T8192 d128), packed.
        dict(name="prefill_long_r2", op="prefill", R=2, N=16384, pattern="even", Hk=16, Hv=16, dk=128, dv=128, io="bf16"),
        # Throughput prefill: many prompts at once.
        dict(name="prefill_n65536", op="prefill", R=96, N=65536, pattern="ragged", Hk=8, Hv=16, dk=128, dv=128, io="bf16"),
        # fp32 tensors (evaluation against a reference), odd lengths, small heads.
        dict(name="prefill_fp32_d64", op="prefill", R=6, N=611, pattern="ragged", Hk=4, Hv=8, dk=64, dv=64, io="fp32"),
        # One token for each of four requests: a decode step that latency bounds.
        dict(name="decode_r4", op="decode", R=4, N=4, pattern="even", Hk=16, Hv=16, dk=128, dv=128, io="bf16"),
        # The library's own decode workload (256 sequences, 16 heads), through a pool.
        dict(name="decode_r256", op="decode", R=256, N=256, pattern="even", Hk=16, Hv=16, dk=128, dv=128, io="bf16"),
        # A few drafted tokens for each request, shared key heads.
        dict(name="decode_few_r128", op="decode", R=128, N=400, pattern="few", Hk=4, Hv=16, dk=128, dv=128, io="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("plan", "step", "prefill", "prefill", "decode"))
    if op == "plan":
        R = _log_uniform(rng, 1, 8000)
        N = max(R, _log_uniform(rng, 16, 250000))
        return dict(op=op, R=R, N=N, pattern=rng.choice(("decode", "mixed", "ragged")), rows=N + rng.choice((0, 1, 7, 1000)),
                    lens=rng.randrange(1 << 20))
    c = dict(op=op, dk=rng.choice((64, 128)), dv=rng.choice((64, 128)), io="bf16", lens=rng.randrange(1 << 20))
    c["Hk"] = rng.choice((1, 2, 4, 8, 16))
    c["Hv"] = c["Hk"] * rng.choice((1, 2, 4)) if c["Hk"] <= 4 else 16
    if op == "decode":
        c["R"] = _log_uniform(rng, 1, 256)
        c["pattern"] = rng.choice(("even", "few"))
        c["N"] = c["R"] if c["pattern"] == "even" else c["R"] * rng.randint(1, 4)
        if rng.random() < 0.3:
            c["io"], c["dk"], c["dv"] = "fp32", rng.choice((16, 32, 64, 128)), rng.choice((16, 32, 64, 128))
    elif op == "prefill" and rng.random() < 0.25:
        c["io"], c["dk"], c["dv"] = "fp32", rng.choice((16, 32, 64, 128)), rng.choice((16, 32, 64, 128))
        c["R"] = _log_uniform(rng, 1, 12)
        c["pattern"] = "ragged"
        c["N"] = max(c["R"], _log_uniform(rng, 16, 1500))
    else:
        c["R"] = _log_uniform(rng, 1, 64)
        c["pattern"] = "mixed" if op == "step" else rng.choice(("ragged", "even"))
        c["N"] = max(c["R"], _log_uniform(rng, 64, 30000 if c["R"] >= 4 else 8000))
    return c


def _lengths(case):
    """The requests' lengths: the case's alone, so that its work is known. They add up to N
    (a plan's "mixed" and "ragged" hold ending requests, -1, besides)."""
    R, N, pattern = case["R"], case["N"], case["pattern"]
    rng = random.Random(case.get("lens", 1) * 7919 + R * 31 + N)
    if pattern == "even":
        return [N * (r + 1) // R - N * r // R for r in range(R)]
    if pattern == "few":      # 1 to 4 drafted tokens, an idle request now and then
        w = [rng.choice((1, 2, 3, 4)) for _ in range(R)]
    elif pattern == "decode":
        w = [1.0 if rng.random() < 0.9 else 0.0 for _ in range(R)]
    elif pattern == "mixed":  # most requests decode one token, a few bring a prompt
        w = [0.0 if rng.random() < 0.9 else math.exp(rng.uniform(0, 3)) for _ in range(R)]
    else:                     # lengths over a factor of about a hundred
        w = [math.exp(rng.uniform(0, 4.6)) for _ in range(R)]
    if pattern == "few":
        lens = w
        while sum(lens) != N:
            r = rng.randrange(R)
            lens[r] = max(0, lens[r] + (1 if sum(lens) < N else -1))
    else:
        base = 1 if pattern == "mixed" else 0
        left, total = N - base * R, sum(w)
        if not total:
            w[rng.randrange(R)] = total = 1.0
        cum, lens = 0.0, []
        for x in w:
            a = int(left * cum / total)
            cum += x
            lens.append(base + int(left * min(1.0, cum / total)) - a)
        lens[max(range(R), key=lambda r: lens[r])] += N - sum(lens)
    if case["op"] == "plan" and pattern != "decode":
        for r in range(3, R, 17):  # ended: gives its slot back
            take, lens[r] = max(0, lens[r]), -1
            lens[r - 1] += take
    return lens


def _seen(case):
    """Tokens absorbed before this step: every third request of a prefill is new."""
    R = case["R"]
    if case["op"] == "decode":
        return [100 + r for r in range(R)]
    return [0 if r % 3 == 0 else 10 + r for r in range(R)]


def work(case):
    R = case["R"]
    lens, seen = _lengths(case), _seen(case)
    b = f = 0
    if case["op"] in ("plan", "step"):
        rows = case.get("rows", case["N"])
        b += 4 * (3 * R) + 4 * (3 * R + 1) + 8 * rows     # lengths, seen, slots in; offsets, slots, order, two words a row out
    if case["op"] != "plan":
        e = 2 if case["io"] == "bf16" else 4
        Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        n, S = sum(lens), Hv * dv * dk * 4
        b += n * (e * (2 * Hk * dk + 2 * Hv * dv) + 8 * Hv)
        b += sum(S * (2 if s else 1) for x, s in zip(lens, seen) if x > 0)
        f += n * Hv * 6 * dk * dv                          # S k, the rank-one update, S q
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs

def _io(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda", torch.cuda.current_device())
    R, lens, seen = case["R"], _lengths(case), _seen(case)
    pool = R + R // 4 + 2
    rows = case.get("rows", case["N"])
    ints = dict(dtype=torch.int32, device=dev)
    s = dict(op=case["op"], R=R, rows=rows, pool=pool, lens=lens)
    perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    s["lengths"], s["seen"] = torch.tensor(lens, **ints), torch.tensor(seen, **ints)
    # a new request has no slot yet where a plan is made; the pool's other slots are free
    fresh = (s["seen"] == 0) & (s["lengths"] > 0) if case["op"] in ("plan", "step") else torch.zeros(R, dtype=torch.bool, device=dev)
    s["slots"] = torch.where(fresh, torch.full_like(s["seen"], -1), perm[:R])
    s["free_slots"] = torch.full((pool,), -1, **ints)
    spare = torch.cat([perm[:R][fresh], perm[R:]])
    s["free_slots"][:spare.numel()] = spare
    s["free_count"] = torch.tensor([spare.numel()], **ints)
    if case["op"] != "plan":
        Hk, Hv, dk, dv, io = case["Hk"], case["Hv"], case["dk"], case["dv"], _io(case)
        n = rows
        q = torch.randn(n, Hk, dk, generator=gen, device=dev)
        k = torch.randn(n, Hk, dk, generator=gen, device=dev)
        k = k / k.norm(dim=-1, keepdim=True)
        v = torch.randn(n, Hv, dv, generator=gen, device=dev)
        fused = torch.cat([q.reshape(n, -1), k.reshape(n, -1), v.reshape(n, -1)], 1).to(io)
        s["q"] = fused[:, :Hk * dk].view(n, Hk, dk)
        s["k"] = fused[:, Hk * dk:2 * Hk * dk].view(n, Hk, dk)
        s["v"] = fused[:, 2 * Hk * dk:].view(n, Hv, dv)
        s["gate"] = torch.sigmoid(torch.randn(n, Hv, generator=gen, device=dev) + 4)
        s["beta"] = torch.sigmoid(torch.randn(n, Hv, generator=gen, device=dev))
        s["states"] = torch.randn(pool, Hv, dv, dk, generator=gen, device=dev) * 0.02
        s["dims"] = (Hk, Hv, dk, dv, io)
        s["blocks"] = _blocks(lens, dev)
    if own:
        import gated_delta_rule_causal_gb300 as la
        Hk, Hv, dk, dv = (case.get(x, y) for x, y in (("Hk", 1), ("Hv", 1), ("dk", 64), ("dv", 64)))
        s["handle"] = la.PackedHandle(max_requests=R, max_tokens=rows, slots=pool, H_k=Hk, H_v=Hv, d_k=dk, d_v=dv,
                                      io=case.get("io", "bf16"))
        s["plan"] = s["handle"].new_plan()
        if case["op"] in ("prefill", "decode"):
            s["handle"].plan(s["lengths"], s["seen"], s["slots"], s["free_slots"], s["free_count"], tokens=rows, plan=s["plan"])
    return s


def _blocks(lens, dev):
    """The plain form's tables: the requests, longest first, and for each step c the rows of block c of the requests
    that have one (rows past a request's end are marked)."""
    offs = [0]
    for x in lens:
        offs.append(offs[-1] + max(0, x))
    order = sorted((r for r in range(len(lens)) if lens[r] > 0), key=lambda r: -lens[r])
    few = not order or max(lens) <= FEW
    C = 1 if few else BLOCK
    start, count, active = [], [], []
    for c in range((max(lens) + C - 1) // C if order else 0):
        a = [r for r in order if lens[r] > c * C]
        active.append(len(a))
        start += [offs[r] + c * C for r in a]
        count += [min(C, lens[r] - c * C) for r in a]
    t = torch.arange(C, device=dev)
    start, count = torch.tensor(start, device=dev).view(-1, 1), torch.tensor(count, device=dev).view(-1, 1)
    valid = t < count
    return dict(order=torch.tensor(order, dtype=torch.long, device=dev), active=active, few=few, rows=torch.where(valid, start + t, start), valid=valid)


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        h, res = s["handle"], []
        if s["op"] in ("plan", "step"):
            p = h.plan(s["lengths"], s["seen"], s["slots"], s["free_slots"], s["free_count"], tokens=s["rows"], plan=s["plan"])
            res += [p.counts, p.offsets, p.state_slots, p.order, p.token_request, p.token_position, s["slots"], s["free_slots"], s["free_count"]]
        if s["op"] != "plan":
            step = h.decode_step if s["op"] == "decode" else h.forward
            res += [step(s["plan"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["states"]), s["states"]]
        return res
    res, slots = [], s["slots"]
    if s["op"] in ("plan", "step"):
        res += _plain_plan(s)
        slots = res[2]
    if s["op"] != "plan":
        res += _plain_rule(s, slots)
    return res


def _plain_plan(s):
    """counts (rows used, requests taking part, free slots left, faults), offsets, the state slot of every request that
    takes part, their order (most 32-token blocks first, to a power of two), and for every row its request and position."""
    R, rows, S, dev = s["R"], s["rows"], s["pool"], s["lengths"].device
    lens, seen, slots, free, count = s["lengths"].long(), s["seen"].long(), s["slots"].long(), s["free_slots"], s["free_count"]
    r = torch.arange(R, device=dev)
    n = lens.clamp(min=0)
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), n.cumsum(0)]).clamp(max=rows + 1)
    fits = off[1:] <= rows
    inside = (slots >= 0) & (slots < S)
    at = torch.where(inside, slots, S)
    owner = torch.full((S + 1,), R, device=dev).scatter_reduce(0, at, r, "amin")
    mine = inside & (owner[at] == r)
    ends = (lens < 0) & mine
    c0 = count.long()
    push = torch.where(ends, c0 + ends.long().cumsum(0) - 1, S).clamp(max=S)
    stack = torch.cat([free.long(), free.new_zeros(1).long()]).scatter(0, push, slots)[:S]
    c1 = c0 + ends.long().sum()
    need = (lens > 0) & (slots == -1) & (seen == 0) & fits
    pop = c1 - need.long().cumsum(0)
    got = need & (pop >= 0)
    new = stack[pop.clamp(min=0)]
    now = torch.where(got, new, torch.where(ends, -1, slots))
    part = (lens > 0) & fits & (got | mine)
    faults = ((lens > 0) & ~fits).any().long() + 2 * (need & ~got).any().long() + 4 * ((slots >= S) | (slots < -1)).any().long() \
        + 8 * (inside & ~mine).any().long() + 16 * ((lens > 0) & (slots == -1) & (seen != 0)).any().long()
    left = (c1 - got.long().sum())
    use = torch.where(part, now, -1)
    blocks = (n + 31) // 32
    key = torch.frexp(blocks.float()).exponent * part       # whole numbers below 2^24: exact
    order = torch.sort(key, descending=True, stable=True).indices
    row = torch.arange(rows, device=dev)
    req = torch.searchsorted(off[1:].contiguous(), row, right=True)
    used = row < off[R].clamp(max=rows)
    used = used & (req < R)
    reqc = req.clamp(max=R - 1)
    used = used & fits[reqc]
    pos = torch.where(used, seen[reqc] + row - off[reqc], -1)
    counts = torch.stack([off[R].clamp(max=rows), part.long().sum(), left.view(()), faults])
    s["slots"].copy_(now)
    s["free_slots"].copy_(stack)
    s["free_count"].copy_(left)
    i32 = [x.to(torch.int32) for x in (counts, off, use, order, torch.where(used, req, -1), pos)]
    return i32 + [s["slots"], s["free_slots"], s["free_count"]]


def _plain_rule(s, slots):
    Hk, Hv, dk, dv, io = s["dims"]
    b = s["blocks"]
    order, rows, valid = b["order"], b["rows"], b["valid"]
    out = torch.zeros(s["rows"], Hv, dv, dtype=io, device=s["q"].device)
    at = slots.long()[order]
    S = s["states"][at] * (s["seen"][order] != 0).float()[:, None, None, None]
    C = rows.shape[1] if rows.numel() else 1
    rep = Hv // Hk
    heads = lambda x: x[rows].float().permute(0, 2, 1, 3)   # [block, heads, C, d]  # noqa: E731
    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    live = valid[:, None, :].float()
    beta = s["beta"][rows].permute(0, 2, 1) * live
    if b["few"]:
        gate = s["gate"][rows].permute(0, 2, 1)
        o, lo = torch.empty_like(v), 0
        for a in b["active"]:
            g, bt = gate[lo:lo + a, :, 0, None, None], beta[lo:lo + a, :, 0, None]
            kk, qq = k[lo:lo + a, :, 0, :, None], q[lo:lo + a, :, 0, :, None]
            X = S[:a] * g
            u = bt * (v[lo:lo + a, :, 0] - (X @ kk).squeeze(-1))
            X = X + u[..., None] * kk.transpose(-1, -2)
            o[lo:lo + a, :, 0] = (X @ qq).squeeze(-1)
            S[:a] = X
            lo += a
    else:
        G = (torch.log(s["gate"].double())[rows].permute(0, 2, 1) * live).cumsum(-1)
        D = (G[..., :, None] - G[..., None, :]).clamp(max=0.0).float().exp()
        low = torch.ones(C, C, device=D.device).tril()
        A = (k @ k.transpose(-1, -2)) * D * beta[..., :, None] * low.tril(-1)
        P = (q @ k.transpose(-1, -2)) * D * low
        T, M = torch.eye(C, device=D.device) - A, A
        for _ in range(5):                                  # (I + A)^-1 = (I - A)(I + A^2)(I + A^4)...
            M = M @ M
            T = T + T @ M
        gam = G.float().exp()
        U0, W = T @ (beta[..., None] * v), T @ ((beta * gam)[..., None] * k)
        qg, kg = q * gam[..., None], k * (G[..., -1:] - G).float().exp()[..., None]
        gC = gam[..., -1, None, None]
        o, lo = torch.empty_like(v), 0
        for a in b["active"]:
            i = slice(lo, lo + a)
            X = S[:a]
            u = U0[i] - W[i] @ X.transpose(-1, -2)
            o[i] = qg[i] @ X.transpose(-1, -2) + P[i] @ u
            S[:a] = gC[i] * X + u.transpose(-1, -2) @ kg[i]
            lo += a
    out[rows[valid]] = o.permute(0, 2, 1, 3)[valid].to(io)
    s["states"].index_copy_(0, at, S)
    return [out, s["states"]]


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    """Token by token in 64 bits; None for a plan's whole numbers."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    Hk, Hv, dk, dv, _ = s["dims"]
    lens = s["lens"]
    idx = sorted((r for r in range(len(lens)) if lens[r] > 0), key=lambda r: -lens[r])
    first = {}
    at = 0
    for r, x in enumerate(lens):
        first[r] = at
        at += max(0, x)
    dev = s["q"].device
    states = s["states"].double()
    out = torch.zeros(s["rows"], Hv, dv, dtype=torch.float64, device=dev)
    slots = _slots_given(s)
    pick = torch.tensor(idx, dtype=torch.long, device=dev)
    begin = torch.tensor([first[r] for r in idx], dtype=torch.long, device=dev)
    X = states[slots[pick]]
    X[s["seen"][pick] == 0] = 0.0
    head = torch.arange(Hv, device=dev) * Hk // Hv
    alive = [0] * (max(lens) + 1)
    for r in idx:
        alive[lens[r] - 1] += 1
    a = len(idx)
    for t in range(max(lens)):
        row = begin[:a] + t
        k, q, v = s["k"][row].double()[:, head], s["q"][row].double()[:, head], s["v"][row].double()
        g, bt = s["gate"][row].double(), s["beta"][row].double()
        Y = X[:a]
        Y.mul_(g[:, :, None, None])
        err = v - torch.matmul(Y, k.unsqueeze(-1)).squeeze(-1)
        Y.addcmul_((bt[:, :, None] * err).unsqueeze(-1), k.unsqueeze(-2))
        out[row] = torch.matmul(Y, q.unsqueeze(-1)).squeeze(-1)
        a -= alive[t]
    states[slots[pick]] = X
    res = [out, states]
    return [None] * 9 + res if case["op"] == "step" else res


def _slots_given(s):
    """The slots of a step's requests: new ones take the free list's last entries in the requests' order."""
    got, free, n = s["slots"].tolist(), s["free_slots"].tolist(), int(s["free_count"])
    for r in range(s["R"]):
        if got[r] < 0 and s["lens"][r] > 0:
            n -= 1
            got[r] = free[n]
    return torch.tensor(got, dtype=torch.long, device=s["q"].device)
