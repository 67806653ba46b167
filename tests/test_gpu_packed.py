"""The packed gated delta rule on the GPU against plain float64 references:
plans against their definition, exactly; outputs and states within what the
kernels' roundings can add up to (bounds in _packed.py)."""
import random

import numpy as np
import pytest

import _packed as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gated_delta_rule_causal_gb300 as la  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    la.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plans

class PlanCase:
    def __init__(self, lengths, seen, slots, free, count, pool, rows, max_requests=None, max_tokens=None):
        self.args = (lengths, seen, slots, free, count, pool, rows)
        R = len(lengths)
        self.h = la.PackedHandle(max_requests=max_requests or max(R, 1), max_tokens=max_tokens or max(rows, 1), slots=pool,
                                 H_k=1, H_v=1, d_k=16, d_v=16)
        self.dev = [i32(lengths), i32(seen), i32(slots), i32(free), i32([count])]

    def run(self, **kw):
        return self.h.plan(*self.dev, tokens=self.args[-1], **kw)

    def check(self, plan):
        want = ref.plan(*self.args)
        torch.cuda.synchronize()
        for name in ("counts", "offsets", "state_slots", "order", "token_request", "token_position"):
            assert getattr(plan, name).tolist() == want[name], name
        assert self.dev[2].tolist() == want["slots"]
        assert self.dev[3].tolist() == want["free_slots"]
        assert self.dev[4].tolist() == want["free_count"]
        return want


def serving_case(R, rows, seed, long=False):
    """Consistent slots: live requests own different ones, the others are free."""
    rng = random.Random(seed)
    pool = R + R // 3 + 2
    perm = list(range(pool))
    rng.shuffle(perm)
    lengths, seen, slots = [], [], []
    left = rows
    for r in range(R):
        new = rng.random() < 0.3
        n = rng.choice((0, 1, 1, 1, 2, 31, 32, 33, 64, 65, 130) if not long else (1, 700, 3, 4096, 64))
        n = min(n, left)
        left -= n
        if not new and rng.random() < 0.15:
            n = -rng.randint(1, 3)
        lengths.append(n)
        seen.append(0 if new else rng.randint(0, 5000))
        slots.append(-1 if new else perm.pop())
    lengths[0] += max(0, left - 5) if R > 2 and lengths[0] >= 0 else 0
    return PlanCase(lengths, seen, slots, perm + [0] * (pool - len(perm)), len(perm), pool, rows)


@pytest.mark.parametrize("R,rows", [(1, 1), (1, 5000), (2, 64), (7, 33), (31, 200), (33, 4096), (64, 4097), (1000, 9000),
                                    (1024, 12345), (1025, 8192), (2500, 30001), (16384, 40000)])
def test_plan_of_a_serving_step(R, rows):
    c = serving_case(R, rows, seed=R * 7 + rows)
    want = c.check(c.run())
    assert want["counts"][3] == 0
    assert c.h.last_launches() == 1


def test_plan_of_nothing():
    c = PlanCase([], [], [], [3, 1], 1, 2, 6)
    want = c.check(c.run())
    assert want["counts"] == [0, 0, 1, 0] and want["token_request"] == [-1] * 6
    c = PlanCase([0, 0], [1, 0], [1, -1], [0, 0], 1, 2, 0, max_tokens=4)
    c.check(c.run())


def test_plan_in_a_buffer_of_larger_maxima_leaves_the_rest():
    c = PlanCase([2, 1], [4, 0], [0, -1], [1, 0, 0], 1, 3, 5, max_requests=50, max_tokens=70)
    plan = c.h.new_plan()
    plan.words.fill_(-77)
    c.check(c.run(plan=plan))
    plan._set(50, 70)
    assert plan.offsets[3:].eq(-77).all() and plan.state_slots[2:].eq(-77).all() and plan.order[2:].eq(-77).all()
    assert plan.token_request[5:].eq(-77).all() and plan.token_position[5:].eq(-77).all()


@pytest.mark.parametrize("name,args,faults", [
    ("rows", ([3, 5, 0, 2], [1, 1, 1, 0], [0, 1, 2, -1], [3, 4, 0, 0, 0], 2, 5, 6), la.LA_PLAN_FAULT_ROWS),
    ("rows saturate", ([2 ** 31 - 1] * 5, [0] * 5, [-1] * 5, [0, 1, 2, 3, 4], 5, 5, 100), la.LA_PLAN_FAULT_ROWS),
    ("no free slot", ([1, 2, 3], [0, 0, 0], [-1, -1, -1], [4, 0, 0, 0, 0], 1, 5, 10), la.LA_PLAN_FAULT_FREE),
    ("outside", ([1, 1, 1, -1], [0, 1, 1, 1], [5, -2, -2 ** 31, 9], [0, 1, 0, 0, 0], 2, 5, 10), la.LA_PLAN_FAULT_SLOT),
    ("claimed twice", ([1, 1, 1], [1, 1, 1], [2, 2, 2], [0, 1, 3, 0, 0], 3, 5, 10), la.LA_PLAN_FAULT_OWNER),
    ("given back twice", ([-1, -1, 1], [1, 1, 1], [2, 2, 2], [0, 1, 3, 0, 0], 3, 5, 10), la.LA_PLAN_FAULT_OWNER),
    ("free and owned", ([1, 4], [0, 3], [-1, 2], [0, 2, 0, 0, 0], 2, 5, 10), la.LA_PLAN_FAULT_OWNER),
    ("free twice", ([1, 4], [0, 0], [-1, -1], [3, 3, 0, 0, 0], 2, 5, 10), la.LA_PLAN_FAULT_OWNER),
    ("free holds nonsense", ([1, 4], [0, 0], [-1, -1], [77, -5, 0, 0, 0], 2, 5, 10), la.LA_PLAN_FAULT_SLOT),
    ("no state", ([1, 4], [9, 0], [-1, 2], [0, 1, 0, 0, 0], 2, 5, 10), la.LA_PLAN_FAULT_STATE),
    ("overflow", ([-1, -1], [1, 1], [2, 3], [0, 1, 2, 3, 4], 5, 5, 10), la.LA_PLAN_FAULT_OVERFLOW),
    ("count above the pool", ([1], [0], [-1], [0, 1, 4], 99, 3, 4), la.LA_PLAN_FAULT_SLOT),
    ("count below zero", ([1], [0], [-1], [0, 1, 4], -99, 3, 4), la.LA_PLAN_FAULT_FREE),
])
def test_plan_faults_drop_the_request_alone(name, args, faults):
    c = PlanCase(*args)
    want = c.check(c.run())
    assert want["counts"][3] == faults


@pytest.mark.parametrize("name,args,faults", [
    ("outside", ([1, 1, -1, 2], [0, 1, 1, 7], [60000, -2, 60000, 59999], [0, 1], 2), la.LA_PLAN_FAULT_SLOT),
    ("claimed twice", ([1, 1, 1], [1, 1, 1], [2, 2, 2], [0, 1, 3], 3), la.LA_PLAN_FAULT_OWNER),
    ("given back twice", ([-1, -1, 1], [1, 1, 1], [2, 2, 2], [0, 1, 3], 3), la.LA_PLAN_FAULT_OWNER),
    ("free and owned", ([1, 4], [0, 3], [-1, 2], [0, 2], 2), la.LA_PLAN_FAULT_OWNER),
    ("free twice", ([1, 4], [0, 0], [-1, -1], [3, 3], 2), la.LA_PLAN_FAULT_OWNER),
    ("back and taken", ([-1, 3, 2], [5, 0, 0], [59999, -1, -1], [7], 1), 0),
])
def test_plan_of_a_pool_whose_claims_do_not_fit_shared_memory(name, args, faults):
    pool = 60000
    lengths, seen, slots, free, count = args
    c = PlanCase(lengths, seen, slots, free + [0] * (pool - len(free)), count, pool, 10)
    assert c.check(c.run())["counts"][3] == faults


# ------------------------------------------------------------------ the rule

def handle_for(lens, Hk, Hv, dk, dv, io, pool, extra_rows=0):
    return la.PackedHandle(max_requests=len(lens), max_tokens=max(1, sum(lens) + extra_rows), slots=pool, H_k=Hk, H_v=Hv,
                           d_k=dk, d_v=dv, io=io)


def draw(lens, Hk, Hv, dk, dv, io, seed, pad=0, extra_rows=0, gates="usual"):
    """Packed inputs of requests, rows strided by `pad` elements between the tensors' own, and a pool."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    n, rnd = sum(lens) + extra_rows, lambda *s: torch.randn(*s, generator=gen, device="cuda")
    k = rnd(n, Hk, dk)
    k = k / k.norm(dim=-1, keepdim=True)
    x = {}
    for name, t, w in (("q", rnd(n, Hk, dk), Hk * dk), ("k", k, Hk * dk), ("v", rnd(n, Hv, dv), Hv * dv)):
        buf = torch.full((n, w + pad), float("nan"), device="cuda", dtype=dt)
        buf[:, :w] = t.reshape(n, w).to(dt)
        x[name] = buf[:, :w].view(n, t.shape[1], t.shape[2])
    x["gate"] = torch.sigmoid(rnd(n, Hv) + 4)
    x["beta"] = torch.sigmoid(rnd(n, Hv))
    if gates == "strong":
        x["gate"] = torch.sigmoid(rnd(n, Hv) * 4)
    elif gates == "zero":
        x["gate"][torch.rand(n, Hv, generator=gen, device="cuda") < 0.2] = 0.0
        x["gate"][torch.rand(n, Hv, generator=gen, device="cuda") < 0.1] = 1e-38
        x["beta"][torch.rand(n, Hv, generator=gen, device="cuda") < 0.2] = 1.0
        x["beta"][torch.rand(n, Hv, generator=gen, device="cuda") < 0.2] = 0.0
    elif gates == "none":
        x["gate"].fill_(1.0)
        x["beta"].fill_(1.0)
    pool = len(lens) + 3
    x["states"] = rnd(pool, Hv, dv, dk) * 0.5
    perm = torch.randperm(pool, generator=gen, device="cuda").tolist()
    x["slots"] = perm[:len(lens)]
    return x, pool


def make_plan(h, lens, seen, slots, rows=None):
    pool = h.slots
    return h.plan(i32(lens), i32(seen), i32(slots), i32([0] * pool), i32([0]), tokens=sum(lens) if rows is None else rows)


def check(x, lens, seen, states_before, out, io, chunk, only=None):
    """Every request's outputs and state against the references (chunk: 1, or the blocks' tokens); returns the largest
    share of a bound used."""
    worst = 0.0
    d = lambda t: t.double().cpu().numpy()   # noqa: E731
    q, k, v, g, b = (d(x[n]) for n in ("q", "k", "v", "gate", "beta"))
    after, before, o = d(x["states"]), d(states_before), d(out)
    Hk, Hv = q.shape[1], v.shape[1]
    row = 0
    for r, n in enumerate(lens):
        if n > 0 and (only is None or r in only):
            s = slice(row, row + n)
            for h in range(Hv):
                hk = h * Hk // Hv
                X0 = before[x["slots"][r], h] if seen[r] else np.zeros_like(before[0, 0])
                args = (q[s, hk], k[s, hk], v[s, h], g[s, h], b[s, h], X0)
                want, X, bo, E = ref.rule_by_blocks(*args, chunk) if chunk > 1 else ref.rule_by_tokens(
                    *args, ref.H if io == "bf16" else ref.F)
                used = np.max(np.abs(o[s, h] - want) / (bo + 1e-30))
                assert used <= 1.0, f"request {r} head {h}: output {used:.3g} of its bound"
                err = np.linalg.norm(after[x["slots"][r], h] - X)
                assert err <= E, f"request {r} head {h}: state off by {err:.3g}, bound {E:.3g}"
                worst = max(worst, used, err / (E + 1e-30))
        row += max(0, n)
    return worst


LENS = [[1], [31, 1, 33], [64, 0, 65, 32], [130, 7, 0, 0, 97, 1], [513]]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("Hk,Hv,dk,dv,chunk", [(1, 1, 64, 64, 32), (2, 4, 128, 128, 32), (1, 3, 128, 64, 32), (2, 2, 64, 128, 32),
                                               (2, 4, 128, 128, 64), (2, 2, 64, 128, 64), (1, 2, 128, 128, 64)])
def test_prefill_by_blocks(lens, Hk, Hv, dk, dv, chunk):
    x, pool = draw(lens, Hk, Hv, dk, dv, "bf16", seed=sum(lens) + dk, pad=8, extra_rows=3)
    h = handle_for(lens, Hk, Hv, dk, dv, "bf16", pool, extra_rows=3)
    seen = [r % 2 * 11 for r in range(len(lens))]
    plan = make_plan(h, lens, seen, x["slots"], rows=sum(lens) + 3)
    before = x["states"].clone()
    out = torch.full((sum(lens) + 3, Hv, dv), -7.5, device="cuda", dtype=torch.bfloat16)
    h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], out=out, chunk=chunk)
    assert h.status() == la.LA_OK and h.last_launches() == 1
    check(x, lens, seen, before, out, "bf16", chunk)
    # rows behind the last request, states of idle requests and of nobody: as they were
    assert out[sum(lens):].eq(-7.5).all()
    others = [s for s in range(pool) if s not in [x["slots"][r] for r, n in enumerate(lens) if n > 0]]
    assert torch.equal(x["states"][others], before[others])


@pytest.mark.parametrize("gates", ["strong", "zero", "none"])
@pytest.mark.parametrize("dk,dv,chunk", [(64, 64, 32), (128, 64, 32), (64, 128, 64), (128, 128, 64)])
def test_prefill_gates(gates, dk, dv, chunk):
    lens = [70, 129]
    x, pool = draw(lens, 1, 2, dk, dv, "bf16", seed=5, gates=gates)
    if gates == "none":   # the same key again and again, and its negative
        x["k"][:, 0] = x["k"][0, 0]
        x["k"][1::3, 0] *= -1
    h = handle_for(lens, 1, 2, dk, dv, "bf16", pool)
    plan = make_plan(h, lens, [0, 3], x["slots"])
    before = x["states"].clone()
    out = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], chunk=chunk)
    assert h.status() == la.LA_OK
    check(x, lens, [0, 3], before, out, "bf16", chunk)


@pytest.mark.parametrize("chunk", [1, 32, 64, 0])
def test_only_requests_that_have_seen_nothing_start_from_zeros(chunk):
    # any other number, a negative one too, goes on from the slot's state (chunk 0: short requests beside the others)
    lens = [70, 2, 40, 1, 9] * 4 if chunk == 0 else [70, 2, 40]
    Hk, Hv = (4, 8) if chunk == 0 else (1, 2)
    x, pool = draw(lens, Hk, Hv, 128, 128, "bf16", seed=17)
    h = handle_for(lens, Hk, Hv, 128, 128, "bf16", pool)
    seen = [(-3, 0, -2 ** 31, -1, 2 ** 31 - 100)[r % 5] for r in range(len(lens))]
    plan = make_plan(h, lens, seen, x["slots"])
    assert plan.counts.tolist() == [sum(lens), len(lens), 0, 0]
    before = x["states"].clone()
    out = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], chunk=chunk)
    assert h.status() == la.LA_OK and h.last_launches() == (2 if chunk == 0 else 1)
    check(x, lens, seen, before, out, "bf16", chunk or 64)


@pytest.mark.parametrize("dk,dv,chunk", [(64, 64, 32), (128, 128, 32), (64, 128, 64), (128, 128, 64), (64, 128, 1)])
def test_gates_above_one_and_below_zero(dk, dv, chunk):
    lens = [67, 130]
    x, pool = draw(lens, 1, 2, dk, dv, "bf16", seed=dk + chunk)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda: torch.rand(sum(lens), 2, generator=gen, device="cuda")   # noqa: E731
    x["gate"] = (0.7 + 0.6 * rnd()) * torch.where(rnd() < 0.5, -1.0, 1.0)   # products of 64 stay below 2^25
    h = handle_for(lens, 1, 2, dk, dv, "bf16", pool)
    plan = make_plan(h, lens, [0, 3], x["slots"])
    before = x["states"].clone()
    out = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], chunk=chunk)
    assert h.status() == la.LA_OK
    check(x, lens, [0, 3], before, out, "bf16", chunk)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_token_by_token_takes_any_finite_gate(io):
    # powers of two whose products leave fp32's range while the states stay inside: with beta 0 states are scaled exactly
    lens, Hv, d = [8, 4], 2, 64
    x, pool = draw(lens, 1, Hv, d, d, io, seed=2)
    x["gate"] = torch.tensor([2.0 ** e for e in (100, 60, -100, -60)] * 3, device="cuda")[:, None].expand(12, Hv).contiguous()
    x["beta"].zero_()
    x["states"] = x["states"].mul(2.0 ** -90)
    h = handle_for(lens, 1, Hv, d, d, io, pool)
    plan = make_plan(h, lens, [1, 1], x["slots"])
    before = x["states"].clone()
    out = h.decode_step(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"])
    assert h.status() == la.LA_OK
    assert torch.equal(x["states"], before) and torch.isfinite(out).all()


@pytest.mark.parametrize("chunk", [1, 32, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nothing_leaks_between_requests(bad, chunk):
    # requests 1 and 3 and the rows behind the last request hold NaN or infinities,
    # as do the slots of new requests and of nobody
    lens, Hk, Hv, dk, dv = [37, 5, 50, 20, 33], 2, 2, 64, 128
    x, pool = draw(lens, Hk, Hv, dk, dv, "bf16", seed=9, extra_rows=40)
    seen = [0, 1, 6, 1, 0]
    starts = np.concatenate([[0], np.cumsum(lens)])
    for a, e in ((starts[1], starts[2]), (starts[3], starts[4]), (starts[5], sum(lens) + 40)):
        for name in ("q", "k", "v", "gate", "beta"):
            x[name][a:e] = bad
    for s in range(pool):
        if s != x["slots"][2]:
            x["states"][s] = bad
    h = handle_for(lens, Hk, Hv, dk, dv, "bf16", pool, extra_rows=40)
    plan = make_plan(h, lens, seen, x["slots"], rows=sum(lens) + 40)
    before = x["states"].clone()
    out = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], chunk=chunk)
    assert h.status() == la.LA_OK
    check(x, lens, seen, before, out, "bf16", chunk, only=(0, 2, 4))


@pytest.mark.parametrize("dk,dv,chunk", [(64, 128, 64), (128, 128, 64), (64, 64, 32), (128, 128, 32)])
def test_a_last_block_is_cleared_in_its_own_tile(dk, dv, chunk):
    # whole blocks, then one whose rows past the request's end hold the next request's NaN: whoever clears them has not
    # looked at the tiles of the blocks before. Many CTAs, so that loads take their time; the requests between the NaN
    # ones give the bits that they give beside finite neighbours
    rng = random.Random(dk + dv)
    blocks = [rng.choice((2, 3, 4, 5, 7)) * chunk + rng.choice((1, 2, chunk // 2, chunk - 1)) for _ in range(24)]
    x, pool = draw(blocks, 8, 16, dk, dv, "bf16", seed=dk * 5 + dv)
    h = handle_for(blocks, 8, 16, dk, dv, "bf16", pool)
    seen = [r % 3 for r in range(len(blocks))]
    plan = make_plan(h, blocks, seen, x["slots"])
    before, starts = x["states"].clone(), np.concatenate([[0], np.cumsum(blocks)])
    args = [x[n] for n in ("q", "k", "v", "gate", "beta")]
    clean = h.forward(plan, *args, x["states"], chunk=chunk)
    assert h.status() == la.LA_OK
    check(x, blocks, seen, before, clean, "bf16", chunk, only=(0, 10))
    for r in range(1, len(blocks), 2):
        for t in args:
            t[starts[r]:starts[r + 1]] = float("nan")
    for _ in range(10):
        states = before.clone()
        out = h.forward(plan, *args, states, chunk=chunk)
        assert h.status() == la.LA_OK
        for r in range(0, len(blocks), 2):
            assert torch.equal(out[starts[r]:starts[r + 1]], clean[starts[r]:starts[r + 1]]), r
            assert torch.equal(states[x["slots"][r]], x["states"][x["slots"][r]]), r


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 64), (64, 16), (128, 128), (16, 128), (128, 32), (64, 64), (32, 16)])
@pytest.mark.parametrize("lens", [[1, 1, 1], [0, 3, 1, 17]], ids=["ones", "few"])
def test_token_by_token(io, dk, dv, lens):
    Hk, Hv = 2, 4
    x, pool = draw(lens, Hk, Hv, dk, dv, io, seed=dk + dv, pad=16, extra_rows=2)
    h = handle_for(lens, Hk, Hv, dk, dv, io, pool, extra_rows=2)
    seen = [r % 2 for r in range(len(lens))]
    plan = make_plan(h, lens, seen, x["slots"], rows=sum(lens) + 2)
    before = x["states"].clone()
    out = torch.full((sum(lens) + 2, Hv, dv), 3.25, device="cuda", dtype=h.dtype)
    h.decode_step(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], out=out)
    assert h.status() == la.LA_OK and h.last_launches() == 1
    check(x, lens, seen, before, out, io, 1)
    assert out[sum(lens):].eq(3.25).all()
    others = [s for s in range(pool) if s not in [x["slots"][r] for r, n in enumerate(lens) if n > 0]]
    assert torch.equal(x["states"][others], before[others])


@pytest.mark.parametrize("io,dk,dv", [("bf16", 128, 128), ("fp32", 128, 16), ("fp32", 64, 64), ("bf16", 16, 128), ("fp32", 32, 32), ("bf16", 64, 128)])
def test_token_by_token_for_many_requests(io, dk, dv):
    # more state rows than a warp each could hold at once
    rng = random.Random(dk + dv)
    lens = [rng.choice((0, 1, 1, 1, 2, 5, 9)) for _ in range(220)]
    x, pool = draw(lens, 2, 8, dk, dv, io, seed=dk * 3 + dv)
    h = handle_for(lens, 2, 8, dk, dv, io, pool)
    seen = [r % 3 for r in range(len(lens))]
    plan = make_plan(h, lens, seen, x["slots"])
    before = x["states"].clone()
    out = h.decode_step(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"])
    assert h.status() == la.LA_OK
    check(x, lens, seen, before, out, io, 1, only=range(0, 220, 7))
    others = [s for s in range(pool) if s not in [x["slots"][r] for r, n in enumerate(lens) if n > 0]]
    assert torch.equal(x["states"][others], before[others])


def test_default_form_by_type():
    # fp32 and small heads have no blockwise form: the default is token by token, bit for bit the decode step
    for io, dk, dv in (("fp32", 64, 64), ("bf16", 32, 64), ("bf16", 64, 32)):
        lens = [40, 3]
        x, pool = draw(lens, 1, 2, dk, dv, io, seed=3)
        h = handle_for(lens, 1, 2, dk, dv, io, pool)
        plan = make_plan(h, lens, [1, 0], x["slots"])
        s1, s2 = x["states"].clone(), x["states"].clone()
        a = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], s1)
        b = h.decode_step(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], s2)
        assert torch.equal(a, b) and torch.equal(s1, s2)
        with pytest.raises(la.LAError) as e:
            h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], s1, chunk=32)
        assert e.value.code == la.LA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dk,dv,chunk", [(128, 128, 64), (64, 128, 64), (128, 128, 32), (64, 64, 32), (128, 64, 32)])
def test_many_requests_and_heads(dk, dv, chunk):
    # more CTAs than are resident, long and short ones mixed; every head of a few requests checked
    rng = random.Random(4)
    lens = [rng.choice((0, 1, 2, 33, 64, 200, 260)) for _ in range(150)]
    x, pool = draw(lens, 4, 8, dk, dv, "bf16", seed=8)
    h = handle_for(lens, 4, 8, dk, dv, "bf16", pool)
    seen = [r % 3 for r in range(len(lens))]
    plan = make_plan(h, lens, seen, x["slots"])
    before = x["states"].clone()
    out = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], chunk=chunk)
    assert h.status() == la.LA_OK
    check(x, lens, seen, before, out, "bf16", chunk, only=range(0, 150, 19))
    # the same inputs again: the same bits
    again = before.clone()
    out2 = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], again, chunk=chunk)
    assert torch.equal(again, x["states"])
    for r in range(150):
        a, e = int(plan.offsets[r]), int(plan.offsets[r + 1])
        assert torch.equal(out[a:e], out2[a:e])


@pytest.mark.parametrize("dk,dv,chunk", [(128, 128, 64), (64, 64, 32), (128, 64, 32)])
def test_a_larger_step_runs_its_short_requests_token_by_token(dk, dv, chunk):
    # bit for bit the two forms' own results; and call after call without a pause, eager and from a graph
    rng = random.Random(dk + dv)
    lens = [rng.choice((0, 1, 1, 2, 3, 4, 4, 5, 6, 40, 130, 300)) for _ in range(45)]
    x, pool = draw(lens, 4, 8, dk, dv, "bf16", seed=dk - dv + 200)
    h = handle_for(lens, 4, 8, dk, dv, "bf16", pool)
    plan = make_plan(h, lens, [r % 2 for r in range(len(lens))], x["slots"])
    args = [x[n] for n in ("q", "k", "v", "gate", "beta")]
    start = x["states"]
    mixed, blocks, tokens = start.clone(), start.clone(), start.clone()
    o1 = h.forward(plan, *args, mixed)
    assert h.last_launches() == 2
    o2 = h.forward(plan, *args, blocks, chunk=chunk)
    assert h.last_launches() == 1
    o3 = h.decode_step(plan, *args, tokens)
    assert h.status() == la.LA_OK
    for r, n in enumerate(lens):
        a, e = int(plan.offsets[r]), int(plan.offsets[r + 1])
        o, st = (o3, tokens) if n <= 4 else (o2, blocks)
        assert torch.equal(o1[a:e], o[a:e]) and torch.equal(mixed[x["slots"][r]], st[x["slots"][r]]), r
    plan = make_plan(h, lens, [5] * len(lens), x["slots"])   # states go on from call to call
    want, got, replayed = start.clone(), start.clone(), start.clone()
    for _ in range(6):
        o1 = h.forward(plan, *args, want)
        torch.cuda.synchronize()
    for _ in range(6):
        o2 = h.forward(plan, *args, got)
    assert torch.equal(got, want)
    out = torch.empty_like(o1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            h.forward(plan, *args, replayed, out=out)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert h.status() == la.LA_OK and torch.equal(replayed, want)
    for r, n in enumerate(lens):
        a, e = int(plan.offsets[r]), int(plan.offsets[r + 1])
        assert torch.equal(o2[a:e], o1[a:e]) and torch.equal(out[a:e], o1[a:e])


# ------------------------------------------------------------------ which form runs

def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dk,dv,share", [(64, 64, 1), (128, 64, 1), (64, 128, 1), (128, 128, 1), (64, 64, 2), (128, 128, 2), (64, 64, 0), (128, 64, 0)])
def test_long_requests_in_blocks_of_32(dk, dv, share):
    # dozens of turns of every ring. CTAs of 32 state rows on more (share 1) or fewer (2) than half of the SMs, each on
    # its own; or more than there are SMs, of 64 rows (0)
    R = 2
    per_head = R * (dv // 32)
    Hv = sms() // (share * per_head) if share else sms() // per_head + 3
    ctas = per_head * Hv
    assert {0: ctas > sms(), 1: sms() / 2 < ctas <= sms(), 2: ctas <= sms() / 2}[share]
    lens = [1003, 1057]
    x, pool = draw(lens, 1, Hv, dk, dv, "bf16", seed=dk + 2 * dv + share, pad=8)
    h = handle_for(lens, 1, Hv, dk, dv, "bf16", pool)
    plan = make_plan(h, lens, [1, 0], x["slots"])
    before, args = x["states"].clone(), [x[n] for n in ("q", "k", "v", "gate", "beta")]
    out = h.forward(plan, *args, x["states"], chunk=32)
    assert h.status() == la.LA_OK
    check(x, lens, [1, 0], before, out, "bf16", 32)
    for _ in range(10):
        again = before.clone()
        assert torch.equal(h.forward(plan, *args, again, chunk=32), out) and torch.equal(again, x["states"])


def test_long_requests_in_blocks_of_64():
    lens = [1003, 1057]
    for dk, Hv in ((64, 11), (128, 11)):
        x, pool = draw(lens, 1, Hv, dk, 128, "bf16", seed=dk, pad=8)
        h = handle_for(lens, 1, Hv, dk, 128, "bf16", pool)
        plan = make_plan(h, lens, [1, 0], x["slots"])
        before, args = x["states"].clone(), [x[n] for n in ("q", "k", "v", "gate", "beta")]
        out = h.forward(plan, *args, x["states"], chunk=64)
        assert h.status() == la.LA_OK
        check(x, lens, [1, 0], before, out, "bf16", 64)
        for _ in range(10):
            again = before.clone()
            assert torch.equal(h.forward(plan, *args, again, chunk=64), out) and torch.equal(again, x["states"])


def even_lengths(R, n):
    return [n * (r + 1) // R - n * r // R for r in range(R)]


def edge_cases():
    """(d_k, requests, tokens, blocks of the default form): both sides of every rule's edge at d_v 128, 16
    value heads."""
    few = sms() // 64            # requests whose CTAs of 32 state rows have an SM each
    full = -(-sms() // 16)       # requests with at least a head per SM
    return [(128, few, 300, 32), (128, few + 1, 256, 32), (128, few + 1, 257, 64),
            (64, full, 8191, 32), (64, full, 8192, 64), (64, full - 1, 8192, 32)]


@pytest.mark.parametrize("case", range(6))
def test_default_blocks_at_the_edges_of_their_rules(case):
    dk, R, n, blocks = edge_cases()[case]
    lens = even_lengths(R, n)
    x, pool = draw(lens, 8, 16, dk, 128, "bf16", seed=n + R)
    h = handle_for(lens, 8, 16, dk, 128, "bf16", pool)
    plan = make_plan(h, lens, [1] * R, x["slots"])
    got = {}
    for chunk in (0, 32, 64):
        states = x["states"].clone()
        got[chunk] = h.forward(plan, *(x[y] for y in ("q", "k", "v", "gate", "beta")), states, chunk=chunk), states
    assert h.status() == la.LA_OK
    same = {c: all(torch.equal(a, b) for a, b in zip(got[0], got[c])) for c in (32, 64)}
    assert same[blocks] and not same[96 - blocks]


def test_a_larger_step_of_64_channels_runs_its_short_requests_beside_blocks_of_64():
    lens = [700, 1, 4, 33, 2] * 12
    R, Hv = len(lens), 16
    assert sum(lens) * Hv >= 1 << 17 and R * Hv > sms()
    x, pool = draw(lens, 8, Hv, 64, 128, "bf16", seed=77)
    h = handle_for(lens, 8, Hv, 64, 128, "bf16", pool)
    plan = make_plan(h, lens, [r % 2 for r in range(R)], x["slots"])
    args = [x[n] for n in ("q", "k", "v", "gate", "beta")]
    mixed, blocks, tokens = (x["states"].clone() for _ in range(3))
    o1 = h.forward(plan, *args, mixed)
    assert h.last_launches() == 2
    o2 = h.forward(plan, *args, blocks, chunk=64)
    o3 = h.decode_step(plan, *args, tokens)
    assert h.status() == la.LA_OK
    at = 0
    for r, n in enumerate(lens):
        o, st = (o3, tokens) if n <= 4 else (o2, blocks)
        s = x["slots"][r]
        assert torch.equal(o1[at:at + n], o[at:at + n]) and torch.equal(mixed[s], st[s]), r
        at += n


@pytest.mark.parametrize("dk,chunk", [(64, 1), (128, 1), (64, 64), (128, 64)])
def test_bits_do_not_depend_on_the_other_requests(dk, chunk):
    # chunk 1 and 64: one request in a step of its own gives what it gives among many others
    rng = random.Random(dk + chunk)
    lens = [rng.choice((1, 3, 20, 64, 130)) for _ in range(60)]
    lens[20] = 150
    x, pool = draw(lens, 4, 8, dk, 128, "bf16", seed=dk)
    h = handle_for(lens, 4, 8, dk, 128, "bf16", pool)
    names, start = ("q", "k", "v", "gate", "beta"), x["states"].clone()
    out = h.forward(make_plan(h, lens, [1] * 60, x["slots"]), *(x[n] for n in names), x["states"], chunk=chunk)
    for r in (0, 20, 59):
        a, s = sum(lens[:r]), x["slots"][r]
        own = start.clone()
        o = h.forward(make_plan(h, [lens[r]], [1], [s]), *(x[n][a:a + lens[r]].clone() for n in names), own, chunk=chunk)
        assert h.status() == la.LA_OK
        assert torch.equal(o, out[a:a + lens[r]]) and torch.equal(own[s], x["states"][s])


def test_a_prompt_in_two_steps_is_the_prompt():
    lens = [200]
    x, pool = draw(lens, 1, 2, 128, 128, "bf16", seed=12)
    h = handle_for(lens, 1, 2, 128, 128, "bf16", pool)
    t = lambda a, e: [x[n][a:e] for n in ("q", "k", "v", "gate", "beta")]   # noqa: E731
    before = x["states"].clone()
    out = torch.empty(200, 2, 128, device="cuda", dtype=torch.bfloat16)
    for a, e in ((0, 77), (77, 78), (78, 200)):
        plan = make_plan(h, [e - a], [a], x["slots"])
        h.forward(plan, *t(a, e), x["states"], out=out[a:e])
    # blocks elsewhere, so the bound of each part's own blocks adds up: three times the one call's is above it
    d = lambda y: y.double().cpu().numpy()   # noqa: E731
    for hd in range(2):
        want, X, bo, E = ref.rule_by_blocks(*(d(x[n])[:, 0] for n in ("q", "k")), d(x["v"])[:, hd],
                                            d(x["gate"])[:, hd], d(x["beta"])[:, hd], np.zeros((128, 128)))
        assert np.all(np.abs(d(out)[:, hd] - want) <= 3 * bo)
        assert np.linalg.norm(d(x["states"])[x["slots"][0], hd] - X) <= 3 * E
    assert not torch.equal(before, x["states"])


def test_offsets_past_32_bits():
    # states: slot 65600 of [2, 128, 128] lies past 2^31 elements; rows: 2^21 rows of 1088 elements
    # lie past 2^31 elements too, before the request that takes part (the first has no slot: no part)
    Hk, Hv, d = 1, 2, 128
    skip, n = 2 ** 21, 70
    pool = 65601
    h = la.PackedHandle(max_requests=2, max_tokens=skip + n, slots=pool, H_k=Hk, H_v=Hv, d_k=d, d_v=d)
    states = torch.zeros(pool, Hv, d, d, device="cuda")
    x, _ = draw([n], Hk, Hv, d, d, "bf16", seed=2)
    wide = torch.zeros(skip + n, 1088, device="cuda", dtype=torch.bfloat16)
    packed = {}
    at = 0
    for name, heads in (("q", Hk), ("k", Hk), ("v", Hv)):
        packed[name] = wide[:, at:at + heads * d].view(skip + n, heads, d)
        packed[name][skip:] = x[name]
        at += heads * d
    for name in ("gate", "beta"):
        packed[name] = torch.ones(skip + n, Hv, device="cuda")
        packed[name][skip:] = x[name]
    slot = pool - 1
    start = torch.randn(Hv, d, d, device="cuda") * 0.5
    plan = h.plan(i32([skip, n]), i32([4, 4]), i32([-1, slot]), i32([0] * pool), i32([0]), tokens=skip + n)
    assert plan.counts.tolist() == [skip + n, 1, 0, la.LA_PLAN_FAULT_STATE]
    out = torch.zeros(skip + n, Hv, d, device="cuda", dtype=torch.bfloat16)
    for chunk in (64, 32, 1):
        states[slot] = start
        h.forward(plan, packed["q"], packed["k"], packed["v"], packed["gate"], packed["beta"], states, out=out, chunk=chunk)
        assert h.status() == la.LA_OK
        y = dict(x, states=states[slot:], slots=[0])
        check(y, [n], [1], start[None], out[skip:], "bf16", chunk)
        assert not out[:skip].any() and not states[:slot].any()


# ------------------------------------------------------------------ a serving loop

class Server:
    """Requests over several steps: the device side through the library, the
    references kept per request in float64."""

    def __init__(self, Hk=2, Hv=4, dk=64, dv=64, pool=9, max_requests=6, max_tokens=200, seed=0):
        self.dims, self.pool, self.R, self.N = (Hk, Hv, dk, dv), pool, max_requests, max_tokens
        self.h = la.PackedHandle(max_requests=max_requests, max_tokens=max_tokens, slots=pool, H_k=Hk, H_v=Hv, d_k=dk, d_v=dv)
        self.states = torch.full((pool, Hv, dv, dk), float("nan"), device="cuda")
        self.lengths, self.seen, self.slots = i32([0] * self.R), i32([0] * self.R), i32([-1] * self.R)
        self.free, self.count = i32(list(range(pool))), i32([pool])
        self.plan = self.h.new_plan()
        self.x, _ = draw([max_tokens], Hk, Hv, dk, dv, "bf16", seed)
        self.out = torch.zeros(max_tokens, Hv, dv, device="cuda", dtype=torch.bfloat16)
        self.want = [None] * self.R    # per request: [tokens, state per head, state error per head]

    def step(self, decode):
        """What a program enqueues for a step; capturable."""
        self.h.plan(self.lengths, self.seen, self.slots, self.free, self.count, tokens=self.N, plan=self.plan)
        f = self.h.decode_step if decode else self.h.forward
        f(self.plan, *(self.x[n] for n in ("q", "k", "v", "gate", "beta")), self.states, out=self.out)

    def feed(self, lens, seed):
        x, _ = draw([self.N], *self.dims, "bf16", seed)
        for n in ("q", "k", "v", "gate", "beta"):
            self.x[n].copy_(x[n])
        self.lengths.copy_(i32(lens))
        self.seen.copy_(i32([w[0] if w else 0 for w in self.want]))

    def check(self, lens, decode):
        torch.cuda.synchronize()
        assert self.h.status() == la.LA_OK and self.plan.counts.tolist()[3] == 0
        Hk, Hv, dk, dv = self.dims
        d = lambda t: t.double().cpu().numpy()   # noqa: E731
        q, k, v, g, b = (d(self.x[n]) for n in ("q", "k", "v", "gate", "beta"))
        states, out, slots, row = d(self.states), d(self.out), self.slots.tolist(), 0
        held = [s for s in slots if s >= 0]
        free = self.free.tolist()[:int(self.count)]
        assert sorted(held + free) == list(range(self.pool))       # no slot lost, none twice
        for r, n in enumerate(lens):
            if n < 0:
                self.want[r] = None
                assert slots[r] == -1
            if n > 0:
                w = self.want[r] or [0, [np.zeros((dv, dk))] * Hv, [0.0] * Hv]
                s, new = slice(row, row + n), [w[0] + n, [], []]
                for h in range(Hv):
                    hk = h * Hk // Hv
                    args = (q[s, hk], k[s, hk], v[s, h], g[s, h], b[s, h], w[1][h])
                    o, X, bo, E = ref.rule_by_tokens(*args, ref.H) if decode else ref.rule_by_blocks(*args)
                    carried = w[2][h] * (1 + np.linalg.norm(q[s, hk], axis=1).max() * n)   # of the state before
                    assert np.all(np.abs(out[s, h] - o) <= bo + carried)
                    E += w[2][h]
                    assert np.linalg.norm(states[slots[r], h] - X) <= E
                    new[1].append(X)
                    new[2].append(E)
                self.want[r] = new
                row += n


STEPS = [([40, 3, 0, 65, 1, 33], False), ([1, 1, 10, 1, 1, 1], False), ([1, 2, 1, 1, 3, 1], True), ([-1, 1, 1, 0, -1, 1], True),
         ([90, 1, 1, 1, 50, 1], False), ([1, 1, 1, 1, 1, 1], True), ([-1] * 6, True), ([5, 0, 0, 0, 0, 100], False)]


def test_serving_steps():
    s = Server()
    for i, (lens, decode) in enumerate(STEPS):
        s.feed(lens, seed=100 + i)
        s.step(decode)
        s.check(lens, decode)


def test_serving_steps_replayed_from_graphs():
    # one graph of a prefill step and one of a decode step, replayed with new lengths, slots and values
    s = Server(seed=1)
    graphs = {}
    side = torch.cuda.Stream()
    for decode in (False, True):
        graphs[decode] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[decode], stream=side):
            s.step(decode)
    for i, (lens, decode) in enumerate(STEPS):
        s.feed(lens, seed=200 + i)
        graphs[decode].replay()
        s.check(lens, decode)


def test_two_servers_on_two_streams():
    # two handles, then one handle with two plans, pools and outputs, at once on two streams
    for shared in (False, True):
        a, b = Server(seed=3), Server(seed=4)
        if shared:
            b.h = a.h
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for i, (lens, decode) in enumerate(STEPS):
            for j, s in enumerate((a, b)):
                s.feed(lens, seed=300 + 10 * i + j)
            torch.cuda.synchronize()
            for s, st in zip((a, b), streams):
                with torch.cuda.stream(st):
                    s.step(decode)
            torch.cuda.synchronize()
            for s in (a, b):
                s.check(lens, decode)


@pytest.mark.parametrize("dk,chunk", [(128, 64), (64, 64), (128, 0), (64, 32)])
def test_large_steps_at_once_on_two_streams(dk, chunk):
    # one handle, two plans, pools and outputs: more CTAs than SMs each, several calls without a pause
    rng = random.Random(dk)
    lens = [rng.choice((1, 4, 64, 129, 200)) for _ in range(30)]
    h, parts = None, []
    for seed in (1, 2):
        x, pool = draw(lens, 8, 16, dk, 128, "bf16", seed=seed)
        h = h or handle_for(lens, 8, 16, dk, 128, "bf16", pool)
        plan = make_plan(h, lens, [7] * 30, x["slots"])
        args = [x[n] for n in ("q", "k", "v", "gate", "beta")]
        want = x["states"].clone()
        for _ in range(6):
            o = h.forward(plan, *args, want, chunk=chunk)
            torch.cuda.synchronize()
        parts.append((plan, args, x["states"], torch.zeros_like(o), want, o, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(6):
        for plan, args, states, out, _, _, st in parts:
            h.forward(plan, *args, states, out=out, chunk=chunk, stream=st)
    torch.cuda.synchronize()
    assert h.status() == la.LA_OK
    for _, _, states, out, want, o, _ in parts:
        assert torch.equal(states, want) and torch.equal(out, o)


def test_a_stream_given_by_argument():
    lens = [50, 9]
    x, pool = draw(lens, 1, 2, 64, 64, "bf16", seed=31)
    h = handle_for(lens, 1, 2, 64, 64, "bf16", pool)
    st = torch.cuda.Stream()
    before = x["states"].clone()
    args = [i32(lens), i32([1, 1]), i32(x["slots"]), i32([0] * pool), i32([0])]
    torch.cuda.synchronize()
    plan = h.plan(*args, tokens=59, stream=st)
    out = h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], stream=st)
    assert h.status(stream=st) == la.LA_OK
    check(x, lens, [1, 1], before, out, "bf16", 32)


# ------------------------------------------------------------------ refusals

def test_python_refuses_wrong_tensors():
    lens = [5, 4]
    x, pool = draw(lens, 2, 2, 64, 64, "bf16", seed=1)
    h = handle_for(lens, 2, 2, 64, 64, "bf16", pool)
    plan = make_plan(h, lens, [0, 0], x["slots"])
    good = [x[n] for n in ("q", "k", "v", "gate", "beta", "states")]
    bad = [(0, x["q"].float()), (0, x["q"].cpu()), (0, x["q"][:8]), (0, x["q"].transpose(1, 2)), (1, x["k"][:, :1]),
           (2, x["v"].transpose(0, 1).contiguous().transpose(0, 1)), (3, x["gate"].half()), (3, x["gate"].t()),
           (4, x["beta"][:, :1]), (5, x["states"].bfloat16()), (5, x["states"][:-1]), (5, x["states"].transpose(2, 3))]
    before = x["states"].clone()
    for i, t in bad:
        args = list(good)
        args[i] = t
        with pytest.raises(ValueError):
            h.forward(plan, *args)
    with pytest.raises(ValueError):
        h.forward(plan, *good, out=torch.empty(9, 2, 64, device="cuda"))
    with pytest.raises(ValueError):
        make_plan(h, [1, 1], [0, 0], [0])
    with pytest.raises(ValueError):
        h.plan(i32([1]), i32([1]).long(), i32([0]), i32([0] * pool), i32([0]), tokens=1)
    with pytest.raises(ValueError):   # a plan of other maxima
        h.forward(handle_for([1], 2, 2, 64, 64, "bf16", pool).new_plan(), *good)
    heads = dict(H_k=1, H_v=1, d_k=16, d_v=16)   # of as many words, laid out otherwise
    one, other = la.PackedHandle(max_requests=2, max_tokens=4, slots=16, **heads), la.PackedHandle(max_requests=2, max_tokens=8, slots=8, **heads)
    assert one.new_plan().words.numel() == other.new_plan().words.numel()
    with pytest.raises(ValueError):
        one.plan(i32([1]), i32([0]), i32([-1]), i32([0] * 16), i32([1]), tokens=1, plan=other.new_plan())
    torch.cuda.synchronize()
    assert torch.equal(before, x["states"])


def test_a_buffer_without_a_plan_is_refused():
    for n in (0, 1, 9):
        x, pool = draw([9], 2, 2, 64, 64, "bf16", seed=1)
        h = handle_for([9], 2, 2, 64, 64, "bf16", pool)
        with pytest.raises(ValueError, match="no step has been planned|shape"):
            h.forward(h.new_plan(), *(x[y][:n] for y in ("q", "k", "v", "gate", "beta")), x["states"])
    with pytest.raises(ValueError, match="no step has been planned"):
        h.decode_step(h.new_plan(), *(x[y][:0] for y in ("q", "k", "v", "gate", "beta")), x["states"])


def test_the_library_refuses_before_it_launches():
    lens = [5, 4]
    x, pool = draw(lens, 2, 2, 64, 64, "bf16", seed=1)
    h = handle_for(lens, 2, 2, 64, 64, "bf16", pool)
    plan = make_plan(h, lens, [0, 0], x["slots"])
    out = torch.zeros(9, 2, 64, device="cuda", dtype=torch.bfloat16)
    P = [plan.words.data_ptr(), *(x[n].data_ptr() for n in ("q", "k", "v", "gate", "beta", "states")), out.data_ptr()]
    L, stream = la.lib(), torch.cuda.current_stream().cuda_stream
    call = lambda p=P, R=2, n=9, s=(128, 128, 128), chunk=0: L.la_packed_forward(h._h, *p, R, n, *s, chunk, stream)   # noqa: E731
    for i in range(8):
        assert call([None if j == i else y for j, y in enumerate(P)]) == la.LA_ERR_INVALID_ARG
        assert call([y + (2 if i in (4, 5) else 8) if j == i else y for j, y in enumerate(P)]) == la.LA_ERR_MISALIGNED
    assert call(R=-1) == call(n=-1) == call(R=3) == call(n=10) == la.LA_ERR_INVALID_ARG
    assert call(s=(127, 128, 128)) == call(s=(128, 0, 128)) == call(s=(128, 128, -128)) == la.LA_ERR_INVALID_ARG
    assert call(s=(129, 128, 128)) == call(s=(128, 132, 128)) == la.LA_ERR_MISALIGNED
    assert call(s=(1 << 40, 128, 128)) == la.LA_ERR_UNSUPPORTED
    assert call(chunk=64) == call(chunk=2) == call(chunk=-1) == la.LA_ERR_UNSUPPORTED
    assert L.la_packed_last_launches(h._h) == 0 and L.la_packed_last_error(h._h)
    assert call(R=0) == call(n=0) == la.LA_OK and L.la_packed_last_launches(h._h) == 0
    ints = [i32([1, 1]).data_ptr(), i32([1, 1]).data_ptr(), i32([0, 1]).data_ptr(), i32([0] * pool).data_ptr(),
            i32([0]).data_ptr(), plan.words.data_ptr()]
    pl = lambda p=ints, R=2, n=9: L.la_packed_plan(h._h, *p, R, n, stream)   # noqa: E731
    for i in range(6):
        assert pl([None if j == i else y for j, y in enumerate(ints)]) == la.LA_ERR_INVALID_ARG
        assert pl([y + 1 if j == i else y for j, y in enumerate(ints)]) == la.LA_ERR_MISALIGNED
    assert pl([y + 4 if j == 5 else y for j, y in enumerate(ints)]) == la.LA_ERR_MISALIGNED
    assert pl(R=3) == pl(n=10) == pl(R=-1) == pl(n=-1) == la.LA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert not out.any()


def test_a_buffer_no_plan_was_made_in_reaches_nothing():
    # any words: the kernels take only what lies inside the tensors; here no word does
    lens = [40, 20]
    for words in (-1, 0, 2 ** 31 - 1, -2 ** 31, 1000):
        x, pool = draw(lens, 1, 1, 64, 128, "bf16", seed=6)
        h = handle_for(lens, 1, 1, 64, 128, "bf16", pool)
        plan = make_plan(h, lens, [1, 1], x["slots"])
        plan.words.fill_(words)
        before = x["states"].clone()
        out = torch.zeros(60, 1, 128, device="cuda", dtype=torch.bfloat16)
        for chunk in (1, 32, 64):
            h.forward(plan, x["q"], x["k"], x["v"], x["gate"], x["beta"], x["states"], out=out, chunk=chunk)
        assert h.status() == la.LA_OK
        assert not out.any() and torch.equal(before, x["states"])
