"""The packed gated delta rule on the CPU: configurations that are refused,
null handles, the plan buffer's layout, and the reference of the GPU tests
against the oracle and against its own definition."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import _packed as ref
import gated_delta_rule_causal_gb300 as la
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    la.build()
    return la.lib()


GOOD = dict(max_requests=8, max_tokens=100, slots=10, H_k=2, H_v=4, d_k=64, d_v=128, io=0, flags=0, device=0)


def config(**kw):
    return la.la_packed_config(*{**GOOD, **kw}.values())


@pytest.mark.parametrize("change,code", [
    (dict(max_requests=0), la.LA_ERR_INVALID_ARG),
    (dict(max_tokens=0), la.LA_ERR_INVALID_ARG),
    (dict(slots=0), la.LA_ERR_INVALID_ARG),
    (dict(H_k=0), la.LA_ERR_INVALID_ARG),
    (dict(H_v=-4), la.LA_ERR_INVALID_ARG),
    (dict(H_k=3), la.LA_ERR_INVALID_ARG),        # value heads do not divide
    (dict(H_k=8), la.LA_ERR_INVALID_ARG),        # more key heads than value heads
    (dict(io=2), la.LA_ERR_INVALID_ARG),
    (dict(flags=1), la.LA_ERR_INVALID_ARG),
    (dict(d_k=96), la.LA_ERR_UNSUPPORTED),
    (dict(d_v=256), la.LA_ERR_UNSUPPORTED),
    (dict(max_requests=16385), la.LA_ERR_UNSUPPORTED),
    (dict(max_tokens=(1 << 24) + 1), la.LA_ERR_UNSUPPORTED),
])
def test_configurations_refused(lib, change, code):
    h = ctypes.c_void_p()
    c = config(**change)
    assert lib.la_packed_create(ctypes.byref(c), ctypes.byref(h)) == code and not h.value
    assert lib.la_packed_plan_words(ctypes.byref(c)) == 0


def test_null_arguments(lib):
    h = ctypes.c_void_p()
    assert lib.la_packed_create(None, ctypes.byref(h)) == la.LA_ERR_INVALID_ARG
    assert lib.la_packed_create(ctypes.byref(config()), None) == la.LA_ERR_INVALID_ARG
    assert lib.la_packed_plan_words(None) == 0
    n = None
    assert lib.la_packed_plan(n, n, n, n, n, n, n, 1, 1, n) == la.LA_ERR_INVALID_ARG
    assert lib.la_packed_forward(n, n, n, n, n, n, n, n, n, 1, 1, 8, 8, 8, 0, n) == la.LA_ERR_INVALID_ARG
    assert lib.la_packed_decode_step(n, n, n, n, n, n, n, n, n, 1, 1, 8, 8, 8, n) == la.LA_ERR_INVALID_ARG
    assert lib.la_packed_status(n, n) == la.LA_ERR_INVALID_ARG
    assert lib.la_packed_last_launches(n) == 0
    assert lib.la_packed_last_error(n) == b"null handle"
    lib.la_packed_destroy(n)


def test_create_without_gpu_reports_cuda(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    h = ctypes.c_void_p()
    assert lib.la_packed_create(ctypes.byref(config()), ctypes.byref(h)) == la.LA_ERR_CUDA and not h.value


@pytest.mark.parametrize("R,N,S", [(1, 1, 1), (8, 100, 10), (5, 4097, 3), (16384, 1 << 24, 7)])
def test_plan_sections_agree_with_the_header(lib, tmp_path, R, N, S):
    # the binding's views against the C macros, and the sections against the buffer's size
    src = tmp_path / "words.c"
    src.write_text('#include "la.h"\n#include <stdio.h>\nint main(void) { printf("%d %d %lld %lld %lld %lld\\n", LA_PLAN_COUNTS, '
                   f"LA_PLAN_OFFSETS, LA_PLAN_SLOTS({R}), LA_PLAN_ORDER({R}), LA_PLAN_TOKEN_REQUEST({R}), "
                   f"LA_PLAN_TOKEN_POSITION({R}, {N})); return 0; }}\n")
    exe = tmp_path / "words"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    at = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    words = lib.la_packed_plan_words(ctypes.byref(config(max_requests=R, max_tokens=N, slots=S)))
    assert all(x % 4 == 0 for x in at) and words % 4 == 0
    assert words >= at[-1] + N + S
    p = la.PackedPlan(config(max_requests=R, max_tokens=N, slots=S), words, "cpu")
    p._set(R, N)
    views = (p.counts, p.offsets, p.state_slots, p.order, p.token_request, p.token_position)
    assert [v.storage_offset() for v in views] == at
    assert [v.numel() for v in views] == [4, R + 1, R, R, N, N]


def test_a_plan_has_sections_once_a_step_is_planned(lib):
    c = config()
    p = la.PackedPlan(c, lib.la_packed_plan_words(ctypes.byref(c)), "cpu")
    for name in ("counts", "offsets", "state_slots", "order", "token_request", "token_position"):
        with pytest.raises(ValueError, match="no step has been planned"):
            getattr(p, name)
    p._set(0, 0)
    assert p.counts.numel() == 4 and p.offsets.numel() == 1 and p.order.numel() == 0


def test_fault_numbers_agree():
    src = open(os.path.join(ROOT, "include", "la.h")).read()
    for name in ("ROWS", "FREE", "SLOT", "OWNER", "STATE", "OVERFLOW"):
        value = int(re.search(rf"LA_PLAN_FAULT_{name} = (\d+)", src).group(1))
        assert value == getattr(la, "LA_PLAN_FAULT_" + name) == getattr(ref, "FAULT_" + name)


@pytest.mark.parametrize("T", [1, 31, 32, 33, 100])
def test_reference_is_the_oracles_rule(T):
    rng = np.random.default_rng(T)
    dk, dv = 64, 16
    q, k, v = rng.standard_normal((T, dk)), rng.standard_normal((T, dk)), rng.standard_normal((T, dv))
    k /= np.linalg.norm(k, axis=1, keepdims=True)
    g, b = rng.uniform(0.3, 1.0, T), rng.uniform(0, 1, T)
    X = rng.standard_normal((dv, dk))
    r = oracle.run("gdn", q[None, None], k[None, None], v[None, None], g[None, None], b[None, None], X.reshape(1, 1, -1))
    for f, arg in ((ref.rule_by_blocks, 32), (ref.rule_by_tokens, ref.H)):
        o, Y, bo, E = f(q, k, v, g, b, X, arg)
        np.testing.assert_allclose(o, r.o[0, 0], rtol=0, atol=1e-11)
        np.testing.assert_allclose(Y.ravel(), r.state.ravel(), rtol=0, atol=1e-11)
        # the bounds say something: far below the values themselves
        assert np.all(bo > 0) and np.linalg.norm(bo) < 0.25 * np.linalg.norm(o) and E < 2e-2 * np.linalg.norm(Y)


def test_reference_plan_by_hand():
    p = ref.plan([3, -1, 2, 0, 4], [5, 9, 0, 1, 0], [7, 2, -1, 4, -1], [8, 6, 0, 0, 0, 0, 0, 0, 0], 1, 9, 12)
    assert p["offsets"] == [0, 3, 3, 5, 5, 9]
    assert p["slots"] == [7, -1, 2, 4, 8] and p["free_count"] == [0]      # 2 comes back on top, then 8
    assert p["state_slots"] == [7, -1, 2, -1, 8] and p["counts"] == [9, 3, 0, 0]
    assert p["order"] == [0, 2, 4, 1, 3]
    assert p["token_request"] == [0, 0, 0, 2, 2, 4, 4, 4, 4, -1, -1, -1]
    assert p["token_position"] == [5, 6, 7, 0, 1, 0, 1, 2, 3, -1, -1, -1]
