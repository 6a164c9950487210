"""The operators around the sequential head, on the CPU: their 64-bit
definitions against differences, closed forms and each other, and the host
checks of every entry point, which answer before any launch."""
import ctypes
import os
import re

import numpy as np
import pytest

import draft_sampling_verification_head_b200 as sd
from oracle import head_ops as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)


# ---- definitions ------------------------------------------------------------------
def test_embed_grad_is_the_transpose_of_embed():
    rng = np.random.default_rng(0)
    table, ids = rng.standard_normal((11, 5)), np.array([3, 0, 3, -1, 10, 11, 3])
    d = rng.standard_normal((len(ids), 5))
    g, _, n = H.embed_grad(ids, d, 0.5, np.zeros_like(table))
    assert n.sum() == 5 and n[3] == 3
    # <embed(table), d> is linear in the table: its gradient is embed_grad(d)
    for v in range(11):
        e = np.zeros_like(table)
        e[v, 2] = 1.0
        assert np.isclose((H.embed(e, ids, 0.5) * d).sum(), g[v, 2], atol=1e-14)


def _scan_loss(gate, x, h0, lens, dh, dl):
    h, last, _, _ = H.gated_scan(gate, x, h0, lens)
    return np.nansum(np.where(np.isnan(h), 0.0, h) * dh) + (last * dl).sum()


def test_scan_gradient_against_differences():
    rng = np.random.default_rng(1)
    B, T, D = 3, 7, 2
    gate, x, dh = (rng.standard_normal((B, T, D)) for _ in range(3))
    h0, dl = rng.standard_normal((B, D)), rng.standard_normal((B, D))
    lens = np.array([7, 0, 4])
    (dg, dx, d0), _ = H.gated_scan_grad(gate, x, h0, lens, dh, dl)
    eps = 1e-6
    for name, a, g in (("gate", gate, dg), ("x", x, dx), ("h0", h0, d0)):
        for at in np.ndindex(a.shape):
            keep = a[at]
            a[at] = keep + eps
            up = _scan_loss(gate, x, h0, lens, dh, dl)
            a[at] = keep - eps
            down = _scan_loss(gate, x, h0, lens, dh, dl)
            a[at] = keep
            # central differences: truncation ~ eps^2, cancellation ~ 1e-16 / eps
            assert abs((up - down) / (2 * eps) - g[at]) < 1e-8, (name, at)


def test_scan_closed_forms():
    """A constant gate gives a geometric mean of the inputs; a saturated one
    keeps the state, or copies the input."""
    T = 9
    x = np.arange(1.0, T + 1).reshape(1, T, 1)
    h, last, _, _ = H.gated_scan(np.zeros((1, T, 1)), x, np.zeros((1, 1)), np.array([T]))
    want = sum(0.5 ** (T - t) * (t + 1) for t in range(T))
    assert np.isclose(last[0, 0], want, atol=1e-12)
    _, last, _, _ = H.gated_scan(np.full((1, T, 1), 800.0), x, np.ones((1, 1)), np.array([T]))
    assert last[0, 0] == 1.0
    with np.errstate(over="ignore"):
        h, _, _, _ = H.gated_scan(np.full((1, T, 1), -800.0), x, np.ones((1, 1)), np.array([T]))
    assert np.array_equal(h, x)


def test_w4_packing_is_a_bijection_and_matches_the_stated_layout():
    rng = np.random.default_rng(2)
    for r in (32, 96, 128, 160, 256):
        codes = rng.integers(0, 16, (5, r))
        wq = H.w4_pack(codes)
        assert wq.shape == (5, -(-r // 128) * 64)
        assert np.array_equal(H.w4_unpack(wq, r), codes)
        if r % 128 == 0:  # the header's words: 16 bytes hold one word of each 32 features
            nat = codes[:, 0::2] | codes[:, 1::2] << 4
            t = nat.reshape(5, r // 128, 4, 4, 4).transpose(0, 1, 3, 2, 4).reshape(5, -1)
            assert np.array_equal(wq, t)


def test_verify_probs_preserves_the_target_distribution():
    """Exact law by integrating the uniforms out: with one draft drawn from q,
    the emitted token has the target's distribution."""
    rng = np.random.default_rng(3)
    V, n = 5, 4000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    got = np.zeros(V)
    grid = (np.arange(n) + 0.5) / n
    for d in range(V):
        # share of accepted u, then the residual law of the rest on a fine grid
        acc = np.mean([u * q[d] < p[d] for u in grid])
        got[d] += q[d] * acc
        if acc < 1:
            t = np.broadcast_to(np.stack([p, p]), (n, 2, V))
            o, tau, _, _ = H.verify_probs(t, np.broadcast_to(q, (n, 1, V)), np.full((n, 1), d),
                                          np.full((n, 1), 1 - 1e-9), grid)
            assert np.all(tau == 1)
            got += q[d] * (1 - acc) * np.bincount(o[:, 0], minlength=V) / n
    # each grid average is off by at most a few of its n cells
    assert np.max(np.abs(got - p)) < 3 * V / n


def test_verify_probs_worked_cases():
    p = np.array([[[0.25, 0.25, 0.5, 0.0], [0.5, 0.5, 0.0, 0.0], [0.0, 0.0, 0.0, 1.0]]])
    q = np.array([[[0.5, 0.25, 0.25, 0.0], [0.25, 0.25, 0.25, 0.25]]])
    d = np.array([[0, 1]])
    # u q = p is not accepted; the residual at 0 is (0, 0, 1/4, 0)
    o, tau, pd, qd = H.verify_probs(p, q, d, np.array([[0.5, 0.0]]), np.array([0.9]))
    assert o.tolist() == [[2, -1, -1]] and tau[0] == 1 and pd[0, 0] == 0.25 and np.isnan(pd[0, 1])
    o, tau, _, _ = H.verify_probs(p, q, d, np.array([[0.49, 0.5]]), np.array([0.0]))
    assert o.tolist() == [[0, 1, 3]] and tau[0] == 3
    # length 1: the bonus comes from row 1; u total = a boundary goes past it
    o, tau, _, _ = H.verify_probs(p, q, d, np.array([[0.0, 0.0]]), np.array([0.5]), [1])
    assert o.tolist() == [[0, 1, -1]] and tau[0] == 2
    o, tau, _, _ = H.verify_probs(p, q, d, np.array([[0.0, 0.0]]), np.array([0.5]), [0])
    assert o.tolist() == [[2, -1, -1]] and tau[0] == 1
    # a row without mass
    o, tau, _, _ = H.verify_probs(p * 0, q, d, np.array([[0.0, 0.0]]), np.array([0.5]))
    assert o.tolist() == [[-1, -1, -1]] and tau[0] == 0


# ---- host checks --------------------------------------------------------------------
STRUCTS = [("spec_embed_params", sd.SpecEmbedParams), ("spec_scan_params", sd.SpecScanParams),
           ("spec_w4_params", sd.SpecW4Params), ("spec_probs_params", sd.SpecProbsParams)]


@pytest.mark.parametrize("name,mirror", STRUCTS, ids=[s[0] for s in STRUCTS])
def test_struct_mirrors_match_the_c_compiler(name, mirror, tmp_path):
    import shutil
    import subprocess
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "specdec.h")).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
    ctype = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    fields = [(n, ctype[t]) for t, n in re.findall(r"\b(int\d+_t|float)\s+(\w+)\s*;", body)]
    assert fields == list(mirror._fields_)
    if shutil.which("gcc") is None:
        pytest.skip("no host C compiler")
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "specdec.h"', "int main(void) {",
             f'  printf("%zu\\n", sizeof({name}));']
    lines += [f'  printf("%zu\\n", offsetof({name}, {n}));' for n, _ in fields]
    (tmp_path / "p.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "p"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "p.c"),
                    "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, n).offset for n, _ in fields]


def _call(fn, p, *args):
    return getattr(sd.lib(), fn)(None if p is None else ctypes.byref(p.c()), *args)


def _embed(**kw):
    d = dict(n=4, V=10, D=8)
    d.update(kw)
    return sd.EmbedParams(**d)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(V=0), dict(D=0), dict(D=65537),
                                dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(table_stride=7), dict(row_stride=-8)])
@pytest.mark.parametrize("fn", ["spec_embed", "spec_embed_grad"])
def test_embed_rejects_bad_parameters(fn, kw):
    p = _embed(**kw)
    assert _call(fn, p, FAKE, FAKE, FAKE, FAKE, None) == sd.SPEC_ERR_INVALID_ARG
    assert sd.workspace_size(p) == 0


@pytest.mark.parametrize("fn", ["spec_embed", "spec_embed_grad"])
def test_embed_rejects_bad_pointers(fn):
    odd = ctypes.c_void_p(0x10001)
    for k in range(3):
        args = [FAKE] * 4
        args[k] = None
        assert _call(fn, _embed(), *args, None) == sd.SPEC_ERR_INVALID_ARG
        args[k] = odd
        assert _call(fn, _embed(), *args, None) == sd.SPEC_ERR_INVALID_ARG
    assert _call(fn, _embed(), FAKE, FAKE, FAKE, None, None) == sd.SPEC_ERR_WORKSPACE
    assert _call(fn, _embed(), FAKE, FAKE, FAKE, ctypes.c_void_p(0x10010), None) == sd.SPEC_ERR_WORKSPACE
    assert _call(fn, None, FAKE, FAKE, FAKE, FAKE, None) == sd.SPEC_ERR_INVALID_ARG


def test_embed_without_tokens_is_no_work():
    assert _call("spec_embed", _embed(n=0), None, None, None, FAKE, None) == sd.SPEC_OK
    assert _call("spec_embed_grad", _embed(n=0, accumulate=True), None, None, None, FAKE,
                 None) == sd.SPEC_OK
    assert sd.last_launch_count() == 0


@pytest.mark.parametrize("fn", ["spec_embed", "spec_embed_grad"])
def test_embed_refuses_more_tokens_than_its_indices_hold(fn):
    p = _embed(n=2**30 + 1)
    assert _call(fn, p, FAKE, FAKE, FAKE, FAKE, None) == sd.SPEC_ERR_UNSUPPORTED
    assert sd.workspace_size(p) == 0
    assert sd.workspace_size(_embed(n=2**30)) > 0


def _scan(**kw):
    d = dict(B=2, T=5, D=8)
    d.update(kw)
    return sd.ScanParams(**d)


def test_scan_host_checks():
    bad, ws = sd.SPEC_ERR_INVALID_ARG, sd.SPEC_ERR_WORKSPACE

    def fwd(p, gate=FAKE, x=FAKE, h0=None, ln=None, h=FAKE, hl=None, st=None, w=FAKE):
        return _call("spec_gated_scan", p, gate, x, h0, ln, h, hl, st, w, None)

    def bwd(p, w=FAKE, **kw):
        a = dict(gate=FAKE, x=FAKE, h0=None, ln=None, st=FAKE, dh=FAKE, dl=None, dg=FAKE, dx=FAKE, d0=None)
        a.update(kw)
        return _call("spec_gated_scan_grad", p, *a.values(), w, None)

    for kw in (dict(B=0), dict(T=-1), dict(D=0), dict(gate_stride=7), dict(x_stride=3), dict(h_stride=-1)):
        assert fwd(_scan(**kw)) == bad and bwd(_scan(**kw)) == bad, kw
    assert fwd(_scan(B=70000, D=70000)) == sd.SPEC_ERR_UNSUPPORTED
    assert fwd(None) == bad and bwd(None) == bad
    assert fwd(_scan(), gate=None) == bad and fwd(_scan(), x=None) == bad
    assert fwd(_scan(), h=None) == bad  # nothing to write
    assert fwd(_scan(), w=None) == ws and bwd(_scan(), w=None) == ws
    odd = ctypes.c_void_p(0x10001)
    assert fwd(_scan(), gate=odd) == bad and fwd(_scan(), h0=ctypes.c_void_p(0x10002)) == bad
    for k in ("gate", "x", "st", "dh", "dg", "dx"):
        assert bwd(_scan(), **{k: None}) == bad, k
    # no steps: nothing to do unless the last state or its gradient is wanted
    assert fwd(_scan(T=0), gate=None, x=None) == sd.SPEC_OK
    assert bwd(_scan(T=0), gate=None, x=None, st=None, dh=None, dg=None, dx=None) == sd.SPEC_OK


def test_w4_host_checks():
    bad, uns = sd.SPEC_ERR_INVALID_ARG, sd.SPEC_ERR_UNSUPPORTED

    def run(x=FAKE, prev=None, wq=FAKE, wscale=FAKE, base=None, out=FAKE, w=FAKE, **kw):
        d = dict(B=2, r=64, V=10, group=32, x_rows=3)
        d.update(kw)
        return _call("spec_bias_w4", sd.W4Params(**d), x, prev, wq, wscale, base, out, w, None)

    for kw in (dict(B=0), dict(r=0), dict(V=0), dict(r=65600), dict(x_stride=63), dict(base_stride=9),
               dict(out_stride=9), dict(x=None), dict(wq=None), dict(wscale=None), dict(out=None),
               dict(prev=FAKE, x_rows=0), dict(wq=ctypes.c_void_p(0x10008)),
               dict(out=ctypes.c_void_p(0x10002))):
        assert run(**kw) == bad, kw
    for kw in (dict(group=16), dict(group=48, r=96), dict(r=80), dict(group=128), dict(B=65537),
               dict(V=2**30 + 1)):
        assert run(**kw) == uns, kw
    assert run(w=None) == sd.SPEC_ERR_WORKSPACE
    p = sd.W4Params(B=1, r=64, V=10, group=32)
    assert _call("spec_w4_quantize", p, None, 1, FAKE, FAKE, None) == bad
    assert _call("spec_w4_quantize", p, FAKE, 7, FAKE, FAKE, None) == bad


def test_verify_probs_host_checks():
    bad = sd.SPEC_ERR_INVALID_ARG

    def run(at=None, v=None, w=FAKE, **kw):
        d = dict(B=2, K=3, V=10)
        d.update(kw)
        args = [FAKE] * 5 + [None] + [FAKE] * 2 + [None, None, w]
        if at is not None:
            args[at] = v
        return _call("spec_verify_probs", sd.ProbsParams(**d), *args, None)

    for kw in (dict(B=0), dict(K=0), dict(K=1025), dict(V=0), dict(target_stride=9), dict(draft_stride=-1)):
        assert run(**kw) == bad, kw
    assert run(V=2**30 + 1) == sd.SPEC_ERR_UNSUPPORTED
    for k in (0, 1, 2, 3, 4, 6, 7):
        assert run(at=k) == bad, k
    assert run(at=2, v=ctypes.c_void_p(0x10002)) == bad
    assert run(w=None) == sd.SPEC_ERR_WORKSPACE


# ---- the binding's checks of layouts (no GPU: they look at shapes and strides only) ----
def _rows_ok(t, rows, stride, width):
    try:
        sd._check_rows("t", t, rows, stride, width)
        return True
    except ValueError:
        return False


def test_binding_accepts_rows_where_the_call_looks_for_them():
    import torch
    ok = _rows_ok
    assert ok(torch.zeros(6, 5), 6, 5, 5) and ok(torch.zeros(30), 6, 5, 5)
    assert ok(torch.zeros(2, 3, 5), 6, 5, 5)
    assert ok(torch.zeros(6, 8), 6, 8, 5)            # whole storage, longer rows
    assert ok(torch.zeros(6, 8)[:, :5], 6, 8, 5)     # its view
    assert ok(torch.zeros(2, 3, 8)[..., :5], 6, 8, 5)
    assert ok(torch.zeros(1, 5).expand(1, 5), 1, 5, 5) and ok(torch.empty(0), 0, 5, 5)
    assert ok(torch.zeros(6, 1), 6, 1, 1)


def test_binding_refuses_rows_that_lie_elsewhere():
    import torch
    ok = _rows_ok
    assert not ok(torch.zeros(6, 8)[:, :5], 6, 5, 5)          # dense rows are expected
    assert not ok(torch.zeros(6, 5), 6, 8, 5)                 # wider ones are
    assert not ok(torch.zeros(5, 6).t(), 6, 5, 5)             # columns
    assert not ok(torch.zeros(2, 4, 5)[:, :3], 6, 5, 5)       # a gap between sequences
    assert not ok(torch.zeros(5, 5), 6, 5, 5) and not ok(torch.zeros(29), 6, 5, 5)
    assert not ok(torch.zeros(1, 5).expand(6, 5), 6, 5, 5)    # one row for all
    assert not ok(torch.zeros(12)[::2], 1, 6, 6)
    assert not ok(torch.zeros(4, 8)[:, :4], 4, 4, 4)          # drafts of a longer block


def test_parameter_objects_copy_with_a_structure_of_their_own():
    import copy
    import pickle
    p = sd.ProbsParams(B=2, K=3, V=10)
    assert p.c().V == 10
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert q == p and q.c() is not p.c() and q.c().V == 10


# ---- parameter objects used by several threads ---------------------------------------
class _SlowLibrary:
    """The library, whose first workspace size is asked for takes until `go`."""

    def __init__(self, real):
        import threading
        self.real, self.asked, self.go, self.first = real, threading.Event(), threading.Event(), True

    def __getattr__(self, name):
        f = getattr(self.real, name)
        if not name.endswith("_workspace_size"):
            return f

        def size(p):
            if self.first:
                self.first = False
                self.asked.set()
                assert self.go.wait(20)
            return f(p)
        return size


def test_threads_see_a_parameter_object_whole(monkeypatch):
    """While one thread still asks for the size, another gets the true one, and
    both keep the address of one structure."""
    import threading
    want = sd.workspace_size(sd.EmbedParams(n=200000, V=32000, D=256))
    assert want > sd.SPEC_WORKSPACE_MIN
    slow = _SlowLibrary(sd.lib())
    monkeypatch.setattr(sd, "_lib", slow)
    p, got = sd.EmbedParams(n=200000, V=32000, D=256), []
    t = threading.Thread(target=lambda: got.append(sd.workspace_size(p)))
    t.start()
    assert slow.asked.wait(20)
    try:
        assert sd.workspace_size(p) == want
    finally:
        slow.go.set()
        t.join()
    assert got == [want] and sd.workspace_size(p) == want
    assert p._calls.at == ctypes.addressof(p._calls.c)


def test_many_threads_ask_a_fresh_parameter_object():
    import sys
    import threading
    every = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        want = sd.workspace_size(sd.EmbedParams(n=50000, V=1000, D=64))
        for _ in range(200):
            p, got, gate = sd.EmbedParams(n=50000, V=1000, D=64), [], threading.Barrier(3)

            def ask():
                gate.wait()
                got.append((sd.workspace_size(p), p._calls.at))
            ts = [threading.Thread(target=ask) for _ in range(3)]
            for t in ts:
                t.start()
            for t in ts:
                t.join()
            assert got == [(want, ctypes.addressof(p._calls.c))] * 3
    finally:
        sys.setswitchinterval(every)


def test_a_library_that_is_missing_at_first_leaves_nothing_behind(monkeypatch):
    p = sd.EmbedParams(n=50000, V=1000, D=64)
    real = sd.lib()

    def fails(*_):
        raise RuntimeError("not built")
    with monkeypatch.context() as m:
        m.setattr(sd, "lib", fails)
        with pytest.raises(RuntimeError):
            sd.workspace_size(p)
    assert sd.workspace_size(p) == real.spec_embed_workspace_size(ctypes.byref(p.c()))


def test_a_changed_copy_of_the_structure_changes_no_call():
    p = sd.EmbedParams(n=50000, V=1000, D=64)
    need = sd.workspace_size(p)
    p.c().n = 2**29
    assert p.c().n == 50000 and sd.lib().spec_embed_workspace_size(p._calls.at) == need


# ---- workspace sizes by device --------------------------------------------------------
def test_workspace_sizes_belong_to_a_device(monkeypatch):
    """The recurrence's scratch grows with the device's multiprocessors, and is
    unknown without one: what one device needs is not taken for another's."""
    p = sd.ScanParams(B=1, T=60000, D=64)
    now, sizes = [0], {0: 0, 1: 5000, 2: 9000}
    monkeypatch.setattr(sd.ScanParams, "_size", lambda self: sizes[now[0]])

    def need(dev):  # as the calls look it up
        return p._calls.need.get(dev) or sd._need(p, dev)

    assert sd.workspace_size(p) == 0 and need(0) == 0
    sizes[0] = 7000  # a device has come up since
    assert sd.workspace_size(p) == 7000 and need(0) == 7000
    for dev in (1, 2, 0, 1):
        now[0] = dev
        assert need(dev) == sizes[dev] == sd.workspace_size(p)


# ---- sequences without steps ------------------------------------------------------------
def test_scan_without_steps_and_without_a_last_state():
    """h [B, 0, D] and the states are empty, and empty tensors lie at address 0: no
    work, as for the gradient, and no missing output."""
    none = [None] * 7
    assert _call("spec_gated_scan", _scan(T=0), *none, FAKE, None) == sd.SPEC_OK
    assert sd.last_launch_count() == 0
    assert _call("spec_gated_scan", _scan(T=1), FAKE, FAKE, *none[2:], FAKE, None) == sd.SPEC_ERR_INVALID_ARG
    assert _call("spec_gated_scan", _scan(T=0), *none, None, None) == sd.SPEC_ERR_WORKSPACE
