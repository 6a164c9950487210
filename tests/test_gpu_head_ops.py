"""The operators around the sequential head against their 64-bit definitions
(needs a B200): sizes from one token on, odd widths, strides, empty sequences
and rows, masked places that hold NaN, refusals, streams and graphs.

Tolerances count roundings, with u = 2^-24 (half a step of fp32): a sum of n
fp32 terms is off by at most n u times the sum of their magnitudes, an output
type adds half of its step."""
import numpy as np
import pytest
import torch

import draft_sampling_verification_head_b200 as sd
from oracle import head_ops as H

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
# gates: exponential, sum, reciprocal, product, each within a few units, and the
# two roundings of a step: 16 u bounds them with room for the split evaluation,
# whose products of gates carry one such error per step as the recurrence does
STEP = 16 * U
GUARD = -77.0
# the recurrence may flush what lies below 2^-126 to zero, a few dozen times
TINY = 1e-36


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sd.lib()


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def rand(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(DT[dtype]).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol, what=""):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], want[bad][:3], np.broadcast_to(tol, got.shape)[bad][:3])


def strided(t, extra):
    """The same rows in storage whose rows are `extra` elements further apart,
    guard values between them; (view of the whole storage, rows view)."""
    n, d = t.shape
    whole = torch.full((n, d + extra), GUARD, dtype=t.dtype, device=t.device)
    whole[:, :d] = t
    return whole, whole[:, :d]


# ---------------------------------------------------------------------------
# lookup and its gradient
# ---------------------------------------------------------------------------
EMBED = [(1, 1, 1), (3, 7, 5), (64, 500, 256), (257, 33, 250), (5, 2, 1030), (1000, 3, 64),
         (4097, 900, 36), (70, 100, 4104), (4096, 1500, 70), (2100, 3000, 256),
         (65537, 700, 33), (140000, 1000, 6)]


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("rows", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,D", EMBED)
def test_embed(n, V, D, dtype, rows, pad):
    g = gen(n + V + D)
    whole, table = strided(rand(g, V, D, dtype=dtype), pad)
    ids = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    if n > 2:
        ids[1] = -1
    out = torch.full((n, D + pad), GUARD, dtype=DT[rows], device="cuda")
    p = sd.EmbedParams(n=n, V=V, D=D, dtype=dtype, row_dtype=rows, scale=0.3,
                       table_stride=D + pad, row_stride=D + pad)
    ws = sd.make_workspace(p)
    sd.embed(p, table, ids.cuda(), out, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    want = H.embed(np64(table), ids.numpy(), float(np.float32(0.3)))
    # one product, then the output's rounding
    within(out[:, :D], want, np.abs(want) * (half_step(rows) + 2 * U) + 1e-38)
    assert bool((out[:, D:] == GUARD).all())


def _embed_grad(n, V, D, dtype, rows, pad, acc, ids, g, scale=0.3):
    drows_w, drows = strided(rand(g, n, D, dtype=rows), pad)
    init = rand(g, V, D, dtype=dtype)
    dt_w, dtable = strided(init, pad)
    p = sd.EmbedParams(n=n, V=V, D=D, dtype=dtype, row_dtype=rows, scale=scale, accumulate=acc,
                       table_stride=D + pad, row_stride=D + pad)
    ws = sd.make_workspace(p)
    sd.embed_grad(p, ids.cuda(), drows, dt_w, ws)
    st = sd.sync_status(ws)
    s = float(np.float32(scale))
    start = np64(init) if acc else np.zeros((V, D))
    want, mag, count = H.embed_grad(ids.numpy(), np64(drows), s, start)
    # count - 1 sums, the scale, the add to the table, the output's rounding
    tol = (count[:, None] + 2) * U * mag + np.abs(want) * half_step(dtype) * (1 + 1e-3) + 1e-38
    if acc:
        tol[count == 0] = 0.0  # rows that no token names stay as they were
    within(dt_w[:, :D], want, tol)
    assert bool((dt_w[:, D:] == GUARD).all())
    return st, dt_w


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype,rows", [("f32", "bf16"), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n,V,D", EMBED)
def test_embed_grad(n, V, D, dtype, rows, pad, acc):
    g = gen(n + V + D + 1)
    # squared uniforms: low tokens come often, many not at all
    ids = (torch.rand(n, generator=g) ** 2 * V).to(torch.int32).clamp_(max=V - 1)
    if n > 2:
        ids[n // 2] = -1
    st, _ = _embed_grad(n, V, D, dtype, rows, pad, acc, ids, g)
    assert st == sd.SPEC_OK


@pytest.mark.parametrize("kind", ["one_token", "all_different", "two_runs", "none"])
@pytest.mark.parametrize("n", [1, 700, 9000, 20000])
def test_embed_grad_token_patterns(n, kind):
    V, D = 30000, 40
    ids = {"one_token": torch.full((n,), 17), "all_different": torch.randperm(V, generator=gen(n))[:n],
           "two_runs": torch.where(torch.arange(n) % 3 == 0, V - 1, 0),
           "none": torch.full((n,), -1)}[kind].to(torch.int32)
    st, _ = _embed_grad(n, V, D, "f32", "bf16", 0, False, ids, gen(n + 5))
    assert st == sd.SPEC_OK


def test_embed_grad_same_bits_every_time():
    n, V, D = 20000, 500, 64
    g = gen(9)
    ids = (torch.rand(n, generator=g) ** 3 * V).to(torch.int32).cuda()
    d = rand(g, n, D, dtype="bf16")
    p = sd.EmbedParams(n=n, V=V, D=D, dtype="f32")
    ws = sd.make_workspace(p)
    got = []
    for _ in range(4):
        out = torch.full((V, D), GUARD, device="cuda")
        sd.embed_grad(p, ids, d, out, ws)
        got.append(out)
    assert all(torch.equal(got[0], o) for o in got[1:])


def test_embed_without_tokens():
    p = sd.EmbedParams(n=0, V=6, D=5, dtype="f32")
    ws = sd.make_workspace(p)
    t = torch.full((6, 5), 3.0, device="cuda")
    none = torch.empty(0, 5, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    sd.embed(p, t, ids, none, ws)
    sd.embed_grad(p, ids, none, t, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK and bool((t == 0).all())


@pytest.mark.parametrize("bad", [-2, 10, 2**31 - 1, -2**31])
def test_embed_reports_tokens_out_of_range(bad):
    """They read and write nothing of the table: zeros out, no gradient."""
    n, V, D = 40, 10, 12
    ids = torch.arange(n, dtype=torch.int32) % V
    ids[7] = bad
    p = sd.EmbedParams(n=n, V=V, D=D, dtype="f32", row_dtype="f32")
    ws = sd.make_workspace(p)
    t, out = rand(gen(1), V, D), torch.full((n, D), GUARD, device="cuda")
    sd.embed(p, t, ids.cuda(), out, ws)
    assert sd.sync_status(ws) == sd.SPEC_ERR_TOKEN_RANGE
    assert bool((out[7] == 0).all())
    st, _ = _embed_grad(n, V, D, "f32", "f32", 0, False, ids, gen(2))
    assert st == sd.SPEC_ERR_TOKEN_RANGE


# ---------------------------------------------------------------------------
# gated recurrence
# ---------------------------------------------------------------------------
SCAN = [(1, 1, 1), (2, 1, 64), (64, 1, 256), (3, 5, 7), (1, 16, 33), (2, 17, 64), (2, 100, 130),
        (5, 65, 2), (1, 1000, 66), (3, 2050, 31), (1, 5000, 8), (40, 33, 257),
        # steps split over the GPU
        (1, 6001, 8), (3, 5205, 31), (2, 5120, 66),
        # sequences that fill the GPU, short ones and longer ones
        (1200, 40, 66), (300, 70, 200)]


def scan_inputs(B, T, D, dtype, seed, ragged, pad=0, std=2.0):
    g = gen(seed)
    flat = [rand(g, B * T, D, dtype=dtype, std=std), rand(g, B * T, D, dtype=dtype)]
    if std > 4:  # saturated gates of both signs
        flat[0] += 1.0
    h0 = rand(g, B, D)
    lens = None
    if ragged:
        lens = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
        lens[0] = T
        if B > 1:
            lens[1] = 0
    n = np.full(B, T) if lens is None else lens.numpy()
    if ragged:  # what lies behind a sequence's end is no input
        for t in flat:
            v = t.view(B, T, D)
            for b in range(B):
                v[b, n[b]:] = float("nan")
    return flat[0], flat[1], h0, lens, n


def clean(t, n, B, T, D):
    """float64 inputs with zeros past each sequence's end."""
    a = np64(t).reshape(B, T, D).copy()
    for b in range(B):
        a[b, n[b]:] = 0.0
    return a


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", SCAN)
def test_gated_scan_and_gradient(B, T, D, dtype, ragged):
    pad = 0 if (B + T + D) % 2 else 5
    for std in (2.0, 30.0):
        gate, x, h0, lens, n = scan_inputs(B, T, D, dtype, B + T + D, ragged, std=std)
        G, X, h064 = clean(gate, n, B, T, D), clean(x, n, B, T, D), np64(h0)
        gw, _ = strided(gate, pad)
        xw, _ = strided(x, 2 * pad)
        h = torch.full((B * T, D + pad), GUARD, dtype=DT[dtype], device="cuda")
        last = torch.full((B, D), GUARD, device="cuda")
        nch = -(-T // sd.SPEC_SCAN_CHUNK)
        states = torch.full((B, nch, D), GUARD, device="cuda")
        p = sd.ScanParams(B=B, T=T, D=D, dtype=dtype, gate_stride=D + pad, x_stride=D + 2 * pad,
                          h_stride=D + pad)
        ws = sd.make_workspace(p)
        ln = None if lens is None else lens.cuda()
        sd.gated_scan(p, gw, xw, h0, ln, h, last, states, ws)
        assert sd.sync_status(ws) == sd.SPEC_OK
        want, wlast, before, _ = H.gated_scan(G, X, h064, n)
        err = H.gated_scan_error(G, X, h064, n, STEP)
        hv = np64(h[:, :D]).reshape(B, T, D)
        live = np.arange(T)[None, :] < n[:, None]
        within(hv[live], want[live], (err[:, 1:] + np.abs(want) * half_step(dtype))[live] + TINY, "h")
        assert np.all(hv[~live] == GUARD)  # as it was
        assert bool((h[:, D:] == GUARD).all())
        within(last, wlast, err[:, T] + TINY, "h_last")
        within(states, before[:, ::sd.SPEC_SCAN_CHUNK], err[:, :T:sd.SPEC_SCAN_CHUNK] + TINY, "states")

        dh, dl = rand(gen(T), B * T, D, dtype=dtype), rand(gen(D), B, D)
        if ragged:
            for b in range(B):
                dh.view(B, T, D)[b, n[b]:] = float("nan")
        dhw, _ = strided(dh, pad)
        dg = torch.full((B * T, D + pad), GUARD, dtype=DT[dtype], device="cuda")
        dx = torch.full((B * T, D + 2 * pad), GUARD, dtype=DT[dtype], device="cuda")
        d0 = torch.full((B, D), GUARD, device="cuda")
        sd.gated_scan_grad(p, gw, xw, h0, ln, states, dhw, dl, dg, dx, d0, ws)
        assert sd.sync_status(ws) == sd.SPEC_OK
        (wg, wx, w0), (eg, ex, e0) = H.gated_scan_grad(G, X, h064, n, np64(dh).reshape(B, T, D),
                                                       np64(dl), STEP)
        hs = half_step(dtype)
        within(np64(dg[:, :D]).reshape(B, T, D), wg, eg + np.abs(wg) * hs + TINY, "dgate")
        within(np64(dx[:, :D]).reshape(B, T, D), wx, ex + np.abs(wx) * hs + TINY, "dx")
        within(d0, w0, e0 + np.abs(w0) * U + TINY, "dh0")
        assert bool((dg[:, D:] == GUARD).all()) and bool((dx[:, D:] == GUARD).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_optional_arguments(dtype):
    """No initial state, no lengths, single outputs: the same numbers."""
    B, T, D = 3, 50, 40
    gate, x, _, _, n = scan_inputs(B, T, D, dtype, 4, False)
    p = sd.ScanParams(B=B, T=T, D=D, dtype=dtype)
    ws = sd.make_workspace(p)
    h, last = torch.empty(B, T, D, dtype=DT[dtype], device="cuda"), torch.empty(B, D, device="cuda")
    states = torch.empty(B, 4, D, device="cuda")
    zero = torch.zeros(B, D, device="cuda")
    sd.gated_scan(p, gate, x, zero, torch.full((B,), T, dtype=torch.int32).cuda(), h, last, states, ws)
    h2, last2, st2 = torch.empty_like(h), torch.empty_like(last), torch.empty_like(states)
    sd.gated_scan(p, gate, x, None, None, h2, None, None, ws)
    sd.gated_scan(p, gate, x, None, None, None, last2, None, ws)
    sd.gated_scan(p, gate, x, None, None, None, None, st2, ws)
    assert torch.equal(h, h2) and torch.equal(last, last2) and torch.equal(states, st2)
    dh = rand(gen(3), B, T, D, dtype=dtype)
    a = [torch.empty_like(h), torch.empty_like(h), torch.empty_like(last)]
    b = [torch.empty_like(h), torch.empty_like(h)]
    sd.gated_scan_grad(p, gate, x, zero, None, states, dh, zero, *a, ws)
    sd.gated_scan_grad(p, gate, x, None, None, states, dh, None, *b, None, ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_scan_steps_in_place_equal_the_sequence():
    """Decoding: T = 1 calls whose state goes out over the state that came in
    give the sequence's numbers to rounding."""
    B, T, D = 6, 20, 48
    gate, x, h0, _, n = scan_inputs(B, T, D, "f32", 8, False)
    g3, x3 = gate.view(B, T, D), x.view(B, T, D)
    p1, p = sd.ScanParams(B=B, T=1, D=D, dtype="f32"), sd.ScanParams(B=B, T=T, D=D, dtype="f32")
    ws = sd.make_workspace(p)
    state = h0.clone()
    for t in range(T):
        sd.gated_scan(p1, g3[:, t].contiguous(), x3[:, t].contiguous(), state, None, None, state, None, ws)
    last = torch.empty_like(h0)
    sd.gated_scan(p, gate, x, h0, None, None, last, None, ws)
    G, X = clean(gate, n, B, T, D), clean(x, n, B, T, D)
    e = H.gated_scan_error(G, X, np64(h0), n, STEP)[:, T]
    within(state, np64(last), 2 * e)


@pytest.mark.parametrize("B,T,D,dtype", [(1, 4099, 40, "bf16"), (2, 2048, 7, "f32"), (2, 700, 64, "bf16"),
                                       (1, 6099, 40, "bf16"), (2, 5130, 7, "f32")])
def test_scan_state_in_place_over_long_sequences(B, T, D, dtype):
    """The last state written over the first one: the same bits as apart."""
    gate, x, h0, _, _ = scan_inputs(B, T, D, dtype, 12, False)
    p = sd.ScanParams(B=B, T=T, D=D, dtype=dtype)
    ws = sd.make_workspace(p)
    h, last = torch.empty(B, T, D, dtype=DT[dtype], device="cuda"), torch.empty(B, D, device="cuda")
    h2, state = torch.empty_like(h), h0.clone()
    sd.gated_scan(p, gate, x, h0, None, h, last, None, ws)
    sd.gated_scan(p, gate, x, state, None, h2, state, None, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    assert torch.equal(h, h2) and torch.equal(last, state)


def test_scan_no_steps_and_bad_lengths():
    B, D = 3, 9
    p = sd.ScanParams(B=B, T=0, D=D, dtype="f32")
    ws = sd.make_workspace(p)
    h0, last = rand(gen(1), B, D), torch.empty(B, D, device="cuda")
    empty = torch.empty(0, device="cuda")
    sd.gated_scan(p, empty, empty, h0, None, None, last, None, ws)
    assert torch.equal(last, h0)
    d0 = torch.empty(B, D, device="cuda")
    sd.gated_scan_grad(p, empty, empty, None, None, empty, empty, h0, empty, empty, d0, ws)
    assert torch.equal(d0, h0) and sd.sync_status(ws) == sd.SPEC_OK
    T = 4
    p = sd.ScanParams(B=B, T=T, D=D, dtype="f32")
    gate, x = rand(gen(2), B, T, D), rand(gen(3), B, T, D)
    good, got = torch.empty(B, D, device="cuda"), torch.empty(B, D, device="cuda")
    sd.gated_scan(p, gate, x, h0, torch.tensor([4, 0, 2], dtype=torch.int32).cuda(), None, good, None, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    sd.gated_scan(p, gate, x, h0, torch.tensor([9, -5, 2], dtype=torch.int32).cuda(), None, got, None, ws)
    assert sd.sync_status(ws) == sd.SPEC_ERR_INVALID_ARG
    assert torch.equal(good, got)  # clamped


# ---------------------------------------------------------------------------
# 4-bit vocabulary product
# ---------------------------------------------------------------------------
W4 = [(1, 32, 1, 32), (1, 64, 17, 64), (2, 128, 100, 128), (3, 96, 1000, 32), (1, 256, 5003, 32),
      (7, 320, 129, 64), (16, 384, 2000, 128), (17, 256, 333, 64), (33, 128, 70, 32),
      (5, 4096, 300, 128), (16, 2080, 65, 32), (8, 1024, 4096, 64),
      # vocabularies that fill the GPU
      (1, 32, 9472, 32), (1, 256, 9999, 32), (16, 384, 20001, 128), (3, 96, 40010, 32), (17, 320, 9601, 64),
      (9, 640, 12345, 128), (10, 64, 30000, 64), (33, 128, 19000, 32)]


def w4_inputs(B, r, V, group, dtype, sdtype, g):
    codes = torch.randint(0, 16, (V, r), generator=g).numpy()
    wq = torch.from_numpy(H.w4_pack(codes)).cuda()
    wscale = (torch.rand(V, r // group, generator=g) * 0.02 + 0.001).to(DT[sdtype]).cuda()
    return codes, wq, wscale


@pytest.mark.parametrize("lookup,based", [(False, False), (True, True)])
@pytest.mark.parametrize("dtype,sdtype,odtype", [("bf16", "bf16", "f32"), ("f32", "f32", "f32"),
                                                 ("bf16", "f32", "bf16"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("B,r,V,group", W4)
def test_bias_w4(B, r, V, group, dtype, sdtype, odtype, lookup, based):
    g = gen(B + r + V)
    codes, wq, wscale = w4_inputs(B, r, V, group, dtype, sdtype, g)
    pad = 3 if based else 0
    rows = 11 if lookup else B
    xw, xv = strided(rand(g, rows, r, dtype=dtype), pad)
    prev = torch.randint(0, rows, (B,), generator=g, dtype=torch.int32) if lookup else None
    bdt = dtype
    base = strided(rand(g, B, V, dtype=bdt), pad) if based else None
    out = torch.full((B, V + pad), GUARD, dtype=DT[odtype], device="cuda")
    p = sd.W4Params(B=B, r=r, V=V, group=group, dtype=dtype, scale_dtype=sdtype, base_dtype=bdt,
                    out_dtype=odtype, x_rows=rows, x_stride=r + pad, base_stride=V + pad,
                    out_stride=V + pad)
    ws = sd.make_workspace(p)
    sd.bias_w4(p, xw, None if prev is None else prev.cuda(), wq, wscale,
               None if base is None else base[0], out, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    X = np64(xv) if prev is None else np64(xv)[prev.numpy()]
    b64 = np64(base[1]) if based else np.zeros((B, V))
    want, mag = H.bias_w4(X, codes, np64(wscale), group, b64)
    # r products and their sums in an order of the hardware's, which may cut
    # instead of round (2 u each), one scale per group, the groups' sum, the base
    tol = (2 * r + 2 * (r // group) + 2) * U * mag + np.abs(want) * half_step(odtype) + 1e-38
    within(out[:, :V], want, tol)
    assert bool((out[:, V:] == GUARD).all())


def test_bias_w4_in_place_and_token_range():
    B, r, V, group = 4, 128, 250, 32
    g = gen(5)
    codes, wq, wscale = w4_inputs(B, r, V, group, "bf16", "bf16", g)
    x = rand(g, 6, r, dtype="bf16")
    z = rand(g, B, V)
    want, _ = H.bias_w4(np64(x)[[2, 0, 5, 0]], codes, np64(wscale), group, np64(z))
    p = sd.W4Params(B=B, r=r, V=V, group=group, base_dtype="f32", out_dtype="f32", x_rows=6)
    ws = sd.make_workspace(p)
    out = torch.empty_like(z)
    good = torch.tensor([2, 0, 5, 0], dtype=torch.int32).cuda()
    sd.bias_w4(p, x, good, wq, wscale, z, out, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    bad = torch.tensor([2, -1, 7, 0], dtype=torch.int32).cuda()  # clamped to 0 and 5
    sd.bias_w4(p, x, bad, wq, wscale, z, z, ws)
    assert sd.sync_status(ws) == sd.SPEC_ERR_TOKEN_RANGE
    assert torch.equal(z, out)
    within(out, want, 1e-3)


def test_bias_w4_infinities_and_nan_stay_in_their_rows():
    B, r, V, group = 3, 64, 40, 32
    g = gen(6)
    for dtype in ("f32", "bf16"):
        codes, wq, wscale = w4_inputs(B, r, V, group, dtype, "f32", g)
        codes[:, 3] = np.where(codes[:, 3] == 8, 9, codes[:, 3])
        wq = torch.from_numpy(H.w4_pack(codes)).cuda()
        x = rand(g, B, r, dtype=dtype)
        x[0, 3], x[2, 60] = float("inf"), float("nan")
        out = torch.empty(B, V, device="cuda")
        p = sd.W4Params(B=B, r=r, V=V, group=group, dtype=dtype, scale_dtype="f32")
        sd.bias_w4(p, x, None, wq, wscale, None, out, sd.make_workspace(p))
        o = np64(out)
        assert np.array_equal(o[0], np.where(codes[:, 3] > 8, np.inf, -np.inf))
        assert np.isfinite(o[1]).all() and np.isnan(o[2]).all()


@pytest.mark.parametrize("wd", ["f32", "bf16"])
@pytest.mark.parametrize("sdt", ["f32", "bf16"])
@pytest.mark.parametrize("r,V,group", [(64, 100, 32), (256, 777, 128), (160, 33, 32), (128, 1, 64)])
def test_w4_quantize(r, V, group, sdt, wd):
    W = rand(gen(r + V), r, V, dtype=wd, std=0.02)
    W[:group, 0] = 0.0
    p = sd.W4Params(B=1, r=r, V=V, group=group, scale_dtype=sdt)
    wq, wscale = sd.w4_quantize(p, W)
    codes = H.w4_unpack(wq.cpu().numpy(), r)
    w = np64(W).T.reshape(V, r // group, group)
    m = np.abs(w).max(-1)
    s = np64(wscale)
    within(s, m / 7, m / 7 * (half_step(sdt) + 2 * U) + 1e-38)
    assert np.all(codes[0, :group] == 8)
    # half a code of rounding (bf16 scales may lie half a step below max / 7:
    # then the largest weights are clamped by that much)
    back = (codes.reshape(V, -1, group) - 8) * s[..., None]
    within(back, w, s[..., None] * (0.5 + 7 * half_step(sdt) + 1e-4) + 1e-38)
    full = H.w4_pack(codes)
    assert np.array_equal(full, wq.cpu().numpy())  # padding holds code 8


# ---------------------------------------------------------------------------
# verification from probabilities
# ---------------------------------------------------------------------------
def probs_inputs(B, K, V, dtype, ddtype, seed, sigma=0.7):
    g = gen(seed)
    core = torch.randn(B, K + 1, V, generator=g) * 2
    q = torch.softmax(core[:, :K], -1).to(DT[ddtype])
    t = torch.softmax(core + sigma * torch.randn(B, K + 1, V, generator=g), -1).to(DT[dtype])
    d = torch.multinomial(q.float().reshape(B * K, V) + 1e-30, 1, generator=g).view(B, K).to(torch.int32)
    return t, q, d, torch.rand(B, K, generator=g), torch.rand(B, generator=g), g


def run_probs(t, q, d, ua, ud, kb=None, pad=(0, 0), dtype="f32", ddtype="f32"):
    B, K, V = q.shape
    p = sd.ProbsParams(B=B, K=K, V=V, dtype=dtype, draft_dtype=ddtype,
                       target_stride=V + pad[0], draft_stride=V + pad[1])
    ws = sd.make_workspace(p)
    tw, _ = strided(t.reshape(-1, V).cuda(), pad[0])
    qw, _ = strided(q.reshape(-1, V).cuda(), pad[1])
    out = torch.full((B, K + 1), -9, dtype=torch.int32, device="cuda")
    tau = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    pd, qd = torch.full((B, K), GUARD, device="cuda"), torch.full((B, K), GUARD, device="cuda")
    sd.verify_probs(p, tw, qw, d.cuda(), ua.cuda(), ud.cuda(),
                    None if kb is None else torch.as_tensor(kb, dtype=torch.int32).cuda(), out, tau,
                    pd, qd, ws)
    return sd.sync_status(ws), out.cpu().numpy(), tau.cpu().numpy(), np64(pd), np64(qd)


def same_probs(got, t, q, d, ua, ud, kb=None):
    st, out, tau, pd, qd = got
    wo, wt, wp, wq = H.verify_probs(t.double().numpy(), q.double().numpy(), d.numpy(), ua.numpy(),
                                    ud.numpy(), kb)
    assert np.array_equal(out, wo), np.argwhere(out != wo)[:4]
    assert np.array_equal(tau, wt)
    skipped = np.zeros(len(tau), bool) if kb is None else np.asarray(kb) < 0
    for got_, want in ((pd, wp), (qd, wq)):
        assert np.array_equal(got_[~skipped], want[~skipped], equal_nan=True)
        assert np.all(got_[skipped] == GUARD)
    return st


PROBS = [(1, 1, 1), (1, 4, 1024), (3, 2, 7), (5, 3, 1001), (9, 5, 4099), (2, 16, 32000), (300, 2, 257),
         (1, 3, 151936), (4, 1, 40003)]


@pytest.mark.parametrize("pad", [(0, 0), (5, 3)])
@pytest.mark.parametrize("dtype,ddtype", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("B,K,V", PROBS)
def test_verify_probs(B, K, V, dtype, ddtype, pad):
    t, q, d, ua, ud, g = probs_inputs(B, K, V, dtype, ddtype, B + K + V)
    assert same_probs(run_probs(t, q, d, ua, ud, None, pad, dtype, ddtype), t, q, d, ua, ud) == sd.SPEC_OK
    kb = torch.randint(-1, K + 1, (B,), generator=g).numpy()
    assert same_probs(run_probs(t, q, d, ua, ud, kb, pad, dtype, ddtype), t, q, d, ua, ud, kb) == sd.SPEC_OK


def test_verify_probs_ends_of_the_uniforms():
    """u = 0 takes the first token with mass and accepts what has any; the
    largest float below 1 takes the last; drafts equal to the target all pass."""
    B, K, V = 6, 3, 500
    t, q, d, ua, ud, _ = probs_inputs(B, K, V, "f32", "f32", 3)
    t[:, :, :40] = 0.0
    t[:, :, 460:] = 0.0
    top = float(np.nextafter(np.float32(1), np.float32(0)))
    for a in (0.0, top):
        for u in (0.0, top):
            ua.fill_(a), ud.fill_(u)
            assert same_probs(run_probs(t, q, d, ua, ud), t, q, d, ua, ud) == sd.SPEC_OK
    q = t[:, :K].clone()
    d = torch.multinomial(q.reshape(-1, V), 1).view(B, K).to(torch.int32)
    ua.fill_(top)
    st, out, tau, _, _ = run_probs(t, q, d, ua, ud)
    assert np.all(tau == K + 1)


def test_verify_probs_masked_places_and_empty_rows():
    """NaN, infinite and negative probabilities carry no mass; a residual
    without mass draws from p; a row without any emits -1 and is reported."""
    B, K, V = 5, 2, 301
    t, q, d, ua, ud, _ = probs_inputs(B, K, V, "f32", "f32", 4)
    t[0, :, 5], t[0, :, 6], t[0, :, 7] = float("nan"), float("inf"), -1.0
    q[0, :, 9] = float("nan")
    q[0, :, 10] = float("inf")
    d[0] = 11
    ua[0] = 0.999
    t[0, 0, 11] = 0.0
    q[1] = t[1, :K] + 1e-3          # q above p everywhere: no residual
    ua[1] = 0.9999999
    assert same_probs(run_probs(t, q, d, ua, ud), t, q, d, ua, ud) == sd.SPEC_OK
    t[2] = 0.0
    t[3, 0] = 0.0
    got = run_probs(t, q, d, ua, ud)
    assert same_probs(got, t, q, d, ua, ud) == sd.SPEC_ERR_INVALID_ARG
    assert got[1][2, 0] == -1 and got[2][2] == 0


def test_verify_probs_reports_bad_drafts_and_lengths():
    B, K, V = 4, 3, 100
    t, q, d, ua, ud, _ = probs_inputs(B, K, V, "f32", "f32", 5)
    ua.fill_(0.0)
    d2 = d.clone()
    d2[1, 1], d2[2, 0] = V, -1
    assert same_probs(run_probs(t, q, d2, ua, ud), t, q, d2, ua, ud) == sd.SPEC_ERR_TOKEN_RANGE
    kb = np.array([3, 9, 0, 1])
    assert same_probs(run_probs(t, q, d, ua, ud, kb), t, q, d, ua, ud, kb) == sd.SPEC_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# the chain, streams, graphs, refusals
# ---------------------------------------------------------------------------
def test_a_head_trains_and_decodes_with_them():
    """A gated recurrent head end to end: rows of U by token, the recurrence, the
    4-bit vocabulary product on base logits, probabilities, verification; then
    the gradient of U and of the gates' rows back through recurrence and lookup,
    against the 64-bit definitions chained the same way."""
    B, T, D, V = 3, 12, 64, 400
    g = gen(21)
    fac = rand(g, V, D)
    Wg = rand(g, V, D)
    ids = torch.randint(0, V, (B * T,), generator=g, dtype=torch.int32)
    pe = sd.EmbedParams(n=B * T, V=V, D=D, dtype="f32", row_dtype="f32", scale=1.0)
    we = sd.make_workspace(pe)
    x, gate = torch.empty(B, T, D, device="cuda"), torch.empty(B, T, D, device="cuda")
    sd.embed(pe, fac, ids.cuda(), x, we)
    sd.embed(pe, Wg, ids.cuda(), gate, we)
    ps = sd.ScanParams(B=B, T=T, D=D, dtype="f32")
    ws = sd.make_workspace(ps)
    h, last = torch.empty(B, T, D, device="cuda"), torch.empty(B, D, device="cuda")
    states = torch.empty(B, 1, D, device="cuda")
    sd.gated_scan(ps, gate, x, None, None, h, last, states, ws)
    G, X = np64(Wg)[ids.numpy()].reshape(B, T, D), np64(fac)[ids.numpy()].reshape(B, T, D)
    n, zero = np.full(B, T), np.zeros((B, D))
    wh, wlast, _, _ = H.gated_scan(G, X, zero, n)
    within(last, wlast, H.gated_scan_error(G, X, zero, n, STEP)[:, T])

    W = rand(g, D, V, std=0.1)
    pw = sd.W4Params(B=B, r=D, V=V, group=32, dtype="f32", scale_dtype="f32", base_dtype="f32")
    wq, wscale = sd.w4_quantize(pw, W)
    base, z = rand(g, B, V), torch.empty(B, V, device="cuda")
    ww = sd.make_workspace(pw)
    sd.bias_w4(pw, last, None, wq, wscale, base, z, ww)
    wz, mag = H.bias_w4(np64(last), H.w4_unpack(wq.cpu().numpy(), D), np64(wscale), 32, np64(base))
    within(z, wz, (2 * D + 2 * (D // 32) + 2) * U * mag + 1e-38)

    q = torch.softmax(z, -1)[:, None]
    t = torch.softmax(z[:, None] + 0.5 * rand(g, B, 2, V), -1)
    d = torch.multinomial(q[:, 0].cpu(), 1, generator=g).to(torch.int32)
    ua, ud = torch.rand(B, 1, generator=g), torch.rand(B, generator=g)
    assert same_probs(run_probs(t.cpu(), q.cpu(), d, ua, ud), t.cpu(), q.cpu(), d, ua, ud) == sd.SPEC_OK

    dl = rand(g, B, D)
    dg, dx, dh = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(x)
    sd.gated_scan_grad(ps, gate, x, None, None, states, dh, dl, dg, dx, None, ws)
    dU = torch.empty(V, D, device="cuda")
    sd.embed_grad(pe, ids.cuda(), dx, dU, we)
    (_, wx, _), (_, ex, _) = H.gated_scan_grad(G, X, zero, n, np.zeros((B, T, D)), np64(dl), STEP)
    wU, mag, cnt = H.embed_grad(ids.numpy(), wx.reshape(-1, D), 1.0, np.zeros((V, D)))
    eU, _, _ = H.embed_grad(ids.numpy(), ex.reshape(-1, D), 1.0, np.zeros((V, D)))
    within(dU, wU, eU + (cnt[:, None] + 2) * U * mag + 1e-38)
    for w in (we, ws, ww):
        assert sd.sync_status(w) == sd.SPEC_OK


def _every_call(seed, V=3000):
    """One call of each operator with its output tensors: (name, call(stream), outputs)."""
    g = gen(seed)
    calls = []
    n, D = 9000, 64
    ids = (torch.rand(n, generator=g) ** 2 * V).to(torch.int32).cuda()
    pe = sd.EmbedParams(n=n, V=V, D=D, dtype="f32")
    we, table, d = sd.make_workspace(pe), rand(g, V, D), rand(g, n, D, dtype="bf16")
    rows, dt = torch.empty(n, D, dtype=torch.bfloat16, device="cuda"), torch.empty(V, D, device="cuda")
    calls.append(("embed", lambda s: sd.embed(pe, table, ids, rows, we, s), [rows]))
    calls.append(("embed_grad", lambda s: sd.embed_grad(pe, ids, d, dt, we, s), [dt]))
    B, T, C = 2, 300, 96
    ps = sd.ScanParams(B=B, T=T, D=C)
    wsp = sd.make_workspace(ps)
    gate, x, dh = (rand(g, B, T, C, dtype="bf16") for _ in range(3))
    h, dg, dx = (torch.empty_like(gate) for _ in range(3))
    last, st = torch.empty(B, C, device="cuda"), torch.empty(B, -(-T // 16), C, device="cuda")
    calls.append(("scan", lambda s: sd.gated_scan(ps, gate, x, None, None, h, last, st, wsp, s), [h, last, st]))
    st0 = torch.empty_like(st)
    sd.gated_scan(ps, gate, x, None, None, h, last, st0, wsp)
    calls.append(("scan_grad", lambda s: sd.gated_scan_grad(ps, gate, x, None, None, st0, dh, None, dg, dx, None,
                                                            wsp, s), [dg, dx]))
    pw = sd.W4Params(B=3, r=256, V=V, group=64)
    wq, sc = sd.w4_quantize(pw, rand(g, 256, V))
    xw, z = rand(g, 3, 256, dtype="bf16"), torch.empty(3, V, device="cuda")
    ww = sd.make_workspace(pw)
    calls.append(("w4", lambda s: sd.bias_w4(pw, xw, None, wq, sc, None, z, ww, s), [z]))
    t, q, dr, ua, ud, _ = probs_inputs(4, 3, V, "f32", "f32", seed)
    t, q, dr, ua, ud = (v.cuda() for v in (t, q, dr, ua, ud))
    pp = sd.ProbsParams(B=4, K=3, V=V)
    out, tau = torch.empty(4, 4, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    calls.append(("verify", lambda s: sd.verify_probs(pp, t, q, dr, ua, ud, None, out, tau, None, None, wsp, s),
                  [out, tau]))
    return calls


def test_other_streams_and_graphs_give_the_same_bits():
    calls = _every_call(31)
    want = {}
    for name, call, outs in calls:
        call(None)
        want[name] = [o.clone() for o in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for name, call, outs in calls:
        for o in outs:
            o.zero_()
        side.wait_stream(torch.cuda.current_stream())
        call(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for name, call, outs in calls:
            call(torch.cuda.current_stream())
    for _ in range(2):
        for _, _, outs in calls:
            for o in outs:
                o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name, _, outs in calls:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name


def test_two_graphs_share_a_workspace_in_turn():
    a, b = _every_call(41), _every_call(42)
    want = []
    for calls in (a, b):
        for _, call, outs in calls:
            call(None)
            want.append([o.clone() for o in outs])
    graphs = []
    for calls in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _, call, _ in calls:
                call(torch.cuda.current_stream())
        graphs.append(gr)
    for k in (0, 1, 0, 1):
        graphs[k].replay()
    torch.cuda.synchronize()
    for (_, _, outs), w in zip(a + b, want):
        assert all(torch.equal(o, v) for o, v in zip(outs, w))


def test_operators_share_a_workspace_with_the_cycle():
    """spec_embed and spec_verify_probs touch only the status: a cycle before and
    after them on the same workspace gives the same tokens."""
    import synth
    w = synth.Workload("hs", B=5, K=3, V=1000, r=64, dtype="bf16", sigma=0.6, seed=71, uw_std=0.3)
    d = {k: v.cuda() for k, v in synth.make(w).items()}
    p = sd.Params(B=w.B, K=w.K, V=w.V, r=w.r, seed=13, cycle=1)
    ws = sd.make_workspace(p)

    def cycle():
        o = sd.alloc_outputs(p)
        sd.cycle(p, d["base"], d["target"], d["U"], d["W"], d["last_token"], o["draft"], o["out"],
                 o["tau"], o["p_draft"], o["q_draft"], ws)
        assert sd.sync_status(ws) == sd.SPEC_OK
        return o["out"]

    first = cycle()
    ids = torch.arange(5, dtype=torch.int32).cuda()
    pe = sd.EmbedParams(n=5, V=w.V, D=64)
    rows = torch.empty(5, 64, dtype=torch.bfloat16, device="cuda")
    sd.embed(pe, d["U"], ids, rows, ws)
    assert torch.equal(rows, d["U"][:5])
    t, q, dr, ua, ud, _ = probs_inputs(3, 2, 500, "f32", "f32", 7)
    out, tau = torch.empty(3, 3, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    sd.verify_probs(sd.ProbsParams(B=3, K=2, V=500), *(v.cuda() for v in (t, q, dr, ua, ud)), None, out, tau,
                    None, None, ws)
    assert torch.equal(first, cycle())


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("bad", [-2, 50, 2**31 - 1, -2**31])
def test_embed_grad_of_many_positions_reports_tokens_out_of_range(bad, acc):
    """The others' sums are as without it."""
    n, V, D = 9000, 50, 12
    ids = torch.randint(0, V, (n,), generator=gen(5), dtype=torch.int32)
    ids[[0, 4111, n - 1]] = bad
    st, _ = _embed_grad(n, V, D, "f32", "bf16", 0, acc, ids, gen(6))
    assert st == sd.SPEC_ERR_TOKEN_RANGE


# ---------------------------------------------------------------------------
# rows whose offsets pass 32 bits
# ---------------------------------------------------------------------------
FAR = 2**30  # elements between rows: the fifth one lies past 2^32


@pytest.fixture(scope="module")
def far_buffers():
    if torch.cuda.get_device_properties(0).total_memory < 40 * 2**30:
        pytest.skip("needs 18 GB")
    yield [torch.empty(4 * FAR + 2**23, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.empty_cache()


def far(buf, t, stride, at=0):
    """The rows of t (or space for them) `stride` elements apart: the flat view that a
    call takes, and its rows."""
    n, d = t.shape
    flat = buf[at:at + (n - 1) * stride + d]
    rows = flat.as_strided((n, d), (stride, 1))
    rows.copy_(t)
    return flat, rows


def test_embed_far_rows(far_buffers):
    a, b = far_buffers
    V, D, n = 5, 72, 5
    t, ids = rand(gen(1), V, D, dtype="bf16"), torch.tensor([4, 0, 3, 4, 1], dtype=torch.int32).cuda()
    dense = sd.EmbedParams(n=n, V=V, D=D, scale=0.5)
    p = sd.EmbedParams(n=n, V=V, D=D, scale=0.5, table_stride=FAR, row_stride=FAR)
    ws, want = sd.make_workspace(p), torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    sd.embed(dense, t, ids, want, ws)
    table, _ = far(a, t, FAR)
    out, rows = far(b, torch.zeros_like(want), FAR)
    sd.embed(p, table, ids, out, ws)
    assert torch.equal(rows, want)
    sd.embed_grad(dense, ids, want, t, ws)
    dtable, drows = far(a, torch.ones_like(t), FAR)
    sd.embed_grad(p, ids, out, dtable, ws)
    assert torch.equal(drows, t) and sd.sync_status(ws) == sd.SPEC_OK


def test_embed_grad_far_rows_sorted(far_buffers):
    a, b = far_buffers
    n, V, D, stride = 2050, 5, 40, 2**21
    assert (n - 1) * stride > 2**32 - 1 and n > 2048
    drows, t = rand(gen(1), n, D, dtype="bf16"), torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, V, (n,), generator=gen(2), dtype=torch.int32).cuda()
    p = sd.EmbedParams(n=n, V=V, D=D, table_stride=FAR, row_stride=stride)
    ws = sd.make_workspace(p)
    sd.embed_grad(sd.EmbedParams(n=n, V=V, D=D), ids, drows, t, ws)
    flat, _ = far(a, drows, stride)
    dtable, got = far(b, torch.ones_like(t), FAR)
    sd.embed_grad(p, ids, flat, dtable, ws)
    assert torch.equal(got, t) and sd.sync_status(ws) == sd.SPEC_OK


def test_gated_scan_far_rows(far_buffers):
    a, b = far_buffers
    T, D = 5, 70
    g = gen(3)
    gate, x, dh = (rand(g, T, D, dtype="bf16") for _ in range(3))
    h0 = rand(g, 1, D)
    p = sd.ScanParams(B=1, T=T, D=D, gate_stride=FAR, x_stride=FAR, h_stride=FAR)
    dense = sd.ScanParams(B=1, T=T, D=D)
    ws = sd.make_workspace(p)
    h, dg, dx = (torch.empty_like(gate) for _ in range(3))
    last, states, d0 = (torch.empty(1, D, device="cuda") for _ in range(3))
    sd.gated_scan(dense, gate, x, h0, None, h, last, states, ws)
    sd.gated_scan_grad(dense, gate, x, h0, None, states, dh, last, dg, dx, d0, ws)
    fg, fx, fd = far(a, gate, FAR)[0], far(a, x, FAR, 256)[0], far(a, dh, FAR, 512)[0]
    fh, got = far(b, torch.zeros_like(h), FAR)
    last2, states2, d02 = (torch.empty(1, D, device="cuda") for _ in range(3))
    sd.gated_scan(p, fg, fx, h0, None, fh, last2, states2, ws)
    assert torch.equal(got, h) and torch.equal(last, last2) and torch.equal(states, states2)
    (f1, got1), (f2, got2) = far(b, torch.ones_like(h), FAR), far(b, torch.ones_like(h), FAR, 256)
    sd.gated_scan_grad(p, fg, fx, h0, None, states, fd, last, f1, f2, d02, ws)
    assert torch.equal(got1, dg) and torch.equal(got2, dx) and torch.equal(d0, d02)
    assert sd.sync_status(ws) == sd.SPEC_OK


def test_bias_w4_far_rows(far_buffers):
    a, b = far_buffers
    B, r, V = 5, 64, 75
    g = gen(4)
    codes, wq, wscale = w4_inputs(B, r, V, 64, "bf16", "f32", g)
    x, base = rand(g, B, r, dtype="bf16"), rand(g, B, V, dtype="bf16")
    kw = dict(B=B, r=r, V=V, group=64, dtype="bf16", scale_dtype="f32", base_dtype="bf16", out_dtype="bf16")
    dense, p = sd.W4Params(**kw), sd.W4Params(x_stride=FAR, base_stride=FAR, out_stride=FAR, **kw)
    ws, want = sd.make_workspace(p), torch.empty_like(base)
    sd.bias_w4(dense, x, None, wq, wscale, base, want, ws)
    out, got = far(b, torch.zeros_like(base), FAR)
    sd.bias_w4(p, far(a, x, FAR)[0], None, wq, wscale, far(a, base, FAR, 256)[0], out, ws)
    assert torch.equal(got, want) and sd.sync_status(ws) == sd.SPEC_OK


def test_bias_w4_codes_past_32_bits(far_buffers):
    """The last tokens of a factor of more than 2^32 bytes, alone and among all."""
    r, tail = 4096, 64
    V = 2**32 // (r // 2) + 2 * tail
    g = gen(5)
    codes, wq, sc = w4_inputs(1, r, tail, 128, "bf16", "bf16", g)
    allq = far_buffers[0].view(torch.uint8)[:V * (r // 2)].view(V, r // 2)
    allq[:-tail].zero_()
    allq[-tail:] = wq
    scales = torch.zeros(V, r // 128, dtype=torch.bfloat16, device="cuda")
    scales[-tail:] = sc
    x = rand(g, 1, r, dtype="bf16")
    kw = dict(B=1, r=r, group=128, dtype="bf16", scale_dtype="bf16", out_dtype="f32")
    small, big = sd.W4Params(V=tail, **kw), sd.W4Params(V=V, **kw)
    ws = sd.make_workspace(big)
    want, got = torch.empty(1, tail, device="cuda"), torch.empty(1, V, device="cuda")
    sd.bias_w4(small, x, None, wq, sc, None, want, ws)
    sd.bias_w4(big, x, None, allq, scales, None, got, ws)
    # the features may be split over another number of warps: fp32 sums of r terms
    w = (codes.astype(np.float64) - 8) * np.repeat(np64(sc), 128, axis=1)
    tol = 2 * r * U * (np.abs(w) @ np.abs(np64(x)[0]))
    within(got[0, -tail:], np64(want)[0], tol)
    assert bool((got[0, :-tail] == 0).all()) and sd.sync_status(ws) == sd.SPEC_OK


def test_verify_probs_far_rows(far_buffers):
    a, b = far_buffers
    B, K, V = 1, 4, 1003
    for seed in range(6):
        t, q, d, ua, ud, _ = probs_inputs(B, K, V, "bf16", "bf16", seed, sigma=0.2)
        if seed < 3:
            ua[:] = 0.0  # all accepted: the bonus row is the far one
        want = run_probs(t, q, d, ua, ud, None, (0, 0), "bf16", "bf16")
        p = sd.ProbsParams(B=B, K=K, V=V, dtype="bf16", draft_dtype="bf16", target_stride=FAR, draft_stride=FAR)
        ws = sd.make_workspace(p)
        out, tau = torch.empty(B, K + 1, dtype=torch.int32).cuda(), torch.empty(B, dtype=torch.int32).cuda()
        pd, qd = torch.empty(B, K).cuda(), torch.empty(B, K).cuda()
        sd.verify_probs(p, far(a, t[0].cuda(), FAR)[0], far(b, q[0].cuda(), FAR)[0], d.cuda(), ua.cuda(),
                        ud.cuda(), None, out, tau, pd, qd, ws)
        for got, w in zip((sd.sync_status(ws), out.cpu().numpy(), tau.cpu().numpy(), np64(pd), np64(qd)), want):
            assert np.array_equal(got, w, equal_nan=isinstance(w, np.ndarray) and w.dtype == np.float64)


def test_binding_refuses_what_the_library_cannot_see():
    p = sd.EmbedParams(n=4, V=10, D=8, dtype="f32", row_dtype="f32")
    ws = sd.make_workspace(p)
    t, ids, rows = torch.zeros(10, 8).cuda(), torch.zeros(4, dtype=torch.int32).cuda(), torch.zeros(4, 8).cuda()
    with pytest.raises(ValueError):
        sd.embed(p, t.cpu(), ids, rows, ws)
    with pytest.raises(ValueError):
        sd.embed(p, t, ids.long(), rows, ws)
    with pytest.raises(ValueError):
        sd.embed(p, t[:9].clone(), ids, rows, ws)
    with pytest.raises(ValueError):
        sd.embed(p, t, ids, torch.zeros(8, 4).cuda().t(), ws)
    with pytest.raises(sd.SpecError):
        sd.embed(p, t, ids, rows, ws[:100])

# ---------------------------------------------------------------------------
# forms that the shapes above do not reach
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype,rows", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n,V,D", [
    # whole warps and several blocks of columns, pieces of 16 to 128 positions
    (5000, 300, 520), (9000, 700, 1001), (40000, 500, 512), (131072, 2000, 256),
    # three passes of the sort
    (5000, 2**18, 4), (9000, 300001, 12),
    # behind one tile a CTA, and twice that
    (131073, 1000, 8), (262145, 900, 4)])
def test_embed_grad_of_many_positions(n, V, D, dtype, rows, pad, acc):
    g = gen(n + D)
    ids = (torch.rand(n, generator=g) ** 2 * V).to(torch.int32).clamp_(max=V - 1)
    ids[torch.rand(n, generator=g) < 0.4] = V // 3  # a run through many pieces
    ids[n // 2] = -1
    st, _ = _embed_grad(n, V, D, dtype, rows, pad, acc, ids, g)
    assert st == sd.SPEC_OK


def test_embed_grad_far_rows_of_many_positions(far_buffers):
    """Row offsets past 2^32 in the sums of the sorted list: dense rows' bits."""
    a, b = far_buffers
    n, V, D, stride = 4098, 5, 40, 2**20
    assert (n - 1) * stride > 2**32 - 1 and n > 4096
    drows, t = rand(gen(1), n, D, dtype="bf16"), torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, V, (n,), generator=gen(2), dtype=torch.int32).cuda()
    p = sd.EmbedParams(n=n, V=V, D=D, table_stride=FAR, row_stride=stride)
    ws = sd.make_workspace(p)
    sd.embed_grad(sd.EmbedParams(n=n, V=V, D=D), ids, drows, t, ws)
    flat, _ = far(a, drows, stride)
    dtable, got = far(b, torch.ones_like(t), FAR)
    sd.embed_grad(p, ids, flat, dtable, ws)
    assert torch.equal(got, t) and sd.sync_status(ws) == sd.SPEC_OK
    want, mag, count = H.embed_grad(ids.cpu().numpy(), np64(drows), 1.0, np.zeros((V, D)))
    within(got, want, (count[:, None] + 2) * U * mag + np.abs(want) * half_step("bf16") * (1 + 1e-3))


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 2, 8])
@pytest.mark.parametrize("B,T,D", [(1, 16, 64), (2, 100, 136), (5, 65, 8), (40, 33, 256), (3, 2050, 64),
                                   # steps split over the GPU
                                   (1, 6000, 256), (2, 5121, 72),
                                   # sequences that fill the GPU
                                   (1200, 40, 128), (300, 70, 192)])
def test_gated_scan_rows_in_vectors(B, T, D, pad, dtype, ragged):
    """Widths and strides of whole pairs (2) and of 16 bytes (0, 8)."""
    gate, x, h0, lens, n = scan_inputs(B, T, D, dtype, B + T + D + pad, ragged)
    G, X, h064 = clean(gate, n, B, T, D), clean(x, n, B, T, D), np64(h0)
    gw, xw = strided(gate, pad)[0], strided(x, 2 * pad)[0]
    h = torch.full((B * T, D + pad), GUARD, dtype=DT[dtype], device="cuda")
    last = torch.full((B, D), GUARD, device="cuda")
    states = torch.full((B, -(-T // sd.SPEC_SCAN_CHUNK), D), GUARD, device="cuda")
    p = sd.ScanParams(B=B, T=T, D=D, dtype=dtype, gate_stride=D + pad, x_stride=D + 2 * pad,
                      h_stride=D + pad)
    ws = sd.make_workspace(p)
    ln = None if lens is None else lens.cuda()
    sd.gated_scan(p, gw, xw, h0, ln, h, last, states, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    want, wlast, before, _ = H.gated_scan(G, X, h064, n)
    err = H.gated_scan_error(G, X, h064, n, STEP)
    live, hs = np.arange(T)[None, :] < n[:, None], half_step(dtype)
    hv = np64(h[:, :D]).reshape(B, T, D)
    within(hv[live], want[live], (err[:, 1:] + np.abs(want) * hs)[live] + TINY, "h")
    assert np.all(hv[~live] == GUARD) and bool((h[:, D:] == GUARD).all())
    within(last, wlast, err[:, T] + TINY, "h_last")
    within(states, before[:, ::sd.SPEC_SCAN_CHUNK], err[:, :T:sd.SPEC_SCAN_CHUNK] + TINY, "states")

    dh, dl = rand(gen(T), B * T, D, dtype=dtype), rand(gen(D), B, D)
    for b in range(B):
        dh.view(B, T, D)[b, n[b]:] = float("nan")
    dg = torch.full((B * T, D + pad), GUARD, dtype=DT[dtype], device="cuda")
    dx = torch.full((B * T, D + 2 * pad), GUARD, dtype=DT[dtype], device="cuda")
    d0 = torch.full((B, D), GUARD, device="cuda")
    sd.gated_scan_grad(p, gw, xw, h0, ln, states, strided(dh, pad)[0], dl, dg, dx, d0, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    (wg, wx, w0), (eg, ex, e0) = H.gated_scan_grad(G, X, h064, n, np64(dh).reshape(B, T, D),
                                                   np64(dl), STEP)
    within(np64(dg[:, :D]).reshape(B, T, D), wg, eg + np.abs(wg) * hs + TINY, "dgate")
    within(np64(dx[:, :D]).reshape(B, T, D), wx, ex + np.abs(wx) * hs + TINY, "dx")
    within(d0, w0, e0 + np.abs(w0) * U + TINY, "dh0")
    assert bool((dg[:, D:] == GUARD).all()) and bool((dx[:, D:] == GUARD).all())


@pytest.mark.parametrize("K,V", [(257, 40), (600, 97), (1024, 33)])
def test_verify_probs_long_blocks(K, V):
    """More positions than a CTA tests at a time: rejections and bad drafts in
    every part of the block, lengths that end in any of them."""
    B = 12
    t, q, d, ua, ud, g = probs_inputs(B, K, V, "f32", "f32", K, sigma=0.0)
    q = t[:, :K].clone()
    d = torch.multinomial(q.reshape(B * K, V), 1, generator=g).view(B, K).to(torch.int32)
    ua = torch.rand(B, K, generator=g) * 0.99  # all pass, but for:
    for b, j in enumerate([0, 100, 255, 256, K - 1, K // 2]):
        t[b, j, d[b, j]] = 0.0
    d2 = d.clone()
    d2[6, 256], d2[7, 3] = V, -5
    assert same_probs(run_probs(t, q, d, ua, ud), t, q, d, ua, ud) == sd.SPEC_OK
    assert same_probs(run_probs(t, q, d2, ua, ud), t, q, d2, ua, ud) == sd.SPEC_ERR_TOKEN_RANGE
    kb = np.array([K, K, K, K, K, K, -1, 256, 255, 257, K - 1, 0])
    assert same_probs(run_probs(t, q, d, ua, ud, kb), t, q, d, ua, ud, kb) == sd.SPEC_OK


# ---------------------------------------------------------------------------
# waits that run out
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("n,V,D", [(9000, 50, 12), (70000, 300000, 8)])
def test_embed_grad_after_a_wait_that_ran_out(n, V, D, acc):
    """The workspace's abort word, set beforehand, ends the sort's first wait in
    every CTA.  The launches behind it must not use the lists, which hold
    anything here: no row is added, the status tells, and the next call on the
    same workspace is right."""
    g = gen(11)
    ids = torch.randint(0, V, (n,), generator=g, dtype=torch.int32).cuda()
    d, init = rand(g, n, D, dtype="bf16"), rand(g, V, D)
    p = sd.EmbedParams(n=n, V=V, D=D, dtype="f32", accumulate=acc)
    want, ws = init.clone(), sd.make_workspace(p)
    sd.embed_grad(p, ids, d, want, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    head = ws[:256].view(torch.int32)  # status, three diagnostics, barrier, spare, exits, abort
    assert bool((head == 0).all())
    ws[256:] = 0xFF
    head[7] = 1
    got = init.clone()
    sd.embed_grad(p, ids, d, got, ws)
    assert sd.sync_status(ws) == sd.SPEC_ERR_TIMEOUT
    assert torch.equal(got, init if acc else torch.zeros_like(init))
    assert head[4:8].tolist() == [0, 0, 0, 0]
    head[:4] = 0
    got = init.clone()
    sd.embed_grad(p, ids, d, got, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK and torch.equal(got, want)

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(5, 200, 72), (2, 2050, 64), (1, 4999, 40)])
def test_scan_after_waits_that_ran_out(B, T, D, dtype):
    """Joins between CTAs that give up at once: the call ends, the status tells,
    nothing outside the outputs is written, and the next call is right."""
    gate, x, h0, lens, n = scan_inputs(B, T, D, dtype, 3, True, std=1.0)
    gate, x = torch.nan_to_num(gate), torch.nan_to_num(x)
    dh, dl = rand(gen(4), B * T, D, dtype=dtype), rand(gen(5), B, D)
    p = sd.ScanParams(B=B, T=T, D=D, dtype=dtype, h_stride=D + 8)
    ws, ln = sd.make_workspace(p), lens.cuda()

    def both(states):
        h = torch.full((B * T, D + 8), GUARD, dtype=DT[dtype], device="cuda")
        out = [torch.full((B, D), GUARD, device="cuda")]
        sd.gated_scan(p, gate, x, h0, ln, h, out[0], states, ws)
        first = sd.sync_status(ws)
        dg, dx = torch.empty_like(gate), torch.empty_like(x)
        d0 = torch.empty(B, D, device="cuda")
        sd.gated_scan_grad(p, gate, x, h0, ln, states, strided(dh, 8)[0], dl, dg, dx, d0, ws)
        return first, sd.sync_status(ws), h, [out[0], dg, dx, d0]

    states = torch.zeros(B, -(-T // sd.SPEC_SCAN_CHUNK), D, device="cuda")
    want = both(states)
    assert want[:2] == (sd.SPEC_OK, sd.SPEC_OK)
    try:
        sd._check(sd.lib().spec_debug_scan_polls(0), "spec_debug_scan_polls")
        gave = both(states.clone())
    finally:
        sd.lib().spec_debug_scan_polls(-1)
    assert gave[:2] == (sd.SPEC_ERR_TIMEOUT, sd.SPEC_ERR_TIMEOUT)
    late = (torch.arange(T)[None, :] >= torch.from_numpy(n)[:, None]).view(-1).cuda()
    assert bool((gave[2][late] == GUARD).all()) and bool((gave[2][:, D:] == GUARD).all())
    sd.workspace_init(ws)
    again = both(states)
    assert again[:2] == (sd.SPEC_OK, sd.SPEC_OK) and torch.equal(again[2], want[2])
    assert all(torch.equal(a, b) for a, b in zip(again[3], want[3]))


def test_calls_without_scratch_take_any_workspace():
    """The lookup of many rows and the verification on the smallest workspace and
    on another operator's; the gradient refuses them."""
    n, V, D = 9000, 300, 24
    g = gen(15)
    t, ids = rand(g, V, D), torch.randint(0, V, (n,), generator=g, dtype=torch.int32).cuda()
    p = sd.EmbedParams(n=n, V=V, D=D, dtype="f32", row_dtype="f32")
    pr, q, d, ua, ud, _ = (v.cuda() if isinstance(v, torch.Tensor) else v
                           for v in probs_inputs(3, 2, 500, "f32", "f32", 7))
    pp = sd.ProbsParams(B=3, K=2, V=500)
    for other in (pp, sd.ScanParams(B=2, T=3, D=4), sd.W4Params(B=1, r=32, V=8, group=32)):
        ws, rows = sd.make_workspace(other), torch.empty(n, D, device="cuda")
        assert sd.workspace_size(p) > ws.numel()
        sd.embed(p, t, ids, rows, ws)
        out, tau = torch.empty(3, 3, dtype=torch.int32).cuda(), torch.empty(3, dtype=torch.int32).cuda()
        sd.verify_probs(pp, pr, q, d, ua, ud, None, out, tau, None, None, ws)
        assert sd.sync_status(ws) == sd.SPEC_OK and torch.equal(rows, t[ids.long()])
        with pytest.raises(sd.SpecError):
            sd.embed_grad(p, ids, rows, t, ws)


def like_definition(got, want, tol, what):
    """The same NaN and infinities, and finite values within tol."""
    got = np64(got) if isinstance(got, torch.Tensor) else got
    for f in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(f(got), f(want)), (what, f.__name__, np.argwhere(f(got) != f(want))[:4])
    fin = np.isfinite(want)
    within(got[fin], want[fin], tol[fin], what)


@pytest.mark.parametrize("std", [2.0, 30.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(2, 16, 64), (2, 500, 64), (2, 2050, 40), (1, 6000, 64), (2, 6001, 33),
                                   (1200, 60, 66)])
def test_scan_infinities_stay(B, T, D, dtype, std):
    """Infinite states, inputs and gradients over hundreds of steps, after which
    the product of the gates is below any fp32 number, and NaN beside them."""
    gate, x, h0, _, n = scan_inputs(B, T, D, dtype, 77, False, std=std)
    inf, nan, mid = float("inf"), float("nan"), T // 3
    xv, gv = x.view(B, T, D), gate.view(B, T, D)
    h0[:, 0], h0[:, 1] = inf, -inf
    xv[:, mid, 2], xv[:, 3, 3], xv[:, T - 2, 3] = inf, -inf, inf  # channel 3 ends in NaN
    xv[:, mid, 4], gv[:, mid + 1, 5] = nan, nan
    gv[:, ::2, 6], gv[:, 1::2, 6], gv[:, :, 7], gv[:, :, 8] = 300.0, -300.0, 200.0, -200.0
    xv[:, 5, 6], xv[:, 5, 7], xv[:, 5, 8] = inf, -inf, inf
    dh, dl = rand(gen(1), B, T, D, dtype=dtype), rand(gen(2), B, D)
    # what infinities are multiplied by keeps its sign whatever the rounding: delta
    # of the infinite states, and h_{t-1} - x_t (h is a mean of smaller inputs)
    dh[..., :9], dl[:, :9] = dh[..., :9].abs() + 0.5, dl[:, :9].abs() + 0.5
    xv[..., 9:13] = torch.exp2(torch.arange(1, T + 1) * (60.0 / T)).to(xv)[:, None]
    h0[:, 9:13] = 0.0
    dl[:, 9], dl[:, 10] = inf, nan
    dh[:, T // 2, 11], dh[:, T - 1, 12], dh[:, 2, 12] = -inf, inf, -inf
    G, X, h064 = clean(gate, n, B, T, D), clean(x, n, B, T, D), np64(h0)
    # Gates count as held in -87 .. 87: that moves f and 1 - f by up to e^-87 = 1.6e-38
    # and a result by that times the inputs, which are up to 2^60 here, so TINY, made
    # for inputs around 1, does not hold it; the definition is taken of the held gates.
    G = np.clip(G, -87.0, 87.0)
    p = sd.ScanParams(B=B, T=T, D=D, dtype=dtype)
    ws = sd.make_workspace(p)
    h, last = torch.empty(B, T, D, dtype=DT[dtype], device="cuda"), torch.empty(B, D, device="cuda")
    states = torch.empty(B, -(-T // sd.SPEC_SCAN_CHUNK), D, device="cuda")
    sd.gated_scan(p, gate, x, h0, None, h, last, states, ws)
    dg, dx, d0 = torch.empty_like(h), torch.empty_like(h), torch.empty_like(last)
    sd.gated_scan_grad(p, gate, x, h0, None, states, dh, dl, dg, dx, d0, ws)
    assert sd.sync_status(ws) == sd.SPEC_OK
    hs = half_step(dtype)
    with np.errstate(all="ignore"):
        want, wlast, before, _ = H.gated_scan(G, X, h064, n)
        err = H.gated_scan_error(G, X, h064, n, STEP)
        (wg, wx, w0), (eg, ex, e0) = H.gated_scan_grad(G, X, h064, n, np64(dh), np64(dl), STEP)
        like_definition(h, want, err[:, 1:] + np.abs(want) * hs + TINY, "h")
        like_definition(last, wlast, err[:, T] + TINY, "h_last")
        like_definition(states, before[:, ::sd.SPEC_SCAN_CHUNK], err[:, :T:sd.SPEC_SCAN_CHUNK] + TINY, "states")
        like_definition(dx, wx, ex + np.abs(wx) * hs + TINY, "dx")
        # an infinite delta times h_{t-1} - x_t: where two bf16 inputs in a row are equal
        # and the gate is saturated, that difference is smaller than its error, which
        # is h's bound and the subtraction's rounding, so it may be 0 or of either sign
        known = ~(np.isinf(wx) & (np.abs(before - X) <= err[:, :T] + U * (np.abs(before) + np.abs(X))))
        assert known.mean() > 0.99
        like_definition(np64(dg)[known], wg[known], (eg + np.abs(wg) * hs + TINY)[known], "dgate")
        like_definition(d0, w0, e0 + np.abs(w0) * U + TINY, "dh0")


@pytest.mark.parametrize("wd", ["f32", "bf16"])
@pytest.mark.parametrize("sdt", ["f32", "bf16"])
def test_w4_quantize_infinities_and_nan(sdt, wd):
    """An infinite weight takes the code of its sign under the largest scale, a NaN
    the code of 0; the other groups and tokens are as without them."""
    r, V, group = 128, 40, 32
    W = rand(gen(8), r, V, dtype=wd, std=0.02)
    p = sd.W4Params(B=1, r=r, V=V, group=group, scale_dtype=sdt)
    wq0, s0 = sd.w4_quantize(p, W)
    inf = float("inf")
    W[3, 0], W[70, 1], W[40, 2], W[41, 2], W[5, 3] = inf, -inf, inf, -inf, float("nan")
    wq, s = sd.w4_quantize(p, W)
    codes, was = H.w4_unpack(wq.cpu().numpy(), r), H.w4_unpack(wq0.cpu().numpy(), r)
    top = np64(torch.tensor(torch.finfo(torch.float32).max / 7).to(DT[sdt]))
    want, ws = was.copy(), np64(s0)
    for v, part in ((0, 0), (1, 2), (2, 1)):
        want[v, part * group:(part + 1) * group], ws[v, part] = 8, top
    want[0, 3], want[1, 70], want[2, 40], want[2, 41] = 15, 1, 15, 1
    assert np.array_equal(codes[:3], want[:3])
    # fp32's largest number through 7: the division's and the type's rounding
    within(np64(s)[:3], ws[:3], ws[:3] * (half_step(sdt) + 2 * U))
    W[5, 3] = 0.0
    wqn, sn = sd.w4_quantize(p, W)
    assert torch.equal(wq[3:], wqn[3:]) and torch.equal(s[3:], sn[3:]) and codes[3, 5] == 8
    assert torch.equal(wq[4:], wq0[4:]) and torch.equal(s[4:], s0[4:]) and bool(torch.isfinite(s).all())


def test_an_earlier_calls_error_is_not_reported_again():
    """spec_sync_status on a capturing stream is an error; the calls after it launch,
    and say so, the operators' and the other ones."""
    import ctypes
    cu = ctypes.CDLL("libcuda.so.1")
    calls = _every_call(51)
    big, ids = torch.randn(64, 200, device="cuda"), torch.arange(50, dtype=torch.int32).cuda()
    pe = sd.EmbedParams(n=50, V=64, D=200, dtype="f32", row_dtype="f32")
    pl = sd.ScanParams(B=1, T=6000, D=8)
    we, wl = sd.make_workspace(pe), sd.make_workspace(pl)
    gate = torch.zeros(1, 6000, 8, dtype=torch.bfloat16, device="cuda")
    last, out = torch.empty(1, 8, device="cuda"), torch.empty(64, 200, device="cuda")
    calls += [("embed_grad of few", lambda s: sd.embed_grad(pe, ids, big, out, we, s), [out]),
              ("split scan", lambda s: sd.gated_scan(pl, gate, gate, None, None, None, last, None, wl, s), [last]),
              ("quantize", lambda s: sd.w4_quantize(sd.W4Params(B=1, r=64, V=200, group=64), big, s),
               [])]
    f = torch.randn(4200, 64, device="cuda")
    d, bias = torch.zeros(4200, 1, dtype=torch.int32, device="cuda"), torch.zeros(4200, 64, device="cuda")
    ctr = torch.arange(64, dtype=torch.int32, device="cuda").view(8, 8)
    ph, tau, vo = torch.zeros(8, 4, dtype=torch.int32, device="cuda"), torch.zeros_like(d[:, 0]), torch.zeros_like(d)
    vo = vo.expand(-1, 2).contiguous()
    pf, pb = (sd.Params(B=4200, K=1, V=64, r=64, dtype=t, draft_dtype="f32") for t in ("f32", "bf16"))
    wf, wb = sd.make_workspace(pf), sd.make_workspace(pb)
    b16 = f.bfloat16()
    calls += [("philox", lambda s: sd.debug_philox(ctr[:, :4].contiguous(), ctr[:, 4:6].contiguous(), ph, s), [ph]),
              ("bias f32", lambda s: sd.markov_bias(pf, f[:64], f[64:128], d[:, 0], bias, wf, s), [bias]),
              ("bias bf16", lambda s: sd.markov_bias(pb, b16[:64], b16[64:128], d[:, 0], bias, wb, s), [bias]),
              ("verify", lambda s: sd.verify_block(pf, f.repeat(2, 1), f, d, vo, tau, None, None, wf, s), [vo, tau])]
    for _, call, _ in calls:
        call(None)
    torch.cuda.synchronize()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for name, call, outs in calls:
        call(None)
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph, st = ctypes.c_void_p(), ctypes.c_void_p(side.cuda_stream)
        assert cu.cuStreamBeginCapture_v2(st, 2) == 0  # relaxed
        assert sd.sync_status(we, side) == sd.SPEC_ERR_CUDA
        cu.cuStreamEndCapture(st, ctypes.byref(graph))  # invalidated: no graph
        assert not graph.value
        call(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), name
