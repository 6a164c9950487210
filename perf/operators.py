"""The operators around the sequential head, as cases to be measured.

Each case is one call a serving or training program makes beside the fused
cycle: the scaled lookup of the head's rows by token and its gradient, the
gated recurrence over a sequence of them and its gradient, the product with a
4-bit vocabulary factor, and the verification of a drafted block from
probabilities and given uniform numbers.  With `own` false, `run` computes the
operator with elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}
ZIPF = 1.1  # exponent of the token frequencies, as in the synthetic workloads


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the last committed tokens of a serving batch: 64 rows of a rank-256 factor
        dict(name="embed_64_tokens", op="embed", n=64, V=129280, D=256, dtype="bf16", rows="bf16",
             scale=1.0),
        # a training batch of 8 x 8192 tokens, 32-bit table to bf16 rows, scaled by sqrt(D)
        dict(name="embed_65536_tokens", op="embed", n=65536, V=32000, D=1024, dtype="f32",
             rows="bf16", scale=32.0),
        # a small training step that adds to a running 32-bit gradient; odd row width
        dict(name="embed_grad_1000_tokens", op="embed_grad", n=1000, V=32000, D=250, dtype="f32",
             rows="bf16", scale=1.0, accumulate=True),
        # the whole gradient of the rank-256 factor for 8 x 16384 tokens
        dict(name="embed_grad_131072_tokens", op="embed_grad", n=131072, V=129280, D=256,
             dtype="f32", rows="bf16", scale=16.0, accumulate=False),
        # one decoding step of 64 sequences: the state in, the state out
        dict(name="scan_one_step", op="scan", B=64, T=1, D=256, dtype="bf16", state=True,
             ragged=False),
        # one long document: 65536 steps of one sequence
        dict(name="scan_65536_steps", op="scan", B=1, T=65536, D=256, dtype="bf16", state=False,
             ragged=False),
        # a padded batch in 32 bits, odd sizes, sequences of different lengths
        dict(name="scan_grad_ragged", op="scan_grad", B=5, T=1537, D=200, dtype="f32", state=True,
             ragged=True),
        # a training batch
        dict(name="scan_grad_8x8192", op="scan_grad", B=8, T=8192, D=1024, dtype="bf16",
             state=False, ragged=False),
        # the Markov bias of one sequence with its vocabulary factor in 4 bits
        dict(name="w4_markov_1_row", op="w4", B=1, r=256, V=129280, group=32, dtype="bf16",
             lookup=True, base=False),
        # the output product of 16 decoding rows, added to base logits
        dict(name="w4_head_16_rows", op="w4", B=16, r=4096, V=151936, group=128, dtype="bf16",
             lookup=False, base=True),
        # the smallest block: one sequence, four drafts
        dict(name="verify_1x4x1024", op="verify", B=1, K=4, V=1024, dtype="f32", sigma=0.5,
             ragged=False),
        # a large serving batch
        dict(name="verify_256x8x151936", op="verify", B=256, K=8, V=151936, dtype="f32", sigma=0.5,
             ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "scan", "scan_grad", "w4", "verify"])
    ty = rng.choice(["f32", "bf16"])
    if op in ("embed", "embed_grad"):
        V = rng.choice([32000, 129280, 151936, _log(rng, 1000, 152000)])
        D = rng.choice([64, 128, 256, 512, 1024, rng.randint(1, 1500)])
        n = _log(rng, 1, min(131072, (1 << 26) // D))
        scale = rng.choice([1.0, math.sqrt(D), 0.125])
        c = dict(op=op, n=n, V=V, D=D, dtype=ty, rows=rng.choice(["f32", "bf16"]), scale=scale)
        if op == "embed_grad":
            if V * D > 1 << 26:
                c["V"] = V = (1 << 26) // D
            c["accumulate"] = rng.random() < 0.5
            c["dtype"] = "f32" if c["accumulate"] else ty
        return c
    if op in ("scan", "scan_grad"):
        D = rng.choice([64, 128, 256, 1024, rng.randint(1, 1500)])
        B = _log(rng, 1, 256)
        T = _log(rng, 1, max(2, min(65536, (1 << 25) // (B * D))))
        return dict(op=op, B=B, T=T, D=D, dtype=ty, state=rng.random() < 0.5,
                    ragged=rng.random() < 0.4)
    if op == "w4":
        group = rng.choice([32, 64, 128])
        r = group * rng.randint(1, 4096 // group)
        V = rng.choice([32000, 129280, 151936, rng.randint(1, 152000)])
        return dict(op=op, B=rng.randint(1, 16), r=r, V=V, group=group, dtype=ty,
                    lookup=rng.random() < 0.3, base=rng.random() < 0.5)
    V = rng.choice([32000, 129280, 151936, rng.randint(8, 152000)])
    K = rng.randint(1, 16)
    B = _log(rng, 1, min(256, max(1, (1 << 28) // (V * K))))
    return dict(op=op, B=B, K=K, V=V, dtype=ty, sigma=rng.choice([0.2, 0.5, 1.0]),
                ragged=rng.random() < 0.4)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _zipf_cdf(V):
    w = torch.arange(1, V + 1, dtype=torch.float64, device="cuda").pow(-ZIPF).cumsum(0)
    return w / w[-1]


def _tokens(g, n, V):
    """Tokens by Zipf frequencies, their ranks spread over the vocabulary."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(_zipf_cdf(V), u).clamp_(max=V - 1)
    return torch.randperm(V, generator=g, device="cuda")[rank].to(torch.int32)


def _lens(g, B, T):
    """Lengths from 0 to T, both among them where there is room."""
    n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = T
    if B > 2:
        n[1] = 0
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op, "case": case}

    def normal(*shape, dtype="f32", std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(DT[dtype])

    if op in ("embed", "embed_grad"):
        n, V, D = case["n"], case["V"], case["D"]
        s["ids"] = _tokens(g, n, V)
        if op == "embed":
            s["table"] = normal(V, D, dtype=case["dtype"])
            s["rows"] = torch.empty(n, D, dtype=DT[case["rows"]], device="cuda")
        else:
            s["drows"] = normal(n, D, dtype=case["rows"])
            s["dtable"] = normal(V, D, dtype=case["dtype"])
    elif op in ("scan", "scan_grad"):
        B, T, D, ty = case["B"], case["T"], case["D"], case["dtype"]
        # gates that keep a state for some tens of steps
        s["gate"] = (torch.randn(B, T, D, generator=g, device="cuda") + 2.0).to(DT[ty])
        s["x"] = normal(B, T, D, dtype=ty)
        s["h0"] = normal(B, D) if case["state"] else None
        s["len"] = _lens(g, B, T) if case["ragged"] else None
        s["h"] = torch.zeros(B, T, D, dtype=DT[ty], device="cuda")
        s["h_last"] = torch.zeros(B, D, device="cuda")
        if op == "scan_grad":
            s["dh"] = normal(B, T, D, dtype=ty)
            s["dh_last"] = normal(B, D) if case["state"] else None
            # what the forward pass kept for the gradient: the state before every 16th step
            s["states"] = _boundary_states(s["gate"], s["x"], s["h0"], s["len"])
            s["dgate"], s["dx"] = torch.empty_like(s["gate"]), torch.empty_like(s["x"])
            s["dh0"] = torch.empty(B, D, device="cuda")
            s["h"] = s["h_last"] = None
    elif op == "w4":
        B, r, V, group, ty = case["B"], case["r"], case["V"], case["group"], case["dtype"]
        rp = -(-r // 128) * 128
        q = torch.randint(1, 16, (V, r), generator=g, device="cuda", dtype=torch.uint8)
        s["wscale"] = (torch.rand(V, r // group, generator=g, device="cuda") * 0.01 + 0.001).to(DT[ty])
        s["wq"] = _pack(q, rp)
        s["x"] = normal(1000 if case["lookup"] else B, r, dtype=ty)
        s["prev"] = (torch.randint(0, 1000, (B,), generator=g, device="cuda", dtype=torch.int32)
                     if case["lookup"] else None)
        s["base"] = normal(B, V, dtype=ty, std=2.0) if case["base"] else None
        s["out"] = torch.empty(B, V, device="cuda")
    else:
        B, K, V, ty = case["B"], case["K"], case["V"], case["dtype"]
        core = torch.randn(B, K + 1, V, generator=g, device="cuda") * 2.0
        core -= 1.1 * torch.log(torch.arange(1, V + 1, device="cuda"))
        s["q"] = torch.softmax(core[:, :K], -1).to(DT[ty])
        e = torch.rand(B, K, V, generator=g, device="cuda")
        e = e.clamp_(min=1e-30).log_().neg_().log_().neg_()
        s["draft"] = (core[:, :K] + e).argmax(-1).to(torch.int32)
        del e
        core += torch.randn(B, K + 1, V, generator=g, device="cuda") * case["sigma"]
        s["p"] = torch.softmax(core, -1).to(DT[ty])
        del core
        s["u_accept"] = torch.rand(B, K, generator=g, device="cuda")
        s["u_draw"] = torch.rand(B, generator=g, device="cuda")
        s["verify_len"] = (torch.randint(0, K + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
                           if case["ragged"] else None)
        s["out"] = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
        s["tau"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["p_draft"] = torch.empty(B, K, device="cuda")
        s["q_draft"] = torch.empty(B, K, device="cuda")
    return s


def _pack(q, rp):
    """4-bit codes [V, r] in the packed layout: two codes a byte, the lower
    feature in the lower half; in each run of 128 features the sixteen 4-byte
    words w are stored in the order 4 * (w % 4) + w // 4; features past r hold
    the code of zero, 8."""
    V, r = q.shape
    full = torch.full((V, rp), 8, dtype=torch.uint8, device=q.device)
    full[:, :r] = q
    by = full[:, 0::2] | (full[:, 1::2] << 4)
    return by.view(V, rp // 128, 4, 4, 4).transpose(2, 3).contiguous().view(V, rp // 2)


def _doubling(f, z):
    """h_t = f_t h_{t-1} + z_t from a zero state, along dimension 1, by
    doubling strides."""
    f, h = f.clone(), z.clone()
    k = 1
    while k < h.shape[1]:
        h[:, k:] += f[:, k:] * h[:, :-k].clone()
        f[:, k:] *= f[:, :-k].clone()
        k *= 2
    return h


def _live(n, B, T):
    """[B, T, 1]: which steps belong to their sequence."""
    if n is None:
        return None
    return (torch.arange(T, device=n.device)[None, :] < n[:, None])[..., None]


def _states(gate, x, h0, n):
    """The recurrence in 32 bits: the state after every step, [B, T, D]; past a
    sequence's end the state stays."""
    f = 1 / (1 + torch.exp(-gate.float()))
    z = x.float() / (1 + torch.exp(gate.float()))
    live = _live(n, *gate.shape[:2])
    if live is not None:
        f, z = torch.where(live, f, 1.0), torch.where(live, z, 0.0)
    if h0 is not None:
        z[:, 0] += f[:, 0] * h0
    return _doubling(f, z)


def _before(h, h0):
    """The state before every step, from the state after every step."""
    first = torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None]
    return torch.cat([first, h[:, :-1]], 1)


def _boundary_states(gate, x, h0, n):
    return _before(_states(gate, x, h0, n), h0)[:, ::16].contiguous()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)(s)


def _plain(s):
    op, c = s["op"], s["case"]
    if op == "embed":
        s["rows"].copy_(s["table"][s["ids"].long()].float() * c["scale"])
        return s["rows"]
    if op == "embed_grad":
        d = s["dtable"]
        if c["accumulate"]:
            d.index_add_(0, s["ids"].long(), s["drows"].float(), alpha=c["scale"])
        else:
            acc = torch.zeros(d.shape, device="cuda")
            acc.index_add_(0, s["ids"].long(), s["drows"].float())
            d.copy_(acc * c["scale"])
        return d
    if op == "scan":
        h = _states(s["gate"], s["x"], s["h0"], s["len"])
        s["h_last"].copy_(h[:, -1])
        live = _live(s["len"], *h.shape[:2])
        s["h"].copy_(h if live is None else torch.where(live, h, s["h"].float()))
        return s["h"], s["h_last"]
    if op == "scan_grad":
        gate, x, dh = s["gate"].float(), s["x"].float(), s["dh"].float()
        B, T, _ = gate.shape
        before = _before(_states(s["gate"], s["x"], s["h0"], s["len"]), s["h0"])
        f, i = 1 / (1 + torch.exp(-gate)), 1 / (1 + torch.exp(gate))
        live = _live(s["len"], B, T)
        fl = f
        if live is not None:
            dh, fl = torch.where(live, dh, 0.0), torch.where(live, f, 1.0)
        # delta_t = dh_t + f_{t+1} delta_{t+1}; the last state's gradient enters at the end
        dh = dh.flip(1)
        fr = fl.flip(1)
        decay = torch.cat([torch.ones_like(fr[:, :1]), fr[:, :-1]], 1)
        if s["dh_last"] is not None:
            dh[:, 0] += s["dh_last"]
        delta = _doubling(decay, dh).flip(1)
        s["dh0"].copy_(fl[:, 0] * delta[:, 0])
        if live is not None:
            delta = torch.where(live, delta, 0.0)
        s["dx"].copy_(delta * i)
        s["dgate"].copy_(delta * (before - x) * f * i)
        return s["dgate"], s["dx"], s["dh0"]
    if op == "w4":
        V, r = s["out"].shape[1], c["r"]
        by = s["wq"].view(V, -1, 4, 4, 4).transpose(2, 3).reshape(V, -1)
        w = torch.stack([by & 15, by >> 4], -1).view(V, -1)[:, :r].float() - 8
        w = (w.view(V, -1, c["group"]) * s["wscale"].float()[..., None]).view(V, r)
        x = s["x"] if s["prev"] is None else s["x"][s["prev"].long()]
        z = x.float() @ w.t()
        s["out"].copy_(z if s["base"] is None else z + s["base"].float())
        return s["out"]
    p, q, d = s["p"], s["q"], s["draft"].long()
    B, K = d.shape
    b, i = torch.arange(B, device="cuda"), torch.arange(K, device="cuda")
    kb = torch.full((B,), K, device="cuda") if s["verify_len"] is None else s["verify_len"].long()
    pd = p[b[:, None], i, d].double()
    qd = q[b[:, None], i, d].double()
    ok = (s["u_accept"].double() * qd < pd) & (i < kb[:, None])
    j = ok.long().cumprod(1).sum(1)
    pj = p[b, j].double()
    pj = torch.where((pj > 0) & (pj < math.inf), pj, 0.0)
    res = pj - q[b, j.clamp(max=K - 1)].double()
    res = torch.where((res > 0) & (j < kb)[:, None], res, 0.0)
    mass = torch.where(res.sum(1, keepdim=True) > 0, res, pj)
    cum = mass.cumsum(1)
    tok = torch.searchsorted(cum, (s["u_draw"].double() * cum[:, -1])[:, None], right=True)[:, 0]
    last = mass.shape[1] - 1 - (mass.flip(1) > 0).int().argmax(1)
    tok = torch.minimum(tok, last)
    at = torch.arange(K + 1, device="cuda")
    tokens = torch.cat([d, d[:, :1]], 1)
    out = torch.where(at < j[:, None], tokens, torch.where(at == j[:, None], tok[:, None], -1))
    s["out"].copy_(out)
    s["tau"].copy_(j + 1)
    tested = (i <= j[:, None]) & (i < kb[:, None])
    s["p_draft"].copy_(torch.where(tested, pd, math.nan))
    s["q_draft"].copy_(torch.where(tested, qd, math.nan))
    return s["out"], s["tau"], s["p_draft"], s["q_draft"]


_kept = {}  # parameters and workspace, which a program makes once for a shape


def _own(s):
    import draft_sampling_verification_head_b200 as sd

    op, c = s["op"], s["case"]
    kept = _kept.setdefault(tuple(sorted(c.items())), {})
    if not kept:
        if op in ("embed", "embed_grad"):
            kept["p"] = sd.EmbedParams(n=c["n"], V=c["V"], D=c["D"], dtype=c["dtype"],
                                       row_dtype=c["rows"], scale=c["scale"],
                                       accumulate=c.get("accumulate", False))
        elif op in ("scan", "scan_grad"):
            kept["p"] = sd.ScanParams(B=c["B"], T=c["T"], D=c["D"], dtype=c["dtype"])
        elif op == "w4":
            kept["p"] = sd.W4Params(B=c["B"], r=c["r"], V=c["V"], group=c["group"],
                                    dtype=c["dtype"], scale_dtype=c["dtype"], base_dtype=c["dtype"],
                                    x_rows=s["x"].shape[0])
        else:
            kept["p"] = sd.ProbsParams(B=c["B"], K=c["K"], V=c["V"], dtype=c["dtype"],
                                       draft_dtype=c["dtype"])
        kept["ws"] = sd.make_workspace(kept["p"])
    p, ws = kept["p"], kept["ws"]
    if op == "embed":
        sd.embed(p, s["table"], s["ids"], s["rows"], ws)
        return s["rows"]
    if op == "embed_grad":
        sd.embed_grad(p, s["ids"], s["drows"], s["dtable"], ws)
        return s["dtable"]
    if op == "scan":
        sd.gated_scan(p, s["gate"], s["x"], s["h0"], s["len"], s["h"], s["h_last"], None, ws)
        return s["h"], s["h_last"]
    if op == "scan_grad":
        sd.gated_scan_grad(p, s["gate"], s["x"], s["h0"], s["len"], s["states"], s["dh"],
                           s["dh_last"], s["dgate"], s["dx"], s["dh0"], ws)
        return s["dgate"], s["dx"], s["dh0"]
    if op == "w4":
        sd.bias_w4(p, s["x"], s["prev"], s["wq"], s["wscale"], s["base"], s["out"], ws)
        return s["out"]
    sd.verify_probs(p, s["p"], s["q"], s["draft"], s["u_accept"], s["u_draw"], s["verify_len"],
                    s["out"], s["tau"], s["p_draft"], s["q_draft"], ws)
    return s["out"], s["tau"], s["p_draft"], s["q_draft"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _distinct(n, V):
    """Expected number of different tokens among n."""
    w = np.arange(1, V + 1, dtype=np.float64) ** -ZIPF
    return float(np.sum(-np.expm1(n * np.log1p(-np.minimum(w / w.sum(), 1 - 1e-12)))))


def work(case):
    op, c = case["op"], case
    if op in ("embed", "embed_grad"):
        n, V, D = c["n"], c["V"], c["D"]
        d = _distinct(n, V)
        rows = n * D * ES[c["rows"]] + 4 * n
        if op == "embed":
            return {"bytes": rows + d * D * ES[c["dtype"]], "flops": n * D}
        table = 2 * d * D if c["accumulate"] else V * D
        return {"bytes": rows + table * ES[c["dtype"]], "flops": n * D + d * D}
    if op in ("scan", "scan_grad"):
        part = 0.5 if c["ragged"] and c["B"] > 2 else 1.0  # steps inside their sequences
        e, s = c["B"] * c["T"] * c["D"] * part, 4 * c["B"] * c["D"]
        if op == "scan":
            return {"bytes": 3 * e * ES[c["dtype"]] + s * (2 if c["state"] else 1), "flops": 8 * e}
        return {"bytes": 5 * e * ES[c["dtype"]] + 4 * e / 16 + s * (3 if c["state"] else 1),
                "flops": 18 * e}
    if op == "w4":
        B, r, V, es = c["B"], c["r"], c["V"], ES[c["dtype"]]
        return {"bytes": V * r / 2 + V * r / c["group"] * es + B * r * es
                + B * V * (4 + (es if c["base"] else 0)), "flops": 2 * B * r * V}
    # the block's probabilities at the drafts, then the two rows of its first rejection
    B, K, V, es = c["B"], c["K"], c["V"], ES[c["dtype"]]
    accept = {0.2: 0.92, 0.5: 0.80, 1.0: 0.62}[c["sigma"]]
    k = K / 2 if c["ragged"] else K
    rejected = 1 - accept ** k
    return {"bytes": B * V * es * (1 + rejected) + B * K * (4 + 4 + 64) + 4 * B * (3 * K + 3),
            "flops": 2 * B * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _exact_embed(c, s):
    return s["table"].index_select(0, s["ids"].to(torch.int64)).double().mul_(c["scale"])


def _exact_embed_grad(c, s):
    ids, d = s["ids"].cpu().numpy(), s["drows"].double().cpu().numpy()
    out = s["dtable"].double().cpu().numpy() if c["accumulate"] else np.zeros((c["V"], c["D"]))
    order = np.argsort(ids, kind="stable")
    tok, start = np.unique(ids[order], return_index=True)
    out[tok] += c["scale"] * np.add.reduceat(d[order], start, axis=0)
    return out


def _exact_scan(c, s):
    g, x = s["gate"], s["x"]
    B, T, D = g.shape
    h = torch.zeros(B, D, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    out = s["h"].double()
    n = None if s["len"] is None else s["len"].long()
    for t in range(T):
        f = torch.sigmoid(g[:, t].double())
        new = f * h + (1 - f) * x[:, t].double()
        if n is None:
            h = new
            out[:, t] = h
        else:
            in_it = (n > t)[:, None]
            h = torch.where(in_it, new, h)
            out[:, t] = torch.where(in_it, h, out[:, t])
    return out, h


def _exact_scan_grad(c, s):
    g, x, dh = s["gate"], s["x"], s["dh"]
    B, T, D = g.shape
    zero = torch.zeros(B, D, dtype=torch.float64, device="cuda")
    h = zero if s["h0"] is None else s["h0"].double()
    n = torch.full((B,), T, device="cuda") if s["len"] is None else s["len"].long()
    before = torch.empty(B, T, D, dtype=torch.float64, device="cuda")
    for t in range(T):
        before[:, t] = h
        f = torch.sigmoid(g[:, t].double())
        h = torch.where((n > t)[:, None], f * h + (1 - f) * x[:, t].double(), h)
    dg, dx = torch.zeros_like(before), torch.zeros_like(before)
    carry = zero if s["dh_last"] is None else s["dh_last"].double()
    for t in reversed(range(T)):
        in_it = (n > t)[:, None]
        f = torch.sigmoid(g[:, t].double())
        delta = carry + dh[:, t].double()
        dx[:, t] = torch.where(in_it, delta * (1 - f), zero)
        dg[:, t] = torch.where(in_it, delta * (before[:, t] - x[:, t].double()) * f * (1 - f), zero)
        carry = torch.where(in_it, delta * f, carry)
    return dg, dx, carry


def _exact_w4(c, s):
    V, r, group = c["V"], c["r"], c["group"]
    x = s["x"].double() if s["prev"] is None else s["x"].double()[s["prev"].long()]
    out = torch.zeros(c["B"], V, dtype=torch.float64, device="cuda")
    if s["base"] is not None:
        out += s["base"].double()
    for k in range(0, r, 32):  # 32 features: four words of eight codes
        word = s["wq"].view(V, -1, 16, 4)[:, k // 128]
        part = (k % 128) // 32
        for w in range(4):
            four = word[:, 4 * w + part].to(torch.int64)
            for half in range(2):
                code = ((four >> (4 * half)) & 15).double() - 8
                at = k + 8 * w + half + 2 * torch.arange(4, device="cuda")
                out += (x[:, at] @ code.t()) * s["wscale"][:, k // group].double()
    return out


def _exact_verify(c, s):
    d, ua, ud = (s[k].cpu().numpy() for k in ("draft", "u_accept", "u_draw"))
    B, K = d.shape
    out, tau = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32)
    kb = [K] * B if s["verify_len"] is None else s["verify_len"].tolist()
    at = torch.from_numpy(d).to(device="cuda", dtype=torch.int64)[..., None]
    pd = s["p"][:, :K].gather(2, at)[..., 0].double().cpu().numpy()
    qd = s["q"].gather(2, at)[..., 0].double().cpu().numpy()
    seen = np.full((2, B, K), np.nan)
    for b in range(B):
        j = 0
        while j < kb[b]:
            seen[:, b, j] = pd[b, j], qd[b, j]
            if not float(ua[b, j]) * qd[b, j] < pd[b, j]:
                break
            out[b, j] = d[b, j]
            j += 1
        m = s["p"][b, j].double().cpu().numpy()
        if j < kb[b]:
            res = np.maximum(m - s["q"][b, j].double().cpu().numpy(), 0)
            m = res if res.sum() > 0 else m
        cum = np.cumsum(m)
        past = np.nonzero(cum > float(ud[b]) * cum[-1])[0]
        out[b, j] = past[0] if len(past) else np.nonzero(m)[0][-1]
        tau[b] = j + 1
    return torch.from_numpy(out), torch.from_numpy(tau), seen[0], seen[1]
