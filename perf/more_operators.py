"""What the operators of linear-attention layers are measured on.

The token mixers whose states the decode entry points keep, over whole sequences:
linear attention with a decay for each head (forward, backward, single tokens),
the gated delta rule (forward, backward), and the rotary positions of their
queries and keys.  ``run`` computes a case in elementary torch operations where
``own`` is false and through the library's entry points where it is true;
``exact`` is the definition in 64 bits, token by token.

Values are drawn as the repository's workloads draw them: q, k rows of unit norm
(the delta rule) or N(0, 1) (linear attention), v ~ N(0, 1), beta = sigmoid(N(0, 1)),
states ~ N(0, 0.1); gates log g = -A softplus(N(0, 1) + bias) with A = exp(U[0, ln 16])
and softplus(bias) uniform on [1e-3, 1e-1].
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64          # tokens per block of the plain forms


# ---------------------------------------------------------------- the cases

def listed():
    lin = dict(kheads=32, vheads=32, dk=128, dv=128, io="bf16", decay="head", initial=True)
    gdn = dict(kheads=16, vheads=32, dk=128, dv=128, io="bf16", initial=True)
    return [
        # one decode step of 256 requests: every state is read and written once
        dict(lin, op="lin_step", name="lin_step_b256", batch=256),
        # one long prompt that continues from a cached state
        dict(lin, op="lin_fwd", name="lin_fwd_prompt", tokens=4096, seqs=1, even=True),
        # a serving engine's prefill batch: uneven prompts packed one after another
        dict(lin, op="lin_fwd", name="lin_fwd_packed", tokens=16383, seqs=13, even=False),
        # a training micro-batch with a gate for every token, narrow keys: 8 sequences of 1024
        dict(lin, op="lin_bwd", name="lin_bwd_train", tokens=8192, seqs=8, even=True, dk=64,
             decay="token", initial=False),
        # a few short prompts of a tiny fp32 model: latency is what counts
        dict(gdn, op="gdn_fwd", name="gdn_fwd_tiny", tokens=61, seqs=4, even=False, kheads=2,
             vheads=4, dk=64, dv=64, io="f32"),
        # one long prompt of a layer with the decode workload's heads
        dict(gdn, op="gdn_fwd", name="gdn_fwd_prompt", tokens=4096, seqs=1, even=True),
        # the packed prefill batch of the same layer
        dict(gdn, op="gdn_fwd", name="gdn_fwd_packed", tokens=16383, seqs=13, even=False),
        # its training step on two uneven sequences that continue from states
        dict(gdn, op="gdn_bwd", name="gdn_bwd_uneven", tokens=1291, seqs=2, even=False),
        # and on a micro-batch of 8 sequences of 1024
        dict(gdn, op="gdn_bwd", name="gdn_bwd_train", tokens=8192, seqs=8, even=True,
             initial=False),
        # the decode step's queries and keys of 64 requests far into their contexts
        dict(op="rot_fwd", name="rot_step_b64", tokens=64, heads=48, dim=128, rotary=128,
             interleaved=False, far=1 << 20, io="bf16", inplace=True),
        # queries and keys of the packed prefill batch
        dict(op="rot_fwd", name="rot_packed", tokens=16383, heads=64, dim=128, rotary=128,
             interleaved=False, far=1 << 15, io="bf16", inplace=False),
        # their gradient in training, interleaved pairs in half of each head
        dict(op="rot_bwd", name="rot_bwd_train", tokens=8192, heads=48, dim=128, rotary=64,
             interleaved=True, far=1024, io="bf16", inplace=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_bwd", "lin_step", "gdn_fwd", "gdn_fwd", "gdn_bwd", "gdn_bwd",
                     "rot_fwd", "rot_bwd"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("rot"):
        dim = 8 * _log(rng, 4, 32)
        heads = _log(rng, 1, 64)
        return dict(op=op, tokens=_log(rng, 1, min(16383, 16383 * 64 * 64 // (heads * dim))),
                    heads=heads, dim=dim, rotary=rng.choice([dim, dim, 2 * _log(rng, 2, dim // 2)]),
                    interleaved=rng.random() < 0.5, far=_log(rng, 256, 1 << 20), io=io,
                    inplace=rng.random() < 0.3)
    kheads = _log(rng, 1, 16)
    vheads = kheads * rng.choice([1, 1, 2, 4] if kheads <= 8 else [1, 2])
    dk = rng.choice([64, 128, 128])
    dv = rng.choice([64, 128, 128]) if op.startswith("lin") else dk
    c = dict(op=op, kheads=kheads, vheads=vheads, dk=dk, dv=dv, io=io, initial=rng.random() < 0.6)
    if op.startswith("lin"):
        c["decay"] = rng.choice(["head", "token", "none"])
    if op == "lin_step":
        c.update(batch=_log(rng, 1, 256), initial=True)
        return c
    most = 8192 * 32 * 128 * 128 // (vheads * dk * dv) // (8 if io == "f32" else 1)
    if op.endswith("bwd"):
        most //= 2
    tokens = _log(rng, 3, min(8192, most))
    c.update(tokens=tokens, seqs=_log(rng, 1, min(24, tokens)), even=False)
    return c


# ---------------------------------------------------------------- the inputs

def _lengths(c):
    """Sequence lengths by the case alone: equal, or uneven with some of 1 and 0."""
    T, n = c["tokens"], c["seqs"]
    if c["even"]:
        return [T // n] * n
    r = random.Random(T * 1009 + n)
    w = [math.exp(r.gauss(0.0, 0.8)) for _ in range(n)]
    lens = [int(T * v / sum(w)) for v in w]
    if n >= 4:
        lens[1], lens[2] = 1, 0
    lens[0] += T - sum(lens)
    return lens


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _uniform(g, shape, lo, hi):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32) * (hi - lo) + lo


def _gates(g, rows, H):
    bias = torch.log(torch.expm1(_uniform(g, H, 1e-3, 1e-1)))
    step = torch.nn.functional.softplus(_normal(g, (rows, H), torch.float32) + bias)
    return -torch.exp(_uniform(g, H, 0.0, math.log(16.0))) * step


def _heads(s, g, c, rows):
    """q, k, v and the gates of so many tokens."""
    HK, HV, K, V, io = c["kheads"], c["vheads"], c["dk"], c["dv"], DT[c["io"]]
    q, k = _normal(g, (rows, HK, K), torch.float32), _normal(g, (rows, HK, K), torch.float32)
    if c["op"].startswith("gdn"):
        q, k = q / q.norm(dim=2, keepdim=True), k / k.norm(dim=2, keepdim=True)
        s["log_g"], s["beta"] = _gates(g, rows, HV), torch.sigmoid(_normal(g, (rows, HV), torch.float32))
    else:   # decays from one part in 256 a token to a half
        s["log_g"] = {"head": -torch.exp(_uniform(g, HV, math.log(2.0 ** -8), math.log(0.7))),
                      "token": _gates(g, rows, HV), "none": None}[c["decay"]]
    s.update(q=q.to(io), k=k.to(io), v=_normal(g, (rows, HV, V), io))


def _frequencies(c):
    return torch.tensor([10000.0 ** (-2.0 * i / c["rotary"]) for i in range(c["rotary"] // 2)],
                        dtype=torch.float32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"].startswith("rot"):
        # the tokens' rows are a slice of the projection's wider rows
        io, T = DT[c["io"]], c["tokens"]
        row = _normal(g, (T, (c["heads"] + 2) * c["dim"]), io)
        s["x"] = row[:, :c["heads"] * c["dim"]].unflatten(1, (c["heads"], c["dim"]))
        s["positions"] = torch.randint(0, c["far"], (T,), generator=g, device="cuda")
        s["freqs"] = _frequencies(c)
        if c["inplace"]:   # in place, on a copy made within the pass: the same work on both sides
            s["buffer"] = torch.empty_like(s["x"])
        return s
    HV, K, V = c["vheads"], c["dk"], c["dv"]
    if c["op"] == "lin_step":
        nb = c["batch"]
        order = list(range(nb))
        random.Random(seed).shuffle(order)
        _heads(s, g, c, nb)
        s.update(state=_normal(g, (nb, HV, V, K), torch.float32, 0.1),
                 new_state=torch.empty((nb, HV, V, K), dtype=torch.float32, device="cuda"),
                 slot_idx=torch.tensor(order, dtype=torch.int32, device="cuda"))
        return s
    lens = _lengths(c)
    n, rows = len(lens), -(-max(lens) // CHUNK) * CHUNK
    starts = [0]
    for v in lens:
        starts.append(starts[-1] + v)
    s["lens"], s["starts"] = lens, starts
    s["cu_seqlens"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    at = torch.arange(rows, device="cuda")[None, :]
    s["live"] = at < torch.tensor(lens, device="cuda")[:, None]            # [n, rows]
    s["pad"] = torch.where(s["live"], at + s["cu_seqlens"][:-1, None], 0)
    s["back"] = torch.nonzero(s["live"].reshape(-1)).reshape(-1)           # packed token -> padded row
    _heads(s, g, c, c["tokens"])
    order = list(range(n))
    random.Random(seed).shuffle(order)
    s["slot_idx"] = torch.tensor(order, dtype=torch.int32, device="cuda")
    s["initial"] = s["has_initial"] = None
    if c["initial"]:   # every third sequence starts afresh
        s["initial"] = _normal(g, (n, HV, V, K), torch.float32, 0.1)
        s["has_initial"] = torch.tensor([i % 3 != 2 for i in range(n)], device="cuda").to(torch.uint8)
    if c["op"].endswith("fwd"):
        s["final"] = torch.empty((n, HV, V, K), dtype=torch.float32, device="cuda")
    else:
        s["do"] = _normal(g, s["v"].shape, DT[c["io"]])
        s["dfinal"] = _normal(g, (n, HV, V, K), torch.float32, 0.1) if c["initial"] else None
    return s


# ------------------------------------------------------------ the plain forms

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return _PLAIN[c["op"]](s, c)


def _run_own(s, c):
    import linear_recurrence_amd as R
    op = c["op"]
    if op.startswith("rot"):
        x, out = s["x"], None
        if c["inplace"]:
            x = out = s["buffer"].copy_(s["x"])
        fn = R.rotary_forward if op == "rot_fwd" else R.rotary_backward
        return fn(x, s["positions"], s["freqs"], interleaved=c["interleaved"], out=out)
    if op == "lin_step":
        o = R.linear_attention_decode(s["state"], s["slot_idx"], s["q"], s["k"], s["v"], s["log_g"],
                                      new_state=s["new_state"])
        return o, s["new_state"]
    seq = dict(cu_seqlens=s["cu_seqlens"], initial_state=s["initial"], has_initial=s["has_initial"],
               slot_idx=s["slot_idx"])
    if op == "lin_fwd":
        o = R.linear_attention_forward(s["q"], s["k"], s["v"], s["log_g"], final_state=s["final"], **seq)
        return o, s["final"]
    if op == "gdn_fwd":
        o = R.gdn_scan_forward(s["q"], s["k"], s["v"], s["log_g"], s["beta"], final_state=s["final"], **seq)
        return o, s["final"]
    if op == "lin_bwd":
        g = R.linear_attention_backward(s["do"], s["q"], s["k"], s["v"], s["log_g"],
                                        dfinal_state=s["dfinal"], **seq)
    else:
        g = R.gdn_scan_backward(s["do"], s["q"], s["k"], s["v"], s["log_g"], s["beta"],
                                dfinal_state=s["dfinal"], **seq)
    return {k: v for k, v in g.items() if v is not None}


def _plain_rot(s, c):
    x = s["buffer"].copy_(s["x"]) if c["inplace"] else s["x"]
    angle = s["positions"].double()[:, None] * s["freqs"].double()   # [T, rotary/2]
    if c["op"] == "rot_bwd":
        angle = -angle
    co, si = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.clone()
    part, half = x[..., :c["rotary"]].float(), c["rotary"] // 2
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        y[..., 0:c["rotary"]:2] = (a * co - b * si).to(x.dtype)
        y[..., 1:c["rotary"]:2] = (a * si + b * co).to(x.dtype)
    else:
        a, b = part[..., :half], part[..., half:]
        y[..., :half] = (a * co - b * si).to(x.dtype)
        y[..., half:c["rotary"]] = (a * si + b * co).to(x.dtype)
    return y


def _plain_step(s, c):
    r, at = c["vheads"] // c["kheads"], s["slot_idx"].long()
    q, k = (s[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    S = s["state"][at]
    if s["log_g"] is not None:
        S = S * torch.exp(s["log_g"])[..., None, None]
    S = S + s["v"].float()[..., :, None] * k[..., None, :]
    s["new_state"][at] = S
    o = (S * q[..., None, :]).sum(-1) * c["dk"] ** -0.5
    return o.to(s["v"].dtype), s["new_state"]


def _chunks(s, t):
    """Packed [T, H, ...] -> fp32 [n, chunks, H, 64, ...], zeros behind a sequence's end."""
    t = t.float()[s["pad"]] * s["live"][(...,) + (None,) * (t.dim() - 1)]
    t = t.unflatten(1, (-1, CHUNK))
    return t.transpose(2, 3).contiguous()


def _packed(s, t):
    """[n, chunks, H, 64, ...] -> packed [T, H, ...]."""
    return t.transpose(2, 3).flatten(0, 2)[s["back"]]


def _start(s, c, dev):
    n, HV, K, V = len(s["lens"]), c["vheads"], c["dk"], c["dv"]
    if s["initial"] is None:
        return torch.zeros((n, HV, K, V), device=dev)
    S = s["initial"][s["slot_idx"].long()] * s["has_initial"][:, None, None, None]
    return S.transpose(2, 3).contiguous()


def _pieces(s, c):
    """What both directions need of every chunk, and the states before them."""
    r, T, dev = c["vheads"] // c["kheads"], c["tokens"], s["q"].device
    p = dict(Q=_chunks(s, s["q"]).repeat_interleave(r, 2) * c["dk"] ** -0.5,
             K=_chunks(s, s["k"]).repeat_interleave(r, 2), V=_chunks(s, s["v"]))
    lg = s["log_g"]
    lg = torch.zeros(c["vheads"], device=dev) if lg is None else lg
    G = _chunks(s, lg.expand(T, c["vheads"])).double().cumsum(3)
    low = torch.ones((CHUNK, CHUNK), device=dev).tril().bool()
    gap = (G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)
    p["gam"] = torch.exp(gap.float())                                      # [n, c, H, 64, 64]
    p["eG"], p["eT"] = torch.exp(G.float())[..., None], torch.exp((G[..., -1:] - G).float())[..., None]
    p["all"] = torch.exp(G[..., -1].float())[..., None, None]
    p["P"] = p["gam"] * (p["Q"] @ p["K"].transpose(-1, -2))
    p["delta"] = c["op"].startswith("gdn")
    if p["delta"]:
        p["beta"] = _chunks(s, s["beta"])[..., None]
        p["M"] = (p["gam"] * (p["K"] @ p["K"].transpose(-1, -2))).tril(-1)
        A = p["beta"] * p["M"]
        Ti = torch.eye(CHUNK, device=dev).expand(A.shape).clone()
        for i in range(1, CHUNK):   # (I + A)^-1, a row at a time
            Ti[..., i, :i] = -(A[..., i:i + 1, :i] @ Ti[..., :i, :i])[..., 0, :]
        p["T"] = Ti
    S, states, D, O = _start(s, c, dev), [], [], []
    for j in range(p["V"].shape[1]):
        states.append(S)
        d = p["V"][:, j]
        if p["delta"]:
            d = p["T"][:, j] @ (p["beta"][:, j] * (d - p["eG"][:, j] * (p["K"][:, j] @ S)))
        if c["op"].endswith("fwd"):
            O.append(p["eG"][:, j] * (p["Q"][:, j] @ S) + p["P"][:, j] @ d)
        D.append(d)
        S = p["all"][:, j] * S + (p["eT"][:, j] * p["K"][:, j]).transpose(-1, -2) @ d
    p.update(S=states, D=D, O=O, end=S)
    return p


def _plain_fwd(s, c):
    p = _pieces(s, c)
    s["final"][s["slot_idx"].long()] = p["end"].transpose(2, 3)
    return _packed(s, torch.stack(p["O"], 1)).to(s["v"].dtype), s["final"]


def _plain_bwd(s, c):
    p, io, r = _pieces(s, c), s["v"].dtype, c["vheads"] // c["kheads"]
    dO = _chunks(s, s["do"])
    dS = torch.zeros_like(p["end"]) if s["dfinal"] is None else s["dfinal"].transpose(2, 3)
    dQ, dK, dV, dB, dG = [], [], [], [], []
    tr = lambda t: t.transpose(-1, -2)  # noqa: E731
    for j in reversed(range(dO.shape[1])):
        Q, K, P, D, S, o = p["Q"][:, j], p["K"][:, j], p["P"][:, j], p["D"][j], p["S"][j], dO[:, j]
        eG, eT, gam, al = p["eG"][:, j], p["eT"][:, j], p["gam"][:, j], p["all"][:, j]
        dP = o @ tr(D)                                    # i: output, j: token
        dD = tr(P) @ o + eT * (K @ dS)
        into = eG * (o @ tr(S))                           # gradient of Q through the state
        out = eT * (D @ tr(dS))                           # gradient of K through the state
        N = gam * dP
        dq, dk = into + N @ K, out + tr(N) @ Q
        W = P * dP
        give, take = (into * Q).sum(-1), (out * K).sum(-1)
        total = (al * S * dS).sum((-1, -2)) + take.sum(-1)
        dS = al * dS + tr(eG * Q) @ o
        if p["delta"]:
            b, M = p["beta"][:, j], p["M"][:, j]
            dX = tr(p["T"][:, j]) @ dD
            dA = -(dX @ tr(D))
            back = eG * (dX @ tr(S))
            L = b * gam.tril(-1) * dA
            dk = dk - b * back + (L + tr(L)) @ K
            W = W + b * M * dA
            give = give - b[..., 0] * (back * K).sum(-1)
            dB.append((dX * p["V"][:, j]).sum(-1) - (back * K).sum(-1) + (M * dA).sum(-1))
            dS = dS - tr(eG * K) @ (b * dX)
            dD = b * dX
        g = (W.sum(-1) - W.sum(-2) + give - take).double()
        g[..., -1] += total
        dG.append(g.flip(-1).cumsum(-1).flip(-1).float())
        dQ.append(dq)
        dK.append(dk)
        dV.append(dD)
    whole = lambda t: _packed(s, torch.stack(t[::-1], 1))  # noqa: E731
    share = lambda t: t.unflatten(1, (c["kheads"], r)).sum(2)  # noqa: E731
    out = dict(dq=(share(whole(dQ)) * c["dk"] ** -0.5).to(io), dk=share(whole(dK)).to(io),
               dv=whole(dV).to(io))
    dg = whole(dG)
    if p["delta"]:
        out.update(dlog_g=dg, dbeta=whole(dB))
    elif s["log_g"] is not None:
        out["dlog_decay"] = dg if s["log_g"].dim() == 2 else dg.sum(0)
    if s["initial"] is not None:
        out["dinitial_state"] = (dS * s["has_initial"][:, None, None, None]).transpose(2, 3).contiguous()
    return out


_PLAIN = dict(lin_step=_plain_step, lin_fwd=_plain_fwd, lin_bwd=_plain_bwd, gdn_fwd=_plain_fwd,
              gdn_bwd=_plain_bwd, rot_fwd=_plain_rot, rot_bwd=_plain_rot)


# -------------------------------------------------------------- what it takes

def work(case):
    c = case
    es = 2 if c["io"] == "bf16" else 4
    if c["op"].startswith("rot"):
        n = c["tokens"] * c["heads"] * c["dim"]
        return dict(bytes=2 * n * es + 8 * c["tokens"] + 2 * c["rotary"],
                    flops=3 * c["tokens"] * c["heads"] * c["rotary"])
    HK, HV, K, V = c["kheads"], c["vheads"], c["dk"], c["dv"]
    delta, back = c["op"].startswith("gdn"), c["op"].endswith("bwd")
    rows = c["batch"] if c["op"] == "lin_step" else c["tokens"]
    qk, v, st = rows * HK * K * es, rows * HV * V * es, HV * V * K * 4
    gates = 0 if c.get("decay") == "none" else HV * 4 if c.get("decay") == "head" else rows * HV * 4
    gates += rows * HV * 4 if delta else 0
    if c["op"] == "lin_step":
        return dict(bytes=2 * qk + 2 * v + gates + 2 * rows * st, flops=rows * HV * K * V * 5)
    lens = _lengths(c)
    begun = sum(i % 3 != 2 for i in range(len(lens))) if c["initial"] else 0
    if not back:
        return dict(bytes=2 * qk + 2 * v + gates + (begun + len(lens)) * st,
                    flops=rows * HV * K * V * (6 if delta else 4))
    states = begun + 2 * len(lens) if c["initial"] else 0
    return dict(bytes=4 * qk + 3 * v + 2 * gates + states * st,
                flops=rows * HV * K * V * (16 if delta else 10))


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"].startswith("rot"):
        return _exact_rot(s, c)
    if c["op"] == "lin_step":
        return _exact_step(s, c)
    return _exact_seq(s, c)


def _exact_rot(s, c):
    x, half = s["x"].double(), c["rotary"] // 2
    y = x.clone()
    sign = 1.0 if c["op"] == "rot_fwd" else -1.0
    for i in range(half):
        turn = s["positions"].double() * float(s["freqs"][i])
        co, si = torch.cos(turn)[:, None], sign * torch.sin(turn)[:, None]
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        y[..., a], y[..., b] = x[..., a] * co - x[..., b] * si, x[..., b] * co + x[..., a] * si
    return y


def _exact_step(s, c):
    r = c["vheads"] // c["kheads"]
    o = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
    new = torch.empty(s["state"].shape, dtype=torch.float64, device="cuda")
    for b, slot in enumerate(s["slot_idx"].tolist()):
        S = s["state"][slot].double()
        if s["log_g"] is not None:
            g = s["log_g"] if s["log_g"].dim() == 1 else s["log_g"][b]
            S = S * torch.exp(g.double())[:, None, None]
        q, k = (s[n][b].double().repeat_interleave(r, 0) for n in ("q", "k"))
        S = S + s["v"][b].double()[:, :, None] * k[:, None, :]
        new[slot] = S
        o[b] = (S * q[:, None, :]).sum(2) / math.sqrt(c["dk"])
    return o, new


def _exact_seq(s, c):
    """One token of every sequence at a time, S [sequences, HV, V, K]; the
    backward pass takes the states of 32 tokens at a time."""
    delta, back, f64 = c["op"].startswith("gdn"), c["op"].endswith("bwd"), torch.float64
    HK, HV, T, n, r = c["kheads"], c["vheads"], c["tokens"], len(s["lens"]), c["vheads"] // c["kheads"]
    scale = 1.0 / math.sqrt(c["dk"])
    q, k = (s[m].double().repeat_interleave(r, 1) for m in ("q", "k"))
    v = s["v"].double()
    lg = s["log_g"]
    g = torch.ones((T, HV), dtype=f64, device="cuda") if lg is None else \
        torch.exp(lg.double()).expand(T, HV)
    beta = s["beta"].double() if delta else None
    S = torch.zeros((n, HV, c["dv"], c["dk"]), dtype=f64, device="cuda")
    if s["initial"] is not None:
        for i, slot in enumerate(s["slot_idx"].tolist()):
            if int(s["has_initial"][i]):
                S[i] = s["initial"][slot].double()
    starts = torch.tensor(s["starts"][:-1], device="cuda")
    lens = torch.tensor(s["lens"], device="cuda")
    # the longest first: token t is one of the first `live` of them
    order = torch.argsort(lens, descending=True)
    starts, S = starts[order], S[order]
    count = sorted(s["lens"], reverse=True)
    most = count[0]
    live = [sum(m > t for m in count) for t in range(most)]
    o = torch.zeros(v.shape, dtype=f64, device="cuda")

    def step(S, t):
        m = live[t]
        at = starts[:m] + t
        S1 = S[:m] * g[at][:, :, None, None]
        e = v[at]
        if delta:
            e = e - (S1 * k[at][:, :, None, :]).sum(3)
        d = beta[at][:, :, None] * e if delta else e
        return at, S1, e, d, S1 + d[:, :, :, None] * k[at][:, :, None, :]

    kept = []
    for t in range(most):
        if back and t % 32 == 0:
            kept.append(S.clone())
        at, _, _, _, S2 = step(S, t)
        if not back:
            o[at] = scale * (S2 * q[at][:, :, None, :]).sum(3)
        S[:live[t]] = S2
    put = torch.empty_like(order)
    put[order] = torch.arange(n, device="cuda")
    if not back:
        final = torch.empty_like(S)
        final[s["slot_idx"].long()] = S[put]
        return o, final
    do = s["do"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g).contiguous(), torch.zeros((T, HV), dtype=f64, device="cuda")
    dS = torch.zeros_like(S) if s["dfinal"] is None else s["dfinal"].double()[order]
    for b in reversed(range(len(kept))):
        S, seen = kept[b], []
        for t in range(32 * b, min(32 * b + 32, most)):
            seen.append(step(S, t))
            S = torch.cat([seen[-1][4], S[live[t]:]])
        for at, S1, e, d, S2 in reversed(seen):
            m = at.shape[0]
            dS[:m] += scale * do[at][:, :, :, None] * q[at][:, :, None, :]
            dq[at] = scale * (S2 * do[at][:, :, :, None]).sum(2)
            dd = (dS[:m] * k[at][:, :, None, :]).sum(3)
            dk[at] = (dS[:m] * d[:, :, :, None]).sum(2)
            if delta:
                db[at] = (dd * e).sum(2)
                dd = beta[at][:, :, None] * dd
                dk[at] -= (S1 * dd[:, :, :, None]).sum(2)
                dS[:m] -= dd[:, :, :, None] * k[at][:, :, None, :]
            dv[at] = dd
            dg[at] = (dS[:m] * S1).sum((2, 3))
            dS[:m] *= g[at][:, :, None, None]
    share = lambda t: t.reshape(T, HK, r, -1).sum(2)  # noqa: E731
    out = dict(dq=share(dq), dk=share(dk), dv=dv)
    if delta:
        out.update(dlog_g=dg, dbeta=db)
    elif lg is not None:
        out["dlog_decay"] = dg if lg.dim() == 2 else dg.sum(0)
    if s["initial"] is not None:
        out["dinitial_state"] = dS[put] * s["has_initial"].double()[:, None, None, None]
    return out
