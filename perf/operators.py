"""What the operators around the decode step are measured on.

A Mamba2 layer's prefill and training operators: the gated linear recurrence
over whole sequences (forward and backward), the short causal convolution in
front of it (forward, backward, one decode step) and the root-mean-square norm
around it (residual, gate, 8-bit output, backward).  ``run`` computes a case in
elementary torch operations where ``own`` is false and through the library's
entry points where it is true; ``exact`` is the definition in 64 bits.

Values are drawn as the repository's workloads draw them: x, z, dt_raw ~
N(0, 1), B, C ~ N(0, 1)/4, A = -exp(U[0, ln 16]), softplus(dt_bias) uniform on
[1e-3, 1e-1], D ~ N(0, 1), states ~ N(0, 0.1).
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64          # tokens per block of the plain scan
EPS = 1e-5
E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases

def listed():
    scan = dict(op="scan_fwd", headdim=64, dstate=128, groups=1, io="bf16", state="f32")
    grad = dict(op="scan_bwd", headdim=64, dstate=128, groups=1, io="bf16", initial=False)
    return [
        # a few short prompts of the tiny fp32 model: latency is what counts
        dict(scan, name="scan_fwd_tiny", tokens=61, seqs=4, even=False, heads=8, dstate=16,
             io="f32", initial=True, gate=True),
        # one long prompt of a 2.7B-like layer (80 heads) that continues from a cached state
        dict(scan, name="scan_fwd_prompt", tokens=4096, seqs=1, even=True, heads=80,
             initial=True, gate=False),
        # a serving engine's prefill batch: uneven prompts packed one after another
        dict(scan, name="scan_fwd_packed", tokens=16383, seqs=13, even=False, heads=80,
             state="bf16", initial=True, gate=False),
        # the tiny fp32 model's training step
        dict(grad, name="scan_bwd_tiny", tokens=96, seqs=3, even=False, heads=8, dstate=16,
             io="f32", initial=True),
        # the grouped layer (128 heads, 8 groups) on two uneven sequences
        dict(grad, name="scan_bwd_grouped", tokens=1291, seqs=2, even=False, heads=128,
             groups=8, initial=True),
        # a training micro-batch of a 2.7B-like layer: 8 sequences of 2048
        dict(grad, name="scan_bwd_train", tokens=16384, seqs=8, even=True, heads=80),
        # the convolution in the decode step of 512 requests (x, B and C channels together)
        dict(op="conv_step", name="conv_step_b512", batch=512, channels=5376, width=4, io="bf16"),
        # the same channels over the packed prefill batch
        dict(op="conv_fwd", name="conv_fwd_packed", tokens=16383, seqs=13, even=False,
             channels=5376, width=4, io="bf16", initial=True),
        # and in training
        dict(op="conv_bwd", name="conv_bwd_train", tokens=16384, seqs=8, even=True,
             channels=5376, width=4, io="bf16", initial=False),
        # the gated norm of a decode batch in front of an 8-bit out-projection
        dict(op="norm_fwd", name="norm_gate_fp8_b64", rows=64, dim=5120, group=5120, io="bf16",
             gate=True, residual="none", out="fp8", scales="row"),
        # the block's norm with the fp32 residual's addition, 8-bit output, over a prefill batch
        dict(op="norm_fwd", name="norm_add_fp8_packed", rows=16383, dim=2560, group=2560,
             io="bf16", gate=False, residual="f32", out="fp8", scales="block"),
        # the grouped gated norm's backward pass in training
        dict(op="norm_bwd", name="norm_gate_bwd", rows=8192, dim=8192, group=1024, io="bf16",
             gate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_bwd", "scan_fwd", "scan_bwd", "conv_step", "conv_fwd",
                     "conv_bwd", "norm_fwd", "norm_fwd", "norm_bwd"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("scan"):
        groups = rng.choice([1, 1, 2, 4, 8])
        heads = groups * max(1, _log(rng, 2, 96) // groups)
        headdim, dstate = rng.choice([32, 64, 64, 128]), rng.choice([16, 32, 64, 128, 128, 256])
        most = 16384 * 80 * 64 * 128 // (heads * headdim * dstate)
        if io == "f32":
            most //= 8
        if op == "scan_bwd":
            most //= 2
        tokens = _log(rng, 3, max(4, min(8192, most)))
        c = dict(op=op, tokens=tokens, seqs=_log(rng, 1, min(24, tokens)), even=False, heads=heads,
                 headdim=headdim, dstate=dstate, groups=groups, io=io,
                 initial=rng.random() < 0.6)
        if op == "scan_fwd":
            c.update(state=rng.choice(["f32", "bf16"]), gate=rng.random() < 0.5)
        return c
    if op == "conv_step":
        return dict(op=op, batch=_log(rng, 1, 512), channels=_log(rng, 33, 5376),
                    width=rng.choice([2, 3, 4]), io=io)
    if op.startswith("conv"):
        tokens = _log(rng, 3, 8192)
        return dict(op=op, tokens=tokens, seqs=_log(rng, 1, min(24, tokens)), even=False,
                    channels=rng.choice([8 * _log(rng, 4, 672), _log(rng, 33, 2000)]),
                    width=rng.choice([2, 3, 4]), io=io, initial=rng.random() < 0.6)
    blocks = rng.choice([1, 1, 2, 4, 8])
    if op == "norm_fwd":
        out = rng.choice(["io", "fp8"])
        scales = rng.choice(["row", "block"])
        dim = blocks * 128 * _log(rng, 1, 64 // blocks) if out == "fp8" and scales == "block" \
            else blocks * _log(rng, 40, 8192 // blocks)
        return dict(op=op, rows=_log(rng, 1, 8192), dim=dim, group=dim // blocks, io=io,
                    gate=rng.random() < 0.5, residual=rng.choice(["none", "f32", "io"]), out=out,
                    scales=scales)
    dim = blocks * _log(rng, 40, 8192 // blocks)
    return dict(op=op, rows=_log(rng, 1, 4096), dim=dim, group=dim // blocks, io=io,
                gate=rng.random() < 0.5)


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


def _uniform(g, n, lo, hi):
    return torch.rand(n, generator=g, device="cuda", dtype=torch.float32) * (hi - lo) + lo


def _scan_params(g, H):
    bias = torch.log(torch.expm1(_uniform(g, H, 1e-3, 1e-1)))
    return dict(A=-torch.exp(_uniform(g, H, 0.0, math.log(16.0))),
                D=_normal(g, (H,), torch.float32), dt_bias=bias)


def _plan(s, c):
    lens = _lengths(c)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s["lens"], s["starts"] = lens, starts
    s["cu_seqlens"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    return lens, starts


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"].startswith("scan"):
        T, H, P, N, G, io = c["tokens"], c["heads"], c["headdim"], c["dstate"], c["groups"], DT[c["io"]]
        lens, starts = _plan(s, c)
        n, rows = len(lens), -(-max(lens) // CHUNK) * CHUNK
        at = torch.arange(rows, device="cuda")[None, :]
        ln = torch.tensor(lens, device="cuda")[:, None]
        s["live"] = at < ln                                            # [n, rows]
        s["pad"] = torch.where(s["live"], at + s["cu_seqlens"][:-1, None], 0)
        s["back"] = torch.nonzero(s["live"].reshape(-1)).reshape(-1)   # packed token -> padded row
        s.update(_scan_params(g, H), x=_normal(g, (T, H, P), io), dt=_normal(g, (T, H), io),
                 B=_normal(g, (T, G, N), io, 0.25), C=_normal(g, (T, G, N), io, 0.25))
        order = list(range(n))
        random.Random(seed).shuffle(order)
        s["slot_idx"] = torch.tensor(order, dtype=torch.int32, device="cuda")
        s["initial"] = s["has_initial"] = None
        if c["initial"]:   # every third sequence starts afresh
            st = DT[c["state"]] if c["op"] == "scan_fwd" else torch.float32
            s["initial"] = _normal(g, (n, H, P, N), st, 0.1)
            s["has_initial"] = torch.tensor([i % 3 != 2 for i in range(n)], device="cuda").to(torch.uint8)
        if c["op"] == "scan_fwd":
            s["z"] = _normal(g, (T, H, P), io) if c["gate"] else None
            s["final"] = torch.empty((n, H, P, N), dtype=DT[c["state"]], device="cuda")
        else:
            s["dy"] = _normal(g, (T, H, P), io)
            s["dfinal"] = _normal(g, (n, H, P, N), torch.float32, 0.1) if c["initial"] else None
    elif c["op"].startswith("conv"):
        C, W, io = c["channels"], c["width"], DT[c["io"]]
        s["weight"], s["bias"] = _normal(g, (C, W), torch.float32, 0.5), _normal(g, (C,), torch.float32, 0.5)
        if c["op"] == "conv_step":
            nb = c["batch"]
            order = list(range(nb))
            random.Random(seed).shuffle(order)
            s.update(x=_normal(g, (nb, C), io), conv_state=_normal(g, (nb, W - 1, C), io),
                     slot_idx=torch.tensor(order, dtype=torch.int32, device="cuda"),
                     new_state=torch.empty((nb, W - 1, C), dtype=io, device="cuda"))
        else:
            lens, starts = _plan(s, c)
            n, T = len(lens), c["tokens"]
            s.update(x=_normal(g, (T, C), io), initial=None)
            if c["initial"]:
                s["initial"] = _normal(g, (n, W - 1, C), io)
            # rows of cat([initial states, x]) that each token's window reads
            of = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(lens, device="cuda"))
            first = s["cu_seqlens"][:-1].long()[of]
            pos = torch.arange(T, device="cuda") - first
            j = torch.arange(W, device="cuda")[None, :]
            p = pos[:, None] - (W - 1) + j
            s["window"] = torch.where(p >= 0, n * (W - 1) + first[:, None] + p,
                                      of[:, None] * (W - 1) + p + W - 1)
            ln = torch.tensor(lens, device="cuda")[:, None]
            i = torch.arange(n, device="cuda")[:, None]
            q = ln - (W - 1) + torch.arange(W - 1, device="cuda")[None, :]
            s["last"] = torch.where(q >= 0, n * (W - 1) + s["cu_seqlens"][:-1, None] + q,
                                    i * (W - 1) + q + W - 1)
            s["final"] = torch.empty((n, W - 1, C), dtype=io, device="cuda")
            if c["op"] == "conv_bwd":
                s["dy"] = _normal(g, (T, C), io)
    else:
        R, M, io = c["rows"], c["dim"], DT[c["io"]]
        s.update(x=_normal(g, (R, M), io), weight=1.0 + _normal(g, (M,), torch.float32, 0.2),
                 z=_normal(g, (R, M), io) if c["gate"] else None)
        if c["op"] == "norm_fwd":
            res = c["residual"]
            s["residual"] = None if res == "none" else _normal(g, (R, M), DT["f32"] if res == "f32" else io, 3.0)
        else:
            s["dy"] = _normal(g, (R, M), io)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    return (_OWN if own else _PLAIN)[c["op"]](s, c)


def _own_scan_fwd(s, c):
    import linear_recurrence_amd as R
    y = R.ssu_scan_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                           dt_bias=s["dt_bias"], cu_seqlens=s["cu_seqlens"],
                           initial_state=s["initial"], has_initial=s["has_initial"],
                           final_state=s["final"], slot_idx=s["slot_idx"])
    return y, s["final"]


def _own_scan_bwd(s, c):
    import linear_recurrence_amd as R
    got = R.ssu_scan_backward(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"],
                              dt_bias=s["dt_bias"], cu_seqlens=s["cu_seqlens"],
                              initial_state=s["initial"], has_initial=s["has_initial"],
                              slot_idx=s["slot_idx"], dfinal_state=s["dfinal"])
    return {k: v for k, v in got.items() if v is not None}


def _own_conv_step(s, c):
    import linear_recurrence_amd as R
    y = R.causal_conv_decode(s["x"], s["conv_state"], s["weight"], bias=s["bias"],
                             slot_idx=s["slot_idx"], new_state=s["new_state"])
    return y, s["new_state"]


def _own_conv_fwd(s, c):
    import linear_recurrence_amd as R
    y = R.causal_conv_forward(s["x"], s["weight"], bias=s["bias"], cu_seqlens=s["cu_seqlens"],
                              initial_state=s["initial"], final_state=s["final"])
    return y, s["final"]


def _own_conv_bwd(s, c):
    import linear_recurrence_amd as R
    got = R.causal_conv_backward(s["dy"], s["x"], s["weight"], bias=s["bias"],
                                 cu_seqlens=s["cu_seqlens"], initial_state=s["initial"])
    return {k: v for k, v in got.items() if v is not None}


def _own_norm_fwd(s, c):
    import linear_recurrence_amd as R
    fp8 = c["out"] == "fp8"
    got = R.rms_norm_forward(s["x"], s["weight"], z=s["z"], residual=s["residual"],
                             group_size=c["group"], eps=EPS,
                             out_dtype=torch.float8_e4m3fn if fp8 else None,
                             scale_block=128 if fp8 and c["scales"] == "block" else 0)
    return {k: v for k, v in got.items() if v is not None}


def _own_norm_bwd(s, c):
    import linear_recurrence_amd as R
    got = R.rms_norm_backward(s["dy"], s["x"], s["weight"], z=s["z"], group_size=c["group"], eps=EPS)
    return {k: v for k, v in got.items() if v is not None}


_OWN = dict(scan_fwd=_own_scan_fwd, scan_bwd=_own_scan_bwd, conv_step=_own_conv_step,
            conv_fwd=_own_conv_fwd, conv_bwd=_own_conv_bwd, norm_fwd=_own_norm_fwd,
            norm_bwd=_own_norm_bwd)


# ---------------------------------------------------------------- plain forms

def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _scan_f32(x, dt, A, B, C, D, dt_bias, init, live, pad, back, G):
    """The recurrence in blocks of CHUNK tokens, 32 bits, the decays' angles in 64.

    x [T, H, P], dt [T, H], B, C [T, G, N]; init [n, H, P, N].  Returns
    (y [T, H, P], final states [n, H, P, N])."""
    n, rows = pad.shape
    H, P, N = x.shape[1], x.shape[2], B.shape[2]
    c, q, e = rows // CHUNK, CHUNK, H // G
    m = live.to(torch.float32)
    d = _softplus(dt + dt_bias)[pad] * m[..., None]                                   # [n, rows, H]
    xp = (x[pad] * m[..., None, None]).reshape(n, c, q, H, P).permute(0, 1, 3, 2, 4)  # [n, c, H, q, P]
    Bp = (B[pad] * m[..., None, None]).reshape(n, c, q, G, N).permute(0, 1, 3, 2, 4)
    Cp = (C[pad] * m[..., None, None]).reshape(n, c, q, G, N).permute(0, 1, 3, 2, 4)
    dp = d.reshape(n, c, q, H).permute(0, 1, 3, 2)                                    # [n, c, H, q]
    cum = torch.cumsum(dp.double() * A.double()[None, None, :, None], dim=-1)
    tri = torch.ones(q, q, dtype=torch.bool, device=x.device).tril()
    gap = (cum[..., :, None] - cum[..., None, :]).to(torch.float32)
    decay = torch.exp(gap.masked_fill(~tri, float("-inf")))                           # [n, c, H, q, q]
    cb = torch.matmul(Cp, Bp.transpose(-1, -2).contiguous()).repeat_interleave(e, 2)
    y = torch.matmul(decay * cb * dp[..., None, :], xp.contiguous())
    tail = torch.exp((cum[..., -1:] - cum).to(torch.float32)) * dp
    Bh, Ch = Bp.repeat_interleave(e, 2), Cp.repeat_interleave(e, 2)
    add = torch.matmul((xp * tail[..., None]).transpose(-1, -2).contiguous(), Bh.contiguous())
    # states before each block: the initial one, then what the blocks add
    total = torch.cumsum(torch.cat([torch.zeros_like(cum[:, :1, :, -1]), cum[..., -1]], 1), 1)  # [n, c+1, H]
    total = total.permute(0, 2, 1)
    tri = torch.ones(c + 1, c + 1, dtype=torch.bool, device=x.device).tril()
    over = (total[..., :, None] - total[..., None, :]).to(torch.float32)
    over = torch.exp(over.masked_fill(~tri, float("-inf")))                           # [n, H, c+1, c+1]
    both = torch.cat([init[:, None], add], 1).permute(0, 2, 1, 3, 4).reshape(n, H, c + 1, P * N)
    states = torch.matmul(over, both.contiguous()).reshape(n, H, c + 1, P, N).permute(0, 2, 1, 3, 4)
    y = y + torch.matmul(Ch.contiguous(), states[:, :-1].transpose(-1, -2).contiguous()) \
        * torch.exp(cum.to(torch.float32))[..., None]
    y = y + D[None, None, :, None, None] * xp
    y = y.permute(0, 1, 3, 2, 4).reshape(n * rows, H, P)[back]
    return y, states[:, -1]


def _start(s, c):
    n = len(s["lens"])
    if s["initial"] is None:
        return torch.zeros((n, c["heads"], c["headdim"], c["dstate"]), device="cuda")
    got = s["initial"][s["slot_idx"].long()].float()
    return torch.where(s["has_initial"].bool()[:, None, None, None], got, torch.zeros_like(got))


def _plain_scan_fwd(s, c):
    y, last = _scan_f32(s["x"].float(), s["dt"].float(), s["A"], s["B"].float(), s["C"].float(), s["D"],
                        s["dt_bias"], _start(s, c), s["live"], s["pad"], s["back"], c["groups"])
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    final = torch.empty_like(s["final"])
    final[s["slot_idx"].long()] = last.to(final.dtype)
    return y.to(s["x"].dtype), final


def _plain_scan_bwd(s, c):
    io = s["x"].dtype
    ins = dict(x=s["x"].float(), dt=s["dt"].float(), A=s["A"], B=s["B"].float(), C=s["C"].float(), D=s["D"],
               dt_bias=s["dt_bias"], init=_start(s, c))
    ins = {k: v.detach().clone().requires_grad_(True) for k, v in ins.items()}
    y, last = _scan_f32(**ins, live=s["live"], pad=s["pad"], back=s["back"], G=c["groups"])
    up = [s["dy"].float()] + ([s["dfinal"]] if s["dfinal"] is not None else [])
    got = dict(zip(ins, torch.autograd.grad([y, last][:len(up)], list(ins.values()), up)))
    out = {"d" + k: got[k].to(io) for k in ("x", "dt", "B", "C")}
    out.update({"d" + k: got[k] for k in ("A", "D", "dt_bias")})
    if s["initial"] is not None:   # no gradient where a sequence started afresh
        out["dinitial_state"] = got["init"] * s["has_initial"][:, None, None, None]
    return out


def _plain_conv_step(s, c):
    old = s["conv_state"][s["slot_idx"].long()]
    win = torch.cat([old, s["x"][:, None]], 1)
    y = _silu((win.float() * s["weight"].t()[None]).sum(1) + s["bias"])
    new = torch.empty_like(s["new_state"])
    new[s["slot_idx"].long()] = win[:, 1:]
    return y.to(s["x"].dtype), new


def _conv_f32(x, weight, bias, init, window):
    rows = torch.cat([init.reshape(-1, x.shape[1]), x])
    return _silu((rows[window] * weight.t()[None]).sum(1) + bias)


def _conv_start(s, c):
    if s["initial"] is not None:
        return s["initial"]
    return torch.zeros((len(s["lens"]), c["width"] - 1, c["channels"]), dtype=s["x"].dtype, device="cuda")


def _plain_conv_fwd(s, c):
    init = _conv_start(s, c)
    y = _conv_f32(s["x"].float(), s["weight"], s["bias"], init.float(), s["window"])
    return y.to(s["x"].dtype), torch.cat([init.reshape(-1, c["channels"]), s["x"]])[s["last"]]


def _plain_conv_bwd(s, c):
    io = s["x"].dtype
    ins = dict(x=s["x"].float(), weight=s["weight"], bias=s["bias"], init=_conv_start(s, c).float())
    ins = {k: v.detach().clone().requires_grad_(True) for k, v in ins.items()}
    y = _conv_f32(**ins, window=s["window"])
    got = dict(zip(ins, torch.autograd.grad(y, list(ins.values()), s["dy"].float())))
    out = dict(dx=got["x"].to(io), dweight=got["weight"], dbias=got["bias"])
    if s["initial"] is not None:
        out["dinitial_state"] = got["init"].to(io)
    return out


def _norm_f32(h, weight, z, group):
    u = h if z is None else h * _silu(z)
    v = u.reshape(u.shape[0], -1, group)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return (v * r).reshape(u.shape) * weight


def _plain_norm_fwd(s, c):
    h, out = s["x"].float(), {}
    if s["residual"] is not None:
        out["residual"] = (h + s["residual"].float()).to(s["residual"].dtype)
        h = out["residual"].float()
    y = _norm_f32(h, s["weight"], None if s["z"] is None else s["z"].float(), c["group"])
    if c["out"] != "fp8":
        out["out"] = y.to(s["x"].dtype)
        return out
    v = y.reshape(y.shape[0], -1, 128 if c["scales"] == "block" else y.shape[1])
    top = v.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    out["out"] = (v / scale).clamp(-E4M3_MAX, E4M3_MAX).reshape(y.shape).to(torch.float8_e4m3fn)
    out["scale"] = scale.squeeze(-1)
    return out


def _plain_norm_bwd(s, c):
    io = s["x"].dtype
    ins = dict(h=s["x"].float(), weight=s["weight"])
    if s["z"] is not None:
        ins["z"] = s["z"].float()
    ins = {k: v.detach().clone().requires_grad_(True) for k, v in ins.items()}
    y = _norm_f32(ins["h"], ins["weight"], ins.get("z"), c["group"])
    got = dict(zip(ins, torch.autograd.grad(y, list(ins.values()), s["dy"].float())))
    out = dict(dx=got["h"].to(io), dweight=got["weight"])
    if s["z"] is not None:
        out["dz"] = got["z"].to(io)
    return out


_PLAIN = dict(scan_fwd=_plain_scan_fwd, scan_bwd=_plain_scan_bwd, conv_step=_plain_conv_step,
              conv_fwd=_plain_conv_fwd, conv_bwd=_plain_conv_bwd, norm_fwd=_plain_norm_fwd,
              norm_bwd=_plain_norm_bwd)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    e = 2 if c["io"] == "bf16" else 4
    if c["op"].startswith("scan"):
        T, H, P, N, G, n = c["tokens"], c["heads"], c["headdim"], c["dstate"], c["groups"], c["seqs"]
        xs, bs, st = T * H * P * e, T * G * N * e, n * H * P * N
        if c["op"] == "scan_fwd":
            se = 2 if c["state"] == "bf16" else 4
            b = xs * (3 if c["gate"] else 2) + 2 * bs + T * H * e + st * se * (2 if c["initial"] else 1)
            return {"bytes": b + 12 * H, "flops": 5.0 * T * H * P * N}
        b = 3 * xs + 4 * bs + 2 * T * H * e + (3 * 4 * st if c["initial"] else 0)
        return {"bytes": b + 24 * H, "flops": 14.0 * T * H * P * N}
    if c["op"].startswith("conv"):
        C, W = c["channels"], c["width"]
        if c["op"] == "conv_step":
            return {"bytes": c["batch"] * C * e * 2 * W + 4 * C * (W + 1), "flops": 2.0 * W * c["batch"] * C}
        T, n = c["tokens"], c["seqs"]
        if c["op"] == "conv_fwd":
            return {"bytes": e * C * (2 * T + n * (W - 1) * (2 if c["initial"] else 1)) + 4 * C * (W + 1),
                    "flops": 2.0 * W * T * C}
        return {"bytes": e * C * (3 * T + n * (W - 1) * (2 if c["initial"] else 0)) + 8 * C * (W + 1),
                "flops": 6.0 * W * T * C}
    R, M = c["rows"], c["dim"]
    if c["op"] == "norm_fwd":
        re = {"none": 0, "f32": 8, "io": 2 * e}[c["residual"]]
        oe = 1 if c["out"] == "fp8" else e
        return {"bytes": R * M * (e * (2 if c["gate"] else 1) + re + oe) + 4 * M, "flops": 8.0 * R * M}
    return {"bytes": R * M * e * (5 if c["gate"] else 3) + 8 * M, "flops": 16.0 * R * M}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _f64(s, *names):
    return [None if s[k] is None else s[k].double() for k in names]


def _padded(v, s):
    """[T, ...] packed -> [longest, n, ...] with zeros, one step's rows together."""
    out = torch.zeros((max(s["lens"]), len(s["lens"])) + tuple(v.shape[1:]), dtype=v.dtype, device=v.device)
    for i, (a, n) in enumerate(zip(s["starts"], s["lens"])):
        out[:n, i] = v[a:a + n]
    return out


def _packed(v, s):
    return torch.cat([v[:n, i] for i, n in enumerate(s["lens"])])


def _exact_inputs(s, c):
    A, bias, raw = _f64(s, "A", "dt_bias", "dt")
    raw = raw + bias
    dt = _padded(torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())), s)   # 0 past the end
    H, G = c["heads"], c["groups"]
    head = torch.arange(H, device="cuda") // (H // G)
    S = torch.zeros((len(s["lens"]), H, c["headdim"], c["dstate"]), dtype=torch.float64, device="cuda")
    if s["initial"] is not None:
        for i, slot in enumerate(s["slot_idx"].tolist()):
            if int(s["has_initial"][i]):
                S[i] = s["initial"][slot].double()
    return A, raw, dt, _padded(s["x"], s), _padded(s["B"], s), _padded(s["C"], s), head, S


def _exact_scan_fwd(s, c):
    A, _, dt, x, B, C, head, S = _exact_inputs(s, c)
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    g = torch.exp(dt * A)
    for t in range(x.shape[0]):
        S.mul_(g[t, :, :, None, None])
        S.addcmul_((dt[t, :, :, None] * x[t].double())[..., None], B[t].double()[:, head, None, :])
        y[t] = (S @ C[t].double()[:, head, :, None])[..., 0]
    y = _packed(y, s) + s["D"].double()[:, None] * s["x"].double()
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    final = torch.zeros(s["final"].shape, dtype=torch.float64, device="cuda")
    for i, slot in enumerate(s["slot_idx"].tolist()):
        final[slot] = S[i]
    return y, final


def _exact_scan_bwd(s, c):
    A, raw, dt, x, B, C, head, S = _exact_inputs(s, c)
    dy = _padded(s["dy"], s)
    steps, n, H, G = x.shape[0], x.shape[1], c["heads"], c["groups"]
    g = torch.exp(dt * A)

    def forward(S, t):
        return g[t, :, :, None, None] * S + (dt[t, :, :, None] * x[t].double())[..., None] \
            * B[t].double()[:, head, None, :]

    every, marks = 32, []
    for t in range(steps):
        if t % every == 0:
            marks.append(S.clone())
        S = forward(S, t)
    L = torch.zeros_like(S) if s["dfinal"] is None else s["dfinal"].double()
    dx = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(B.shape, dtype=torch.float64, device="cuda")
    dC, ddt, da = torch.zeros_like(dB), torch.zeros_like(dt), torch.zeros_like(dt)
    for k in reversed(range(len(marks))):
        t0, t1 = k * every, min(steps, k * every + every)
        before = [marks[k]]
        for t in range(t0, t1):
            before.append(forward(before[-1], t))
        for t in reversed(range(t0, t1)):
            u, b, cc, o = x[t].double(), B[t].double()[:, head], C[t].double()[:, head], dy[t].double()
            dC[t] = (o[:, :, None, :] @ before[t + 1 - t0])[:, :, 0].reshape(n, G, H // G, -1).sum(2)
            L = L + o[..., None] * cc[:, :, None, :]
            Lb = (L @ b[..., None])[..., 0]
            dx[t] = dt[t][..., None] * Lb
            ddt[t] = (Lb * u).sum(-1)
            dB[t] = (dt[t][..., None] * (u[:, :, None, :] @ L)[:, :, 0]).reshape(n, G, H // G, -1).sum(2)
            L = g[t, :, :, None, None] * L
            da[t] = (L * before[t - t0]).sum((-1, -2))
    o, u = s["dy"].double(), s["x"].double()
    step = _packed(ddt + da * A, s) * torch.sigmoid(raw)
    out = dict(dx=_packed(dx, s) + s["D"].double()[:, None] * o, ddt=step, dB=_packed(dB, s), dC=_packed(dC, s),
               dA=(da * dt).sum((0, 1)), dD=(o * u).sum((0, 2)), ddt_bias=step.sum(0))
    if s["initial"] is not None:
        out["dinitial_state"] = L * s["has_initial"].double()[:, None, None, None]
    return out


def _exact_conv_step(s, c):
    W = c["width"]
    y = s["bias"].double()[None].expand(c["batch"], -1).clone()
    new = torch.zeros(s["new_state"].shape, dtype=torch.float64, device="cuda")
    slot = s["slot_idx"].long()
    for j in range(W):
        tap = s["x"].double() if j == W - 1 else s["conv_state"][slot, j].double()
        y += s["weight"][:, j].double() * tap
        if j:
            new[slot, j - 1] = tap
    return y * torch.sigmoid(y), new


def _conv_parts(s, c):
    """Each sequence's rows behind its W - 1 earlier ones, and the convolution's sums, in 64 bits."""
    W = c["width"]
    for i, (a, n) in enumerate(zip(s["starts"], s["lens"])):
        old = torch.zeros((W - 1, c["channels"]), dtype=torch.float64, device="cuda")
        if s["initial"] is not None:
            old += s["initial"][i].double()
        rows = torch.cat([old, s["x"][a:a + n].double()])
        v = s["bias"].double()[None].expand(n, -1).clone()
        for j in range(W):
            v += s["weight"][:, j].double() * rows[j:j + n]
        yield i, a, n, rows, v


def _exact_conv_fwd(s, c):
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    final = torch.zeros(s["final"].shape, dtype=torch.float64, device="cuda")
    for i, a, n, rows, v in _conv_parts(s, c):
        y[a:a + n] = v * torch.sigmoid(v)
        final[i] = rows[n:]
    return y, final


def _exact_conv_bwd(s, c):
    W, C = c["width"], c["channels"]
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dw, db = torch.zeros((C, W), dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    di = torch.zeros((len(s["lens"]), W - 1, C), dtype=torch.float64, device="cuda")
    for i, a, n, rows, v in _conv_parts(s, c):
        sg = torch.sigmoid(v)
        dv = s["dy"][a:a + n].double() * sg * (1.0 + v * (1.0 - sg))
        db += dv.sum(0)
        dr = torch.zeros_like(rows)
        for j in range(W):
            dw[:, j] += (dv * rows[j:j + n]).sum(0)
            dr[j:j + n] += dv * s["weight"][:, j].double()
        dx[a:a + n], di[i] = dr[W - 1:], dr[:W - 1]
    out = dict(dx=dx, dweight=dw, dbias=db)
    if s["initial"] is not None:
        out["dinitial_state"] = di
    return out


def _exact_norm_fwd(s, c):
    x, w, z, res = _f64(s, "x", "weight", "z", "residual")
    out, h = {}, x
    if res is not None:
        out["residual"] = h + res
        h = out["residual"].to(s["residual"].dtype).double()   # the norm reads the residual as stored
    u = h if z is None else h * z * torch.sigmoid(z)
    y = torch.empty_like(u)
    for k in range(0, c["dim"], c["group"]):
        part = u[:, k:k + c["group"]]
        y[:, k:k + c["group"]] = part / torch.sqrt(part.square().mean(1, keepdim=True) + EPS)
    y = y * w
    if c["out"] != "fp8":
        out["out"] = y
        return out
    b = 128 if c["scales"] == "block" else c["dim"]
    top = torch.stack([y[:, k:k + b].abs().amax(1) for k in range(0, c["dim"], b)], 1)
    out["scale"] = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    out["out"] = y / out["scale"].repeat_interleave(b, 1)
    return out


def _exact_norm_bwd(s, c):
    x, w, z, dy = _f64(s, "x", "weight", "z", "dy")
    sg = None if z is None else torch.sigmoid(z)
    u = x if z is None else x * z * sg
    du, dw = torch.empty_like(u), torch.empty_like(w)
    for k in range(0, c["dim"], c["group"]):
        p, o, q = u[:, k:k + c["group"]], dy[:, k:k + c["group"]], w[k:k + c["group"]]
        r = 1.0 / torch.sqrt(p.square().mean(1, keepdim=True) + EPS)
        dw[k:k + c["group"]] = (o * p * r).sum(0)
        t = o * q
        du[:, k:k + c["group"]] = r * (t - p * r * r * (t * p).mean(1, keepdim=True))
    out = dict(dx=du if z is None else du * z * sg, dweight=dw)
    if z is not None:
        out["dz"] = du * x * sg * (1.0 + z * (1.0 - sg))
    return out


_EXACT = dict(scan_fwd=_exact_scan_fwd, scan_bwd=_exact_scan_bwd, conv_step=_exact_conv_step,
              conv_fwd=_exact_conv_fwd, conv_bwd=_exact_conv_bwd, norm_fwd=_exact_norm_fwd,
              norm_bwd=_exact_norm_bwd)
