"""Linear-attention layers on the library's operators: packed prefill, decode, training.

    python examples/linear_attention_layer.py

builds one layer of each kind with random weights: "linear" turns queries and
keys by their positions and runs linear attention with a constant decay per
head; "delta" convolves queries, keys and values, brings queries and keys to unit
length and runs the gated delta rule, its gates from the input.  Each prefills a
packed batch of uneven prompts, decodes a few tokens from the states that the
prefill left in the pools, and takes a training step.  Only the projections are
library matrix products; the gates, one number per head, are torch expressions.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_amd as R  # noqa: E402


class LinearAttentionLayer:
    def __init__(self, kind="linear", width=128, k_heads=2, v_heads=4, dim=64, conv=4,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        if kind not in ("linear", "delta"):
            raise ValueError("kind must be 'linear' or 'delta'")
        g = torch.Generator().manual_seed(seed)
        self.delta = kind == "delta"
        self.HK, self.HV, self.K, self.W = k_heads, v_heads, dim, conv
        self.qk, self.inner = 2 * k_heads * dim, v_heads * dim
        self.chan = self.qk + self.inner                     # q, k and v
        self.dtype = dtype

        def rnd(*shape, scale=1.0, dt=torch.float32):
            return (torch.randn(*shape, generator=g) * scale).to(dt).to(device)
        proj = self.chan + self.inner + (2 * v_heads if self.delta else 0)
        self.p = dict(
            norm=torch.ones(width, device=device), w_in=rnd(proj, width, scale=width ** -0.5, dt=dtype),
            gate_norm=torch.ones(self.inner, device=device),
            w_out=rnd(width, self.inner, scale=self.inner ** -0.5, dt=dtype))
        if self.delta:
            self.p.update(conv=rnd(self.chan, conv, scale=0.5), A=torch.rand(v_heads, generator=g).to(device) + 0.2,
                          bias=rnd(v_heads))
            # a norm over each head with this weight leaves rows of length one
            self.unit = torch.full((self.qk,), dim ** -0.5, device=device)
        else:
            at = torch.arange(v_heads, dtype=torch.float32)
            self.p["log_decay"] = torch.log1p(-torch.exp2(-3.0 - 5.0 * at / v_heads)).to(device)
            self.freqs, self.amplitude = R.rotary_frequencies(dim // 2, device=device)

    def pools(self, slots):
        """(convolution states or None, recurrent states) for this many requests."""
        dev = self.p["w_in"].device
        conv = torch.zeros(slots, self.W - 1, self.chan, dtype=self.dtype, device=dev) if self.delta else None
        return conv, torch.zeros(slots, self.HV, self.K, self.K, dtype=torch.float32, device=dev)

    def _split(self, row):
        """q, k and v together, the output's gate, and the gates' inputs (delta)."""
        return row[:, :self.chan], row[:, self.chan:self.chan + self.inner], row[:, self.chan + self.inner:]

    def _values(self, qkv):
        return qkv[:, self.qk:].unflatten(1, (self.HV, self.K))

    def _pair(self, qk):
        return (qk[:, :self.qk // 2].unflatten(1, (self.HK, self.K)),
                qk[:, self.qk // 2:self.qk].unflatten(1, (self.HK, self.K)))

    def _gates(self, ab):
        a, b = ab.float().chunk(2, 1)
        log_g = -self.p["A"] * torch.nn.functional.softplus(a + self.p["bias"])
        return log_g, torch.sigmoid(b).contiguous()

    def _turned(self, qkv, positions):
        return R.rotary_forward(qkv[:, :self.qk].unflatten(1, (2 * self.HK, self.K)), positions, self.freqs,
                                amplitude=self.amplitude).flatten(1)

    def _unit(self, act):
        return R.rms_norm_forward(act[:, :self.qk], self.unit, group_size=self.K, eps=1e-6 / self.K)["out"]

    def prefill(self, x, residual, positions, cu_seqlens, pools=None, slots=None, has_initial=None):
        """x [tokens, width], the fp32 residual stream and the tokens' positions ->
        (the layer's output, the new residual stream, what the backward pass
        needs, which takes sequences that begin here).  The states continue
        from and go back to their slots of `pools`."""
        p = self.p
        conv_pool, pool = pools or (None, None)
        state = dict(cu_seqlens=cu_seqlens, initial_state=pool, has_initial=has_initial, slot_idx=slots,
                     final_state=pool)
        n1 = R.rms_norm_forward(x, p["norm"], residual=residual)
        row = n1["out"] @ p["w_in"].t()
        qkv, z, ab = self._split(row)
        keep = dict(h=n1["residual"], n1=n1["out"], row=row, pos=positions, cu=cu_seqlens, whole=not pools)
        if self.delta:
            act = R.causal_conv_forward(qkv, p["conv"], **{**state, "initial_state": conv_pool,
                                                           "final_state": conv_pool})
            qk, (log_g, beta) = self._unit(act), self._gates(ab)
            y = R.gdn_scan_forward(*self._pair(qk), self._values(act), log_g, beta, **state)
            keep.update(act=act, log_g=log_g, beta=beta)
        else:
            qk = self._turned(qkv, positions)
            y = R.linear_attention_forward(*self._pair(qk), self._values(qkv), p["log_decay"], **state)
        y = y.flatten(1)
        n2 = R.rms_norm_forward(y, p["gate_norm"], z=z, group_size=self.K)["out"]
        keep.update(qk=qk, y=y, n2=n2)
        return n2 @ p["w_out"].t(), n1["residual"], keep

    def decode(self, x, residual, positions, pools, slots):
        """One token of every request, its states updated in place."""
        p = self.p
        n1 = R.rms_norm_forward(x, p["norm"], residual=residual)
        qkv, z, ab = self._split(n1["out"] @ p["w_in"].t())
        if self.delta:
            act = R.causal_conv_decode(qkv, pools[0], p["conv"], slot_idx=slots)
            log_g, beta = self._gates(ab)
            q, k = (t.contiguous() for t in self._pair(self._unit(act)))
            y = R.gdn_standard_decode(pools[1], slots, q, k, self._values(act).contiguous(), log_g.exp(), beta,
                                      out_dtype=self.dtype)
        else:
            y = R.linear_attention_decode(pools[1], slots, *self._pair(self._turned(qkv, positions)),
                                          self._values(qkv), p["log_decay"])
        n2 = R.rms_norm_forward(y.flatten(1), p["gate_norm"], z=z, group_size=self.K)["out"]
        return n2 @ p["w_out"].t(), n1["residual"]

    def backward(self, dout, dresidual, k):
        """Gradients of the parameters, and of x (the residual's is the same)."""
        if not k["whole"]:
            raise ValueError("this prefill continued sequences: the backward pass takes whole ones")
        p = self.p
        qkv, z, ab = self._split(k["row"])
        g = dict(w_out=dout.t() @ k["n2"])
        n2 = R.rms_norm_backward(dout @ p["w_out"], k["y"], p["gate_norm"], z=z, group_size=self.K)
        dy = n2["dx"].unflatten(1, (self.HV, self.K))
        if self.delta:
            s = R.gdn_scan_backward(dy, *self._pair(k["qk"]), self._values(k["act"]), k["log_g"], k["beta"],
                                    cu_seqlens=k["cu"])
            dqk = torch.cat([s["dq"].flatten(1), s["dk"].flatten(1)], 1)
            unit = R.rms_norm_backward(dqk, k["act"][:, :self.qk], self.unit, group_size=self.K, eps=1e-6 / self.K)
            c = R.causal_conv_backward(torch.cat([unit["dx"], s["dv"].flatten(1)], 1), qkv, p["conv"],
                                       cu_seqlens=k["cu"])
            a = ab[:, :self.HV].float() + p["bias"]
            da = -s["dlog_g"] * p["A"] * torch.sigmoid(a)
            db = s["dbeta"] * k["beta"] * (1 - k["beta"])
            g.update(conv=c["dweight"], bias=da.sum(0),
                     A=-(s["dlog_g"] * torch.nn.functional.softplus(a)).sum(0))
            drow = torch.cat([c["dx"], n2["dz"], da.to(self.dtype), db.to(self.dtype)], 1)
        else:
            s = R.linear_attention_backward(dy, *self._pair(k["qk"]), self._values(qkv), p["log_decay"],
                                            cu_seqlens=k["cu"])
            dqk = torch.cat([s["dq"], s["dk"]], 1)
            R.rotary_backward(dqk, k["pos"], self.freqs, amplitude=self.amplitude, out=dqk)
            g["log_decay"] = s["dlog_decay"]
            drow = torch.cat([dqk.flatten(1), s["dv"].flatten(1), n2["dz"]], 1)
        # the first norm read the fp32 residual stream
        n1 = R.rms_norm_backward((drow @ p["w_in"]).float(), k["h"], p["norm"])
        g.update(gate_norm=n2["dweight"], w_in=drow.t() @ k["n1"], norm=n1["dweight"])
        return g, n1["dx"] + dresidual


def main():
    dev = torch.device("cuda")
    gen = torch.Generator().manual_seed(1)
    lens, steps, width = [300, 1, 77, 1500], 4, 128
    full = [n + steps for n in lens]
    T = sum(full)
    cu = lambda n: torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device=dev)  # noqa: E731
    x = torch.randn(T, width, generator=gen).to(torch.bfloat16).to(dev)
    res, dout = torch.randn(T, width, generator=gen).to(dev), torch.randn(T, width, generator=gen).to(dev)
    pos = torch.cat([torch.arange(n) for n in full]).to(torch.int32).to(dev)
    at = [sum(full[:i]) for i in range(len(lens))]
    prompt = torch.cat([torch.arange(a, a + n) for a, n in zip(at, lens)]).to(dev)
    slots = torch.tensor([4, 0, 5, 2], dtype=torch.int32, device=dev)
    none = torch.zeros(len(lens), dtype=torch.uint8, device=dev)
    found = {}
    for kind in ("linear", "delta"):
        # the whole sequences at once, against prompts and then token by token
        layer = LinearAttentionLayer(kind)
        want, _, keep = layer.prefill(x, res, pos, cu(full))
        pools = layer.pools(6)
        layer.prefill(x[prompt], res[prompt], pos[prompt], cu(lens), pools, slots, none)
        worst = 0.0
        for t in range(steps):
            rows = torch.tensor([a + n + t for a, n in zip(at, lens)], device=dev)
            got, _ = layer.decode(x[rows], res[rows], pos[rows], pools, slots)
            worst = max(worst, float((got - want[rows]).float().norm() / want[rows].float().norm()))
        grads, _ = layer.backward((dout / T).to(torch.bfloat16), torch.zeros_like(res), keep)
        for k, g in grads.items():
            layer.p[k] = (layer.p[k].float() - 0.1 * g.float()).to(layer.p[k].dtype)
        found[kind] = worst, {k: float(g.float().norm()) for k, g in grads.items()}
        print(f"{kind}: prefill, then {steps} decode steps against the whole: relative difference {worst:.4f}; "
              f"{len(grads)} gradients")
    return found


if __name__ == "__main__":
    main()
