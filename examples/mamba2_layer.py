"""A Mamba2 layer on the library's operators: packed prefill, decode, training.

    python examples/mamba2_layer.py

builds one layer with random weights, prefills a packed batch of uneven prompts
(norm with residual, projection, convolution, scan, gated norm, projection),
decodes a few tokens from the states that the prefill left in the pools, and
takes training steps on a regression target.  Only the two projections are
library matrix products.
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_amd as R  # noqa: E402


class Mamba2Layer:
    def __init__(self, width=128, nheads=8, headdim=64, dstate=128, ngroups=2, conv=4,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.P, self.N, self.G, self.W = nheads, headdim, dstate, ngroups, conv
        self.inner, self.bc = nheads * headdim, ngroups * dstate
        self.chan = self.inner + 2 * self.bc                  # x, B and C go through the convolution
        self.group = self.inner // ngroups                    # the gated norm's group
        self.dtype = dtype

        def rnd(*shape, scale=1.0, dt=torch.float32):
            return (torch.randn(*shape, generator=g) * scale).to(dt).to(device)
        proj = 2 * self.inner + 2 * self.bc + nheads
        bias = torch.rand(nheads, generator=g) * 0.099 + 0.001
        self.p = dict(
            norm=torch.ones(width, device=device),
            w_in=rnd(proj, width, scale=width ** -0.5, dt=dtype),
            conv=rnd(self.chan, conv, scale=0.5), conv_bias=rnd(self.chan, scale=0.1),
            A=-torch.exp(torch.rand(nheads, generator=g) * math.log(16.0)).to(device),
            D=rnd(nheads), dt_bias=torch.log(torch.expm1(bias)).to(device),
            gate_norm=torch.ones(self.inner, device=device),
            w_out=rnd(width, self.inner, scale=self.inner ** -0.5, dt=dtype))

    def pools(self, slots):
        """(convolution states, scan states) for this many requests."""
        dev = self.p["w_in"].device
        return (torch.zeros(slots, self.W - 1, self.chan, dtype=self.dtype, device=dev),
                torch.zeros(slots, self.H, self.P, self.N, dtype=torch.float32, device=dev))

    def _split(self, row):
        """z, the convolution's channels and dt as slices of the projection's rows."""
        return row[:, :self.inner], row[:, self.inner:self.inner + self.chan], row[:, self.inner + self.chan:]

    def _heads(self, xbc):
        at = self.inner
        return (xbc[:, :at].unflatten(1, (self.H, self.P)),
                xbc[:, at:at + self.bc].unflatten(1, (self.G, self.N)),
                xbc[:, at + self.bc:].unflatten(1, (self.G, self.N)))

    def prefill(self, x, residual, cu_seqlens, pools=None, slots=None, has_initial=None, train=False):
        """x [tokens, width] and the fp32 residual stream -> (the layer's output,
        the new residual stream, what the backward pass needs).  The sequences'
        states continue from and go back to their slots of `pools`; those with
        has_initial[i] = 0 start from zeros.  With pools, a backward pass needs
        train=True, which copies the states that this call replaces."""
        p = self.p
        conv_pool, scan_pool = pools or (None, None)
        first = {}
        if pools and train:
            at = slots.long() if slots is not None else torch.arange(len(cu_seqlens) - 1, device=x.device)
            first = dict(conv=conv_pool[at], scan=scan_pool[at])
        n1 = R.rms_norm_forward(x, p["norm"], residual=residual)
        row = n1["out"] @ p["w_in"].t()
        z, xbc, dt = self._split(row)
        act = R.causal_conv_forward(xbc, p["conv"], bias=p["conv_bias"], cu_seqlens=cu_seqlens,
                                    initial_state=conv_pool, has_initial=has_initial, slot_idx=slots,
                                    final_state=conv_pool)
        xs, B, C = self._heads(act)
        y = R.ssu_scan_forward(xs, dt, p["A"], B, C, D=p["D"], dt_bias=p["dt_bias"],
                               cu_seqlens=cu_seqlens, initial_state=scan_pool, has_initial=has_initial,
                               final_state=scan_pool, slot_idx=slots).flatten(1)
        n2 = R.rms_norm_forward(y, p["gate_norm"], z=z, group_size=self.group)["out"]
        keep = dict(h=n1["residual"], n1=n1["out"], row=row, act=act, y=y, n2=n2, cu=cu_seqlens,
                    first=first, has=has_initial if first else None, whole=not pools or train)
        return n2 @ p["w_out"].t(), n1["residual"], keep

    def decode(self, x, residual, pools, slots):
        """One token of every request, its states updated in place."""
        p = self.p
        n1 = R.rms_norm_forward(x, p["norm"], residual=residual)
        z, xbc, dt = self._split(n1["out"] @ p["w_in"].t())
        act = R.causal_conv_decode(xbc, pools[0], p["conv"], bias=p["conv_bias"], slot_idx=slots)
        xs, B, C = (t.contiguous() for t in self._heads(act))
        y = R.ssu_standard_decode(pools[1], slots, xs, dt.contiguous(), p["A"], B, C, D=p["D"],
                                  dt_bias=p["dt_bias"])
        n2 = R.rms_norm_forward(y.flatten(1).to(self.dtype), p["gate_norm"], z=z,
                                group_size=self.group)["out"]
        return n2 @ p["w_out"].t(), n1["residual"]

    def backward(self, dout, dresidual, k):
        """Gradients of the parameters, and of x (the residual's is the same)."""
        if not k["whole"]:
            raise ValueError("the initial states were replaced: prefill with train=True")
        p = self.p
        first = k["first"]  # by sequence, not by slot
        z, xbc, dt = self._split(k["row"])
        xs, B, C = self._heads(k["act"])
        g = dict(w_out=dout.t() @ k["n2"])
        n2 = R.rms_norm_backward(dout @ p["w_out"], k["y"], p["gate_norm"], z=z, group_size=self.group)
        s = R.ssu_scan_backward(n2["dx"].unflatten(1, (self.H, self.P)), xs, dt, p["A"], B, C, D=p["D"],
                                dt_bias=p["dt_bias"], cu_seqlens=k["cu"],
                                initial_state=first.get("scan"), has_initial=k["has"])
        dact = torch.cat([s["dx"].flatten(1), s["dB"].flatten(1), s["dC"].flatten(1)], 1)
        c = R.causal_conv_backward(dact, xbc, p["conv"], bias=p["conv_bias"], cu_seqlens=k["cu"],
                                   initial_state=first.get("conv"), has_initial=k["has"])
        drow = torch.cat([n2["dz"], c["dx"], s["ddt"]], 1)
        # the first norm read the fp32 residual stream
        n1 = R.rms_norm_backward((drow @ p["w_in"]).float(), k["h"], p["norm"])
        g.update(gate_norm=n2["dweight"], A=s["dA"], D=s["dD"], dt_bias=s["ddt_bias"],
                 conv=c["dweight"], conv_bias=c["dbias"], w_in=drow.t() @ k["n1"], norm=n1["dweight"])
        return g, n1["dx"] + dresidual


def main():
    dev = torch.device("cuda")
    layer = Mamba2Layer()
    gen = torch.Generator().manual_seed(1)
    lens = [300, 1, 77, 512]
    T, width = sum(lens) + len(lens) * 4, 128
    cu = lambda n: torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device=dev)  # noqa: E731
    x = torch.randn(T, width, generator=gen).to(torch.bfloat16).to(dev)
    res = torch.randn(T, width, generator=gen).to(dev)
    # the whole sequences at once, against prompts and then token by token
    full = [n + 4 for n in lens]
    want, _, _ = layer.prefill(x, res, cu(full))
    at = [sum(full[:i]) for i in range(len(lens))]
    prompt = torch.cat([torch.arange(a, a + n) for a, n in zip(at, lens)]).to(dev)
    pools, slots = layer.pools(6), torch.tensor([4, 0, 5, 2], dtype=torch.int32, device=dev)
    none = torch.zeros(len(lens), dtype=torch.uint8, device=dev)
    layer.prefill(x[prompt], res[prompt], cu(lens), pools, slots, none)
    worst = 0.0
    for t in range(4):
        rows = torch.tensor([a + n + t for a, n in zip(at, lens)], device=dev)
        got, _ = layer.decode(x[rows], res[rows], pools, slots)
        worst = max(worst, float((got - want[rows]).float().norm() / want[rows].float().norm()))
    print(f"prefill, then 4 decode steps against the whole: relative difference {worst:.4f}")
    target = torch.randn(T, width, generator=gen).to(dev)
    zero = torch.zeros_like(res)
    first = None
    for step in range(20):
        out, h, keep = layer.prefill(x, res, cu(full))
        err = out.float() - target
        loss = float(err.square().mean())
        first = loss if first is None else first
        grads, _ = layer.backward((2.0 / err.numel() * err).to(torch.bfloat16), zero, keep)
        for k, g in grads.items():
            layer.p[k] = (layer.p[k].float() - 4.0 * g.float()).to(layer.p[k].dtype)
    print(f"training: loss {first:.4f} -> {loss:.4f} in 20 steps")
    return worst, first, loss


if __name__ == "__main__":
    main()
