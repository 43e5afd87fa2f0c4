"""The example layer trained from states that are not zero: its gradients against
automatic differentiation in 64 bits of the layer written token by token."""

import pytest
import torch

from test_gpu_layer import example  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def _silu(v):
    return v * torch.sigmoid(v)


def _norm(v, w, group):
    u = v.unflatten(1, (-1, group))
    return (u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-5)).flatten(1) * w


def _plain(layer, p, x, res, lens, conv, scan):
    """conv [n, W-1, channels] and scan [n, H, P, N]: each sequence's first states."""
    row = _norm(x + res, p["norm"], x.shape[1]) @ p["w_in"].t()
    z, xbc, dt = layer._split(row)
    dt = torch.nn.functional.softplus(dt + p["dt_bias"])
    out, a = [], 0
    head = torch.arange(layer.H) // (layer.H // layer.G)
    for i, n in enumerate(lens):
        rows = torch.cat([conv[i], xbc[a:a + n]])
        act = _silu(sum(p["conv"][:, j] * rows[j:j + n] for j in range(layer.W)) + p["conv_bias"])
        xs, B, C = layer._heads(act)
        S = scan[i]
        for t in range(n):
            d = dt[a + t]
            S = torch.exp(d * p["A"])[:, None, None] * S \
                + (d[:, None] * xs[t])[:, :, None] * B[t][head][:, None, :]
            out.append(((S * C[t][head][:, None, :]).sum(-1) + p["D"][:, None] * xs[t]).flatten())
        a += n
    y = torch.stack(out) * _silu(z)
    return _norm(y, p["gate_norm"], layer.group) @ p["w_out"].t()


@pytest.mark.parametrize("which", ["all", "some", "by sequence"])
def test_gradients_from_states(example, which):  # noqa: F811
    """fp32; the tolerance is that of the same layer from zero states: seven steps of
    2^-16 of what each adds up, 1.1e-4 of a gradient's norm."""
    lens, n = [70, 1, 9], 3
    layer = example.Mamba2Layer(width=32, nheads=4, headdim=32, dstate=16, dtype=torch.float32)
    g = torch.Generator().manual_seed(4)
    x, res, dout = (torch.randn(sum(lens), 32, generator=g) for _ in range(3))
    pools = layer.pools(n if which == "by sequence" else 5)
    for q in pools:
        q.copy_(torch.randn(q.shape, generator=g))
    slots = None if which == "by sequence" else torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    has = torch.tensor([1, 1, 0], dtype=torch.uint8, device="cuda") if which == "some" else None
    at = torch.arange(n) if slots is None else slots.cpu().long()
    keeps = torch.ones(n) if has is None else has.cpu().float()
    conv, scan = (q.double().cpu()[at] * keeps.double().view(-1, *[1] * (q.dim() - 1)) for q in pools)
    cu = torch.tensor([0, 70, 71, 80], dtype=torch.int32, device="cuda")
    out, _, keep = layer.prefill(x.cuda(), res.cuda(), cu, pools, slots, has, train=True)
    got, dx = layer.backward(dout.cuda(), torch.zeros(80, 32, device="cuda"), keep)
    p = {k: v.double().cpu().requires_grad_() for k, v in layer.p.items()}
    xd = x.double().requires_grad_()
    want = _plain(layer, p, xd, res.double(), lens, conv, scan)
    want.backward(dout.double())

    def near(a, b, name):
        off = (a.double().cpu() - b).norm() / b.norm()
        assert off < 1.1e-4, f"{name}: {off:.3g}"
    near(out, want.detach(), "out")
    near(dx, xd.grad, "dx")
    for k in p:
        near(got[k], p[k].grad, k)


def test_backward_without_the_states_is_refused(example):  # noqa: F811
    layer = example.Mamba2Layer(width=32, nheads=2, headdim=32, dstate=16, dtype=torch.float32)
    x = torch.randn(6, 32, device="cuda")
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    _, _, keep = layer.prefill(x, x, cu, layer.pools(1))
    with pytest.raises(ValueError, match="train=True"):
        layer.backward(x, x, keep)
