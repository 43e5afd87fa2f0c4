"""The example layer: its operators together, prefill against decode and the
gradients of a whole layer against automatic differentiation in 64 bits."""

import importlib.util
import os

import pytest
import torch

import linear_recurrence_amd as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    R.load()
    spec = importlib.util.spec_from_file_location(
        "mamba2_layer", os.path.join(ROOT, "examples", "mamba2_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(layer, p, x, res, lens):
    """The layer token by token, in whatever precision the tensors have."""
    def silu(v):
        return v * torch.sigmoid(v)

    def norm(v, w, group):
        u = v.unflatten(1, (-1, group))
        return (u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-5)).flatten(1) * w
    row = norm(x + res, p["norm"], x.shape[1]) @ p["w_in"].t()
    z, xbc, dt = layer._split(row)
    dt = torch.nn.functional.softplus(dt + p["dt_bias"])
    out, a = [], 0
    head = torch.arange(layer.H) // (layer.H // layer.G)
    for n in lens:
        rows = torch.cat([torch.zeros(layer.W - 1, layer.chan, dtype=x.dtype), xbc[a:a + n]])
        act = silu(sum(p["conv"][:, j] * rows[j:j + n] for j in range(layer.W)) + p["conv_bias"])
        xs, B, C = layer._heads(act)
        S = torch.zeros(layer.H, layer.P, layer.N, dtype=x.dtype)
        for t in range(n):
            d = dt[a + t]
            S = torch.exp(d * p["A"])[:, None, None] * S \
                + (d[:, None] * xs[t])[:, :, None] * B[t][head][:, None, :]
            out.append(((S * C[t][head][:, None, :]).sum(-1) + p["D"][:, None] * xs[t]).flatten())
        a += n
    y = torch.stack(out) * silu(z)
    return norm(y, p["gate_norm"], layer.group) @ p["w_out"].t()


def test_layer_gradients(example):
    """fp32, so that only the operators' own rounding counts: each of the seven
    steps between output and gradient is off by at most 2^-16 of what it adds
    up (tests of the operators), and 2^-16 * 7 is 1.1e-4 of a gradient's norm."""
    lens = [70, 1, 9]
    layer = example.Mamba2Layer(width=32, nheads=4, headdim=32, dstate=16, dtype=torch.float32)
    g = torch.Generator().manual_seed(3)
    x, res, dout = (torch.randn(sum(lens), 32, generator=g) for _ in range(3))
    cu = torch.tensor([0, 70, 71, 80], dtype=torch.int32, device="cuda")
    out, _, keep = layer.prefill(x.cuda(), res.cuda(), cu)
    got, dx = layer.backward(dout.cuda(), torch.zeros(80, 32, device="cuda"), keep)
    p = {k: v.double().cpu().requires_grad_() for k, v in layer.p.items()}
    xd = x.double().requires_grad_()
    want = _plain(layer, p, xd, res.double(), lens)
    want.backward(dout.double())

    def near(a, b, name):
        off = (a.double().cpu() - b).norm() / b.norm()
        assert off < 1.1e-4, f"{name}: {off:.3g}"
    near(out, want.detach(), "out")
    near(dx, xd.grad, "dx")
    for k in p:
        near(got[k], p[k].grad, k)


def test_layer_prefill_then_decode_and_training(example):
    """bf16: between the two paths every intermediate tensor (six of them) may
    round the other way, by at most 2^-8 each."""
    worst, first, last = example.main()
    assert worst < 6 * 2.0 ** -8
    assert last < first
