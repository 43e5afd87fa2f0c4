"""The example of linear-attention layers: the operators together, prefill against
decode, and the gradients of a whole layer against automatic differentiation in 64
bits and against differences."""

import importlib.util
import math
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
        "linear_attention_layer", os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(layer, p, x, res, pos, lens):
    """The layer token by token, in whatever precision the tensors have."""
    def norm(v, w, group, eps=1e-5):
        u = v.unflatten(1, (-1, group))
        return (u * torch.rsqrt(u.square().mean(-1, keepdim=True) + eps)).flatten(1) * w
    silu = torch.nn.functional.silu
    row = norm(x + res, p["norm"], x.shape[1]) @ p["w_in"].t()
    qkv, z, ab = layer._split(row)
    head = torch.arange(layer.HV) // (layer.HV // layer.HK)
    if layer.delta:
        a, b = ab.chunk(2, 1)
        decay = torch.exp(-p["A"] * torch.nn.functional.softplus(a + p["bias"]))
        beta = torch.sigmoid(b)
        parts, at = [], 0
        for n in lens:
            rows = torch.cat([torch.zeros(layer.W - 1, layer.chan, dtype=x.dtype), qkv[at:at + n]])
            parts.append(silu(sum(p["conv"][:, j] * rows[j:j + n] for j in range(layer.W))))
            at += n
        qkv = torch.cat(parts)
        qk = norm(qkv[:, :layer.qk], layer.K ** -0.5, layer.K, 1e-6 / layer.K)
    else:
        half = layer.freqs.shape[0]
        u = qkv[:, :layer.qk].unflatten(1, (2 * layer.HK, layer.K))
        turn = (pos.double()[:, None] * layer.freqs.double().cpu())[:, None, :]
        lo, hi = u[..., :half], u[..., half:2 * half]
        qk = torch.cat([lo * turn.cos() - hi * turn.sin(), hi * turn.cos() + lo * turn.sin(),
                        u[..., 2 * half:]], -1).flatten(1)
        decay, beta = torch.exp(p["log_decay"]).expand(len(x), -1), None
    q, k = (t[:, head] for t in layer._pair(qk))
    v = layer._values(qkv)
    out, at = [], 0
    for n in lens:
        S = torch.zeros(layer.HV, layer.K, layer.K, dtype=x.dtype)
        for t in range(at, at + n):
            S = decay[t][:, None, None] * S
            d = v[t] if beta is None else beta[t][:, None] * (v[t] - (S * k[t][:, None, :]).sum(-1))
            S = S + d[:, :, None] * k[t][:, None, :]
            out.append(((S * q[t][:, None, :]).sum(-1) / math.sqrt(layer.K)).flatten())
        at += n
    y = torch.stack(out) * silu(z)
    return norm(y, p["gate_norm"], layer.K) @ p["w_out"].t()


def _case(example, kind):
    lens = [70, 1, 9]
    layer = example.LinearAttentionLayer(kind, width=32, dtype=torch.float32)
    g = torch.Generator().manual_seed(3)
    x, res, dout = (torch.randn(sum(lens), 32, generator=g) for _ in range(3))
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    cu = torch.tensor([0, 70, 71, 80], dtype=torch.int32, device="cuda")
    return layer, lens, x, res, dout, pos, cu


@pytest.mark.parametrize("kind", ["linear", "delta"])
def test_layer_gradients(example, kind):
    """fp32, so that only the operators' own rounding counts: each of the nine
    steps between output and gradient is off by at most 2^-16 of what it adds up
    (tests of the operators), and 2^-16 * 9 is 1.4e-4 of a gradient's norm."""
    layer, lens, x, res, dout, pos, cu = _case(example, kind)
    out, _, keep = layer.prefill(x.cuda(), res.cuda(), pos.cuda(), cu)
    got, dx = layer.backward(dout.cuda(), torch.zeros(80, 32, device="cuda"), keep)
    p = {k: v.double().cpu().requires_grad_() for k, v in layer.p.items()}
    xd = x.double().requires_grad_()
    want = _plain(layer, p, xd, res.double(), pos, lens)
    want.backward(dout.double())

    def near(a, b, name):
        off = (a.double().cpu() - b).norm() / b.norm()
        assert off < 1.4e-4, f"{name}: {off:.3g}"
    near(out, want.detach(), "out")
    near(dx, xd.grad, "dx")
    assert set(got) == set(p)
    for k in p:
        near(got[k], p[k].grad, k)


@pytest.mark.parametrize("kind", ["linear", "delta"])
def test_layer_differences(example, kind):
    """Along a direction over all parameters the output moves as the gradients
    say.  With steps of +-h the difference of sum(out * dout) is off by the
    outputs' rounding, 2 * 9 * 2^-24 * |out| |dout| / (2h) at most if every step's
    error agrees, and by h^2 / 6 of the third derivative."""
    layer, lens, x, res, dout, pos, cu = _case(example, kind)
    x, res, pos, dout = x.cuda(), res.cuda(), pos.cuda(), dout.cuda()
    out, _, keep = layer.prefill(x, res, pos, cu)
    grads, _ = layer.backward(dout, torch.zeros_like(res), keep)
    gen = torch.Generator().manual_seed(4)
    way = {k: torch.randn(v.shape, generator=gen).cuda() * v.abs().mean() for k, v in layer.p.items()}
    want = sum(float((way[k].double() * grads[k].double()).sum()) for k in way)
    start = dict(layer.p)

    def at(h):
        layer.p = {k: v + h * way[k] for k, v in start.items()}
        return float((layer.prefill(x, res, pos, cu)[0].double() * dout.double()).sum())
    h = 2.0 ** -8
    one, two = (at(h) - at(-h)) / (2 * h), (at(2 * h) - at(-2 * h)) / (4 * h)
    layer.p = start
    # the two steps' difference is 3 h^2 / 6 of the third derivative: one's own part is a third of it
    bound = 2 * 9 * 2.0 ** -24 * float(out.norm() * dout.norm()) / (2 * h) + abs(two - one)
    assert abs(one - want) < bound, (one, want, bound)


def test_layer_prefill_then_decode_and_training(example):
    """bf16: between the two paths every intermediate tensor (seven of them) may
    round the other way, by at most 2^-8 each."""
    for kind, (worst, norms) in example.main().items():
        assert worst < 7 * 2.0 ** -8, (kind, worst)
        assert all(math.isfinite(n) and n > 0 for n in norms.values()), (kind, norms)
