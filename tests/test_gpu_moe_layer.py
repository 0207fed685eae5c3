"""The mixture-of-experts example: its gradients against a binary64 autograd
of the same layer without any rounding, for the same choice of experts.

Tolerance.  An e4m3 code is within 2^-4 of its value.  Between the layer's
input and a gradient lie at most eight such roundings (operands of the two
GEMMs forward and of the two backward); they are independent of each other, so
they meet as a root of squares: sqrt(8) 2^-4 = 0.18 of a gradient's norm, to
which bf16 (2^-8 each) adds little: 0.2."""
import importlib.util
import os

import pytest
import torch

import fp8_precision_quantization_amd as mx
from tests.gpu_util import device

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer_step.py")
    spec = importlib.util.spec_from_file_location("moe_layer_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(params, x, chosen, topk, aux):
    """(out, loss) in binary64 with the given choice."""
    y = torch.nn.functional.layer_norm(x, x.shape[1:], params["norm_w"], params["norm_b"], 1e-5)
    probs = torch.softmax(y @ params["router"].T, 1)
    e = probs.shape[1]
    gates = probs.gather(1, chosen)
    gates = gates / gates.sum(1, keepdim=True)
    out = x
    for i in range(e):
        h = y @ params["w1"][i].T
        g, u = h.chunk(2, 1)
        share = (gates * (chosen == i)).sum(1, keepdim=True)
        out = out + share * ((torch.nn.functional.silu(g) * u) @ params["w2"][i].T)
    counts = torch.bincount(chosen.reshape(-1), minlength=e).double()
    loss = e / (topk * x.shape[0] ** 2) * (counts * probs.sum(0)).sum()
    return out, aux * loss


@pytest.mark.parametrize("tokens,model,hidden,experts,topk", [(96, 128, 64, 4, 2), (333, 256, 192, 8, 3), (1, 128, 64, 2, 1)])
def test_gradients(tokens, model, hidden, experts, topk):
    dev = device()
    layer = _example().MoELayer(model, hidden, experts, topk, dev, seed=tokens, aux=0.5)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(tokens, model, generator=g).bfloat16()
    dout = torch.randn(tokens, model, generator=g)
    out, loss, kept = layer.forward(x.to(dev))
    dx, grads = layer.backward(dout.to(dev), kept)
    again_dx, again = layer.backward(dout.to(dev), kept)
    assert torch.equal(dx, again_dx) and all(torch.equal(grads[k], again[k]) for k in grads)

    params = {k: v.double().cpu().requires_grad_() for k, v in layer.params.items()}
    xr = x.double().requires_grad_()
    want, want_loss = _plain(params, xr, kept["chosen"].long().cpu(), topk, 0.5)
    ((want * dout.double()).sum() + want_loss).backward()

    def near(got, ref, name):
        ref = ref.detach()
        off = (got.double().cpu() - ref).norm() / max(float(ref.norm()), 1e-6)
        assert float(off) <= 0.2, (name, float(off))

    near(out, want, "out")
    near(0.5 * loss, want_loss.reshape(1), "loss")
    near(dx, xr.grad, "dx")
    for name in params:
        near(grads[name], params[name].grad, name)


def test_example_learns(capsys, monkeypatch):
    m = _example()
    monkeypatch.setattr("sys.argv", ["moe_layer_step.py", "--tokens", "512", "--model", "256", "--hidden", "128",
                                     "--experts", "4", "--steps", "3"])
    m.main()
    errors = [float(line.split()[3]) for line in capsys.readouterr().out.splitlines() if line.startswith("step")]
    assert len(errors) == 3 and errors[2] < errors[1] < errors[0]
