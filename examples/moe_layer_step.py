"""Training steps of a mixture-of-experts layer whose activations are kept in
8 bits: layer norm, router, two grouped GEMMs per expert around a gated
activation, and the gradients of all of it.

    out[t] = x[t] + sum_j gate[t, j] * W2_e (silu(g) * u),
    (g, u) = W1_e norm(x)[t],  e = chosen[t, j]

What the backward pass needs of the activations is x, the row statistics, and
three 8-bit checkpoints: of the norm's output (written by the norm, gathered
into expert order, and at once the first GEMM's operand), of the gated
activation's input (written by the activation) and of its output (the second
GEMM's operand).  No call reads device memory on the host.

    python examples/moe_layer_step.py [--tokens 4096 --model 1024 --hidden 512
                                       --experts 8 --topk 2 --steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_precision_quantization_amd as mx  # noqa: E402

ALIGN = 32   # rows of an expert are padded to whole MX blocks


class MoELayer:
    """Weights in float32; w1 (E, 2 F, C), w2 (E, C, F), router (E, C)."""

    def __init__(self, model, hidden, experts, topk, device, seed=0, aux=0.01):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(device)

        self.topk, self.aux = topk, torch.full((1,), aux, device=device)
        self.params = {
            "norm_w": 1.0 + normal(model, scale=0.1), "norm_b": normal(model, scale=0.1),
            "router": normal(experts, model, scale=model ** -0.5),
            "w1": normal(experts, 2 * hidden, model, scale=model ** -0.5),
            "w2": normal(experts, model, hidden, scale=hidden ** -0.5),
        }

    def forward(self, x):
        """x (T, C) bf16 -> (out float32 (T, C), balance loss (1), kept)."""
        p = self.params
        t, c = x.shape
        experts, topk = p["router"].shape[0], self.topk
        y, mean, rstd, q, s = mx.mx_layernorm(x, p["norm_w"], p["norm_b"], checkpoint=True, raw=True)
        logits = y.float() @ p["router"].T
        chosen, gates, lse, counts, ends, balance, loss = mx.mx_router_balance(logits, topk, normalize=True, align=ALIGN)

        # a slot in expert order for every (token, choice)
        flat = chosen.reshape(-1).long()
        order = torch.argsort(flat, stable=True)
        before = torch.cumsum(counts, 0) - counts
        begin = torch.cat([ends.new_zeros(1), ends[:-1]])
        slot = torch.empty_like(flat)
        sorted_e = flat[order]
        slot[order] = begin[sorted_e] + torch.arange(t * topk, device=x.device) - before[sorted_e]
        rows = (t * topk + experts * (ALIGN - 1) + ALIGN - 1) // ALIGN * ALIGN

        def to_slots(a):
            out = a.new_zeros((rows, a.shape[1]))
            out[slot] = a.repeat_interleave(topk, 0)
            return out

        q1, s1 = to_slots(q), to_slots(s)
        h = self._grouped(q1, s1, *self._weight(p["w1"]), ends)
        a, qh, sh = mx.mx_gated_act(h, "silu", raw=True)
        q2, s2 = mx.mx_cast_dim0_dim1(a, dim1=False, raw=True)[:2]
        o = self._grouped(q2, s2, *self._weight(p["w2"]), ends)
        picked = o[slot].reshape(t, topk, c).float()
        out = x.float() + (gates[:, :, None] * picked).sum(1)
        kept = dict(x=x, mean=mean, rstd=rstd, q=q, s=s, logits=logits, lse=lse, chosen=chosen, gates=gates,
                    balance=balance, ends=ends, slot=slot, q1=q1, s1=s1, qh=qh, sh=sh, q2=q2, s2=s2, picked=picked)
        return out, loss, kept

    def backward(self, dout, kept):
        """Gradients (dx, {parameter: gradient}) of sum(dout * out) + aux * loss."""
        p, k, topk = self.params, kept, self.topk
        t, c = dout.shape
        dgates = (dout[:, None, :] * k["picked"]).sum(2)
        do = torch.zeros((k["q1"].shape[0], c), dtype=torch.bfloat16, device=dout.device)
        do[k["slot"]] = (k["gates"][:, :, None] * dout[:, None, :]).reshape(t * topk, c).bfloat16()
        dw2 = mx.mx_wgrad_checkpoint(do, k["q2"], k["s2"], k["ends"])
        da = self._dgrad(do, p["w2"], k["ends"])
        dh, = mx.mx_gated_act_backward(da, k["qh"], k["sh"], "silu")
        dw1 = mx.mx_wgrad_checkpoint(dh, k["q1"], k["s1"], k["ends"])
        dslots = self._dgrad(dh, p["w1"], k["ends"])
        dlogits = mx.mx_router_balance_backward(k["logits"], k["lse"], k["chosen"], k["gates"], k["balance"], dgates,
                                                self.aux, normalize=True)
        drouter = mx.mx_wgrad_checkpoint(dlogits.bfloat16(), k["q"], k["s"])
        dy = dslots[k["slot"]].reshape(t, topk, c).float().sum(1) + dlogits @ p["router"]
        dx, dnw, dnb = mx.mx_layernorm_backward(dy.bfloat16(), k["x"], p["norm_w"], k["mean"], k["rstd"])
        return dout + dx.float(), {"norm_w": dnw, "norm_b": dnb, "router": drouter, "w1": dw1, "w2": dw2}

    @staticmethod
    def _weight(w):
        """(E, N, K) float32 -> its codes along K and their blocked scales."""
        e, n, k = w.shape
        q, s = mx.mx_cast_dim0_dim1(w.bfloat16().reshape(e * n, k), dim1=False, raw=True)[:2]
        return q.reshape(e, n, k), mx.mx_scales_to_blocked(s.reshape(e, n, k // 32), raw=True)

    @staticmethod
    def _grouped(q, s, qw, sw, ends):
        blocked, _ = mx.mx_scales_to_blocked_grouped(s, ends, 0, raw=True)
        out = torch.zeros((q.shape[0], qw.shape[1]), dtype=torch.bfloat16, device=q.device)
        return mx.mx_grouped_gemm_mxfp8(q, blocked, qw, sw, ends, out=out)

    def _dgrad(self, dy, w, ends):
        """dy times the experts' weights, both cast along the summed axis."""
        q, s = mx.mx_cast_dim0_dim1(dy, dim1=False, raw=True)[:2]
        qw, sw = mx.mx_cast_dim1_3d_blocked(w.bfloat16(), raw=True)
        return self._grouped(q, s, qw, sw, ends)


def main():
    ap = argparse.ArgumentParser()
    for name, value in dict(tokens=4096, model=1024, hidden=512, experts=8, topk=2, steps=5).items():
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--rate", type=float, default=0.2)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    layer = MoELayer(a.model, a.hidden, a.experts, a.topk, dev)
    teacher = MoELayer(a.model, a.hidden, a.experts, a.topk, dev, seed=1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(a.tokens, a.model, generator=g).to(dev).bfloat16()
    target = teacher.forward(x)[0]
    for step in range(a.steps):
        out, balance, kept = layer.forward(x)
        d = out - target
        _, grads = layer.backward(d / a.tokens, kept)
        for name, w in layer.params.items():
            w -= a.rate * grads[name]
        print("step %d  error %.5f  balance %.4f" % (step, float(d.square().mean()), float(balance)), flush=True)


if __name__ == "__main__":
    main()
