"""Linear-attention layers with a decay for each head, trained and served with the library's calls.

A layer projects its input to q, k, v and a gate, runs linear attention whose state decays by a fixed
slope of the head, and projects the gated output back.  `LinearAttention` puts the operator under
autograd; between the passes it holds q, k and v in 8 bits (`hold`), which is what such a layer keeps
most memory for.  Serving extends prompts in packed rows and then takes one token of each request over
a pool of states.  Weights are random; a request's next input is its last output.

    python examples/linear_stack.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HIDDEN, HK, HV, K, V = 512, 2, 4, 128, 128


def cumulative(lens):
    out = torch.zeros(len(lens) + 1, dtype=torch.int32)
    out[1:] = torch.tensor(lens).cumsum(0)
    return out.cuda()


def slopes(heads):
    """Log-decays: the heads forget over 8, 16, 32, ... tokens."""
    return -(2.0 ** -(3.0 + torch.arange(heads, device="cuda", dtype=torch.float32)))


class LinearAttention(torch.autograd.Function):
    """gdn.linear_attention with its gradients of q, k, v and h0; hold: torch.int8 or
    torch.float8_e4m3fn for 8-bit checkpoints of q, k and v, None to keep them as they are."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, h0, cu, hold):
        from gated_delta_rule_07_gb300 import gdn
        ctx.dtype, ctx.carried = q.dtype, h0 is not None
        if hold is None:
            kept = (q, k, v)
        else:
            kept = [t for c in gdn.checkpoint_pack(q, k, v, dtype=hold) for t in (c.codes, c.scale)]
        ctx.save_for_backward(log_decay, h0, cu, *kept)
        return gdn.linear_attention(q, k, v, log_decay, h0, cu)

    @staticmethod
    def backward(ctx, dout, dlast):
        from gated_delta_rule_07_gb300 import gdn
        log_decay, h0, cu, *kept = ctx.saved_tensors
        if len(kept) == 6:
            kept = [gdn.Checkpoint(kept[i], kept[i + 1], ctx.dtype) for i in (0, 2, 4)]
        dq, dk, dv, dh0 = gdn.linear_attention_backward(*kept, log_decay, dout.contiguous(), h0,
                                                        dlast.contiguous(), cu)
        return dq, dk, dv, None, dh0 if ctx.carried else None, None, None


class Layer:
    """x -> projections -> linear attention -> gate -> output projection."""

    def __init__(self, gen, requests):
        cols = 2 * HK * K + 2 * HV * V
        self.w_in = (torch.randn(cols, HIDDEN, device="cuda", generator=gen) / HIDDEN ** 0.5).bfloat16()
        self.w_out = (torch.randn(HIDDEN, HV * V, device="cuda", generator=gen)
                      / (HV * V) ** 0.5).bfloat16()
        self.log_decay = slopes(HV)
        self.state = torch.zeros(requests, HV, K, V, device="cuda")
        self.slot = torch.arange(requests, dtype=torch.int32, device="cuda")

    def project(self, x):
        """Slices of one projection's rows: q, k, v and the gate."""
        T = x.shape[0]
        q, k, v, gate = (x @ self.w_in.t()).split([HK * K, HK * K, HV * V, HV * V], dim=1)
        return q.view(T, HK, K), k.view(T, HK, K), v.view(T, HV, V), gate

    def close(self, out, gate):
        # (a state gathers over the slope's span, its outputs are brought back to size)
        out = out * (1 - self.log_decay.exp()).to(out.dtype)[:, None] / 8
        return (out.flatten(1) * gate.sigmoid()) @ self.w_out.t()

    def train(self, x, cu, hold):
        q, k, v, gate = self.project(x)
        out, _ = LinearAttention.apply(q, k, v, self.log_decay, None, cu, hold)
        return self.close(out, gate)

    def extend(self, x, cu):
        from gated_delta_rule_07_gb300 import gdn
        q, k, v, gate = self.project(x)
        out, self.state = gdn.linear_attention(q, k, v, self.log_decay, self.state, cu)
        return self.close(out, gate)

    def step(self, x):
        from gated_delta_rule_07_gb300 import gdn
        q, k, v, gate = self.project(x)
        return self.close(gdn.linear_attention_decode(q, k, v, self.log_decay, self.slot, self.state),
                          gate)


class Stack:
    def __init__(self, requests, layers=3, seed=1):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.layers = [Layer(gen, requests) for _ in range(layers)]

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def run(self, x, call):
        for layer in self.layers:
            x = x + call(layer, self.norm(x))
        return x

    def extend(self, x, lens):
        cu = cumulative(lens)
        return self.run(x, lambda layer, y: layer.extend(y, cu))

    def step(self, x):
        return self.run(x, lambda layer, y: layer.step(y))

    def train(self, x, lens, hold=None):
        cu = cumulative(lens)
        return self.run(x, lambda layer, y: layer.train(y, cu, hold))


def serve(lens=(300, 1, 64, 130), steps=16, seed=1):
    """Prompts and `steps` single tokens fed back, and the same tokens again as the prompts' last ones:
    (outputs of the steps, outputs of the prompts' ends), [requests, steps, HIDDEN]."""
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    prompts = torch.randn(sum(lens), HIDDEN, device="cuda", generator=gen).bfloat16()
    last = (cumulative(lens)[1:] - 1).long()
    stack, fed, outs = Stack(len(lens), seed=seed), [], []
    x = Stack.norm(stack.extend(prompts, list(lens))[last])
    for _ in range(steps):
        fed.append(x)
        y = stack.step(x)
        outs.append(y)
        x = Stack.norm(y)
    again = Stack(len(lens), seed=seed)
    again.extend(prompts, list(lens))
    whole = again.extend(torch.stack(fed, 1).flatten(0, 1), [steps] * len(lens))
    return torch.stack(outs, 1), whole.view(len(lens), steps, HIDDEN)


def gradients(lens=(200, 57, 1), seed=3, hold=None):
    """The gradients of a loss with respect to the input and the layers' weights."""
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(sum(lens), HIDDEN, device="cuda", generator=gen).bfloat16().requires_grad_()
    goal = torch.randn(sum(lens), HIDDEN, device="cuda", generator=gen)
    stack = Stack(len(lens), seed=seed)
    weights = [w.requires_grad_() for layer in stack.layers for w in (layer.w_in, layer.w_out)]
    loss = (stack.train(x, list(lens), hold).float() - goal).square().mean()
    return loss.detach(), torch.autograd.grad(loss, [x, *weights])


def main():
    from gated_delta_rule_07_gb300 import build
    build.build()
    steps, whole = serve()
    off = float((steps.float() - whole.float()).norm() / whole.float().norm())
    print(f"{steps.shape[0]} requests, {steps.shape[1]} steps; the same tokens in one call differ by "
          f"{off:.4f} of their norm")
    _, kept = gradients()
    for hold in (torch.int8, torch.float8_e4m3fn):
        _, held = gradients(hold=hold)
        off = max(float((a.float() - b.float()).norm() / a.float().norm()) for a, b in zip(kept, held))
        print(f"gradients from {hold} checkpoints differ by up to {off:.4f} of their norm")


if __name__ == "__main__":
    main()
