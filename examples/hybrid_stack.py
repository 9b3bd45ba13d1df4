"""A small hybrid stack served and tuned with the library's calls.

Three layers of four carry the gated delta rule's recurrent state, the fourth is softmax attention
over an 8-bit paged cache.  `Stack.extend` takes new tokens of every request in packed rows (a
prompt, a chunk of one, drafted tokens); `Stack.step` takes one token of each.  Both leave the
requests' states, conv inputs and cache pages ready for the next call.  `QkNormRope` puts the norms
and the rotation under autograd.  Weights are random; a request's next input is its last output.

    python examples/hybrid_stack.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HIDDEN = 512
HK, HV, K, V, CONV = 2, 4, 128, 128, 4          # recurrent layers
HQ, HKV, D, ROTARY, PAGE = 8, 2, 128, 64, 32    # attention layer
MAX_TOKENS = 4096                               # positions of a request


def cumulative(lens):
    out = torch.zeros(len(lens) + 1, dtype=torch.int32)
    out[1:] = torch.tensor(lens).cumsum(0)
    return out.cuda()


def rotation_table(positions=MAX_TOKENS, rotary=ROTARY, base=1e6):
    """cos and sin of every position's angles: [positions, rotary] fp32."""
    f = base ** (-torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64) / rotary)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class QkNormRope(torch.autograd.Function):
    """gdn.qk_norm_rope with its gradients of q, k and the norms' weights."""

    @staticmethod
    def forward(ctx, q, k, positions, table, q_weight, k_weight):
        from gated_delta_rule_07_gb300 import gdn
        ctx.save_for_backward(q, k, positions, table, q_weight, k_weight)
        return gdn.qk_norm_rope(q, k, positions, table, q_weight, k_weight)

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        from gated_delta_rule_07_gb300 import gdn
        dq, dk, dqw, dkw = gdn.qk_norm_rope_backward(*ctx.saved_tensors, dq_out.contiguous(),
                                                     dk_out.contiguous())
        return dq, dk, None, None, dqw, dkw


def _weight(gen, rows, cols):
    w = torch.randn(rows, cols, device="cuda", generator=gen) / cols ** 0.5
    return w.bfloat16()


class RecurrentLayer:
    """x -> projections -> conv, norms, gates -> recurrence -> output projection."""

    def __init__(self, gen, requests):
        channels = 2 * HK * K + HV * V
        self.w_in = _weight(gen, channels + 2 * HV, HIDDEN)
        self.w_out = _weight(gen, HIDDEN, HV * V)
        self.conv = 0.5 * torch.randn(channels, CONV, device="cuda", generator=gen)
        self.A_log = torch.randn(HV, device="cuda", generator=gen) - 2.0
        self.dt_bias = torch.zeros(HV, device="cuda")
        self.state = torch.zeros(requests, HV, K, V, device="cuda")
        self.conv_in = torch.zeros(requests, channels, CONV - 1, device="cuda").bfloat16()
        self.slot = torch.arange(requests, dtype=torch.int32, device="cuda")

    def _inputs(self, x, cu):
        from gated_delta_rule_07_gb300 import gdn
        p = x @ self.w_in.t()
        qkv, a, b = p.split([self.conv.shape[0], HV, HV], dim=1)
        q, k, v, g, beta, self.conv_in = gdn.prologue(
            qkv.contiguous(), self.conv, a.contiguous(), b.contiguous(), self.A_log, self.dt_bias,
            HK, HV, K, V, self.conv_in, cu, activation="silu")
        return q, k, v, g, beta

    def extend(self, x, cu):
        from gated_delta_rule_07_gb300 import gdn
        out, self.state = gdn.forward(*self._inputs(x, cu), self.state, cu)
        return out.flatten(1) @ self.w_out.t()

    def step(self, x, cu):
        from gated_delta_rule_07_gb300 import gdn
        out = gdn.decode(*self._inputs(x, cu), self.slot, self.state)
        return out.flatten(1) @ self.w_out.t()


class AttentionLayer:
    """x -> projections -> norms and rotation -> cache -> attention -> gate -> output projection."""

    def __init__(self, gen, requests, dtype=torch.int8):
        from gated_delta_rule_07_gb300 import gdn
        # a head's queries and its gate stand side by side in the projection's rows
        self.w_in = _weight(gen, (2 * HQ + 2 * HKV) * D, HIDDEN)
        self.w_out = _weight(gen, HIDDEN, HQ * D)
        self.q_weight = 1 + 0.1 * torch.randn(D, device="cuda", generator=gen)
        self.k_weight = 1 + 0.1 * torch.randn(D, device="cuda", generator=gen)
        self.table = rotation_table()
        pages = MAX_TOKENS // PAGE
        self.cache = gdn.KVCache.empty(requests * pages, HKV, PAGE, D, dtype)
        order = torch.randperm(requests * pages, generator=torch.Generator().manual_seed(5))
        self.block_table = order.view(requests, pages).int().cuda()

    def project(self, x):
        T, p = x.shape[0], x @ self.w_in.t()
        q_gate, k, v = p.split([2 * HQ * D, HKV * D, HKV * D], dim=1)
        q_gate = q_gate.view(T, HQ, 2 * D)
        return q_gate[..., :D], q_gate[..., D:], k.view(T, HKV, D), v.view(T, HKV, D)

    def extend(self, x, positions, held, cu):
        """`held` [requests]: tokens that each request has in the cache; cu None: one new one each."""
        from gated_delta_rule_07_gb300 import gdn
        q, gate, k, v = self.project(x)
        q, k = gdn.qk_norm_rope(q, k, positions, self.table, self.q_weight, self.k_weight)
        gdn.kv_append(self.cache, k, v, self.block_table, held, cu)
        new = 1 if cu is None else cu[1:] - cu[:-1]
        out, _ = gdn.kv_attention(self.cache, q, self.block_table, held + new, cu)
        return (out * gate.sigmoid()).flatten(1) @ self.w_out.t()


class Stack:
    def __init__(self, requests, seed=1, dtype=torch.int8):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.layers = [RecurrentLayer(gen, requests) for _ in range(3)]
        self.layers.append(AttentionLayer(gen, requests, dtype))
        self.requests = requests
        self.held = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.each = torch.arange(requests + 1, dtype=torch.int32, device="cuda")

    @staticmethod
    def _norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def extend(self, x, lens):
        """x [sum(lens), HIDDEN]: lens[n] >= 1 new tokens of every request; their outputs."""
        cu = cumulative(lens)
        within = torch.cat([torch.arange(n) for n in lens]).int().cuda()
        owner = torch.repeat_interleave(torch.arange(self.requests), torch.tensor(lens)).cuda()
        positions = self.held[owner] + within
        for layer in self.layers[:3]:
            x = x + layer.extend(self._norm(x), cu)
        x = x + self.layers[3].extend(self._norm(x), positions, self.held, cu)
        self.held += cu[1:] - cu[:-1]
        return x

    def step(self, x):
        """x [requests, HIDDEN]: one new token of every request; nothing waits for the host."""
        for layer in self.layers[:3]:
            x = x + layer.step(self._norm(x), self.each)
        x = x + self.layers[3].extend(self._norm(x), self.held, self.held, None)
        self.held += 1
        return x


def serve(lens=(700, 3, 64, 1, 333), steps=24, seed=1, dtype=torch.int8):
    """Prompts, `steps` single tokens fed back, and the same tokens again as a batch of drafted
    ones: (outputs of the steps, outputs of the drafted tokens), [requests, steps, HIDDEN]."""
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    prompts = torch.randn(sum(lens), HIDDEN, device="cuda", generator=gen).bfloat16()
    last = (cumulative(lens)[1:] - 1).long()
    stack, fed, outs = Stack(len(lens), seed, dtype), [], []
    x = Stack._norm(stack.extend(prompts, list(lens))[last])
    for _ in range(steps):
        fed.append(x)
        y = stack.step(x)
        outs.append(y)
        x = Stack._norm(y)
    again = Stack(len(lens), seed, dtype)
    again.extend(prompts, list(lens))
    drafted = again.extend(torch.stack(fed, 1).flatten(0, 1), [steps] * len(lens))
    return torch.stack(outs, 1), drafted.view(len(lens), steps, HIDDEN)


def tune(tokens=256, rounds=30, seed=3):
    """Gradient descent on the norms' weights towards outputs under other weights: the losses."""
    gen = torch.Generator("cuda").manual_seed(seed)
    q = torch.randn(tokens, HQ, D, device="cuda", generator=gen).bfloat16()
    k = torch.randn(tokens, HKV, D, device="cuda", generator=gen).bfloat16()
    positions = torch.arange(tokens, dtype=torch.int32, device="cuda")
    table = rotation_table(tokens)
    goal = [1 + 0.3 * torch.randn(D, device="cuda", generator=gen) for _ in range(2)]
    want = [t.float() for t in QkNormRope.apply(q, k, positions, table, *goal)]
    weights = [torch.ones(D, device="cuda", requires_grad=True) for _ in range(2)]
    losses = []
    for _ in range(rounds):
        got = QkNormRope.apply(q, k, positions, table, *weights)
        loss = sum((a.float() - b).square().mean() for a, b in zip(got, want))
        losses.append(float(loss.detach()))
        for w, g in zip(weights, torch.autograd.grad(loss, weights)):
            w.data -= 0.25 * D * g
    return losses


def main():
    from gated_delta_rule_07_gb300 import build
    build.build()
    steps, drafted = serve()
    off = float((steps.float() - drafted.float()).norm() / drafted.float().norm())
    print(f"{steps.shape[0]} requests, {steps.shape[1]} steps; the same tokens drafted at once "
          f"differ by {off:.4f} of their norm")
    losses = tune()
    print(f"norm weights tuned: loss {losses[0]:.4f} -> {losses[-1]:.6f}")


if __name__ == "__main__":
    main()
