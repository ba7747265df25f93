"""A small hybrid decoder on libkda: a KDA layer and a gated-recurrence layer, alternating, with the fused
norms around them.  It shows the operators as they are used together:

  prefill   packed prompts through kda_forward_segmented and kda_gated_scan_forward, whose final states
            become the slots of two state pools;
  decode    one token per slot through kda_decode_step and kda_gated_scan_step;
  training  the recurrence layer and its norms under autograd (GatedScan and BlockNorm below), a few steps
            of gradient descent.

Run ``python examples/hybrid_decoder.py`` on a GB300: it checks that decoding continues a prefill as a longer
prefill would, and that training lowers its loss.  Weights are random; the projections are plain matrix products.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import context_kda_gb300 as kda  # noqa: E402

HEAD = 128
EPS = 1e-6


def _empty(*shape, like=None, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype if like is None else like.dtype, device="cuda")


class Decoder:
    """'layers' layers, KDA and gated recurrence in turn; the residual stream is fp32, activations bf16."""

    def __init__(self, heads=4, layers=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.width, self.layers = heads, heads * HEAD, layers
        D = self.width

        def matrix(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device="cuda") / rows ** 0.5).to(torch.bfloat16)

        self.proj = []
        for n in range(layers):
            # KDA: q, k, v, output gate, log-decay, beta; recurrence: x, input gate, output gate, log-decay
            cols = 5 * D + heads if n % 2 == 0 else 4 * D
            self.proj.append({"in": matrix(D, cols), "out": matrix(D, D)})
        ones = lambda n: torch.ones(n, device="cuda")
        self.w_pre = [ones(D) for _ in range(layers + 1)]           # the norm before each layer, and the last one
        self.w_head = [ones(HEAD if n % 2 == 0 else D) for n in range(layers)]
        self.w_post = [ones(D) for _ in range(layers)]
        self.ls = [torch.full((D,), 0.5, device="cuda") for _ in range(layers)]

    def new_states(self, slots):
        """A pool of states per layer, one slot a sequence."""
        H, D = self.heads, self.width
        return [torch.zeros(slots, H, HEAD, HEAD, device="cuda") if n % 2 == 0 else torch.zeros(slots, D, device="cuda")
                for n in range(self.layers)]

    def _split(self, n, y):
        """A layer's projections of the normed rows y."""
        D, H = self.width, self.heads
        p = y @ self.proj[n]["in"]
        if n % 2:
            x, i, z, g = p.split(D, dim=1)
            # x is a column range of the projection's rows; gates and decays are made from theirs
            return x, torch.sigmoid(i.float()).to(y.dtype), z, -torch.nn.functional.softplus(g.float() - 2)
        q, k, v, z, g, beta = p.split([D, D, D, D, D, H], dim=1)
        heads = lambda t: t.unflatten(1, (H, HEAD))
        unit = lambda t: torch.nn.functional.normalize(heads(t).float(), dim=-1).to(y.dtype)
        return unit(q), unit(k), heads(v), z, -torch.nn.functional.softplus(heads(g).float() - 4), torch.sigmoid(beta.float())

    def _after(self, n, r, o, z):
        """The head norm with its gate, the output product, then the norm after the layer, the residual and the next
        layer's norm in one pass.  r is updated in place; returns the next normed rows."""
        D = self.width
        gated, y = torch.empty_like(o), torch.empty_like(o)
        kda.kda_block_norm_forward(None, o, z, "sigmoid", HEAD if n % 2 == 0 else 0, self.w_head[n], 1.0, None, None, EPS, gated, None)
        out = gated @ self.proj[n]["out"]
        kda.kda_block_norm_forward(r, out, None, "none", 0, self.w_post[n], 1.0, self.ls[n], self.w_pre[n + 1], EPS, r, y)
        return y

    def _first(self, r):
        y = _empty(*r.shape, dtype=torch.bfloat16)
        kda.kda_block_norm_forward(r, None, None, "none", 0, None, 1.0, None, self.w_pre[0], EPS, None, y)
        return y

    def prefill(self, embedded, lengths):
        """Packed prompts [T, D] (fp32) of the given lengths; returns the last norm's rows and the states after each."""
        T, D = embedded.shape
        H, N = self.heads, len(lengths)
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        plan = kda.kda_plan_segments(cu, 1)
        plan_dev = kda.upload_plan(plan)
        ws = _empty(max(kda.kda_workspace_bytes(plan, H), kda.kda_gated_scan_workspace_bytes(plan, D)), dtype=torch.uint8)
        states = self.new_states(N)
        r = embedded.clone()
        y = self._first(r)
        for n in range(self.layers):
            if n % 2:
                x, i, z, g = self._split(n, y)
                o = _empty(T, D, like=y)
                kda.kda_gated_scan_forward(plan, plan_dev, x, i, g, None, o, states[n], None, ws)
            else:
                q, k, v, z, g, beta = self._split(n, y)
                o = _empty(T, H, HEAD, like=y)
                kda.kda_forward_segmented(plan, plan_dev, H, q, k, v.contiguous(), g, beta, None, 1.0, o, states[n], ws)
                o = o.flatten(1)
            y = self._after(n, r, o, z)
        return y, states

    def step(self, embedded, states, slots):
        """One token per row [B, D] (fp32), row b the next of slots[b] (int32, negative: padding); the states are
        updated in place.  Returns the last norm's rows."""
        B, D = embedded.shape
        r = embedded.clone()
        y = self._first(r)
        for n in range(self.layers):
            if n % 2:
                x, i, z, g = self._split(n, y)
                o = _empty(B, D, like=y)
                kda.kda_gated_scan_step(slots, x, i, g, states[n], o)
            else:
                q, k, v, z, g, beta = self._split(n, y)
                o = _empty(B, self.heads, HEAD, like=y)
                kda.kda_decode_step(slots, q, k, v, g, beta, 1.0, states[n], o)
                o = o.flatten(1)
            y = self._after(n, r, o, z)
        return y


# ---- under autograd ----------------------------------------------------------------------------------------


class GatedScan(torch.autograd.Function):
    """h of kda_gated_scan_forward, with gradients for x, i and g."""

    @staticmethod
    def forward(ctx, plan, plan_dev, ws, x, i, g):
        T, D = x.shape
        h, states = _empty(T, D, like=x), _empty(-(-T // 128), D)
        kda.kda_gated_scan_forward(plan, plan_dev, x, i, g, None, h, None, states, ws)
        ctx.plan, ctx.plan_dev, ctx.ws = plan, plan_dev, ws
        ctx.save_for_backward(x, i, g, states)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, i, g, states = ctx.saved_tensors
        dx, di, dg = torch.empty_like(x), torch.empty_like(i), torch.empty_like(g)
        kda.kda_gated_scan_backward(ctx.plan, ctx.plan_dev, x, i, g, None, states, dh.contiguous(), None, dx, di, dg, None, ctx.ws)
        return None, None, None, dx, di, dg


class BlockNorm(torch.autograd.Function):
    """(r', y) of kda_block_norm_forward, with gradients for r, o, z and the weights.  All but o may be None, as in the call
    (z where the gate is "none"; without w_pre there is no y)."""

    @staticmethod
    def forward(ctx, gate, group, scale, r, o, z, w_post, ls, w_pre):
        r_out, y = torch.empty_like(o if r is None else r), None if w_pre is None else torch.empty_like(o)
        kda.kda_block_norm_forward(r, o, z, gate, group, w_post, scale, ls, w_pre, EPS, r_out, y)
        ctx.how = gate, group, scale, r is not None
        ctx.save_for_backward(r_out, o, z, w_post, ls, w_pre)
        return r_out, y

    @staticmethod
    def backward(ctx, dr_out, dy):
        gate, group, scale, has_r = ctx.how
        r_out, o, z, w_post, ls, w_pre = ctx.saved_tensors
        like = lambda t: None if t is None else torch.empty_like(t)
        dr, do, dz, dw = like(r_out) if has_r else None, like(o), like(z), [like(w) for w in (w_post, ls, w_pre)]
        ws = _empty(kda.kda_block_norm_workspace_bytes(o.shape[1]), dtype=torch.uint8)
        kda.kda_block_norm_backward(r_out, o, z, gate, group, w_post, scale, ls, w_pre, EPS, dr_out.contiguous(),
                                    None if w_pre is None else dy.contiguous(), dr, do, dz, *dw, ws)
        return None, None, None, dr, do, dz, *dw


def train(steps=30, lengths=(700, 90, 300), width=256, seed=0):
    """Gradient descent on one recurrence layer with its norms; returns the losses.  The target is a delayed copy of the
    input, which only a state can give."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, cu = sum(lengths), [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    plan = kda.kda_plan_segments(cu, 1)
    plan_dev = kda.upload_plan(plan)
    ws = _empty(max(16, kda.kda_gated_scan_workspace_bytes(plan, width)), dtype=torch.uint8)
    r = torch.randn(T, width, generator=gen, device="cuda")
    target = torch.zeros_like(r)
    for a, b in zip(cu[:-1], cu[1:]):
        target[a + 1:b] = r[a:b - 1]
    params = [(torch.randn(width, 4 * width, generator=gen, device="cuda") / width ** 0.5).requires_grad_()]
    params += [torch.ones(width, device="cuda", requires_grad=True) for _ in range(3)]
    optimizer = torch.optim.Adam(params, lr=1e-2)
    losses = []
    for _ in range(steps):
        w, w_post, ls, w_pre = params
        x, i, z, g = (r.to(torch.bfloat16) @ w.to(torch.bfloat16)).split(width, dim=1)
        h = GatedScan.apply(plan, plan_dev, ws, x.contiguous(), torch.sigmoid(i), -torch.nn.functional.softplus(g.float()))
        _, y = BlockNorm.apply("silu", 0, 1.0, r, h, z.contiguous(), w_post, ls, w_pre)
        loss = (y.float() - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def decode_error(lengths=(200, 1, 77), new=12, seed=0):
    """The largest difference between the outputs of 'new' decoded tokens per prompt and those of a prefill over prompts
    and tokens together."""
    model = Decoder(seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    rows = [torch.randn(n + new, model.width, generator=gen, device="cuda") for n in lengths]
    want, _ = model.prefill(torch.cat(rows), [n + new for n in lengths])
    _, states = model.prefill(torch.cat([x[:n] for x, n in zip(rows, lengths)]), lengths)
    slots = torch.arange(len(lengths), dtype=torch.int32, device="cuda")
    worst, at = 0.0, [0]
    for n in lengths:
        at.append(at[-1] + n + new)
    for t in range(new):
        got = model.step(torch.stack([x[n + t] for x, n in zip(rows, lengths)]), states, slots)
        expect = torch.stack([want[at[b] + n + t] for b, n in enumerate(lengths)])
        worst = max(worst, float((got.float() - expect.float()).abs().max()))
    return worst


def main():
    error = decode_error()
    print(f"decoding against a longer prefill: largest difference {error:.3f} (outputs of unit size)")
    losses = train()
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    status = kda.kda_device_status()
    if status != 0:
        raise RuntimeError(f"device status {status}")


if __name__ == "__main__":
    main()
