"""A small language model on the token-model operators, as an example of their use together.

    python -m selective_state_space_22_amd.token_model

One gated recurrent layer between a lookup and the same table's transpose:

    x = s E[ids],  y = SiLU(x W_z) scan(x W_u, x W_a, x W_x; lam),  logits = (x + y W_o) E^T.

Training packs documents into rows (``reset`` marks each one's first token) and takes the gradients
of mamba_gated_scan_bwd and mamba_embed_bwd through autograd; generation runs the prompt through the
scan, keeps its last state, and goes on token by token with mamba_gated_state_update and mamba_sample.
The matrix products are torch's.
"""
from __future__ import annotations

import math

import torch

from .lm import (mamba_embed_bwd, mamba_embed_fwd, mamba_gated_scan_bwd, mamba_gated_scan_fwd,
                 mamba_gated_state_update, mamba_sample)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = weight.shape[0], scale
        return mamba_embed_fwd(ids, weight, scale)

    @staticmethod
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        return None, mamba_embed_bwd(ids, dout.contiguous(), ctx.vocab, ctx.scale), None


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, gate_a, gate_x, lam, z, reset):
        out, _, states = mamba_gated_scan_fwd(u, gate_a, gate_x, lam, z=z, reset=reset, return_last_state=False,
                                              return_states=True)
        ctx.save_for_backward(u, gate_a, gate_x, lam, z, reset, states)
        return out

    @staticmethod
    def backward(ctx, dout):
        u, gate_a, gate_x, lam, z, reset, states = ctx.saved_tensors
        g = mamba_gated_scan_bwd(u, gate_a, gate_x, lam, dout.contiguous(), z=z, reset=reset, states=states,
                                 want=("dz",))
        return g["du"], g["dgate_a"], g["dgate_x"], g["dlam"], g["dz"], None


class TokenModel(torch.nn.Module):
    """vocab tokens, width dim; the table and the products in dtype, lam and the states in float32."""

    def __init__(self, vocab, dim, dtype=torch.float32, device="cuda", seed=0):
        super().__init__()
        rng = torch.Generator().manual_seed(seed)
        self.scale = math.sqrt(dim)

        def weight(*shape):
            return torch.nn.Parameter((torch.randn(shape, generator=rng) / self.scale).to(device, dtype))

        self.table = weight(vocab, dim)
        self.w_in = weight(dim, 4 * dim)
        self.w_out = weight(dim, dim)
        # e^{-8 softplus(lam)} evenly from 0.5 to 0.999: channels of short and of long memory
        kappa = -torch.log(torch.linspace(0.5, 0.999, dim)) / 8
        self.lam = torch.nn.Parameter(torch.log(torch.expm1(kappa)).to(device))

    @staticmethod
    def one_document(ids):
        """The reset marks of rows that each hold one document from its first token on."""
        reset = torch.zeros(ids.shape, dtype=torch.bool, device=ids.device)
        reset[:, :1] = True
        return reset

    def inputs(self, x):
        return [p.contiguous() for p in (x @ self.w_in).chunk(4, -1)]

    def forward(self, ids, reset=None):
        """Logits (batch, L, vocab) of ids (batch, L); reset as in mamba_gated_scan_fwd, None: one document a row."""
        reset = self.one_document(ids) if reset is None else reset
        x = _Embedding.apply(ids, self.table, self.scale)
        u, a, g, z = self.inputs(x)
        y = _GatedScan.apply(u, a, g, self.lam, z, reset)
        return (x + y @ self.w_out) @ self.table.t()

    @torch.no_grad()
    def prefill(self, ids):
        """The last token's logits (batch, vocab) and the state behind it."""
        x = mamba_embed_fwd(ids, self.table, self.scale)
        u, a, g, z = self.inputs(x)
        y, state = mamba_gated_scan_fwd(u, a, g, self.lam, z=z, reset=self.one_document(ids))
        return (x[:, -1] + y[:, -1] @ self.w_out) @ self.table.t(), state

    @torch.no_grad()
    def step(self, ids, state):
        """Logits (batch, vocab) behind one more token; state is advanced in place."""
        x = mamba_embed_fwd(ids, self.table, self.scale)
        u, a, g, z = self.inputs(x)
        y = mamba_gated_state_update(state, u, a, g, self.lam, z=z)
        return (x + y @ self.w_out) @ self.table.t()

    @torch.no_grad()
    def generate(self, ids, tokens, generator=None, **filters):
        """ids (batch, L) continued by that many sampled tokens; filters: temperature, top_k, top_p and
        min_p of mamba_sample, one number for all rows each."""
        rows = {k: torch.full((ids.shape[0],), v, dtype=torch.int32 if k == "top_k" else torch.float32,
                              device=ids.device) for k, v in filters.items()}
        logits, state = self.prefill(ids)
        out = []
        for left in range(tokens, 0, -1):
            noise = torch.empty(logits.shape, device=ids.device).exponential_(generator=generator)
            out.append(mamba_sample(logits.contiguous(), noise, return_logprob=False, **rows)[0])
            if left > 1:
                logits = self.step(out[-1], state)
        return torch.stack(out, 1)


def batch_of(rng, rows, length, vocab, period):
    """Rows of packed documents, each a random word of `period` tokens said over and over.
    Returns ids, targets (-100 at a document's last token) and reset."""
    ids = torch.empty((rows, length), dtype=torch.int64)
    reset = torch.zeros((rows, length), dtype=torch.bool)
    for r in range(rows):
        at = 0
        while at < length:
            n = min(length - at, int(torch.randint(4 * period, 8 * period, (1,), generator=rng)))
            word = torch.randint(0, vocab, (period,), generator=rng)
            ids[r, at:at + n] = word.repeat(n // period + 1)[:n]
            reset[r, at] = True
            at += n
    target = torch.full_like(ids, -100)
    target[:, :-1] = torch.where(reset[:, 1:], -100, ids[:, 1:])
    return ids, target, reset


def train(model, steps, rows=16, length=256, period=2, lr=3e-3, seed=1):
    """Cross-entropy of the next token, by AdamW; returns the losses."""
    rng = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    device, vocab, losses = model.table.device, model.table.shape[0], []
    for _ in range(steps):
        ids, target, reset = (t.to(device) for t in batch_of(rng, rows, length, vocab, period))
        logits = model(ids, reset)
        loss = torch.nn.functional.cross_entropy(logits.reshape(-1, vocab).float(), target.reshape(-1))
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    model = TokenModel(vocab=32, dim=128)
    losses = train(model, 300)
    for i in range(0, 300, 50):
        print(f"step {i:4d}  loss {losses[i]:.3f}", flush=True)
    print(f"step  299  loss {losses[-1]:.3f}  (a uniform guess: {math.log(32):.3f})", flush=True)
    prompt = torch.tensor([[3, 17] * 6, [9, 4] * 6], device="cuda")
    gen = torch.Generator("cuda").manual_seed(0)
    print("prompts", prompt.tolist())
    print("go on  ", model.generate(prompt, 8, generator=gen, temperature=0.5, top_p=0.9, top_k=8).tolist())


if __name__ == "__main__":
    main()
