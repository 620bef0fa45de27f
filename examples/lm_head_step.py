"""Trains a small next-token model with the whole optimizer: Muon on the hidden matrices,
and, at the head, layer norm, the linear cross entropy and AdamW with 8-bit moments.

    python -c "import __graft_entry__ as g; g.build()"
    python examples/lm_head_step.py

The model predicts the next symbol of a noisy cyclic sequence from the last two; its loss
falls from log(vocab) towards the sequence's entropy.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_aware_optimizer_muon_gb300 as mm  # noqa: E402

VOCAB, DIM, TOKENS, NOISE = 5003, 256, 2048, 0.1


def batch(gen, dev):
    """(the last two symbols, the next one): next = 7*a + 3*b + 11 mod VOCAB, sometimes noise."""
    pair = torch.randint(0, 64, (TOKENS, 2), generator=gen, device=dev)
    nxt = (7 * pair[:, 0] + 3 * pair[:, 1] + 11) % VOCAB
    noisy = torch.rand(TOKENS, generator=gen, device=dev) < NOISE
    nxt = torch.where(noisy, torch.randint(0, VOCAB, (TOKENS,), generator=gen, device=dev), nxt)
    nxt[:16] = -100                          # a prompt carries no loss
    return pair, nxt


def train(steps=60, seed=0, verbose=True):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.bfloat16).requires_grad_()

    hidden = [normal(2 * DIM, 2 * DIM, std=0.05), normal(DIM, 2 * DIM, std=0.05)]      # Muon
    embed, vocab = normal(VOCAB, DIM, std=0.5), normal(VOCAB, DIM, std=0.02)             # AdamW, 8-bit moments
    gain, shift = torch.ones(DIM, device=dev, dtype=torch.bfloat16), torch.zeros(DIM, device=dev, dtype=torch.bfloat16)
    aux = [embed, vocab, gain.requires_grad_(), shift.requires_grad_()]
    opt = mm.PeriodicMuon([w.detach() for w in hidden], K=3, eta=0.01, lam=0.0, aux_params=[a.detach() for a in aux],
                          aux_lr=3e-3, aux_bits=8, aux_seed=seed)
    losses = []
    for step in range(steps):
        pair, nxt = batch(gen, dev)
        x = embed[pair].view(TOKENS, 2 * DIM)
        x = torch.nn.functional.silu(x @ hidden[0].T) @ hidden[1].T
        loss = mm.linear_cross_entropy(mm.layer_norm(x, gain, shift), vocab, nxt)
        grads = torch.autograd.grad(loss, hidden + aux)
        opt.step([g.contiguous() for g in grads[:2]], [g.contiguous() for g in grads[2:]])
        losses.append(loss.detach())
        if verbose and (step % 10 == 0 or step == steps - 1):
            print(f"step {step:3d}  loss {loss.item():.3f}  (log vocab {math.log(VOCAB):.3f})")
    assert opt.check() == mm.MUON_OK
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    train()
