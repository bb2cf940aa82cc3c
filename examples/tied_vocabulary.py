"""A small language model whose vocabulary table is both its embedding and its LM
head, trained and then searched with this library's operators.

    python examples/tied_vocabulary.py [--steps 300] [--beams 4]

The model: h_t = h_{t-1} / 2 + scale * W[x_t] (a decaying sum of embeddings),
logits z_t = (h_t A) W^T.  A training step looks the tokens up
(`VocabOps.embedding_forward`), takes loss and logit gradient in one call
(`LMLoss.forward_backward`), writes the head's part of W's gradient with a matrix
product and adds the embedding's part to it (`VocabOps.embedding_backward` with
accumulate).  The search takes the best continuations of each prompt's beams
(`VocabOps.beam_step`), lets the beams' hidden states and token histories follow
(`VocabOps.beam_reorder`) and looks up the chosen tokens.

The data follows one rule, x_{t+1} = (5 x_t + 3) mod V, so that the program can say
whether it learned and searched it right.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

V, D, SCALE = 97, 64, 8.0


def follow(x, n):
    """The n tokens after x by the rule, [len(x), n]."""
    out = []
    for _ in range(n):
        x = (5 * x + 3) % V
        out.append(x)
    return torch.stack(out, 1)


def states_of(emb):
    """h_t = h_{t-1} / 2 + e_t over [B, T, D]."""
    h = torch.zeros_like(emb)
    prev = 0.0
    for t in range(emb.shape[1]):
        prev = prev / 2 + emb[:, t]
        h[:, t] = prev
    return h


def states_backward(dh):
    """The gradient of the embeddings from that of the states."""
    de = torch.zeros_like(dh)
    later = 0.0
    for t in reversed(range(dh.shape[1])):
        later = later / 2 + dh[:, t]
        de[:, t] = later
    return de


def train(ops, loss, W, A, steps, batch=16, length=24, seed=0):
    """Adam on W [V, D] and A [D, D] in fp32; the passes in bf16.  Returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.Adam([W, A], lr=0.01)
    W.grad, A.grad = torch.zeros_like(W), torch.zeros_like(A)
    losses = []
    for _ in range(steps):
        first = torch.randint(0, V, (batch,), device="cuda", generator=gen)
        x = torch.cat([first[:, None], follow(first, length)], 1)
        inputs, targets = x[:, :-1].contiguous(), x[:, 1:].contiguous()
        # forward
        Wb, Ab = W.bfloat16(), A.bfloat16()
        emb = ops.embedding_forward(W, inputs, scale=SCALE, out_dtype=torch.bfloat16)
        h = states_of(emb).view(-1, D)
        y = h @ Ab
        logits = y @ Wb.t()
        out = loss.forward_backward(logits, targets.view(-1), grad="inplace")
        # backward: the head's part of W's gradient, then the embedding's on top
        dz = out.grad
        dy = dz @ Wb
        W.grad.copy_(dz.t() @ y)
        A.grad.copy_(h.t() @ dy)
        demb = states_backward((dy @ Ab.t()).view_as(emb))
        ops.embedding_backward(demb, inputs, W.grad, scale=SCALE, accumulate=True)
        opt.step()
        losses.append(out.loss[0])
    return torch.stack(losses).tolist()


def search(ops, W, A, prompts, beams, steps):
    """Beam search from one token a prompt.  Returns (tokens [B, beams, steps], scores [B, beams])."""
    B = prompts.numel()
    Wb, Ab = W.bfloat16(), A.bfloat16()
    tokens = torch.zeros(B * beams, steps, dtype=torch.int64, device="cuda")
    history, spare_history = tokens, torch.zeros_like(tokens)
    last = prompts.repeat_interleave(beams)
    h = torch.zeros(B * beams, D, dtype=torch.bfloat16, device="cuda")
    spare_h = torch.zeros_like(h)
    # one beam is alive to begin with, so that the first step does not pick one token K times
    scores = torch.full((B, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0
    for t in range(steps):
        h = h / 2 + ops.embedding_forward(W, last, scale=SCALE, out_dtype=torch.bfloat16)
        step = ops.beam_step(h @ Ab @ Wb.t(), scores)
        # what each new beam goes on from: its state, and its tokens so far
        ops.beam_reorder([h, history], step.parents, out=[spare_h, spare_history])
        h, spare_h = spare_h, h
        history, spare_history = spare_history, history
        last = step.tokens.view(-1)
        history[:, t] = last
        scores = step.scores
    return history.view(B, beams, steps), scores


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=300, help="training steps")
    ap.add_argument("--beams", type=int, default=4)
    a = ap.parse_args(argv)
    from lm_head_vocab_gb300 import LMLoss, VocabOps
    gen = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(V, D, device="cuda", generator=gen) * 0.05
    A = torch.randn(D, D, device="cuda", generator=gen) * 0.05
    ops, loss = VocabOps(0, max_tokens=4096, max_dim=D, max_rows=256, max_vocab=V), LMLoss(0, max_T=4096, max_segments=1)
    losses = train(ops, loss, W, A, a.steps)
    prompts = torch.arange(0, V, 7, device="cuda")
    tokens, scores = search(ops, W, A, prompts, a.beams, 12)
    want = follow(prompts, 12)
    right = (tokens[:, 0] == want).float().mean().item()
    errors = (ops.device_error(), loss.device_error())
    ops.close()
    loss.close()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} over {a.steps} steps; best beams follow the rule in "
          f"{100 * right:.1f}% of {want.numel()} tokens; their mean score {scores[:, 0].mean().item():.2f}")
    return losses, right, errors


if __name__ == "__main__":
    main()
