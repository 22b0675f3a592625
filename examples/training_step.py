"""A data-parallel training step of R virtual ranks, from the losses to the
update: every rank computes the cross entropy of its own tokens and its
gradients, the balance loss of all ranks' expert routers comes with its
gradients, the gradients are summed over the ranks by an AllReduce, and the
hidden matrix takes an orthogonalised update.

A little language model: tokens are embedded, each of `layers` hidden
matrices adds what it makes of the state, the last state meets the vocabulary.
(The experts themselves are left out: the router learns to spread its tokens.)

    python examples/training_step.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import double_binary_tree_gb300 as vr  # noqa: E402

R, TOKENS, DIM, VOCAB, EXPERTS, TOPK = 4, 256, 256, 2000, 16, 2
B16 = torch.bfloat16


def workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


class Step:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(rows, cols, scale):
            return (scale * torch.randn(rows, cols, generator=g, device="cuda")).to(B16)

        self.g = g
        # a direction that all tokens share, and the router's first expert likes
        common = torch.randn(DIM, generator=g, device="cuda")
        self.embed = (weight(VOCAB, DIM, 1.0) + 0.5 * common).to(B16)
        self.hidden = weight(DIM, DIM, 0.02)
        self.head = weight(VOCAB, DIM, DIM ** -0.5)
        self.router = weight(EXPERTS, DIM, 0.2)
        self.router[0] += (0.03 * common).to(B16)
        self.momentum = torch.zeros(DIM, DIM, device="cuda")
        # what follows what: each token has one likely successor
        self.next = torch.randperm(VOCAB, generator=g, device="cuda")
        # workspaces and buffers, kept for all steps
        x = torch.empty(TOKENS, DIM, device="cuda", dtype=B16)
        self.xent_bytes = vr.vr_linear_xent_workspace_bytes(x, DIM, self.head, DIM, TOKENS, DIM,
                                                            VOCAB, vr.VR_BFLOAT16, 1)
        self.xent_work = workspace(self.xent_bytes)
        self.balance_bytes = vr.vr_balance_loss_workspace_bytes(R, TOKENS, EXPERTS)
        self.balance_work = workspace(self.balance_bytes)
        self.ortho_bytes = vr.vr_orthogonalize_workspace_bytes(1, DIM, DIM, vr.VR_BFLOAT16)
        self.ortho_work = workspace(self.ortho_bytes)

    def batch(self):
        """R ranks' tokens and their successors; the last tokens are padding."""
        tokens = torch.randint(0, VOCAB, (R, TOKENS), generator=self.g, device="cuda")
        targets = self.next[tokens]
        targets[:, -8:] = -100
        return tokens, targets

    def allreduce(self, bufs):
        """The ranks' gradients summed, in place."""
        n = bufs[0].numel()
        vr.vr_allreduce(bufs, bufs, R, n, vr.VR_BFLOAT16, vr.VR_SUM, vr.VR_ALGO_AUTO, 12,
                        512 * 1024, torch.cuda.current_stream())

    def run(self, lr=0.02, head_lr=4.0, router_lr=2.0, coef=0.01):
        stream = torch.cuda.current_stream()
        tokens, targets = self.batch()
        counted = int((targets >= 0).sum())
        x = [self.embed[tokens[r]] for r in range(R)]
        h = [xr + xr @ self.hidden.t() for xr in x]

        # the cross entropy of each rank's tokens: the loss of the whole batch is
        # their sum over all tokens that count
        losses, grads_h, grads_head = [], [], []
        for r in range(R):
            loss = torch.empty(1, device="cuda")
            per_token, lse = (torch.empty(TOKENS, device="cuda") for _ in range(2))
            dh, dw = torch.empty_like(h[r]), torch.empty_like(self.head)
            vr.vr_linear_xent(h[r], DIM, self.head, DIM, targets[r].contiguous(), TOKENS, DIM,
                              VOCAB, vr.VR_BFLOAT16, -100, False, 1.0 / counted, per_token, lse,
                              loss, dh, dw, self.xent_work, self.xent_bytes, stream)
            losses.append(loss / counted)
            grads_h.append(dh)
            grads_head.append(dw)

        # the balance loss of all ranks' routers over the whole batch
        logits = [(hr @ self.router.t()).contiguous() for hr in h]
        masks = [(targets[r] >= 0).to(torch.uint8) for r in range(R)]
        balance = torch.empty(1, device="cuda")
        counts = torch.empty(EXPERTS, device="cuda", dtype=torch.int32)
        dlogits = [torch.empty_like(z) for z in logits]
        vr.vr_balance_loss(logits, EXPERTS, masks, R, TOKENS, EXPERTS, TOPK, vr.VR_BFLOAT16, coef,
                           1.0, balance, counts, None, dlogits, self.balance_work,
                           self.balance_bytes, stream)
        grads_router = [dz.t() @ hr for dz, hr in zip(dlogits, h)]

        # each rank's share of the gradients, then their sum on every rank
        grads_hidden = [(dh.t() @ xr).contiguous() for dh, xr in zip(grads_h, x)]
        for bufs in (grads_head, grads_hidden, grads_router):
            self.allreduce(bufs)

        # the update: momentum orthogonalised for the hidden matrix, plain steps else
        self.momentum.mul_(0.9).add_(grads_hidden[0].float())
        update = self.momentum.to(B16)
        vr.vr_orthogonalize([update], [update], 1, DIM, DIM, vr.VR_BFLOAT16, 5, None, 1e-7, lr,
                            self.ortho_work, self.ortho_bytes, stream)
        self.hidden -= update
        self.head -= head_lr * grads_head[0]
        self.router -= router_lr * grads_router[0]
        return float(sum(losses)), float(balance), counts.tolist()


def main(steps=40):
    step = Step()
    history = []
    for i in range(steps):
        loss, balance, counts = step.run()
        history.append((loss, balance))
        if i % 10 == 0 or i + 1 == steps:
            print("step %3d: cross entropy %.4f, balance %.5f, tokens per expert %d to %d"
                  % (i, loss, balance, min(counts), max(counts)))
    status = vr.vr_stream_status(torch.cuda.current_stream())
    if status:
        raise RuntimeError("device status %d" % status)
    return history


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
