"""A training step of a small mixture of experts on R virtual ranks, from the
tokens to the update: tokens become rows of an embedding table, a router sends
each to its experts, whose products are grouped by expert, and the table, shared
with the output layer, meets the result in the cross entropy.  Back the same
way; the table's and the router's gradients are summed over the ranks by an
AllReduce.  The experts' matrices take an orthogonalised update, everything else
an AdamW step with states in 8 bits.

(The experts see the tokens of all ranks, so that their gradients are sums over
the ranks already.  A token's result is the mean of its experts'.)

    python examples/experts_step.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import double_binary_tree_gb300 as vr  # noqa: E402

R, TOKENS, DIM, INNER, VOCAB, EXPERTS, TOPK = 4, 256, 256, 512, 2000, 16, 2
ROWS = R * TOKENS * TOPK  # of the experts' products, the ignored tokens' last
SCALE = 8.0               # of the embedded tokens
IGNORE = -100
B16, BF = torch.bfloat16, vr.VR_BFLOAT16


def workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


class Step:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.steps = g, 0

        def weight(*shape, scale):
            return scale * torch.randn(*shape, generator=g, device="cuda")

        # what AdamW updates: 32-bit copies, their rounded values, 8-bit states
        self.masters = [weight(VOCAB, DIM, scale=1.0 / SCALE), weight(EXPERTS, DIM, scale=0.05)]
        self.table, self.router = self.params = [w.to(B16) for w in self.masters]
        self.sizes = [w.numel() for w in self.masters]
        self.m, self.v = ([torch.zeros(n, dtype=torch.uint8, device="cuda") for n in self.sizes]
                          for _ in range(2))
        self.ms, self.vs = ([torch.zeros(-(-n // 256), device="cuda") for n in self.sizes]
                            for _ in range(2))
        # the experts' matrices, and their momentum
        self.up = weight(EXPERTS, INNER, DIM, scale=DIM ** -0.5).to(B16)
        self.down = weight(EXPERTS, DIM, INNER, scale=INNER ** -0.5).to(B16)
        self.momentum = [torch.zeros_like(w) for w in (self.up, self.down)]
        # what follows what: each token has one likely successor
        self.next = torch.randperm(VOCAB, generator=g, device="cuda")
        # workspaces, kept for all steps
        x, y = (torch.empty(ROWS, n, device="cuda", dtype=B16) for n in (DIM, INNER))
        h = torch.empty(TOKENS, DIM, device="cuda", dtype=B16)
        self.work = {
            "xent": vr.vr_linear_xent_workspace_bytes(h, DIM, self.table, DIM, TOKENS, DIM, VOCAB,
                                                      BF, 1),
            "balance": vr.vr_balance_loss_workspace_bytes(R, TOKENS, EXPERTS),
            "up": vr.vr_grouped_linear_workspace_bytes(x, DIM, self.up, ROWS, DIM, INNER, EXPERTS,
                                                       BF),
            "down": vr.vr_grouped_linear_workspace_bytes(y, INNER, self.down, ROWS, INNER, DIM,
                                                         EXPERTS, BF),
            "up grad": vr.vr_grouped_linear_grad_workspace_bytes(y, INNER, x, DIM, self.up, ROWS,
                                                                 DIM, INNER, EXPERTS, BF),
            "down grad": vr.vr_grouped_linear_grad_workspace_bytes(x, DIM, y, INNER, self.down,
                                                                   ROWS, INNER, DIM, EXPERTS, BF),
            "embed": vr.vr_embedding_grad_workspace_bytes(TOKENS, DIM, VOCAB, BF),
            "ortho": vr.vr_orthogonalize_workspace_bytes(EXPERTS, INNER, DIM, BF),
        }
        self.work = {k: (workspace(n), n) for k, n in self.work.items()}

    def batch(self):
        """R ranks' tokens and their successors; the last tokens are padding."""
        tokens = torch.randint(0, VOCAB, (R, TOKENS), generator=self.g, device="cuda")
        targets = self.next[tokens]
        tokens[:, -8:] = targets[:, -8:] = IGNORE
        return tokens, targets

    def linear(self, name, x, w, counts, out, inner, outer):
        vr.vr_grouped_linear(x, inner, w, counts, ROWS, inner, outer, EXPERTS, BF, out, outer,
                             *self.work[name], torch.cuda.current_stream())
        return out

    def linear_grad(self, name, dout, x, w, counts, inner, outer):
        dx, dw = torch.zeros(ROWS, inner, device="cuda", dtype=B16), torch.empty_like(w)
        vr.vr_grouped_linear_grad(dout, outer, x, inner, w, counts, ROWS, inner, outer, EXPERTS, BF,
                                  dx, dw, *self.work[name], torch.cuda.current_stream())
        return dx, dw

    def allreduce(self, bufs):
        """The ranks' gradients summed, in place."""
        vr.vr_allreduce(bufs, bufs, R, bufs[0].numel(), BF, vr.VR_SUM, vr.VR_ALGO_AUTO, 12,
                        512 * 1024, torch.cuda.current_stream())

    def gradients(self, tokens, targets, coef=0.01):
        """Losses, the tokens of each expert, and the gradients of table, router,
        up and down."""
        stream = torch.cuda.current_stream()
        counted = int((targets >= 0).sum())
        h = torch.empty(R, TOKENS, DIM, device="cuda", dtype=B16)
        for r in range(R):
            vr.vr_embedding(self.table, DIM, tokens[r], TOKENS, DIM, VOCAB, BF, IGNORE, SCALE, h[r],
                            DIM, stream)

        # the router's choice, and its balance loss over the whole batch
        logits = [(h[r] @ self.router.t()).contiguous() for r in range(R)]
        masks = [(targets[r] >= 0).to(torch.uint8) for r in range(R)]
        balance = torch.empty(1, device="cuda")
        counts = torch.empty(EXPERTS, device="cuda", dtype=torch.int32)
        chosen = torch.empty(R, TOKENS, TOPK, device="cuda", dtype=torch.int32)
        dlogits = [torch.empty_like(z) for z in logits]
        vr.vr_balance_loss(logits, EXPERTS, masks, R, TOKENS, EXPERTS, TOPK, BF, coef, 1.0, balance,
                           counts, list(chosen), dlogits, *self.work["balance"], stream)

        # rows by expert; those of ignored tokens, which chose none, come last
        order = torch.argsort(torch.where(chosen < 0, EXPERTS, chosen).reshape(-1), stable=True)
        token = order // TOPK
        flat = h.view(R * TOKENS, DIM)
        x = flat[token]
        y = self.linear("up", x, self.up, counts,
                        torch.zeros(ROWS, INNER, device="cuda", dtype=B16), DIM, INNER)
        a = y.relu()
        z = self.linear("down", a, self.down, counts,
                        torch.zeros(ROWS, DIM, device="cuda", dtype=B16), INNER, DIM)
        last = flat.float().index_add(0, token, z.float() / TOPK).to(B16).view(R, TOKENS, DIM)

        # the cross entropy of each rank's tokens with the table as output layer
        losses, dtable, dlast = [], [], torch.empty_like(h)
        for r in range(R):
            loss = torch.empty(1, device="cuda")
            per_token, lse = (torch.empty(TOKENS, device="cuda") for _ in range(2))
            dtable.append(torch.empty_like(self.table))
            vr.vr_linear_xent(last[r], DIM, self.table, DIM, targets[r], TOKENS, DIM, VOCAB, BF,
                              IGNORE, False, 1.0 / counted, per_token, lse, loss, dlast[r],
                              dtable[r], *self.work["xent"], stream)
            losses.append(loss / counted)

        # back through the experts
        dflat = dlast.view(R * TOKENS, DIM)
        dz = (dflat[token].float() / TOPK).to(B16)
        da, ddown = self.linear_grad("down grad", dz, a, self.down, counts, INNER, DIM)
        dy = da * (y > 0)
        dx, dup = self.linear_grad("up grad", dy, x, self.up, counts, DIM, INNER)
        dh = dflat.float().index_add(0, token, dx.float()).view(R, TOKENS, DIM)
        dh = torch.stack([dh[r] + (dlogits[r] @ self.router).float() for r in range(R)]).to(B16)

        # the table's gradient as embedding beside the one as output layer
        for r in range(R):
            vr.vr_embedding_grad(dh[r], DIM, tokens[r], TOKENS, DIM, VOCAB, BF, IGNORE, SCALE, True,
                                 dtable[r], *self.work["embed"], stream)
        drouter = [(dlogits[r].t() @ h[r]).contiguous() for r in range(R)]
        for bufs in (dtable, drouter):
            self.allreduce(bufs)
        return float(sum(losses)), float(balance), counts, (dtable[0], drouter[0], dup, ddown)

    def update(self, grads, lr=0.01, expert_lr=0.02):
        stream = torch.cuda.current_stream()
        self.steps += 1
        dtable, drouter, dup, ddown = grads
        vr.vr_adamw(self.params, [dtable, drouter], self.m, self.v, self.ms, self.vs, self.masters,
                    self.sizes, 2, BF, BF, 8, lr, 0.9, 0.99, 1e-8, 0.01, self.steps, 1.0, 17, None,
                    stream)
        for w, momentum, g in zip((self.up, self.down), self.momentum, (dup, ddown)):
            momentum.mul_(0.9).add_(g)
            step = torch.empty_like(w)
            vr.vr_orthogonalize(list(momentum), list(step), EXPERTS, w.shape[1], w.shape[2], BF, 5,
                                None, 1e-7, expert_lr, *self.work["ortho"], stream)
            w -= step

    def run(self):
        loss, balance, counts, grads = self.gradients(*self.batch())
        self.update(grads)
        return loss, balance, counts.tolist()


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
