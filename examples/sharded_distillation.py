"""Distillation of a small language model over p logical ranks.

The teacher writes the text: its logits, sharded over the ranks by vocabulary,
are penalised for what a text already has and masked, and the likeliest entry
is taken.  The student then learns the teacher's likeliest entries at every
position, data parallel up to the last hidden rows and tensor parallel over the
vocabulary:

    x, x W -> RMS norm of x + x W -> (in 8 bits) AllGather -> logits of the own
      shard -> loss against the teacher's entries

and back: the logits' gradient in place, a ReduceScatter of the partial hidden
gradients, the RMS norm's backward pass (whose weight gradient is reduced over
the ranks inside it) and an AllReduce of W's gradient.  The matrix products are
torch.matmul; everything between them is this library.

    python examples/sharded_distillation.py --steps 30
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import collective_communication_primitives_coll_amd as coll  # noqa: E402


class ShardedDistillation:
    def __init__(self, p=4, rows=64, hidden=256, vocab=2000, top=16, temp=2.0, group=64, fp8=True, seed=0, device="cuda"):
        self.p, self.rows, self.hidden, self.vocab, self.top, self.temp = p, rows, hidden, vocab, top, temp
        self.group, self.fp8, self.device = group, fp8, device
        g = torch.Generator().manual_seed(seed)
        f32, bf, u8, i32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32

        def normal(*shape, scale=1.0, dtype=f32):
            return (torch.randn(*shape, generator=g) * scale).to(device=device, dtype=dtype)

        def like(shape, dtype=bf):
            return [torch.empty(shape, device=device, dtype=dtype) for _ in range(p)]

        cut = [vocab * r // p for r in range(p + 1)]
        self.sizes = [b - a for a, b in zip(cut, cut[1:])]
        self.teacher = dict(embedding=normal(vocab, hidden, dtype=bf), out=[normal(hidden, n, scale=2 * hidden ** -0.5, dtype=bf) for n in self.sizes])
        w = normal(hidden, hidden, scale=hidden ** -0.5)
        # fp32 weights, a replica per rank (the output weights: a shard); the products use bf16 copies
        self.w = dict(gamma=[torch.ones(hidden, device=device) for _ in range(p)], w=[w.clone() for _ in range(p)],
                      out=[normal(hidden, n, scale=hidden ** -0.5) for n in self.sizes])
        self.embedding = normal(vocab, hidden, dtype=bf)
        self.grad = {k: [torch.empty_like(t) for t in v] for k, v in self.w.items()}
        all_rows = p * rows
        self.h, self.y, self.dy, self.dw = like((rows, hidden)), like((rows, hidden)), like((rows, hidden)), like((hidden, hidden))
        self.all_y, self.rstd = like((all_rows, hidden)), like(rows, f32)
        row_bytes = coll.coll_ckpt8_row_bytes(hidden, group)
        self.y8, self.all_y8 = like((rows, row_bytes), u8), like((all_rows, row_bytes), u8)
        self.stats, self.loss = like((all_rows, 4), f32), like(all_rows, f32)
        self.t_stats, self.t_logp = like((all_rows, 2), f32), like(all_rows, f32)
        self.t_top, self.t_idx = like((all_rows, top), f32), like((all_rows, top), i32)
        byte = lambda n: torch.empty(n, device=device, dtype=u8)  # noqa: E731
        self.ws_norm = byte(coll.coll_rmsnorm_workspace_bytes(p, rows, hidden))
        self.ws_loss = byte(coll.coll_vocab_distill_workspace_bytes(all_rows, self.sizes, top))
        self.ws_top = byte(coll.coll_vocab_logprob_workspace_bytes(all_rows, self.sizes, top))
        self.given = torch.zeros(all_rows, device=device, dtype=torch.int64)  # no given tokens: alternatives only
        self.dloss = torch.full((all_rows,), temp ** 2 / all_rows, device=device)

    def teacher_logits(self, tokens):
        rows = self.teacher["embedding"][tokens]
        return [rows @ w for w in self.teacher["out"]]

    def teacher_entries(self, logits, n, inv_temp):
        """The n likeliest entries of every row, on every rank: log probabilities and indices."""
        rows = logits[0].shape[0]
        part = lambda ts, k: [t.flatten()[:rows * k].view(rows, k) for t in ts]  # noqa: E731
        top, idx = part(self.t_top, n), part(self.t_idx, n)
        coll.coll_vocab_logprob(logits, self.given[:rows], part(self.t_stats, 2), part(self.t_logp, 1), self.ws_top, top_k=n, top_logp=top,
                                top_idx=idx, inv_temp=inv_temp)
        return top, idx

    def write(self, first, length, allow):
        """Texts of `length` tokens from their first ones, int64 [texts]: the teacher's likeliest token among the allowed
        ones (truth values [vocab]), less likely the more often the text has it."""
        texts = first.numel()
        text = torch.empty(texts, length, dtype=torch.int64, device=self.device)
        text[:, 0] = first
        words = -(-self.vocab // 32)
        bits = torch.zeros(words * 32, dtype=torch.int64)
        bits[:self.vocab] = allow
        mask = (bits.view(words, 32) << torch.arange(32)).sum(1)
        mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(device=self.device, dtype=torch.int32).expand(texts, -1).contiguous()
        per = lambda v: torch.full((texts,), v, device=self.device)  # noqa: E731
        for n in range(1, length):
            logits = self.teacher_logits(text[:, n - 1])
            coll.coll_vocab_adjust(logits, logits, tokens=text[:, :n].contiguous(), offsets=torch.arange(0, texts * n + 1, n, device=self.device),
                                   prompt=torch.ones(texts, dtype=torch.int64, device=self.device), repetition=per(1.2), presence=per(1.0),
                                   frequency=per(0.5), mask=mask)
            text[:, n] = self.teacher_entries(logits, 1, 1.0)[1][0][:, 0]
        return text

    def forward_backward(self, tokens):
        """tokens[r]: int64 [rows].  Returns the mean loss; self.grad gets the gradients, self.dy the embeddings'."""
        p, h, w, grad = self.p, self.hidden, self.w, self.grad
        bf = {k: [t.bfloat16() for t in w[k]] for k in ("w", "out")}
        top, idx = self.teacher_entries(self.teacher_logits(torch.cat(tokens)), self.top, 1.0 / self.temp)
        x = [self.embedding[t] for t in tokens]
        step = [x[r] @ bf["w"][r] for r in range(p)]
        if self.fp8:
            # the rows travel in 8 bits (to the gradient they are what was encoded)
            coll.coll_rmsnorm_fp8(step, w["gamma"], self.y8, h, self.group, residual=x, h=self.h, rstd=self.rstd)
            coll.coll_allgather(self.y8, self.all_y8)
            coll.coll_ckpt8_load(self.all_y8, self.all_y, h, self.group)
        else:
            coll.coll_rmsnorm(step, w["gamma"], self.y, h, residual=x, h=self.h, rstd=self.rstd)
            coll.coll_allgather(self.y, self.all_y)
        logits = [self.all_y[r] @ bf["out"][r] for r in range(p)]
        coll.coll_vocab_distill(logits, idx[0], top[0], self.stats, self.loss, self.ws_loss, inv_temp=1.0 / self.temp)

        coll.coll_vocab_distill_backward(logits, idx[0], top[0], self.stats[0], self.dloss, logits, inv_temp=1.0 / self.temp)
        part = []
        for r in range(p):
            grad["out"][r].copy_(self.all_y[r].t() @ logits[r])
            part.append(logits[r] @ bf["out"][r].t())
        coll.coll_reduce_scatter(part, self.dy)
        # in place: the gradient of x + x W takes the place of the norm's output's
        coll.coll_rmsnorm_backward(self.dy, self.h, self.rstd, w["gamma"], self.dy, grad["gamma"], self.ws_norm, h)
        for r in range(p):
            grad["w"][r].copy_(x[r].t() @ self.dy[r])
            self.dy[r].addmm_(self.dy[r].clone(), bf["w"][r].t())
        coll.coll_allreduce(grad["w"], grad["w"], coll.COLL_SUM)
        return self.loss[0].mean()

    def update(self, lr):
        for k, g in self.grad.items():
            for wt, gt in zip(self.w[k], g):
                wt.sub_(gt, alpha=lr)


def train(steps, lr=2.0, length=32, seed=0, log=print, **sizes):
    m = ShardedDistillation(seed=seed, **sizes)
    g = torch.Generator().manual_seed(seed + 1)
    allow = torch.ones(m.vocab, dtype=torch.bool)
    allow[:10] = False  # what no text may have
    losses = []
    for s in range(steps):
        texts = -(-m.p * m.rows // length)
        text = m.write(torch.randint(10, m.vocab, (texts,), generator=g).to(m.device), length, allow).flatten()[:m.p * m.rows]
        losses.append(float(m.forward_backward(list(text.view(m.p, m.rows)))))
        m.update(lr)
        if log and (s % 10 == 0 or s == steps - 1):
            log(f"step {s}: loss {losses[-1]:.4f}", flush=True)
    return m, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args()
    train(a.steps, a.lr, p=a.ranks)
