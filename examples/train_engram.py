"""Trains a small model around one Engram layer by gradient descent.

    python examples/train_engram.py [steps]

The tiny workload's geometry (2 branches x 256, 6 buckets of 32-wide rows) with
a BF16 table; tokens repeat in phrases, so that the n-gram rows have something
to learn.  Every step runs the library's training operators and updates the
token embedding, the head, the norm weights, wkv and the n-gram rows that the
step touched.  Prints the loss, which falls.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import engram_gram_conditional_gb300 as eg  # noqa: E402
import synth  # noqa: E402
from engram_gram_conditional_gb300.layer import EngramLayerSet  # noqa: E402
from engram_gram_conditional_gb300.training import TrainStep  # noqa: E402


def phrases(w, T, seed):
    """Token ids made of a few phrases in random order."""
    g = np.random.default_rng(seed)
    book = g.integers(0, w.vocab, (8, 6))
    return book[g.integers(0, 8, T // 6 + 2)].reshape(-1)[:T + 1].astype(np.int32)


def run(steps=30, T=300, lr=0.5, seed=0):
    w = synth.WORKLOADS["tiny"]
    model = EngramLayerSet.from_workload(w, synth.token_map(w.vocab, w.vc, w.seed))
    wkv, (wq, wk) = synth.wkv_bf16(w), synth.wq_wk(w)
    kept = model.bind(0, w.table_seeds[0], wkv, wq, wk, flags=eg.BIND_TABLE_BF16)
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda s: (torch.randn(w.vocab, w.d, generator=g, device="cuda") * s).bfloat16()  # noqa: E731
    embedding, head = new(w.d ** -0.5), new(w.d ** -0.5)
    step = TrainStep(model, 0, embedding, head, T)
    tokens = phrases(w, T, seed)
    session = eg.engram_session_create(model.ctx)
    windows = eg.engram_session_append(session, tokens[:-1])
    eg.engram_session_destroy(session)
    ids = torch.from_numpy(tokens[:-1].copy()).cuda()
    labels = torch.from_numpy(tokens[1:].copy()).cuda()
    win = torch.from_numpy(windows.view(np.int32)).cuda()
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    table = kept["table"].view(torch.bfloat16)[:model.rows(0) * w.row_dim].view(-1, w.row_dim)

    def update(p, grad, rate):
        p.copy_((p.float() - rate * grad.float()).to(p.dtype))

    losses = []
    stream = torch.cuda.current_stream()
    for _ in range(steps):
        losses.append(float(step.forward(ids, win, labels, stream).mean()))
        step.backward(ids, win, labels, dloss, stream)
        eg.engram_sync(model.ctx, stream)
        n, r = int(step.token_count), int(step.row_count)
        at = step.token_ids[:n].long()
        embedding[at] = (embedding[at].float() - lr / w.d * step.token_grad[:n]).bfloat16()
        rows = step.row_ids[:r].long()
        table[rows] = (table[rows].float() - lr * step.row_grad[:r]).bfloat16()
        update(head, step.dhead, lr)
        update(kept["wkv"].view(torch.bfloat16), step.dwkv, lr * 1e-6)
        update(kept["wq"], step.dwq.view(-1), lr * 1e-2)
        update(kept["wk"], step.dwk.view(-1), lr * 1e-2)
        # the norm weights' product and the bind-time scans follow the weights
        eg.engram_layer_bind(model.ctx, 0, kept["table"], None, model.rows(0), kept["wkv"], kept["wq"],
                             kept["wk"], eg.BIND_TABLE_BF16)
    model.close()
    return losses


if __name__ == "__main__":
    from engram_gram_conditional_gb300 import build

    build.build()
    for i, x in enumerate(run(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print(f"step {i}: loss {x:.4f}")
