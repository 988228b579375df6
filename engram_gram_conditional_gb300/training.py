"""One training step of a model around an Engram layer.

Token embedding -> hyper-connection branches -> Engram layer -> mean of the
branches -> output head -> cross entropy, and back, through the library's
operators:

  engram_embed              branches from the token embedding
  engram_hash, engram_gather_dequant, engram_prepass
                            rows, their 6,144-vectors, kv
  engram_gate_checkpoint    the gate, its activations kept in 8 bits
  engram_loss               loss and lse, no logits
  engram_loss_backward      gradients of the head and of its input
  engram_gate_backward_checkpoint, engram_project_backward
                            gradients of the norm weights, wkv and the rows
  engram_embed_grad         gradients of the token embedding and the n-gram table,
                            summed over equal ids

torch only allocates, and takes the mean of the branches and its transpose (the
model around the layer).
"""
from __future__ import annotations

import math

import torch

from . import (EMBED_BF16, KV_BF16, KV_F32, engram_embed, engram_embed_grad,
               engram_embed_grad_workspace_bytes, engram_forward_staged_workspace_bytes,
               engram_gate_backward_checkpoint, engram_gate_backward_workspace_bytes,
               engram_gate_checkpoint, engram_gather_dequant, engram_hash, engram_loss,
               engram_loss_backward, engram_loss_backward_workspace_bytes,
               engram_loss_workspace_bytes, engram_prepass, engram_project_backward,
               engram_project_backward_workspace_bytes)


class TrainStep:
    """Buffers and calls of one step for up to ``tokens`` tokens.

    ``model``: an EngramLayerSet with ``layer`` bound; ``embedding`` and ``head``:
    BF16 [vocab][d].  ``kv_format``: how kv waits for the gate (KV_F32 or KV_BF16).

    A step's number of tokens T is that of the ids which forward() is given; what
    the buffers hold past T tokens is left over from longer steps.

    ``stream`` of a call: a torch stream or a handle; None is torch's current one.
    All of a step, the library's calls and torch's alike, runs on it.
    """

    def __init__(self, model, layer: int, embedding, head, tokens: int, *, kv_format=KV_BF16,
                 scale=None):
        g = model.geom
        if tokens < 1:
            raise ValueError("tokens must be at least 1")
        for name, w in (("embedding", embedding), ("head", head)):
            self._check(name, w, 2, (embedding.shape[0], g["d"]), model.device)
        self.model, self.layer, self.embedding, self.head = model, layer, embedding, head
        self.vocab, self.d, self.hc = embedding.shape[0], g["d"], g["hc"]
        self.kv_format, self.scale = kv_format, math.sqrt(g["d"]) if scale is None else scale
        self.tokens = tokens
        self.T = 0  # tokens of the last forward()
        T, nb, K, N, kept = tokens, model.nb, model.K, model.N, (2 * self.hc + 1) * self.d
        bf16, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32

        def new(*shape, dtype=bf16):
            return torch.empty(*shape, dtype=dtype, device=model.device)

        self.hidden, self.out = new(T, self.hc, self.d), new(T, self.hc, self.d)
        self.rows, self.emb = new(T, nb, dtype=i32), new(T, K)
        self.kv = new(T, N, dtype=f32 if kv_format == KV_F32 else bf16)
        self.gates = new(T, self.hc, dtype=f32)
        self.codes, self.scales = new(T, kept, dtype=u8), new(T, kept // 32, dtype=u8)
        self.loss, self.lse = new(T, dtype=f32), new(T, dtype=f32)
        self.x, self.dx, self.dhead = new(T, self.d), new(T, self.d), new(self.vocab, self.d)
        self.dhidden, self.dkv = new(T, self.hc, self.d), new(T, N)
        self.dwq, self.dwk = new(self.hc, self.d, dtype=f32), new(self.hc, self.d, dtype=f32)
        self.demb, self.dwkv = new(T, K), new(N, K)
        self.token_ids, self.token_count = new(T, dtype=i32), new(1, dtype=i32)
        self.token_grad = new(T, self.d, dtype=f32)
        self.row_ids, self.row_count = new(T * nb, dtype=i32), new(1, dtype=i32)
        self.row_grad = new(T * nb, g["row_dim"], dtype=f32)
        ctx = model.ctx
        self.ws = new(max(engram_forward_staged_workspace_bytes(ctx, T),
                          engram_loss_workspace_bytes(T, self.vocab, self.d),
                          engram_loss_backward_workspace_bytes(T, self.vocab, self.d),
                          engram_gate_backward_workspace_bytes(ctx, T),
                          engram_project_backward_workspace_bytes(ctx, T),
                          engram_embed_grad_workspace_bytes(T, self.vocab, self.d),
                          engram_embed_grad_workspace_bytes(T * nb, model.rows(layer),
                                                            g["row_dim"]), 16), dtype=u8)
        # a step may run on another stream than the one whose freed memory this is
        torch.cuda.current_stream(model.device).synchronize()

    def _on(self, stream):
        if stream is None:
            return torch.cuda.current_stream(self.model.device)
        if isinstance(stream, int):
            return (torch.cuda.ExternalStream(stream, self.model.device) if stream else
                    torch.cuda.default_stream(self.model.device))
        return stream

    @staticmethod
    def _check(name, x, size, shape, device):
        """The kernels read as far as the shapes say: a tensor of another number of values, or of
        values that do not have `size` bytes, is refused."""
        if x.element_size() != size or x.numel() != math.prod(shape) or not x.is_contiguous():
            raise ValueError(f"{name}: {list(shape)} of {size} bytes each, contiguous, expected; "
                             f"got {x.dtype} {list(x.shape)}")
        if x.device.type != device.type or (device.index is not None and x.device.index != device.index):
            raise ValueError(f"{name}: on {x.device}, the model is on {device}")

    def _check_step(self, ids, windows, labels, T):
        for name, x, shape in (("ids", ids, (T,)), ("windows", windows, (T, 4)), ("labels", labels, (T,))):
            self._check(name, x, 4, shape, self.model.device)

    def forward(self, ids, windows, labels, stream=None):
        """Loss of each token (fp32 [T]); ids and labels int32 [T], windows int32 [T][4] (an
        image row has slot 0 DEAD), all on the device, T at most ``tokens``."""
        ctx, layer, T = self.model.ctx, self.layer, ids.numel()
        if not 0 < T <= self.tokens:
            raise ValueError(f"{T} tokens: 1 to {self.tokens} are possible")
        self._check_step(ids, windows, labels, T)
        self.T, stream = T, self._on(stream)
        engram_embed(ctx, self.embedding, EMBED_BF16, self.vocab, self.d, ids, T, self.scale, self.hc,
                     self.hidden, stream)
        engram_hash(ctx, layer, windows, T, self.rows, stream)
        engram_gather_dequant(ctx, layer, self.rows, T, self.emb, stream)
        engram_prepass(ctx, layer, windows, T, self.kv, self.kv_format, self.ws, stream)
        engram_gate_checkpoint(ctx, layer, self.kv, self.kv_format, windows, T, self.hidden, self.out,
                               self.gates, self.codes, self.scales, stream)
        with torch.cuda.stream(stream):
            self.x[:T] = self.out[:T].float().mean(1)
        engram_loss(ctx, self.x, self.head, self.vocab, self.d, labels, T, self.loss, self.lse, self.ws,
                    stream)
        return self.loss[:T]

    def backward(self, ids, windows, labels, dloss, stream=None):
        """Gradients of sum(dloss * loss) (dloss fp32 [T]) into this object's buffers: dhead, dwq,
        dwk, dwkv, and the sparse token_ids/token_grad and row_ids/row_grad with their counts.
        ids, windows and labels are those of the forward() before."""
        ctx, layer, T = self.model.ctx, self.layer, self.T
        if T == 0:
            raise ValueError("no forward() to go back through")
        self._check_step(ids, windows, labels, T)
        self._check("dloss", dloss, 4, (T,), self.model.device)
        stream = self._on(stream)
        engram_loss_backward(ctx, self.x, self.head, self.vocab, self.d, labels, T, self.lse, dloss,
                             self.dx, self.dhead, self.ws, stream)
        with torch.cuda.stream(stream):  # the mean's gradient; the gate's call replaces it in place
            self.dhidden[:T] = (self.dx[:T].float() / self.hc).unsqueeze(1)
        engram_gate_backward_checkpoint(ctx, layer, self.codes, self.scales, windows, T, self.dhidden,
                                        self.dhidden, self.dkv, self.dwq, self.dwk, self.ws, stream)
        engram_project_backward(ctx, layer, self.emb, self.dkv, T, self.demb, self.dwkv, self.ws, stream)
        engram_embed_grad(ctx, self.vocab, self.d, ids, T, self.scale, self.hc, self.dhidden,
                          self.token_ids, self.token_count, self.token_grad, 0, self.ws, stream)
        row_dim = self.model.geom["row_dim"]
        engram_embed_grad(ctx, self.model.rows(layer), row_dim, self.rows, T * self.model.nb, 1.0, 1,
                          self.demb, self.row_ids, self.row_count, self.row_grad, 0, self.ws, stream)
