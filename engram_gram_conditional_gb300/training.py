"""One training step of a model around an Engram layer, and the update of its weights.

Token embedding -> hyper-connection branches -> Engram layer -> mean of the
branches (-> norm) -> output head -> cross entropy, and back, through the
library's operators:

  engram_embed              branches from the token embedding
  engram_hash, engram_gather_dequant, engram_prepass
                            rows, their 6,144-vectors, kv
  engram_gate_checkpoint    the gate, its activations kept in 8 bits
  engram_norm, engram_norm_backward
                            with norm weights: mean and root-mean-square norm in one
  engram_loss               loss and lse, no logits
  engram_loss_backward      gradients of the head and of its input
  engram_gate_backward_checkpoint, engram_project_backward
                            gradients of the norm weights, wkv and the rows
  engram_embed_grad         gradients of the token embedding and the n-gram table,
                            summed over equal ids
  engram_grad_norm, engram_adamw, engram_adamw_rows
                            AdamW: the gradients' norm, the update of the weights and of
                            the rows that have a gradient

torch only allocates, and, without norm weights, takes the mean of the branches and
its transpose (the model around the layer).
"""
from __future__ import annotations

import math

import torch

from . import (BF16, EMBED_BF16, F32, KV_BF16, KV_F32, MXFP8, AdamWStep, AdamWTable, adamw_tensors,
               engram_adamw, engram_adamw_rows, engram_embed, engram_embed_grad,
               engram_embed_grad_workspace_bytes, engram_forward_staged_workspace_bytes,
               engram_gate_backward_checkpoint, engram_gate_backward_workspace_bytes,
               engram_gate_checkpoint, engram_gather_dequant, engram_grad_norm,
               engram_grad_norm_workspace_bytes, engram_hash, engram_loss, engram_loss_backward,
               engram_loss_backward_workspace_bytes, engram_loss_workspace_bytes, engram_norm,
               engram_norm_backward, engram_norm_backward_workspace_bytes, engram_prepass,
               engram_project_backward, engram_project_backward_workspace_bytes, grad_parts)


class TrainStep:
    """Buffers and calls of one step for up to ``tokens`` tokens.

    ``model``: an EngramLayerSet with ``layer`` bound; ``embedding`` and ``head``:
    BF16 [vocab][d].  ``kv_format``: how kv waits for the gate (KV_F32 or KV_BF16).
    ``norm``: fp32 [d], the weights of a root-mean-square norm between the mean of the
    branches and the head (epsilon: the model's), or None: the mean goes to the head.

    A step's number of tokens T is that of the ids which forward() is given; what
    the buffers hold past T tokens is left over from longer steps.

    ``stream`` of a call: a torch stream or a handle; None is torch's current one.
    All of a step, the library's calls and torch's alike, runs on it.
    """

    ready = False  # whether the gradients are those of the last forward()

    def __init__(self, model, layer: int, embedding, head, tokens: int, *, kv_format=KV_BF16,
                 scale=None, norm=None):
        g = model.geom
        if tokens < 1:
            raise ValueError("tokens must be at least 1")
        for name, w in (("embedding", embedding), ("head", head)):
            self._check(name, w, 2, (embedding.shape[0], g["d"]), model.device)
        if norm is not None:
            self._check("norm", norm, 4, (g["d"],), model.device)
        self.norm = norm
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
        if norm is not None:
            self.mean, self.dnorm = new(T, self.d), new(self.d, dtype=f32)
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
                          0 if norm is None else engram_norm_backward_workspace_bytes(T, self.d),
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
        if layer in self.model.outdated:
            raise ValueError("the layer's weights changed since it was bound: model.rebind(layer) first")
        self.T, self.ready, stream = T, False, self._on(stream)
        engram_embed(ctx, self.embedding, EMBED_BF16, self.vocab, self.d, ids, T, self.scale, self.hc,
                     self.hidden, stream)
        engram_hash(ctx, layer, windows, T, self.rows, stream)
        engram_gather_dequant(ctx, layer, self.rows, T, self.emb, stream)
        engram_prepass(ctx, layer, windows, T, self.kv, self.kv_format, self.ws, stream)
        engram_gate_checkpoint(ctx, layer, self.kv, self.kv_format, windows, T, self.hidden, self.out,
                               self.gates, self.codes, self.scales, stream)
        if self.norm is None:
            with torch.cuda.stream(stream):
                self.x[:T] = self.out[:T].float().mean(1)
        else:
            engram_norm(ctx, self.out, BF16, self.hc, 1 / self.hc, None, self.norm, T, self.d,
                        self.model.geom["eps"], self.mean, self.x, BF16, None, stream)
        engram_loss(ctx, self.x, self.head, self.vocab, self.d, labels, T, self.loss, self.lse, self.ws,
                    stream)
        return self.loss[:T]

    def backward(self, ids, windows, labels, dloss, stream=None):
        """Gradients of sum(dloss * loss) (dloss fp32 [T]) into this object's buffers: dhead, dwq,
        dwk, dwkv, dnorm (with norm weights), and the sparse token_ids/token_grad and row_ids/row_grad with their counts.
        ids, windows and labels are those of the forward() before."""
        ctx, layer, T = self.model.ctx, self.layer, self.T
        if T == 0:
            raise ValueError("no forward() to go back through")
        self._check_step(ids, windows, labels, T)
        self._check("dloss", dloss, 4, (T,), self.model.device)
        stream = self._on(stream)
        engram_loss_backward(ctx, self.x, self.head, self.vocab, self.d, labels, T, self.lse, dloss,
                             self.dx, self.dhead, self.ws, stream)
        # the mean's gradient; the gate's call replaces it in place
        if self.norm is None:
            with torch.cuda.stream(stream):
                self.dhidden[:T] = (self.dx[:T].float() / self.hc).unsqueeze(1)
        else:
            engram_norm_backward(ctx, self.mean, BF16, self.norm, T, self.d, self.model.geom["eps"],
                                 self.dx, None, self.hc, 1 / self.hc, self.dhidden, None, self.dnorm,
                                 self.ws, stream)
        engram_gate_backward_checkpoint(ctx, layer, self.codes, self.scales, windows, T, self.dhidden,
                                        self.dhidden, self.dkv, self.dwq, self.dwk, self.ws, stream)
        engram_project_backward(ctx, layer, self.emb, self.dkv, T, self.demb, self.dwkv, self.ws, stream)
        engram_embed_grad(ctx, self.vocab, self.d, ids, T, self.scale, self.hc, self.dhidden,
                          self.token_ids, self.token_count, self.token_grad, 0, self.ws, stream)
        row_dim = self.model.geom["row_dim"]
        engram_embed_grad(ctx, self.model.rows(layer), row_dim, self.rows, T * self.model.nb, 1.0, 1,
                          self.demb, self.row_ids, self.row_count, self.row_grad, 0, self.ws, stream)
        self.ready = True


class AdamW:
    """AdamW on the weights of a TrainStep, with the gradients that its backward() left: head, wkv,
    w_q, w_k and the norm's weights as a list, the token embedding and the n-gram table by the rows
    that have a gradient (the others keep their states and are not decayed).

    ``lr`` is a device word: set_lr() changes it, also for a captured graph.  ``max_norm``: the norm
    above which all gradients are scaled down; a step whose norm is not finite is left out and not
    counted.  ``states``: MXFP8 (2.06 bytes a value) or F32 (8).  8 bits make a root of v that
    strays by 15 % around its value (F32 at a beta2 of 0.999: 1.6 %) and an m that is off by 9 %; they
    are the default for the tables' sake, and F32 is the choice where memory allows.  All tensors share
    ``seed``: the head, the token embedding and the table are rounded with the same random bits at
    equal places.  ``masters``: fp32 copies of the BF16
    weights that the steps are taken on (an MXFP8 table has one in any case; they begin as the
    weights are when this object is made).  ``weight_decay`` is that of the BF16 and MXFP8 weights.
    ``lr_scale``: factors of lr by name (head, wkv, wq, wk, norm, embedding, table).

    norm (fp32 [1]) and norms (by name, ``names``) are those of the last step's gradients.
    """

    def __init__(self, step: TrainStep, lr: float, *, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                 max_norm=math.inf, states=MXFP8, masters=True, lr_scale=None, seed=0):
        if states not in (F32, MXFP8):
            raise ValueError("states: F32 or MXFP8")
        model, kept, device = step.model, step.model.tensors[step.layer], step.model.device
        if kept["table"].device.type != "cuda":
            raise ValueError("the n-gram table has to be in device memory")
        if step.head.data_ptr() == step.embedding.data_ptr():
            raise ValueError("head and token embedding are one tensor: their gradients are not joined")
        self.train, self.betas, self.eps, self.max_norm, self.states = step, betas, eps, max_norm, states
        scale = dict.fromkeys(("head", "wkv", "wq", "wk", "norm", "embedding", "table"), 1.0)
        if set(lr_scale or ()) - set(scale):
            raise ValueError(f"lr_scale: names are {sorted(scale)}")
        scale.update(lr_scale or {})
        bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        self.seed = seed

        def state(*shape):
            n = math.prod(shape)
            if states == F32:
                return dict(m=torch.zeros(n, dtype=f32, device=device), v=torch.zeros(n, dtype=f32, device=device))
            return {k: torch.zeros(n if k in "mv" else (n + 31) // 32, dtype=u8, device=device)
                    for k in ("m", "v", "m_scales", "v_scales")}

        def dense(name, param, grad, decay):
            param = param.view(bf16) if param.element_size() == 2 else param
            master = param.float().reshape(-1) if masters and param.dtype == bf16 else None
            return dict(param=param, grad=grad, master=master, lr_scale=scale[name], weight_decay=decay,
                        **state(param.numel()))

        self.dense = {"head": dense("head", step.head, step.dhead, weight_decay),
                      "wkv": dense("wkv", kept["wkv"], step.dwkv, weight_decay),
                      "wq": dense("wq", kept["wq"], step.dwq, 0.0), "wk": dense("wk", kept["wk"], step.dwk, 0.0)}
        if step.norm is not None:
            self.dense["norm"] = dense("norm", step.norm, step.dnorm, 0.0)
        self._list = adamw_tensors(list(self.dense.values()))
        # the tables
        rows, dim = model.rows(step.layer), model.geom["row_dim"]
        table, scales = kept["table"], kept["scales"]
        if scales is None:
            table, master = table.view(bf16)[:rows * dim], None
            if masters:
                master = table.float()
        else:
            table, scales = table[:rows * dim], scales[:rows * dim // 32]
            master = torch.empty(rows * dim, dtype=f32, device=device)
            for i in range(0, rows * dim, 1 << 28):  # in pieces: a table may fill much of the memory
                exps = scales[i // 32:(i + (1 << 28)) // 32].int()
                power = torch.ldexp(torch.ones_like(exps, dtype=f32), exps - 127)
                codes = table[i:i + (1 << 28)].view(torch.float8_e4m3fn).float().view(-1, 32)
                master[i:i + (1 << 28)] = (codes * power.unsqueeze(1)).view(-1)
        embedding = step.embedding.view(bf16)
        self.rows = {
            "embedding": dict(table=embedding, table_format=BF16, rows=step.vocab, dim=step.d,
                              master=embedding.float() if masters else None,
                              lr_scale=scale["embedding"], weight_decay=weight_decay,
                              **state(step.vocab, step.d)),
            "table": dict(table=table, scales=scales, table_format=BF16 if scales is None else MXFP8, rows=rows,
                          dim=dim, master=master, lr_scale=scale["table"], weight_decay=weight_decay,
                          **state(rows, dim))}
        self._tables = {name: AdamWTable(**t) for name, t in self.rows.items()}
        # the gradients' norms
        self.names = [*self.dense, *self.rows]
        self._parts = grad_parts([dict(grad=t["grad"]) for t in self.dense.values()] + [
            dict(grad=step.token_grad, count=step.token_count, dim=step.d),
            dict(grad=step.row_grad, count=step.row_count, dim=dim)])
        new = lambda n, dtype=f32: torch.zeros(n, dtype=dtype, device=device)  # noqa: E731
        self.norms, self.norm, self.factor = new(len(self.names)), new(1), new(1)
        self.lr, self.steps = torch.full((1,), float(lr), device=device), new(1, torch.int32)
        self.ws = new(max(engram_grad_norm_workspace_bytes(self._parts), 16), u8)
        torch.cuda.current_stream(device).synchronize()

    def set_lr(self, lr: float, stream=None):
        with torch.cuda.stream(self.train._on(stream)):
            self.lr.fill_(float(lr))

    def step(self, stream=None, rebind=True):
        """One update with the gradients of the last backward(), which has to be that of the last forward().

        The layer's next use needs what it keeps of its weights made again.  ``rebind``: wait for the
        update and bind the layer (and return what ``model.rebind`` does: True where what was captured
        of the layer has to be captured again).  Without, nothing waits, as a captured step needs: a layer on BF16
        operands (a BF16 table, or bound with BIND_BF16_OPERANDS) is refreshed on the stream, and a
        captured step's replays follow one another like eager ones.  One on FP16 operands has to be
        bound (``model.rebind(layer)``) before its next forward(), which refuses until then; such a
        step is not captured."""
        t = self.train
        if not t.ready:
            raise ValueError("no backward() of the last forward() whose gradients could be used")
        ctx, stream = t.model.ctx, t._on(stream)
        fp16 = t.model.fp16_operands(t.layer)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing() and (rebind or fp16):
                raise ValueError("a captured step: rebind=False, and a layer on BF16 operands (BIND_BF16_OPERANDS)")
        engram_grad_norm(ctx, self._parts, self.max_norm, self.norms, self.norm, self.factor, self.ws, stream)
        with torch.cuda.stream(stream):
            self.steps += torch.isfinite(self.norm)
        step = AdamWStep(beta1=self.betas[0], beta2=self.betas[1], eps=self.eps, seed=self.seed,
                         state_format=self.states, d_lr=self.lr, d_step=self.steps, d_factor=self.factor)
        engram_adamw(ctx, self._list, step, stream)
        engram_adamw_rows(ctx, self._tables["embedding"], t.token_ids, t.token_count, t.tokens, t.token_grad,
                          step, stream)
        engram_adamw_rows(ctx, self._tables["table"], t.row_ids, t.row_count, t.tokens * t.model.nb, t.row_grad,
                          step, stream)
        if rebind:
            stream.synchronize()
            return t.model.rebind(t.layer)
        if fp16:
            t.model.outdated.add(t.layer)
        else:
            t.model.refresh(t.layer, stream)
        return False
