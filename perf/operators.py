"""The operators that train an Engram layer and the model's two ends, as measured cases.

  embed      token embedding lookup with scaling, each row copied into every
             hyper-connection branch; its gradient by sorted tokens, for the token
             embedding and for the rows of an n-gram table
  gate       the gate with an 8-bit checkpoint of its activations (E4M3 codes and
             one E8M0 exponent per 32 values), and the gate's backward pass, from
             that checkpoint or from kept 16/32-bit activations
  project    the backward pass of the wkv projection
  loss       softmax cross entropy of x head^T over a large vocabulary without
             keeping the logits, and its gradient

Geometry, vocabulary and token counts are this repository's workloads
(129,280 tokens, 4 branches x 5,120, 24 rows x 256, prefills of 2,048 and 50,032
tokens, 256 decode sessions), and generic smaller and odd sizes.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False  # set from outside: run() calls the framework's operators where true

VOCAB, HC, D, HEADS, ROW_DIM = 129_280, 4, 5120, 8, 256
EPS = 1e-6
DEAD = -1  # window slot 0 of an image row; also the masked id


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's tokens: latency of a small lookup
        dict(name="embed_decode_256", op="embed", n=256, rows=VOCAB, dim=D, copies=HC,
             table="bf16"),
        # a long prompt's embedding, written to the four branches
        dict(name="embed_prefill_50032", op="embed", n=50_032, rows=VOCAB, dim=D, copies=HC,
             table="bf16"),
        # the token embedding's gradient of a training batch: the four branches' sum, Zipf tokens
        dict(name="embed_grad_tokens_8192", op="embed_grad", n=8192, rows=VOCAB, dim=D, copies=HC,
             dense=False),
        # the n-gram table's gradient of a 50,032-token batch: 24 rows a token, sparse rows
        dict(name="embed_grad_rows_50032x24", op="embed_grad", n=50_032 * 24, rows=64_000_000,
             dim=ROW_DIM, copies=1, dense=False),
        # the training forward: gate, and the activations kept in 8 bits
        dict(name="gate_checkpoint_2048", op="gate_checkpoint", T=2048, hc=HC, d=D, kv="f32"),
        # its backward pass from the checkpoint
        dict(name="gate_backward_checkpoint_2048", op="gate_backward", T=2048, hc=HC, d=D,
             kv="mxfp8"),
        # a short odd sequence from activations kept in 16 bits
        dict(name="gate_backward_bf16_77", op="gate_backward", T=77, hc=HC, d=D, kv="bf16"),
        # both gradients of the projection of a training batch, and of a short odd one
        dict(name="project_backward_2048", op="project_backward", T=2048, hc=HC, d=D, heads=HEADS,
             row_dim=ROW_DIM),
        dict(name="project_backward_333", op="project_backward", T=333, hc=HC, d=D, heads=HEADS,
             row_dim=ROW_DIM),
        # scoring a few tokens (the head is read once), and a training batch's loss
        dict(name="loss_16", op="loss", T=16, vocab=VOCAB, dim=D),
        dict(name="loss_2048", op="loss", T=2048, vocab=VOCAB, dim=D),
        # the loss's gradient of a training batch
        dict(name="loss_backward_2048", op="loss_backward", T=2048, vocab=VOCAB, dim=D),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        sizes = [v for v in c.values() if isinstance(v, int)]
        if c["op"] in ("gate_checkpoint", "gate_backward", "project_backward"):
            sizes += [j * c["d"] for j in range(1, 2 * HC + 2)]
            sizes.append(3 * c.get("heads", 0) * c.get("row_dim", 0))
        if 3072 not in sizes:  # a size that none of this repository's workloads has
            return c


def _draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "gate_checkpoint", "gate_backward",
                     "gate_backward", "project_backward", "loss", "loss_backward"])
    if op == "embed":
        return dict(op=op, n=_log_int(rng, 1, 50_032), rows=_log_int(rng, 1000, VOCAB),
                    dim=8 * _log_int(rng, 8, D // 8), copies=rng.randint(1, HC),
                    table=rng.choice(["bf16", "f32"]))
    if op == "embed_grad":
        if rng.random() < 0.5:  # tokens
            return dict(op=op, n=_log_int(rng, 1, 8192), rows=_log_int(rng, 1000, VOCAB),
                        dim=8 * _log_int(rng, 8, D // 8), copies=rng.randint(1, HC),
                        dense=rng.random() < 0.5)
        return dict(op=op, n=24 * _log_int(rng, 1, 50_032),  # rows of an n-gram table
                    rows=_log_int(rng, 6000, 64_000_000), dim=rng.choice([32, 64, 128, 256]),
                    copies=1, dense=False)
    if op in ("gate_checkpoint", "gate_backward"):
        return dict(op=op, T=_log_int(rng, 1, 2048), hc=rng.randint(1, HC),
                    d=256 * rng.randint(1, D // 256),
                    kv=rng.choice(["f32", "bf16"] if op == "gate_checkpoint"
                                  else ["mxfp8", "f32", "bf16"]))
    if op == "project_backward":
        return dict(op=op, T=_log_int(rng, 1, 2048), hc=rng.randint(1, HC),
                    d=256 * rng.randint(1, D // 256), heads=rng.randint(2, HEADS),
                    row_dim=rng.choice([64, 128, 256]))
    return dict(op=op, T=_log_int(rng, 1, 2048), vocab=_log_int(rng, 1000, VOCAB),
                dim=8 * _log_int(rng, 16, D // 8))


# ---- what a pass cannot do without ----------------------------------------------------------

def _distinct(n, rows):
    """Expected number of different ids among n log-uniform draws from [0, rows)."""
    top = np.arange(1, min(rows, 1 << 16) + 1, dtype=np.float64)
    total = float(-np.expm1(n * np.log1p(-np.minimum(np.log1p(1 / top) / math.log(rows + 1),
                                                     1 - 1e-12))).sum())
    if rows > top.size:  # the tail, on a logarithmic grid
        edge = np.exp(np.linspace(math.log(top.size + 1), math.log(rows + 1), 2000))
        mid = np.sqrt(edge[1:] * edge[:-1])
        total += float((np.diff(edge) * -np.expm1(-n / (mid * math.log(rows + 1)))).sum())
    return min(total, n)


def work(case):
    c, op = case, case["op"]
    if op == "embed":
        size = 2 if c["table"] == "bf16" else 4
        return dict(bytes=4 * c["n"] + _distinct(c["n"], c["rows"]) * c["dim"] * size +
                    2 * c["n"] * c["copies"] * c["dim"], flops=c["n"] * c["dim"])
    if op == "embed_grad":
        out = (c["rows"] * 4 * c["dim"] if c["dense"] else
               _distinct(c["n"], c["rows"]) * (4 * c["dim"] + 4))
        return dict(bytes=4 * c["n"] + 2 * c["n"] * c["copies"] * c["dim"] + out,
                    flops=c["n"] * c["copies"] * c["dim"])
    if op in ("gate_checkpoint", "gate_backward"):
        h, kv = c["T"] * c["hc"] * c["d"], c["T"] * (c["hc"] + 1) * c["d"]
        saved = (h + kv) * 33 / 32
        weights = 8 * c["hc"] * c["d"]
        if op == "gate_checkpoint":
            read = kv * (4 if c["kv"] == "f32" else 2) + 2 * h + weights + 16 * c["T"]
            return dict(bytes=read + 2 * h + saved + 4 * c["T"] * c["hc"], flops=8 * h)
        read = saved if c["kv"] == "mxfp8" else kv * (4 if c["kv"] == "f32" else 2) + 2 * h
        return dict(bytes=read + 2 * h + 2 * h + 2 * kv + 2 * weights + 16 * c["T"], flops=20 * h)
    if op == "project_backward":
        n, k = (c["hc"] + 1) * c["d"], 3 * c["heads"] * c["row_dim"]
        return dict(bytes=2 * (2 * c["T"] * k + c["T"] * n + 2 * n * k), flops=4 * c["T"] * n * k)
    t, v, d = c["T"], c["vocab"], c["dim"]
    if op == "loss":
        return dict(bytes=2 * (t * d + v * d) + 12 * t, flops=2 * t * v * d)
    # the logits are not kept: they are computed again for the gradient
    return dict(bytes=4 * (t * d + v * d) + 12 * t, flops=6 * t * v * d)


# ---- inputs -----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000 + int(seed))


def _normal(g, *shape, sigma=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(dtype)


def _ids(g, n, rows, masked):
    """Log-uniform ids (a Zipf distribution of exponent 1), `masked` of them masked."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(rows + 1)) - 1).long().clamp(0, rows - 1)
    drop = torch.rand(n, generator=g, device="cuda") < masked
    return ids, drop


def _pack(x):
    """MXFP8 of x [..., n]: E4M3 codes and, per 32 values, the smallest E8M0 exponent that
    keeps the largest of them at or below 448."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    exps = (e - 1 - 8 + 127 + (m > 0.875).int()).clamp(0, 254)
    exps = torch.where(m == 0, torch.zeros_like(exps), exps)
    inv = ((254 - exps).to(torch.int32) << 23).view(torch.float32)
    codes = (b * inv.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.reshape(x.shape), exps.to(torch.uint8)


def _unpack(codes, exps):
    s = (exps.int() << 23).view(torch.float32)
    s = torch.where(exps == 0, torch.full_like(s, 2.0 ** -127), s)
    return (codes.float().reshape(*exps.shape, 32) * s.unsqueeze(-1)).reshape(codes.shape)


def _inputs(case, seed):
    """The data of a pass, the same whichever side runs it."""
    c, op, g = case, case["op"], _gen(seed)
    if op == "embed":
        table = torch.empty(c["rows"], c["dim"], device="cuda",
                            dtype=torch.bfloat16 if c["table"] == "bf16" else torch.float32)
        table.normal_(0.0, 0.02, generator=g)
        ids, drop = _ids(g, c["n"], c["rows"], 0.02)
        return dict(table=table, ids=torch.where(drop, DEAD, ids).int(), scale=math.sqrt(c["dim"]))
    if op == "embed_grad":
        ids, drop = _ids(g, c["n"], c["rows"], 0.02)
        if c["dim"] <= ROW_DIM:  # hashed rows: frequency says nothing about the row's place
            ids = ids * 0x9E3779B1 % c["rows"]
        return dict(ids=torch.where(drop, DEAD, ids).int(), scale=math.sqrt(c["dim"]),
                    dout=_normal(g, c["n"], c["copies"], c["dim"], sigma=1e-3))
    if op in ("gate_checkpoint", "gate_backward"):
        T, hc, d = c["T"], c["hc"], c["d"]
        win = torch.randint(0, 1000, (T, 4), generator=g, device="cuda").int()
        win[torch.rand(T, generator=g, device="cuda") < 0.04, 0] = DEAD
        s = dict(windows=win, hidden=_normal(g, T, hc, d),
                 kv=_normal(g, T, (hc + 1) * d, dtype=torch.float32),
                 wq=1 + _normal(g, hc, d, sigma=0.1, dtype=torch.float32),
                 wk=1 + _normal(g, hc, d, sigma=0.1, dtype=torch.float32))
        # keys that agree with the hidden state more or less: the gates' dots spread over
        # +-[0.4, 8], away from 0, where the root's slope grows without bound and no 32-bit
        # sum says what the gradient is
        h, k = s["hidden"].float(), s["kv"][:, :hc * d].reshape(T, hc, d)
        hw = h * (s["wq"] * s["wk"])
        k = k - h * ((hw * k).sum(-1, keepdim=True) / (hw * h).sum(-1, keepdim=True))
        u = torch.rand(T, hc, 1, generator=g, device="cuda") * 2 - 1
        dot = torch.sign(u) * torch.exp(u.abs() * math.log(20)) * 0.4
        s["kv"][:, :hc * d] = (k + dot / math.sqrt(d) * h).reshape(T, hc * d)
        if c["kv"] == "bf16":
            s["kv"] = s["kv"].bfloat16()
        if op == "gate_backward":
            s["dout"] = _normal(g, T, hc, d, sigma=1e-3)
            if c["kv"] == "mxfp8":
                s["codes"], s["scales"] = _pack(torch.cat([s["hidden"].float().reshape(T, hc * d),
                                                           s["kv"]], 1))
                del s["kv"], s["hidden"]
        return s
    if op == "project_backward":
        n, k = (c["hc"] + 1) * c["d"], 3 * c["heads"] * c["row_dim"]
        return dict(emb=_normal(g, c["T"], k, sigma=38.5), dkv=_normal(g, c["T"], n, sigma=1e-3),
                    wkv=_normal(g, n, k, sigma=1 / (math.sqrt(k) * 38.5)),
                    wq=torch.ones(c["hc"], c["d"], device="cuda"),
                    wk=torch.ones(c["hc"], c["d"], device="cuda"))
    T, V, d = c["T"], c["vocab"], c["dim"]
    head = torch.empty(V, d, device="cuda", dtype=torch.bfloat16)
    head.normal_(0.0, 2 / math.sqrt(d), generator=g)
    ids, drop = _ids(g, T, V, 0.05)
    s = dict(x=_normal(g, T, d), head=head, labels=torch.where(drop, -1, ids).int())
    if op == "loss_backward":
        s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
        s["lse"] = torch.cat([torch.logsumexp(x.float() @ head.float().T, 1)
                              for x in s["x"].split(1024)])
    return s


class _Layer:
    """A context with one bound Engram layer, as a user's program keeps it."""

    def __init__(self, hc, d, heads, row_dim, wkv, wq, wk):
        from engram_gram_conditional_gb300.layer import EngramLayerSet

        self.set = EngramLayerSet(1024, 1000, np.arange(1024, dtype=np.uint32) % 1000, [7], [1000],
                                  heads=heads, row_dim=row_dim, hc=hc, d=d, eps=EPS)
        self.set.bind(0, 7, wkv.view(torch.int16), wq, wk)
        self.ctx = self.set.ctx

    def __del__(self):
        torch.cuda.synchronize()
        self.set.close()


def prepare(case, seed):
    c, op = case, case["op"]
    s = _inputs(case, seed)
    s["case"] = c
    if op == "embed_grad":  # buffers that a training program keeps
        rows = c["rows"] if c["dense"] else c["n"]
        s["grad"] = torch.zeros(rows, c["dim"], device="cuda")
        s["unique"] = torch.full((c["n"],), -1, dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if not own:
        return s
    import engram_gram_conditional_gb300 as eg

    if op in ("gate_checkpoint", "gate_backward"):
        n = (c["hc"] + 1) * c["d"]
        wkv = torch.zeros(n, 192, dtype=torch.bfloat16, device="cuda")
        s["layer"] = _Layer(c["hc"], c["d"], 2, 32, wkv, s["wq"], s["wk"])
        need = eg.engram_gate_backward_workspace_bytes(s["layer"].ctx, c["T"])
    elif op == "project_backward":
        s["layer"] = _Layer(c["hc"], c["d"], c["heads"], c["row_dim"], s["wkv"], s["wq"], s["wk"])
        need = eg.engram_project_backward_workspace_bytes(s["layer"].ctx, c["T"])
    else:
        s["layer"] = _Layer(1, 256, 2, 32, torch.zeros(512, 192, dtype=torch.bfloat16, device="cuda"),
                            torch.ones(1, 256, device="cuda"), torch.ones(1, 256, device="cuda"))
        need = {"embed": lambda: 0,
                "embed_grad": lambda: eg.engram_embed_grad_workspace_bytes(c["n"], c["rows"],
                                                                           c["dim"]),
                "loss": lambda: eg.engram_loss_workspace_bytes(c["T"], c["vocab"], c["dim"]),
                "loss_backward": lambda: eg.engram_loss_backward_workspace_bytes(
                    c["T"], c["vocab"], c["dim"])}[op]()
    s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import engram_gram_conditional_gb300 as eg

    c, op, ctx = s["case"], s["case"]["op"], s["layer"].ctx
    stream = torch.cuda.current_stream()
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "embed":
        out = new(c["n"], c["copies"], c["dim"])
        fmt = eg.EMBED_BF16 if c["table"] == "bf16" else eg.EMBED_F32
        eg.engram_embed(ctx, s["table"], fmt, c["rows"], c["dim"], s["ids"], c["n"], s["scale"],
                        c["copies"], out, stream)
        return dict(out=out)
    if op == "embed_grad":
        if c["dense"]:
            eg.engram_embed_grad(ctx, c["rows"], c["dim"], s["ids"], c["n"], s["scale"],
                                 c["copies"], s["dout"], None, None, s["grad"], 0, s["ws"], stream)
            return dict(grad=s["grad"])
        eg.engram_embed_grad(ctx, c["rows"], c["dim"], s["ids"], c["n"], s["scale"], c["copies"],
                             s["dout"], s["unique"], s["count"], s["grad"], 0, s["ws"], stream)
        return dict(unique=s["unique"], count=s["count"], grad=s["grad"])
    if op in ("gate_checkpoint", "gate_backward"):
        T, hc, d = c["T"], c["hc"], c["d"]
        n, kept = (hc + 1) * d, (2 * hc + 1) * d
        fmt = {"f32": eg.KV_F32, "bf16": eg.KV_BF16}.get(c["kv"])
        if op == "gate_checkpoint":
            r = dict(hidden=new(T, hc, d), gates=new(T, hc, dtype=torch.float32),
                     codes=new(T, kept, dtype=torch.uint8),
                     scales=new(T, kept // 32, dtype=torch.uint8))
            eg.engram_gate_checkpoint(ctx, 0, s["kv"], fmt, s["windows"], T, s["hidden"],
                                      r["hidden"], r["gates"], r["codes"], r["scales"], stream)
            r["codes"] = r["codes"].view(torch.float8_e4m3fn)
            return r
        r = dict(dhidden=new(T, hc, d), dkv=new(T, n), dwq=new(hc, d, dtype=torch.float32),
                 dwk=new(hc, d, dtype=torch.float32))
        to = (r["dhidden"], r["dkv"], r["dwq"], r["dwk"], s["ws"], stream)
        if c["kv"] == "mxfp8":
            eg.engram_gate_backward_checkpoint(ctx, 0, s["codes"], s["scales"], s["windows"], T,
                                               s["dout"], *to)
        else:
            eg.engram_gate_backward(ctx, 0, s["kv"], fmt, s["hidden"], s["windows"], T, s["dout"],
                                    *to)
        return r
    if op == "project_backward":
        r = dict(demb=torch.empty_like(s["emb"]), dwkv=torch.empty_like(s["wkv"]))
        eg.engram_project_backward(ctx, 0, s["emb"], s["dkv"], c["T"], r["demb"], r["dwkv"],
                                   s["ws"], stream)
        return r
    T, V, d = c["T"], c["vocab"], c["dim"]
    if op == "loss":
        r = dict(loss=new(T, dtype=torch.float32), lse=new(T, dtype=torch.float32))
        eg.engram_loss(ctx, s["x"], s["head"], V, d, s["labels"], T, r["loss"], r["lse"], s["ws"],
                       stream)
        return r
    r = dict(dx=torch.empty_like(s["x"]), dhead=torch.empty_like(s["head"]))
    eg.engram_loss_backward(ctx, s["x"], s["head"], V, d, s["labels"], T, s["lse"], s["dloss"],
                            r["dx"], r["dhead"], s["ws"], stream)
    return r


def _gate_parts(h, k, wqk, d):
    """h, k [T, hc, d]: (the two norm factors, dot, signed root, gate), each [T, hc, 1]."""
    rh = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    rk = (k.square().mean(-1, keepdim=True) + EPS).rsqrt()
    dot = (h * wqk * k).sum(-1, keepdim=True) * rh * rk / math.sqrt(d)
    root = torch.copysign(dot.abs().clamp_min(1e-6).sqrt(), dot)
    return rh, rk, dot, root, torch.sigmoid(root)


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "embed":
        ids = s["ids"].long()
        row = s["table"][ids.clamp_min(0)].float() * s["scale"]
        row = row * (ids >= 0).unsqueeze(1)
        return dict(out=row.bfloat16().unsqueeze(1).expand(-1, c["copies"], -1).contiguous())
    if op == "embed_grad":
        ids = s["ids"].long()
        rows = s["dout"].float().sum(1) * s["scale"]
        if c["dense"]:
            grad = torch.zeros(c["rows"] + 1, c["dim"], device="cuda")
            grad.index_add_(0, torch.where(ids < 0, c["rows"], ids), rows)
            return dict(grad=grad[:-1])
        at = ids >= 0
        unique, inverse = torch.unique(ids[at], return_inverse=True)
        m = unique.numel()  # the buffers' rows past the distinct ids are not written
        s["unique"][:m] = unique
        s["count"].fill_(m)
        s["grad"][:m].zero_().index_add_(0, inverse, rows[at])
        return dict(unique=s["unique"], count=s["count"], grad=s["grad"])
    if op in ("gate_checkpoint", "gate_backward"):
        T, hc, d = c["T"], c["hc"], c["d"]
        text = (s["windows"][:, 0] != DEAD).reshape(T, 1, 1)
        wqk = s["wq"] * s["wk"]
        if c["kv"] == "mxfp8":
            saved = _unpack(s["codes"], s["scales"])
            h, kv = saved[:, :hc * d].reshape(T, hc, d), saved[:, hc * d:]
        else:
            h, kv = s["hidden"].float(), s["kv"].float()
        k, v = kv[:, :hc * d].reshape(T, hc, d), kv[:, hc * d:].reshape(T, 1, d)
        rh, rk, dot, root, gate = _gate_parts(h, k, wqk, d)
        if op == "gate_checkpoint":
            out = torch.where(text, h + gate * v, h).bfloat16()
            codes, scales = _pack(torch.cat([h.reshape(T, hc * d), kv], 1) * text.reshape(T, 1))
            return dict(hidden=out, gates=(gate * text).reshape(T, hc), codes=codes, scales=scales)
        dy = s["dout"].float()
        dgate = (dy * v).sum(-1, keepdim=True)
        ddot = dgate * gate * (1 - gate) * (dot.abs() > 1e-6) / (2 * root.abs()) * text
        dsum = ddot * rh * rk / math.sqrt(d)
        dh = dy + dsum * wqk * k - ddot * dot * rh.square() / d * h
        dk = dsum * wqk * h - ddot * dot * rk.square() / d * k
        dv = (gate * dy * text).sum(1)
        dwqk = (dsum * h * k).sum(0)
        return dict(dhidden=dh.bfloat16(), dkv=torch.cat([dk.reshape(T, hc * d), dv], 1).bfloat16(),
                    dwq=dwqk * s["wk"], dwk=dwqk * s["wq"])
    if op == "project_backward":
        dkv = s["dkv"].float()
        return dict(demb=(dkv @ s["wkv"].float()).bfloat16(),
                    dwkv=(dkv.T @ s["emb"].float()).bfloat16())
    labels = s["labels"].long()
    counted = (labels >= 0)
    x, head = s["x"].float(), s["head"].float()
    logits = x @ head.T
    at = labels.clamp_min(0).unsqueeze(1)
    if op == "loss":
        top = logits.amax(1, keepdim=True)
        lse = (logits - top).exp().sum(1).log() + top.squeeze(1)
        return dict(loss=(lse - logits.gather(1, at).squeeze(1)) * counted, lse=lse)
    dz = (logits - s["lse"].unsqueeze(1)).exp()
    dz.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    dz *= (s["dloss"] * counted).unsqueeze(1)
    return dict(dx=(dz @ head).bfloat16(), dhead=(dz.T @ x).bfloat16())


# ---- the definitions in 64 bits -----------------------------------------------------------

def exact(case, seed):
    c, op = case, case["op"]
    s = _inputs(case, seed)
    f = torch.float64
    if op == "embed":
        out = torch.zeros(c["n"], c["copies"], c["dim"], dtype=f, device="cuda")
        at = s["ids"] >= 0
        out[at] = (s["table"][s["ids"][at].long()].to(f) * s["scale"]).unsqueeze(1)
        return dict(out=out)
    if op == "embed_grad":
        at = s["ids"] >= 0
        ids, rows = s["ids"][at].long(), s["dout"][at].to(f).sum(1) * s["scale"]
        if c["dense"]:
            return dict(grad=torch.zeros(c["rows"], c["dim"], dtype=f,
                                         device="cuda").index_add_(0, ids, rows))
        unique, inverse = torch.unique(ids, return_inverse=True)
        grad = torch.zeros(c["n"], c["dim"], dtype=f, device="cuda")
        return dict(unique=None, count=None, grad=grad.index_add_(0, inverse, rows))
    if op in ("gate_checkpoint", "gate_backward"):
        return _exact_gate(c, op, s)
    if op == "project_backward":
        dkv = s["dkv"].to(f)
        return dict(demb=torch.mm(dkv, s["wkv"].to(f)), dwkv=torch.mm(dkv.t(), s["emb"].to(f)))
    if op == "loss":
        loss, lse = [], []
        head = s["head"].to(f)
        for x, y in zip(s["x"].split(512), s["labels"].long().split(512)):
            z = torch.mm(x.to(f), head.t())
            lse.append(torch.logsumexp(z, 1))
            own_z = z[torch.arange(len(y), device="cuda"), y.clamp_min(0)]
            loss.append(torch.where(y >= 0, lse[-1] - own_z, torch.zeros_like(own_z)))
        return dict(loss=torch.cat(loss), lse=torch.cat(lse))
    if 6.0 * c["T"] * c["vocab"] * c["dim"] > 9e12:
        return None
    head, dx = s["head"].to(f), []
    dhead = torch.zeros(c["vocab"], c["dim"], dtype=f, device="cuda")
    for i in range(0, c["T"], 512):
        x, y = s["x"][i:i + 512].to(f), s["labels"][i:i + 512].long()
        z = torch.mm(x, head.t())
        p = torch.exp(z - s["lse"][i:i + 512].to(f).unsqueeze(1))
        p[torch.arange(len(y), device="cuda"), y.clamp_min(0)] -= 1
        p *= torch.where(y >= 0, s["dloss"][i:i + 512].to(f), 0.0).unsqueeze(1)
        dx.append(torch.mm(p, head))
        dhead.addmm_(p.t(), x)
    return dict(dx=torch.cat(dx), dhead=dhead)


def _exact_gate(c, op, s):
    """Gates and gradients in 64 bits; the gradients by differentiating the forward step."""
    T, hc, d, f = c["T"], c["hc"], c["d"], torch.float64
    on = s["windows"][:, 0] != DEAD
    if c["kv"] == "mxfp8":
        power = torch.pow(torch.tensor(2.0, dtype=f, device="cuda"), s["scales"].to(f) - 127)
        saved = s["codes"].to(torch.float32).to(f) * power.repeat_interleave(32, 1)
        hidden, kv = saved[:, :hc * d].reshape(T, hc, d), saved[:, hc * d:]
    else:
        hidden, kv = s["hidden"].to(f), s["kv"].to(f)
    wq, wk = s["wq"].to(f), s["wk"].to(f)
    leaves = [t.clone().requires_grad_(op == "gate_backward") for t in (hidden, kv, wq, wk)]
    hidden, kv, wq, wk = leaves
    k, v = kv[:, :hc * d].reshape(T, hc, d), kv[:, hc * d:].reshape(T, 1, d)
    nh = hidden / torch.sqrt(torch.mean(hidden * hidden, 2, keepdim=True) + EPS)
    nk = k / torch.sqrt(torch.mean(k * k, 2, keepdim=True) + EPS)
    dot = torch.sum(nh * wq * nk * wk, 2, keepdim=True) / math.sqrt(d)
    size = torch.where(dot.abs() > 1e-6, dot.abs(), torch.full_like(dot, 1e-6))
    gate = 1 / (1 + torch.exp(-torch.where(torch.signbit(dot), -size.sqrt(), size.sqrt())))
    gate = gate * on.reshape(T, 1, 1)
    out = hidden + gate * v
    if op == "gate_checkpoint":
        return dict(hidden=out, gates=gate.reshape(T, hc), codes=None, scales=None)
    got = torch.autograd.grad(out, leaves, s["dout"].to(f))
    return dict(dhidden=got[0], dkv=got[1], dwq=got[2], dwk=got[3])
