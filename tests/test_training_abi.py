"""Refusals of the training operators (no GPU): arguments are checked before any launch."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import engram_gram_conditional_gb300 as eg
from engram_gram_conditional_gb300.training import TrainStep


@pytest.fixture(scope="module")
def ctx():
    from engram_gram_conditional_gb300 import build

    build.build()
    c = eg.engram_ctx_create(64, 60, np.arange(64, dtype=np.uint32) % 60, [3], [50], heads=2,
                             row_dim=32, hc=2, d=256)
    yield c
    eg.engram_ctx_destroy(c)


A = 1 << 20  # an aligned address that no refused call touches


def refused(status, f, *args):
    with pytest.raises(eg.EngramError) as e:
        f(*args)
    assert e.value.status == status


EMBED = dict(table=A, fmt=eg.EMBED_BF16, rows=10, dim=64, ids=A, n=4, scale=1.0, copies=1, out=A)


@pytest.mark.parametrize("bad", [dict(table=None), dict(ids=None), dict(out=None), dict(table=A + 8),
                                 dict(out=A + 2), dict(ids=A + 1), dict(fmt=2), dict(fmt=-1),
                                 dict(rows=0), dict(rows=2**32 - 1), dict(dim=0), dict(dim=12),
                                 dict(dim=65544), dict(n=-1), dict(n=2**30 + 1), dict(copies=0),
                                 dict(copies=9)])
def test_embed_refuses(ctx, bad):
    a = {**EMBED, **bad}
    refused(eg.EINVAL, eg.engram_embed, ctx, a["table"], a["fmt"], a["rows"], a["dim"], a["ids"],
            a["n"], a["scale"], a["copies"], a["out"])
    refused(eg.EINVAL, eg.engram_embed, None, *list(EMBED.values()))


GRAD = dict(rows=10, dim=64, ids=A, n=4, scale=1.0, copies=1, dout=A, unique=A, count=A, grad=A,
            accumulate=0, ws=A)


@pytest.mark.parametrize("bad", [dict(ids=None), dict(dout=None), dict(grad=None), dict(ws=None),
                                 dict(count=None), dict(accumulate=1), dict(accumulate=2),
                                 dict(dout=A + 4), dict(grad=A + 4), dict(ws=A + 4),
                                 dict(unique=A + 1), dict(dim=4), dict(copies=0), dict(n=-1)])
def test_embed_grad_refuses(ctx, bad):
    refused(eg.EINVAL, eg.engram_embed_grad, ctx, *{**GRAD, **bad}.values())


LOSS = dict(x=A, head=A, vocab=100, dim=64, labels=A, T=4, loss=A, lse=A, ws=A)


@pytest.mark.parametrize("bad", [dict(x=None), dict(head=None), dict(labels=None), dict(ws=None),
                                 dict(x=A + 8), dict(head=A + 8), dict(ws=A + 8), dict(vocab=0),
                                 dict(dim=0), dict(dim=20), dict(T=-1), dict(T=2**24 + 1)])
def test_loss_refuses(ctx, bad):
    refused(eg.EINVAL, eg.engram_loss, ctx, *{**LOSS, **bad}.values())


BACK = dict(x=A, head=A, vocab=100, dim=64, labels=A, T=4, lse=A, dloss=A, dx=A, dhead=A, ws=A)


@pytest.mark.parametrize("bad", [dict(x=None), dict(lse=None), dict(dloss=None), dict(ws=None),
                                 dict(dx=A + 8), dict(dhead=A + 8), dict(vocab=2**30 + 1),
                                 dict(dim=7), dict(T=-1)])
def test_loss_backward_refuses(ctx, bad):
    refused(eg.EINVAL, eg.engram_loss_backward, ctx, *{**BACK, **bad}.values())


def test_layer_operators_need_a_bound_layer(ctx):
    refused(eg.ESTATE, eg.engram_gate_checkpoint, ctx, 0, A, eg.KV_F32, A, 1, A, A, None, A, A)
    refused(eg.ESTATE, eg.engram_gate_backward, ctx, 0, A, eg.KV_F32, A, A, 1, A, A, A, A, A, A)
    refused(eg.ESTATE, eg.engram_gate_backward_checkpoint, ctx, 0, A, A, A, 1, A, A, A, A, A, A)
    refused(eg.ESTATE, eg.engram_project_backward, ctx, 0, A, A, 1, A, A, A)
    refused(eg.EINVAL, eg.engram_gate_checkpoint, ctx, 1, A, eg.KV_F32, A, 1, A, A, None, A, A)
    refused(eg.EINVAL, eg.engram_project_backward, None, 0, A, A, 1, A, A, A)


def test_workspace_sizes(ctx):
    assert eg.engram_embed_grad_workspace_bytes(0, 10, 64) > 0
    assert eg.engram_embed_grad_workspace_bytes(4, 10, 12) == 0
    assert eg.engram_gate_backward_workspace_bytes(ctx, -1) == 0
    assert eg.engram_project_backward_workspace_bytes(ctx, 0) == 0
    assert eg.engram_loss_workspace_bytes(4, 0, 64) == 0
    assert eg.engram_loss_backward_workspace_bytes(0, 100, 64) == 0
    # no logits: the loss keeps two floats per 128 columns, the backward pass one piece
    assert eg.engram_loss_workspace_bytes(2048, 129_280, 5120) < 2048 * 129_280 // 8
    assert eg.engram_loss_backward_workspace_bytes(2048, 129_280, 5120) < 2048 * 129_280 * 2 // 4


def geometry(hc, d, heads, row_dim):
    return eg.engram_ctx_create(64, 60, np.arange(64, dtype=np.uint32) % 60, [3], [50], heads=heads,
                                row_dim=row_dim, hc=hc, d=d)


SIZES = sorted({*range(1, 700), *range(700, 20_000, 61), *(2 ** k + e for k in range(9, 18) for e in (-1, 0, 1))})


@pytest.mark.parametrize("of", ["embed_grad", "gate_backward", "project_backward", "loss", "loss_backward"])
def test_a_workspace_holds_for_every_smaller_batch(of):
    """Sizes never fall as the batch grows."""
    def check(f):
        sizes = [f(n) for n in SIZES]
        assert sizes == sorted(sizes)

    if of == "embed_grad":
        for rows, dim in ((129_280, 5120), (64_000_000, 256), (5000, 40), (100, 8), (70_000, 65_536)):
            check(lambda n: eg.engram_embed_grad_workspace_bytes(n, rows, dim))
    elif of in ("loss", "loss_backward"):
        for vocab, dim in ((1000, 64), (31, 1032), (32_000, 2048), (129_280, 5120), (129_280, 8)):
            check(lambda n: getattr(eg, f"engram_{of}_workspace_bytes")(n, vocab, dim))
    else:
        for g in ((4, 5120, 8, 256), (1, 256, 2, 32), (2, 1280, 4, 128), (8, 2560, 3, 64)):
            c = geometry(*g)
            check(lambda n: getattr(eg, f"engram_{of}_workspace_bytes")(c, n))
            eg.engram_ctx_destroy(c)


def tensors(**bad):
    t = dict(ids=torch.zeros(5, dtype=torch.int32), windows=torch.zeros(5, 4, dtype=torch.int32),
             labels=torch.zeros(5, dtype=torch.int32), dloss=torch.zeros(5))
    return {**t, **bad}


@pytest.mark.parametrize("bad", [dict(ids=torch.zeros(0, dtype=torch.int32)), dict(ids=torch.zeros(9, dtype=torch.int32)),
                                 dict(ids=torch.zeros(5, dtype=torch.int64)),
                                 dict(windows=torch.zeros(4, 4, dtype=torch.int32)),
                                 dict(windows=torch.zeros(4, 5, dtype=torch.int32).t()),
                                 dict(labels=torch.zeros(4, dtype=torch.int32)),
                                 dict(labels=torch.zeros(5, dtype=torch.int64)),
                                 dict(labels=torch.zeros(10, dtype=torch.int32)[::2]),
                                 dict(labels=torch.zeros(5, dtype=torch.int32, device="meta"))])
def test_a_step_refuses_tensors_that_do_not_go_together(bad):
    step = object.__new__(TrainStep)  # (its buffers need a GPU; what is refused reaches none)
    step.model, step.layer, step.tokens, step.T = SimpleNamespace(device=torch.device("cpu"), ctx=None), 0, 8, 0
    t = tensors(**bad)
    with pytest.raises(ValueError):
        step.forward(t["ids"], t["windows"], t["labels"])
    assert step.T == 0
    with pytest.raises(ValueError):
        step.backward(*tensors().values())  # no forward before
    step.T = 5
    t = tensors(**bad) if "ids" not in bad or bad["ids"].numel() else tensors(dloss=torch.zeros(4))
    with pytest.raises(ValueError):
        step.backward(*t.values())


def test_a_step_refuses_weights_of_another_shape():
    model = SimpleNamespace(device=torch.device("cpu"), geom=dict(d=256, hc=2, row_dim=32), ctx=None)
    good = torch.zeros(10, 256, dtype=torch.bfloat16)
    for embedding, head, tokens in ((good, good[:9], 4), (good, good.float(), 4), (good[:, :128], good, 4),
                                    (good, good.t(), 4), (good, good, 0)):
        with pytest.raises(ValueError):
            TrainStep(model, 0, embedding, head, tokens)
