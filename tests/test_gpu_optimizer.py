"""Training steps with an optimizer that follow one another: what a layer keeps of its weights, eager and
captured."""
import math

import pytest
import torch

import engram_gram_conditional_gb300 as eg
from engram_gram_conditional_gb300.training import AdamW, TrainStep
from test_gpu_update import step_inputs, step_model

pytestmark = pytest.mark.gpu


def made(mx_table, flags=0, T=40, **kw):
    s, kept, embedding, head, norm = step_model(mx_table)
    if flags:
        s._flags[0] |= flags
        s.rebind(0)
    step = TrainStep(s, 0, embedding, head, T, norm=norm)
    opt = AdamW(step, 1e-2, max_norm=5.0, weight_decay=0.1, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    return s, kept, step, opt, side, step_inputs(s, T, 2)


def exponent(x):
    return math.frexp(float(x.view(torch.bfloat16).abs().max()))[1]


@pytest.mark.parametrize("mx_table", [False, True])
def test_replays_of_a_captured_step_are_eager_steps(mx_table):
    """Forward, backward and update, replayed, against eager steps that bind the layer each time: every
    step sees all weights as the one before left them (with an MXFP8 table the largest |wkv| passes a
    power of two)."""
    results = []
    for captured in (False, True):
        s, kept, step, opt, side, inputs = made(mx_table, eg.BIND_BF16_OPERANDS if mx_table else 0,
                                                lr_scale=dict(table=300.0))
        begin = exponent(kept["wkv"]), kept["wq"].clone(), kept["table"].clone()
        seen = []

        def once(rebind):
            step.forward(*inputs[:3], side)
            step.backward(*inputs, side)
            opt.step(side, rebind=rebind)

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                once(False)
        for _ in range(4):
            graph.replay() if captured else once(True)
            torch.cuda.synchronize()
            seen += [x.clone() for x in (step.loss, step.kv, step.gates, step.dwq, step.dwkv, step.dhidden)]
        eg.engram_sync(s.ctx)
        assert int(opt.steps) == 4
        assert not torch.equal(begin[1], kept["wq"]) and not torch.equal(begin[2], kept["table"])
        assert not mx_table or exponent(kept["wkv"]) > begin[0]  # (its weights are small: the rate takes them there)
        results.append(seen + [x.clone() for x in (step.head, step.embedding, step.norm, kept["wkv"], kept["wq"],
                                                   kept["wk"], kept["table"])])
        s.close()
    assert all(torch.equal(a, b) for a, b in zip(*results))
    losses = results[1][::6][:4]
    assert not torch.equal(losses[0], losses[1]) and not torch.equal(losses[1], losses[2])


def test_steps_without_a_bind_are_steps_with_one():
    """A layer on BF16 operands is refreshed on the stream; nothing else of it is kept."""
    results = []
    for rebind in (True, False):
        s, kept, step, opt, side, inputs = made(True, eg.BIND_BF16_OPERANDS)
        for _ in range(3):
            step.forward(*inputs[:3], side)
            step.backward(*inputs, side)
            opt.step(side, rebind=rebind)
        torch.cuda.synchronize()
        eg.engram_sync(s.ctx)
        results.append([x.clone() for x in (step.loss, step.gates, kept["wkv"], kept["wq"], kept["table"])])
        s.close()
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_a_layer_on_fp16_operands_is_bound_between_steps():
    """What such a layer keeps is made by a bind alone: a step without one holds up the next
    forward(), and is not captured."""
    s, kept, step, opt, side, inputs = made(True)
    assert s.fp16_operands(0)
    with pytest.raises(eg.EngramError) as e:
        s.refresh(0)
    assert e.value.status == eg.EUNSUPPORTED
    step.forward(*inputs[:3], side)
    step.backward(*inputs, side)
    torch.cuda.synchronize()
    before = kept["wq"].clone()
    for rebind in (False, True):
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(ValueError, match="captured"):
            with torch.cuda.graph(graph, stream=side):
                opt.step(side, rebind=rebind)
    torch.cuda.synchronize()
    assert int(opt.steps) == 0 and torch.equal(before, kept["wq"])
    opt.step(side, rebind=False)
    with pytest.raises(ValueError, match="rebind"):
        step.forward(*inputs[:3], side)
    torch.cuda.synchronize()
    assert int(opt.steps) == 1 and not torch.equal(before, kept["wq"])
    s.rebind(0)
    step.forward(*inputs[:3], side)
    got = step.loss.clone()
    # the same step with the bind in it
    t, _, step2, opt2, _, _ = made(True)
    step2.forward(*inputs[:3], side)
    step2.backward(*inputs, side)
    opt2.step(side)
    step2.forward(*inputs[:3], side)
    torch.cuda.synchronize()
    assert torch.equal(got, step2.loss)
    s.close()
    t.close()


def test_a_captured_forward_holds_over_binds():
    """On FP16 operands: the copy of wkv stays where a graph reads it, also while the layer is bound to
    a table that takes BF16 operands; where exponents change, the bind says so."""
    s, kept, step, opt, side, inputs = made(True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.forward(*inputs[:3], side)

    def replay():
        graph.replay()
        torch.cuda.synchronize()
        return step.kv.clone(), step.loss.clone()

    def eager():
        step.forward(*inputs[:3], side)
        torch.cuda.synchronize()
        return step.kv.clone(), step.loss.clone()

    def same(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))

    first = replay()
    assert same(first, eager())
    # other values of the same size: replays see them
    kept["wkv"].view(torch.bfloat16).neg_()
    kept["wq"].mul_(1.5)
    assert not s.rebind(0)
    changed = replay()
    assert same(changed, eager()) and not torch.equal(first[0], changed[0])
    # a scale far from the others takes the layer off FP16 operands, and back
    scale = int(kept["scales"][0])
    kept["scales"][0] = 30
    assert s.rebind(0) and not s.fp16_operands(0)
    hold = [torch.full((kept["wkv"].numel(),), -1, dtype=torch.int16, device="cuda") for _ in range(8)]
    kept["scales"][0] = scale
    assert s.rebind(0) and s.fp16_operands(0)
    assert same(replay(), changed) and len(hold) == 8
    # another exponent of wkv: captured again
    kept["wkv"].view(torch.bfloat16).mul_(4)
    assert s.rebind(0)
    graph.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.forward(*inputs[:3], side)
    assert same(replay(), eager())
    eg.engram_sync(s.ctx)
    s.close()


def test_a_step_takes_the_gradients_of_the_last_forward():
    """Neither buffers that no backward() wrote nor the gradients of a batch before."""
    s, kept, step, opt, side, inputs = made(False)
    weights = [x.clone() for x in (step.head, step.embedding, kept["wkv"])]
    step.forward(*inputs[:3], side)
    with pytest.raises(ValueError, match="backward"):
        opt.step(side)
    torch.cuda.synchronize()
    assert int(opt.steps) == 0
    assert all(torch.equal(a, b) for a, b in zip(weights, (step.head, step.embedding, kept["wkv"])))
    step.backward(*inputs, side)
    opt.step(side)
    step.forward(*inputs[:3], side)
    with pytest.raises(ValueError, match="backward"):
        opt.step(side)
    torch.cuda.synchronize()
    assert int(opt.steps) == 1
    eg.engram_sync(s.ctx)
    s.close()


@pytest.mark.parametrize("states", ["f32", "mxfp8"])
def test_what_follows_an_update_on_the_stream_reads_the_new_weights(states):
    """Kernels of the layer load wkv and the table before they wait for the kernel before them: the step's
    kernels let them start only when they are done."""
    s, kept, embedding, head, norm = step_model(False)
    T, mx = 64, states == "mxfp8"
    side = torch.cuda.Stream()
    dev = dict(device="cuda")
    emb = torch.randn(T, s.K, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    windows = step_inputs(s, T, 2)[1]
    ws = torch.empty(eg.engram_forward_staged_workspace_bytes(s.ctx, T), dtype=torch.uint8, **dev)
    wkv, rows, dim = kept["wkv"].view(torch.bfloat16), s.rows(0), s.geom["row_dim"]
    table = kept["table"].view(torch.bfloat16)[:rows * dim]

    def state(n):
        if not mx:
            return dict(m=torch.zeros(n, **dev), v=torch.zeros(n, **dev))
        return {k: torch.zeros(n if k in "mv" else n // 32, dtype=torch.uint8, **dev) for k in ("m", "v", "m_scales", "v_scales")}

    fmt = eg.MXFP8 if mx else eg.F32
    dense = eg.adamw_tensors([dict(param=wkv, grad=torch.ones_like(wkv), **state(wkv.numel()))])
    rows_table = eg.AdamWTable(table, rows, dim, eg.BF16, **state(rows * dim))
    ids = torch.arange(rows, dtype=torch.int32, **dev)
    count, grad = torch.tensor([rows], dtype=torch.int32, **dev), torch.ones(rows, dim, **dev)
    got = [torch.empty(T, s.N, **dev) for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(1, 21):
        step = eg.AdamWStep(lr=0.5, step=i, state_format=fmt)  # (every weight moves by 0.5)
        eg.engram_adamw(s.ctx, dense, step, side)
        eg.engram_project(s.ctx, 0, emb, T, got[0], side)
        torch.cuda.synchronize()
        eg.engram_project(s.ctx, 0, emb, T, got[1], side)
        eg.engram_adamw_rows(s.ctx, rows_table, ids, count, rows, grad, step, side)
        eg.engram_prepass(s.ctx, 0, windows, T, got[2], eg.KV_F32, ws, side)
        torch.cuda.synchronize()
        eg.engram_prepass(s.ctx, 0, windows, T, got[3], eg.KV_F32, ws, side)
        torch.cuda.synchronize()
        assert torch.equal(got[0], got[1]) and torch.equal(got[2], got[3]), i
    eg.engram_sync(s.ctx)
    s.close()
