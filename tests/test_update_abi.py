"""Refusals of the norm and the optimizer's operators (no GPU): arguments are checked before any
launch."""
import ctypes as C

import numpy as np
import pytest
import torch

import engram_gram_conditional_gb300 as eg


@pytest.fixture(scope="module")
def ctx():
    from engram_gram_conditional_gb300 import build

    build.build()
    c = eg.engram_ctx_create(64, 60, np.arange(64, dtype=np.uint32) % 60, [3], [50], heads=2,
                             row_dim=32, hc=2, d=256)
    yield c
    eg.engram_ctx_destroy(c)


A = 1 << 20  # an aligned address that no refused call touches
NAN, INF = float("nan"), float("inf")


def refused(status, f, *args):
    with pytest.raises(eg.EngramError) as e:
        f(*args)
    assert e.value.status == status


NORM = dict(x=A, fmt=eg.BF16, copies=2, scale=0.5, res=A, w=A, n=4, dim=64, eps=1e-6, sum=A, y=A,
            y_fmt=eg.MXFP8, scales=A)


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(y=None), dict(scales=None), dict(x=A + 8),
                                 dict(res=A + 8), dict(w=A + 4), dict(sum=A + 2), dict(y=A + 8), dict(fmt=2),
                                 dict(fmt=-1), dict(y_fmt=0), dict(y_fmt=3), dict(copies=0), dict(copies=9),
                                 dict(scale=NAN), dict(scale=INF), dict(n=-1), dict(n=2**30 + 1), dict(dim=0),
                                 dict(dim=12), dict(dim=40), dict(dim=16416), dict(eps=0.0), dict(eps=-1.0),
                                 dict(eps=NAN), dict(eps=INF)])
def test_norm_refuses(ctx, bad):
    refused(eg.EINVAL, eg.engram_norm, ctx, *{**NORM, **bad}.values())
    refused(eg.EINVAL, eg.engram_norm, None, *NORM.values())


BACK = dict(sum=A, fmt=eg.F32, w=A, n=4, dim=40, eps=1e-6, dy=A, dsum=A, copies=2, scale=0.5, dx=A, dres=A,
            dw=A, ws=A)


@pytest.mark.parametrize("bad", [dict(sum=None), dict(w=None), dict(dy=None), dict(ws=None), dict(sum=A + 8),
                                 dict(w=A + 8), dict(dy=A + 8), dict(dsum=A + 8), dict(dx=A + 8),
                                 dict(dres=A + 8), dict(dw=A + 8), dict(ws=A + 8), dict(fmt=2), dict(n=-1),
                                 dict(dim=4), dict(dim=16392), dict(copies=0), dict(scale=INF), dict(eps=0.0)])
def test_norm_backward_refuses(ctx, bad):
    refused(eg.EINVAL, eg.engram_norm_backward, ctx, *{**BACK, **bad}.values())
    refused(eg.EINVAL, eg.engram_norm_backward, None, *BACK.values())


def part(**bad):
    return eg.GradPart(**{**dict(grad=A, count=A, n=10, dim=8, format=eg.F32), **bad})


@pytest.mark.parametrize("bad", [dict(grad=None), dict(grad=A + 8), dict(count=A + 2), dict(dim=0),
                                 dict(format=2), dict(n=1 << 38)])
def test_grad_norm_refuses_a_part(ctx, bad):
    parts = (eg.GradPart * 2)(part(), part(**bad))
    refused(eg.EINVAL, eg.engram_grad_norm, ctx, parts, 1.0, A, A, A, A)


@pytest.mark.parametrize("bad", [dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=NAN), dict(norms=A + 2),
                                 dict(norm=A + 1), dict(factor=A + 2), dict(ws=None), dict(ws=A + 8)])
def test_grad_norm_refuses(ctx, bad):
    a = {**dict(max_norm=1.0, norms=A, norm=A, factor=A, ws=A), **bad}
    refused(eg.EINVAL, eg.engram_grad_norm, ctx, (eg.GradPart * 1)(part()), *a.values())
    refused(eg.EINVAL, eg.engram_grad_norm, None, (eg.GradPart * 1)(part()), 1.0, A, A, A, A)
    f = eg.lib().engram_grad_norm
    assert f(ctx, None, 1, 1.0, A, A, A, A, None) == eg.EINVAL
    assert f(ctx, None, -1, 1.0, A, A, A, A, None) == eg.EINVAL
    assert f(ctx, None, 65537, 1.0, A, A, A, A, None) == eg.EINVAL


def step(**bad):
    return eg.AdamWStep(**{**dict(lr=1e-3, step=1), **bad})


STEPS = [dict(lr=NAN), dict(lr=1e39), dict(beta1=-0.1), dict(beta1=1.0), dict(beta1=NAN), dict(beta2=1.0),
         dict(beta2=-1.0), dict(eps=0.0), dict(eps=-1e-8), dict(eps=1e-39), dict(eps=INF), dict(step=0),
         dict(d_lr=A + 2), dict(d_step=A + 1), dict(d_factor=A + 2), dict(state_format=eg.BF16),
         dict(state_format=3)]


def tensor(**bad):
    return eg.AdamWTensor(**{**dict(param=A, master=A, grad=A, m=A, v=A, m_scales=A, v_scales=A, n=10,
                                    lr_scale=1.0, weight_decay=0.0, param_format=eg.BF16,
                                    grad_format=eg.BF16), **bad})


TENSORS = [dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param=A + 2), dict(master=A + 8),
           dict(grad=A + 8), dict(m=A + 8), dict(v=A + 4), dict(n=(1 << 40) + 1), dict(lr_scale=NAN),
           dict(weight_decay=INF), dict(param_format=eg.MXFP8), dict(grad_format=2),
           dict(param_format=eg.F32)]  # (a master of an fp32 parameter)


@pytest.mark.parametrize("bad", STEPS)
def test_a_step_is_refused(ctx, bad):
    refused(eg.EINVAL, eg.engram_adamw, ctx, (eg.AdamWTensor * 1)(tensor()), step(**bad))
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(), A, A, 4, A, step(**bad))


@pytest.mark.parametrize("bad", TENSORS)
def test_a_tensor_is_refused(ctx, bad):
    refused(eg.EINVAL, eg.engram_adamw, ctx, (eg.AdamWTensor * 2)(tensor(), tensor(**bad)), step())


@pytest.mark.parametrize("bad", [dict(m_scales=None), dict(v_scales=None)])
def test_8_bit_states_need_scales(ctx, bad):
    eight = step(state_format=eg.MXFP8)
    refused(eg.EINVAL, eg.engram_adamw, ctx, (eg.AdamWTensor * 1)(tensor(**bad)), eight)
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(**bad), A, A, 4, A, eight)


def test_adamw_refuses(ctx):
    one = (eg.AdamWTensor * 1)(tensor())
    refused(eg.EINVAL, eg.engram_adamw, None, one, step())
    refused(eg.EINVAL, eg.engram_adamw, ctx, one, None)
    f, s = eg.lib().engram_adamw, step()
    assert f(ctx, None, 1, C.byref(s), None) == eg.EINVAL
    assert f(ctx, one, -1, C.byref(s), None) == eg.EINVAL
    assert f(ctx, one, 65537, C.byref(s), None) == eg.EINVAL
    eg.engram_adamw(ctx, (eg.AdamWTensor * 0)(), s)  # nothing to do
    eg.engram_adamw(ctx, (eg.AdamWTensor * 1)(tensor(n=0, param=None, grad=None, m=None, v=None)), s)


def table(**bad):
    return eg.AdamWTable(**{**dict(table=A, rows=10, dim=64, table_format=eg.MXFP8, m=A, v=A, scales=A, master=A,
                                   m_scales=A, v_scales=A), **bad})


@pytest.mark.parametrize("bad", [dict(table=None), dict(m=None), dict(v=None), dict(table=A + 8), dict(m=A + 8),
                                 dict(master=A + 8), dict(master=None), dict(scales=None), dict(rows=0),
                                 dict(rows=2**32 - 1), dict(dim=0), dict(dim=40), dict(dim=12), dict(dim=65568),
                                 dict(table_format=3), dict(table_format=eg.F32), dict(lr_scale=INF),
                                 dict(weight_decay=NAN)])
def test_rows_refuse_a_table(ctx, bad):
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(**bad), A, A, 4, A, step())


@pytest.mark.parametrize("bad", [dict(ids=None), dict(count=None), dict(grad=None), dict(ids=A + 2),
                                 dict(count=A + 1), dict(grad=A + 8), dict(n=-1), dict(n=2**30 + 1)])
def test_rows_refuse(ctx, bad):
    a = {**dict(ids=A, count=A, n=4, grad=A), **bad}
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(), *a.values(), step())
    refused(eg.EINVAL, eg.engram_adamw_rows, None, table(), A, A, 4, A, step())
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, None, A, A, 4, A, step())
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(), A, A, 4, A, None)
    eight = step(state_format=eg.MXFP8)
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(table_format=eg.BF16, dim=40), A, A, 4, A, eight)
    eg.engram_adamw_rows(ctx, table(), A, A, 0, A, step())  # no rows


def good(**bad):
    f = torch.zeros
    return {**dict(param=f(40, dtype=torch.bfloat16), grad=f(40), m=f(40, dtype=torch.uint8),
                   v=f(40, dtype=torch.uint8), m_scales=f(2, dtype=torch.uint8),
                   v_scales=f(2, dtype=torch.uint8)), **bad}


def test_a_list_of_tensors():
    got = eg.adamw_tensors([good(), good(master=torch.zeros(40), weight_decay=0.5, lr_scale=2.0)])
    assert [t.n for t in got] == [40, 40] and got[1].weight_decay == 0.5 and got[1].lr_scale == 2.0
    assert got[0].master is None and got[0].param_format == eg.BF16 and got[0].grad_format == eg.F32


@pytest.mark.parametrize("bad", [dict(grad=torch.zeros(39)), dict(m=torch.zeros(40)),
                                 dict(m_scales=torch.zeros(1, dtype=torch.uint8)),
                                 dict(master=torch.zeros(40, dtype=torch.bfloat16)),
                                 dict(master=torch.zeros(41)), dict(param=torch.zeros(40, dtype=torch.float16)),
                                 dict(grad=torch.zeros(40, dtype=torch.float64)),
                                 dict(grad=torch.zeros(80)[::2]),
                                 dict(m=torch.zeros(40, dtype=torch.int16), v=torch.zeros(40, dtype=torch.int16))])
def test_a_list_refuses_tensors_that_do_not_go_together(bad):
    refused(eg.EINVAL, eg.adamw_tensors, [good(), good(**bad)])


def test_a_list_goes_with_its_state_format(ctx):
    tensors = eg.adamw_tensors([good()])
    refused(eg.EINVAL, eg.engram_adamw, ctx, tensors, step(state_format=eg.F32))


def test_a_list_of_gradients():
    got = eg.grad_parts([dict(grad=torch.zeros(6, 8)), dict(grad=torch.zeros(6, 8), count=A, dim=8)])
    assert (got[0].n, got[0].dim, got[1].n, got[1].dim, got[1].count) == (48, 1, 6, 8, A)
    refused(eg.EINVAL, eg.grad_parts, [dict(grad=torch.zeros(6, 8), dim=5)])
    refused(eg.EINVAL, eg.grad_parts, [dict(grad=torch.zeros(6, 8).t())])
    refused(eg.EINVAL, eg.grad_parts, [dict(grad=torch.zeros(6, dtype=torch.float16))])


def test_workspace_sizes():
    for dim in (8, 96, 1000, 5120, 16384):
        sizes = [eg.engram_norm_backward_workspace_bytes(n, dim) for n in (*range(0, 900), 5000, 10 ** 6)]
        assert sizes == sorted(sizes) and sizes[0] > 0
    assert eg.engram_norm_backward_workspace_bytes(4, 12) == 0
    assert eg.engram_norm_backward_workspace_bytes(-1, 64) == 0
    lists = lambda n, rows: (eg.GradPart * n)(*[part(n=rows) for _ in range(n)])  # noqa: E731
    for rows in (0, 1, 5000, 10 ** 7):
        sizes = [eg.engram_grad_norm_workspace_bytes(lists(n, rows)) for n in range(0, 900, 7)]
        assert sizes == sorted(sizes)
    sizes = [eg.engram_grad_norm_workspace_bytes(lists(3, n)) for n in (*range(0, 9000, 31), 10 ** 6, 10 ** 9)]
    assert sizes == sorted(sizes) and sizes[-1] < 1 << 20
    assert eg.engram_grad_norm_workspace_bytes(lists(1, 1 << 38)) == 0


def test_a_step_refuses_norm_weights_of_another_shape():
    from types import SimpleNamespace

    from engram_gram_conditional_gb300.training import TrainStep

    model = SimpleNamespace(device=torch.device("cpu"), geom=dict(d=256, hc=2, row_dim=32), ctx=None)
    w = torch.zeros(10, 256, dtype=torch.bfloat16)
    for norm in (torch.ones(255), torch.ones(256, dtype=torch.bfloat16), torch.ones(512)[::2]):
        with pytest.raises(ValueError):
            TrainStep(model, 0, w, w, 4, norm=norm)


def test_an_optimizer_refuses():
    from types import SimpleNamespace

    from engram_gram_conditional_gb300.training import AdamW

    host = SimpleNamespace(model=SimpleNamespace(device=torch.device("cpu"), tensors=[dict(table=torch.zeros(4))]),
                           layer=0)
    with pytest.raises(ValueError):
        AdamW(host, 1e-3, states=eg.BF16)
    with pytest.raises(ValueError):
        AdamW(host, 1e-3)  # a table that is not in device memory


def test_lists_and_structs_keep_their_tensors():
    import gc
    import weakref

    f = torch.zeros
    t = good()
    seen = [weakref.ref(x) for x in t.values()] + [weakref.ref(g := f(8))]
    kept = [eg.adamw_tensors([t]), eg.grad_parts([dict(grad=g)])]
    lr, m = f(1), f(10, 64)
    seen += [weakref.ref(lr), weakref.ref(m)]
    kept += [eg.AdamWStep(d_lr=lr), eg.AdamWTable(m, 10, 64, eg.F32, m, m)]
    del t, g, lr, m
    gc.collect()
    assert all(x() is not None for x in seen)
    kept.clear()
    gc.collect()
    assert all(x() is None for x in seen)


def test_refresh_refuses(ctx):
    refused(eg.EINVAL, eg.engram_layer_refresh, None, 0)
    refused(eg.EINVAL, eg.engram_layer_refresh, ctx, 1)
    refused(eg.EINVAL, eg.engram_layer_refresh, ctx, -1)
    refused(eg.ESTATE, eg.engram_layer_refresh, ctx, 0)  # not bound


def test_a_step_on_an_outdated_layer_is_refused():
    from types import SimpleNamespace

    from engram_gram_conditional_gb300.training import TrainStep

    step = object.__new__(TrainStep)  # (its buffers need a GPU; what is refused reaches none)
    step.model = SimpleNamespace(device=torch.device("cpu"), ctx=None, outdated={1})
    step.layer, step.tokens, step.T = 1, 8, 0
    i32 = torch.int32
    with pytest.raises(ValueError, match="rebind"):
        step.forward(torch.zeros(5, dtype=i32), torch.zeros(5, 4, dtype=i32), torch.zeros(5, dtype=i32))
    assert step.T == 0


def test_an_optimizer_refuses_a_forward_without_its_backward():
    from types import SimpleNamespace

    from engram_gram_conditional_gb300.training import AdamW, TrainStep

    opt = object.__new__(AdamW)  # (its buffers need a GPU; what is refused reaches none)
    opt.train = object.__new__(TrainStep)
    opt.train.model, opt.train.T = SimpleNamespace(ctx=None), 5
    with pytest.raises(ValueError, match="backward"):
        opt.step()


def eight_rows(**bad):
    f = torch.zeros
    u8 = torch.uint8
    return {**dict(table=f(10, 64, dtype=u8), rows=10, dim=64, table_format=eg.MXFP8, m=f(10, 64, dtype=u8),
                   v=f(10, 64, dtype=u8), scales=f(10, 2, dtype=u8), master=f(10, 64), m_scales=f(10, 2, dtype=u8),
                   v_scales=f(24, dtype=u8)), **bad}


@pytest.mark.parametrize("bad", [dict(table=torch.zeros(10, 64)), dict(table=torch.zeros(9, 64, dtype=torch.uint8)),
                                 dict(table=torch.zeros(10, 128, dtype=torch.uint8)[:, ::2]),
                                 dict(table_format=eg.BF16), dict(table_format=eg.F32),
                                 dict(scales=torch.zeros(19, dtype=torch.uint8)), dict(scales=torch.zeros(20)),
                                 dict(master=torch.zeros(10, 64, dtype=torch.bfloat16)), dict(master=torch.zeros(639)),
                                 dict(m=torch.zeros(10, 64)), dict(v=torch.zeros(10, 63, dtype=torch.uint8)),
                                 dict(m=torch.zeros(10, 64, dtype=torch.int16), v=torch.zeros(10, 64, dtype=torch.int16)),
                                 dict(m_scales=torch.zeros(19, dtype=torch.uint8)),
                                 dict(v_scales=torch.zeros(20, dtype=torch.int16))])
def test_a_table_refuses_buffers_that_do_not_go_together(bad):
    assert eg.AdamWTable(**eight_rows()).state_format == eg.MXFP8
    refused(eg.EINVAL, lambda: eg.AdamWTable(**eight_rows(**bad)))


@pytest.mark.parametrize("bad", [dict(d_lr=torch.zeros(1, dtype=torch.float64)), dict(d_lr=torch.zeros(0)),
                                 dict(d_step=torch.zeros(1)), dict(d_step=torch.zeros(1, dtype=torch.int64)),
                                 dict(d_factor=torch.zeros(1, dtype=torch.bfloat16))])
def test_a_step_refuses_words_of_another_type(bad):
    refused(eg.EINVAL, lambda: eg.AdamWStep(**bad))


def test_buffers_that_are_not_on_the_device_are_refused(ctx):
    """Before a kernel gets their addresses."""
    eight, i32 = step(state_format=eg.MXFP8), torch.int32
    refused(eg.EINVAL, eg.engram_adamw, ctx, eg.adamw_tensors([good()]), eight)
    refused(eg.EINVAL, eg.engram_adamw, ctx, (eg.AdamWTensor * 1)(tensor()), step(d_lr=torch.zeros(1)))
    refused(eg.EINVAL, eg.engram_grad_norm, ctx, eg.grad_parts([dict(grad=torch.zeros(8))]), 1.0, A, A, A, A)
    refused(eg.EINVAL, eg.engram_grad_norm, ctx, eg.grad_parts([dict(grad=torch.zeros(8, device="meta"))]), 1.0, A, A, A, A)
    refused(eg.EINVAL, eg.grad_parts, [dict(grad=torch.zeros(8), count=torch.zeros(1, dtype=torch.int64))])
    rows = eg.AdamWTable(**eight_rows())
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, rows, A, A, 4, A, eight)
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, rows, A, A, 4, A, step())  # (fp32 states)
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(), torch.zeros(4, dtype=i32), A, 4, A, step())
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(), A, np.zeros(1, np.int32), 4, A, step())


@pytest.mark.parametrize("bad", [dict(ids=torch.zeros(3, dtype=torch.int32)), dict(ids=torch.zeros(4, dtype=torch.int64)),
                                 dict(count=torch.zeros(1, dtype=torch.int64)), dict(grad=torch.zeros(4, 63)),
                                 dict(grad=torch.zeros(4, 64, dtype=torch.bfloat16))])
def test_rows_refuse_tensors_of_another_size(ctx, bad, monkeypatch):
    monkeypatch.setattr(eg, "_on_device", lambda *a: None)
    a = {**dict(ids=A, count=A, n=4, grad=A), **bad}
    refused(eg.EINVAL, eg.engram_adamw_rows, ctx, table(), *a.values(), step())
