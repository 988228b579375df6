"""The AdamW step where its arithmetic is sensitive: small states and factors, roots and quotients to
their last bit."""
import numpy as np
import pytest
import torch

import engram_gram_conditional_gb300 as eg
from test_gpu_update import check_rows, check_tensor, ctx, listed, on_gpu, run_rows  # noqa: F401 (ctx: the fixture)
from update_reference import HYPER, encode, rnd

pytestmark = pytest.mark.gpu
F32, U8 = torch.float32, torch.uint8
SMALL = 2.0 ** -62


def small_states(seed, *shape):
    """m, and roots between SMALL and 2 SMALL: their squares are normal fp32 numbers, the square of
    their block's scale (2^-70) is not."""
    (m, ms), (v, vs) = encode(rnd(seed, *shape, sigma=SMALL)), encode(SMALL * (1 + rnd(seed + 1, *shape).abs().clamp_max(1)))
    return dict(m=m, v=v, m_scales=ms, v_scales=vs)


@pytest.mark.parametrize("grad,factor", [(SMALL, 1.0), (2.0 ** 50, 2.0 ** -70)])
def test_adamw_of_small_states_or_by_a_small_factor(ctx, grad, factor):  # noqa: F811
    """Roots of 2^-62, and a factor whose square leaves fp32's range while factor x gradient (2^-20) and
    v do not."""
    n = 1 << 16
    t = dict(param=rnd(1, n), master=None, grad=rnd(2, n, sigma=grad), **{k: x[0] for k, x in small_states(3, 1, n).items()})
    gpu = on_gpu(t, n)
    d_factor = torch.tensor([factor], device="cuda")
    s = eg.AdamWStep(**HYPER, step=3, seed=7, state_format=eg.MXFP8, d_factor=d_factor)
    eg.engram_adamw(ctx, listed([gpu], [{}]), s)
    check_tensor(t, gpu, n, 0, True, 3, 7, factor, 1.0, 0.0)


def test_adamw_rows_of_small_states(ctx):  # noqa: F811
    rows, dim = 300, 256
    t = dict(master=None, table=rnd(1, rows, dim), **small_states(2, rows, dim))
    ids, grad = torch.arange(0, rows, 2, dtype=torch.int32), rnd(4, rows // 2, dim, sigma=SMALL)
    gpu = run_rows(ctx, t, rows, dim, "f32", True, ids, len(ids), grad)
    eg.engram_sync(ctx)
    check_rows(t, gpu, rows, dim, "f32", True, ids, grad)
