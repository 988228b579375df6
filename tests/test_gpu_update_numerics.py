"""The AdamW step where its arithmetic is sensitive: small states and factors, roots and quotients to
their last bit."""
import numpy as np
import pytest
import torch

import engram_gram_conditional_gb300 as eg
from test_gpu_update import check_rows, check_tensor, ctx, listed, on_gpu, run_rows  # noqa: F401 (ctx: the fixture)
from update_reference import HYPER, decode, encode, noise_of, rnd

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


def codes_of(x, places, step, seed):
    """Codes and scales of fp32 m and root, rounded with the operator's random numbers."""
    noise = noise_of(places, 0, step, seed)
    return encode(x[0], noise), encode(x[1], noise, True)


def test_roots_of_squares_are_exact(ctx):  # noqa: F811
    """With both betas 0 m is the gradient x, v its square rounded and the root |x|: the rounded root of a
    rounded square is the number itself.  Every x is chosen by its random number: at even places it
    just reaches the next code, at odd ones it just does not, so that a root one unit in the last place
    too low or too high takes another code."""
    n, step, seed = 1 << 18, 3, 11
    places = np.arange(n)
    noise = noise_of(places, 0, step, seed)
    low = np.where(places % 2 == 0, (65536 - np.maximum(noise, 1)) << 4, (65535 - noise) << 4 | 15)
    # 1.xxx in [1, 1.75): three bits that a code keeps, then the 16 that meet the random ones, then 4
    bits = 0x3F800000 | np.random.default_rng(1).integers(0, 6, n) << 20 | low
    g = torch.from_numpy(bits.astype(np.int32).view(np.float32))
    assert np.array_equal(np.sqrt(g.numpy() * g.numpy()), g.numpy())
    new = lambda k, d: torch.zeros(k, dtype=d, device="cuda")  # noqa: E731
    t = dict(param=new(n, F32), grad=g.cuda(), m=new(n, U8), v=new(n, U8), m_scales=new(n // 32, U8),
             v_scales=new(n // 32, U8))
    s = eg.AdamWStep(lr=0.0, beta1=0.0, beta2=0.0, eps=1e-6, step=step, seed=seed, state_format=eg.MXFP8)
    eg.engram_adamw(ctx, eg.adamw_tensors([t]), s)
    for name, (codes, scales) in zip("mv", codes_of((g, g), places, step, seed)):
        assert torch.equal(t[name].cpu(), codes) and torch.equal(t[name + "_scales"].cpu(), scales), name


def test_8_bit_states_are_those_of_rounded_values(ctx):  # noqa: F811
    """m = fma(1 - b1, f, b1 m), v = fma(1 - b2, f^2, b2 r^2) and its root, each rounded once to fp32: the
    codes to the last one."""
    n, step, seed = 1 << 21, 5, 3
    b1, b2, factor = np.float32(HYPER["beta1"]), np.float32(HYPER["beta2"]), np.float32(0.7)
    nb1, nb2 = np.float32(1 - HYPER["beta1"]), np.float32(1 - HYPER["beta2"])
    (mc, ms), (vc, vs) = encode(rnd(1, n, sigma=0.3)), encode(rnd(2, n).abs() + 0.01)
    grad = rnd(3, n)
    f = grad.numpy() * factor
    m, r = (decode(c, e).float().numpy() for c, e in ((mc, ms), (vc, vs)))
    up = lambda x: x.astype(np.float64)  # noqa: E731  (products of two fp32 numbers are exact there)
    m = (up(f) * up(nb1) + up(m * b1)).astype(np.float32)
    v = (up(f * f) * up(nb2) + up(r * r * b2)).astype(np.float32)
    t = dict(param=torch.zeros(n), grad=grad, m=mc, v=vc, m_scales=ms, v_scales=vs)
    t = {k: x.cuda() for k, x in t.items()}
    s = eg.AdamWStep(**HYPER, step=step, seed=seed, state_format=eg.MXFP8, d_factor=torch.tensor([0.7], device="cuda"))
    eg.engram_adamw(ctx, eg.adamw_tensors([t]), s)
    want = codes_of((torch.from_numpy(m), torch.from_numpy(np.sqrt(v))), np.arange(n), step, seed)
    for name, (codes, scales) in zip("mv", want):
        assert torch.equal(t[name].cpu(), codes) and torch.equal(t[name + "_scales"].cpu(), scales), name


def test_fp32_steps_round_their_quotient(ctx):  # noqa: F811
    """With betas and a parameter of 0 and a rate of 1 the new parameter is -g / (|g| + eps): one sum and
    one quotient, each rounded to fp32."""
    n, hyper = 1 << 16, dict(lr=1.0, beta1=0.0, beta2=0.0, eps=0.3)
    g = rnd(5, n)
    want = torch.from_numpy(-(g.numpy() / (np.abs(g.numpy()) + np.float32(0.3))))
    zeros = lambda: torch.zeros(n, device="cuda")  # noqa: E731
    t = dict(param=zeros(), grad=g.cuda(), m=zeros(), v=zeros())
    eg.engram_adamw(ctx, eg.adamw_tensors([t]), eg.AdamWStep(**hyper, step=1))
    assert torch.equal(t["param"].cpu(), want)
    table = eg.AdamWTable(zeros(), n // 64, 64, eg.F32, zeros(), zeros())
    ids = torch.arange(n // 64, dtype=torch.int32, device="cuda")
    count = torch.tensor([n // 64], dtype=torch.int32, device="cuda")
    eg.engram_adamw_rows(ctx, table, ids, count, n // 64, t["grad"], eg.AdamWStep(**hyper, step=1))
    eg.engram_sync(ctx)
    assert torch.equal(table.kept[0].cpu(), want)
