"""The training operators against plain 64-bit formulas, through the C ABI.

Tolerances (u = 2^-8 is a BF16 rounding's relative bound of half an ulp, 2^-9,
doubled for the step to the next binade; eps = 2^-23):
  embed         one BF16 rounding of an fp32 product: |err| <= 2^-8 |ref|
  embed_grad    fp32 sums of m terms: |err| <= (m + 4) 2^-24 sum |term|
  gate          gates 1e-5 + the dot's fp32 error through the root's slope; hidden
                one BF16 rounding plus the gate's error times |v|
  gate backward one BF16 rounding plus 2^-12 of the terms' magnitudes (the fp32
                sums of up to 1,024 columns, twice, through a slope of at most 2)
  products      one BF16 rounding plus K 2^-23 sum |a b|
  loss          dim 2^-23 max_v sum_i |x_i h_vi| + 2^-20 (1 + |ref|)
  loss backward dz is rounded to BF16 once and the sums once more:
                2^-8 (|ref| + sum |dz h|) + K 2^-23 sum |dz h|
"""
import math

import numpy as np
import pytest
import torch

import engram_gram_conditional_gb300 as eg
from engram_gram_conditional_gb300.layer import EngramLayerSet
from engram_gram_conditional_gb300.training import TrainStep
from gate_reference import GateGradients, gate_inputs

pytestmark = pytest.mark.gpu
F = torch.float64


@pytest.fixture(scope="module", autouse=True)
def built():
    from engram_gram_conditional_gb300 import build

    build.build()
    assert torch.cuda.is_available()


def make_layer(hc=1, d=256, heads=2, row_dim=32, wkv=None, wq=None, wk=None, eps=1e-6):
    N, K = (hc + 1) * d, 3 * heads * row_dim
    s = EngramLayerSet(64, 60, np.arange(64, dtype=np.uint32) % 60, [3], [50], heads=heads,
                       row_dim=row_dim, hc=hc, d=d, eps=eps)
    wkv = torch.zeros(N, K, dtype=torch.bfloat16) if wkv is None else wkv
    one = torch.ones(hc, d)
    s.bind(0, 3, wkv.cuda().view(torch.int16), one if wq is None else wq, one if wk is None else wk)
    torch.cuda.synchronize()
    return s


@pytest.fixture(scope="module")
def plain_ctx():
    s = make_layer()
    yield s.ctx
    s.close()


def rnd(seed, *shape, sigma=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sigma).to(dtype)


def ws_of(n):
    return torch.full((max(int(n), 16),), 0xA5, dtype=torch.uint8, device="cuda")


# ---- embedding ------------------------------------------------------------------------

@pytest.mark.parametrize("table", ["f32", "bf16"])
@pytest.mark.parametrize("n,rows,dim,copies", [(1, 1, 8, 1), (1, 5, 5120, 4), (77, 300, 264, 3),
                                               (300, 1000, 40, 8), (5, 9, 2056, 1)])
def test_embed(plain_ctx, table, n, rows, dim, copies):
    w = rnd(n, rows, dim, dtype=torch.float32 if table == "f32" else torch.bfloat16)
    ids = torch.randint(0, rows, (n,), generator=torch.Generator().manual_seed(n)).int()
    ids[n // 2] = -1
    ids[0] = rows - 1
    out = torch.full((n, copies, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    eg.engram_embed(plain_ctx, w.cuda(), eg.EMBED_F32 if table == "f32" else eg.EMBED_BF16, rows,
                    dim, ids.cuda(), n, 1.7, copies, out)
    eg.engram_sync(plain_ctx)
    ref = w.to(F)[ids.clamp_min(0).long()] * 1.7 * (ids >= 0).unsqueeze(1)
    ref = ref.unsqueeze(1).expand(-1, copies, -1)
    assert ((out.cpu().to(F) - ref).abs() <= 2.0 ** -8 * ref.abs()).all()


def test_embed_reports_ids_outside_the_table(plain_ctx):
    w = rnd(0, 10, 64).cuda()
    ids = torch.tensor([3, 10, -1, 9], dtype=torch.int32).cuda()
    out = torch.empty(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    eg.engram_embed(plain_ctx, w, eg.EMBED_BF16, 10, 64, ids, 4, 1.0, 1, out)
    with pytest.raises(eg.EngramError) as e:
        eg.engram_sync(plain_ctx)
    assert e.value.status == eg.EBOUNDS
    assert torch.equal(out[0, 0], w[3]) and torch.equal(out[3, 0], w[9])
    assert not out[1:3].any()
    eg.engram_sync(plain_ctx)


def grad_reference(ids, dout, rows, scale):
    ok = (ids >= 0) & (ids < rows)
    unique, inverse, m = torch.unique(ids[ok].long(), return_inverse=True, return_counts=True)
    src = dout[ok].to(F).sum(1)
    ref = torch.zeros(unique.numel(), dout.shape[2], dtype=F).index_add_(0, inverse, src) * scale
    mag = torch.zeros_like(ref).index_add_(0, inverse, dout[ok].to(F).abs().sum(1)) * abs(scale)
    tol = (m.to(F) * dout.shape[1] + 4).unsqueeze(1) * 2.0 ** -24 * mag
    return unique, ref, tol


def ids_like(kind, n, rows, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((n,), rows - 1)
    elif kind == "distinct":
        ids = torch.randperm(rows, generator=g)[:n]
    elif kind == "masked":
        ids = torch.full((n,), -1)
    else:
        u = torch.rand(n, generator=g, dtype=F)
        ids = (torch.exp(u * math.log(rows + 1)) - 1).long().clamp(0, rows - 1)
        ids[torch.rand(n, generator=g) < 0.05] = -1
    return ids.int()


SPARSE = [("zipf", 1, 7, 8, 1), ("zipf", 33, 300, 64, 2), ("one", 700, 10, 264, 1),
          ("distinct", 500, 600, 32, 1), ("masked", 65, 10, 64, 1), ("zipf", 5000, 129_280, 40, 3),
          ("zipf", 30_000, 64_000_000, 32, 1), ("one", 20_001, 4_000_000_000, 8, 1),
          ("zipf", 8192, 5000, 16, 1), ("zipf", 16_384, 70_000, 8, 1), ("zipf", 16_385, 9, 8, 1),
          ("distinct", 32_768, 32_768, 8, 1), ("zipf", 32_769, 800_000, 8, 1),
          ("zipf", 1_300_000, 40_000_000, 8, 1), ("one", 160_000, 5, 8, 2),
          ("masked", 40_000, 5, 8, 1), ("zipf", 2000, 511, 5120, 4), ("zipf", 2000, 512, 256, 1), ("zipf", 8193, 1, 16, 1)]


@pytest.mark.parametrize("kind,n,rows,dim,copies", SPARSE)
def test_embed_grad_sparse(plain_ctx, kind, n, rows, dim, copies):
    ids = ids_like(kind, n, rows, n)
    if kind == "one":  # (ids are u32: one above 2^31 too)
        ids = torch.full((n,), rows - 1, dtype=torch.int64).numpy().astype(np.uint32).view(np.int32)
        ids = torch.from_numpy(ids.copy())
    dout = rnd(n + 1, n, copies, dim)
    grad = torch.full((n, dim), 7.0, device="cuda")
    unique = torch.full((n,), -5, dtype=torch.int32, device="cuda")
    count = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    ws = ws_of(eg.engram_embed_grad_workspace_bytes(n, rows, dim))
    eg.engram_embed_grad(plain_ctx, rows, dim, ids.cuda(), n, 0.5, copies, dout.cuda(), unique,
                         count, grad, 0, ws)
    eg.engram_sync(plain_ctx)
    wide = torch.from_numpy(ids.numpy().view(np.uint32).astype(np.int64))
    wide[wide == 0xFFFFFFFF] = -1
    u, ref, tol = grad_reference(wide, dout, rows, 0.5)
    m = int(count)
    assert m == u.numel()
    got = torch.from_numpy(unique.cpu().numpy().view(np.uint32).astype(np.int64))
    assert torch.equal(got[:m], u)
    assert (unique[m:] == -5).all() and (grad[m:] == 7.0).all()
    assert ((grad[:m].cpu().to(F) - ref).abs() <= tol).all()


@pytest.mark.parametrize("n,rows,dim,copies", [(1, 3, 8, 1), (900, 130, 264, 4), (4097, 2000, 64, 1)])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_embed_grad_dense(plain_ctx, n, rows, dim, copies, accumulate):
    ids = ids_like("zipf", n, rows, n)
    dout = rnd(n + 1, n, copies, dim)
    before = rnd(5, rows, dim, dtype=torch.float32)
    grad = before.cuda()
    ws = ws_of(eg.engram_embed_grad_workspace_bytes(n, rows, dim))
    eg.engram_embed_grad(plain_ctx, rows, dim, ids.cuda(), n, 2.0, copies, dout.cuda(), None, None,
                         grad, accumulate, ws)
    eg.engram_sync(plain_ctx)
    u, ref, tol = grad_reference(ids.long(), dout, rows, 2.0)
    full = before.to(F) if accumulate else torch.zeros(rows, dim, dtype=F)
    ftol = torch.zeros(rows, dim, dtype=F)
    full[u] += ref
    ftol[u] = tol + 2.0 ** -23 * (full[u].abs() + ref.abs())
    assert ((grad.cpu().to(F) - full).abs() <= ftol).all()


def test_embed_grad_of_no_ids(plain_ctx):
    count = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    grad = torch.ones(4, 8, device="cuda")
    some = torch.zeros(4, dtype=torch.int32, device="cuda")
    eg.engram_embed_grad(plain_ctx, 4, 8, None, 0, 1.0, 1, None, some, count, grad, 0, None)
    eg.engram_sync(plain_ctx)
    assert int(count) == 0 and (grad == 1).all()
    eg.engram_embed_grad(plain_ctx, 4, 8, None, 0, 1.0, 1, None, None, None, grad, 0, None)
    eg.engram_sync(plain_ctx)
    assert not grad.any()


def test_embed_grad_reports_ids_outside_the_table_and_repeats_bit_for_bit(plain_ctx):
    n, rows, dim = 20_000, 50, 64
    ids = ids_like("zipf", n, rows, 1)
    ids[17] = rows + 3
    dout = rnd(2, n, 1, dim).cuda()
    ws = ws_of(eg.engram_embed_grad_workspace_bytes(n, rows, dim))
    runs = []
    for _ in range(2):
        grad = torch.zeros(rows, dim, device="cuda")
        eg.engram_embed_grad(plain_ctx, rows, dim, ids.cuda(), n, 1.0, 1, dout, None, None, grad, 0, ws)
        with pytest.raises(eg.EngramError) as e:
            eg.engram_sync(plain_ctx)
        assert e.value.status == eg.EBOUNDS
        runs.append(grad)
    assert torch.equal(runs[0], runs[1])
    u, ref, tol = grad_reference(ids.long(), dout.cpu(), rows, 1.0)
    assert ((runs[0].cpu().to(F)[u] - ref).abs() <= tol).all()


# ---- gate -----------------------------------------------------------------------------------

def pack_ref(x):
    """Codes and exponents of fp32 x [..., n] by the definition, one block at a time."""
    b = x.double().reshape(-1, 32)
    top = b.abs().amax(1)
    e = torch.zeros(b.shape[0], dtype=torch.int64)
    nz = top > 0
    e[nz] = torch.ceil(torch.log2(top[nz] / 448) - 1e-12).long() + 127
    e = e.clamp(0, 254)
    codes = torch.ldexp(b, (127 - e).unsqueeze(1)).float().to(torch.float8_e4m3fn)
    return codes.reshape(x.shape), e.to(torch.uint8).reshape(*x.shape[:-1], -1)


def unpack_ref(codes, exps):
    v = codes.float().double().reshape(*exps.shape, 32)
    return torch.ldexp(v, (exps.long() - 127).unsqueeze(-1)).reshape(codes.shape)


def gate_problem(T, hc, d, seed, image=(1,)):
    h = rnd(seed, T, hc, d)
    kv = rnd(seed + 1, T, (hc + 1) * d, dtype=torch.float32)
    g = torch.Generator().manual_seed(seed)
    lean = 0.5 * torch.sign(torch.rand(T, hc, 1, generator=g) - 0.5)
    kv[:, :hc * d] += (lean * h.float()).reshape(T, hc * d)  # dots well away from 0
    win = torch.randint(0, 50, (T, 4), generator=g).int()
    for t in image:
        if t < T:
            win[t, 0] = -1
    wq = 1 + rnd(seed + 2, hc, d, sigma=0.1, dtype=torch.float32)
    wk = 1 + rnd(seed + 3, hc, d, sigma=0.1, dtype=torch.float32)
    return h, kv, win, wq, wk


def gate_ref(h, kv, on, wq, wk, eps=1e-6):
    T, hc, d = h.shape
    k, v = kv[:, :hc * d].reshape(T, hc, d), kv[:, hc * d:].reshape(T, 1, d)
    nh = h / torch.sqrt((h * h).mean(2, keepdim=True) + eps)
    nk = k / torch.sqrt((k * k).mean(2, keepdim=True) + eps)
    dot = (nh * wq * nk * wk).sum(2, keepdim=True) / math.sqrt(d)
    size = torch.where(dot.abs() > 1e-6, dot.abs(), torch.full_like(dot, 1e-6))
    root = torch.where(torch.signbit(dot), -size.sqrt(), size.sqrt())
    gate = torch.sigmoid(root) * on
    return h + gate * v, gate, dot


GATE = [(1, 1, 256), (3, 2, 512), (5, 4, 1024), (7, 3, 512), (2, 8, 256), (9, 5, 2816)]


@pytest.mark.parametrize("kv_format", [eg.KV_F32, eg.KV_BF16])
@pytest.mark.parametrize("T,hc,d", GATE)
def test_gate_checkpoint(T, hc, d, kv_format):
    h, kv, win, wq, wk = gate_problem(T, hc, d, 10 * T + hc)
    if kv_format == eg.KV_BF16:
        kv = kv.bfloat16()
    kv[0, :32] = 0                  # a block of zeros
    kv[0, 32:64] *= 2.0 ** -120     # exponents at the bottom of the range
    kv[0, 64] = 448 * 3.0           # a block whose top is the largest code exactly
    kv[0, 65] = 0
    on = (win[:, 0] != -1).to(F).reshape(T, 1, 1)
    if T > 1:
        kv[1] = float("nan")        # image row: its kv is not read
    s = make_layer(hc, d, wq=wq, wk=wk)
    kept = (2 * hc + 1) * d
    out = torch.full((T, hc, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    gates = torch.full((T, hc), float("nan"), device="cuda")
    codes = torch.full((T, kept), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((T, kept // 32), 0x55, dtype=torch.uint8, device="cuda")
    eg.engram_gate_checkpoint(s.ctx, 0, kv.cuda(), kv_format, win.cuda(), T, h.cuda(), out, gates,
                              codes, scales)
    inplace = h.cuda()
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    eg.engram_gate_checkpoint(s.ctx, 0, kv.cuda(), kv_format, win.cuda(), T, inplace, inplace, None,
                              c2, s2)
    eg.engram_sync(s.ctx)
    assert torch.equal(inplace, out) and torch.equal(c2, codes) and torch.equal(s2, scales)
    kvf = torch.nan_to_num(kv.float())
    ref, gate, dot = gate_ref(h.to(F), kvf.to(F), on, wq.to(F), wk.to(F))
    gtol = 1e-5 + 1e-6 / dot.abs().clamp_min(1e-6).sqrt()
    assert ((gates.cpu().to(F) - gate[..., 0]).abs() <= gtol[..., 0]).all()
    v = kvf[:, hc * d:].to(F).reshape(T, 1, d)
    assert ((out.cpu().to(F) - ref).abs() <= 2.0 ** -8 * ref.abs() + gtol * v.abs()).all()
    all_ = torch.cat([h.float().reshape(T, hc * d), kvf], 1) * on.float().reshape(T, 1)
    rc, re = pack_ref(all_)
    assert torch.equal(scales.cpu(), re)
    assert torch.equal(codes.cpu().view(torch.float8_e4m3fn).float(), rc.float())
    s.close()


@pytest.mark.parametrize("kv_format", [eg.KV_F32, eg.KV_BF16])
@pytest.mark.parametrize("T,hc,d", [(700, 2, 256), (320, 4, 5120), (3, 8, 9216), (2, 1, 20_736)])
def test_gate_checkpoint_of_many_and_of_wide_tokens(T, hc, d, kv_format):
    test_gate_checkpoint(T, hc, d, kv_format)


def test_a_dot_that_is_nan_is_taken_for_zero_as_by_engram_gate():
    """max(|dot|, 1e-6) leaves a NaN out (fmax), in the oracle and in every call of the library: the
    branch's gate is that of a dot of 0, engram_gate's and the checkpoint's alike; what is infinite
    or NaN in the activations itself reaches the branch's outputs; other branches and tokens do
    not see it."""
    T, hc, d = 3, 2, 512
    h, kv, win, wq, wk = gate_problem(T, hc, d, 6, image=())
    kv[1, 5] = float("nan")     # a key of branch 0
    h[2, 1, 7] = float("inf")   # hidden of branch 1: rh = 0, dot = 0 inf = NaN
    dy = rnd(9, T, hc, d)
    s = make_layer(hc, d, wq=wq, wk=wk)
    plain, pgates = h.cuda(), torch.empty(T, hc, device="cuda")
    eg.engram_gate(s.ctx, 0, kv.cuda(), win.cuda(), T, plain, pgates)
    out, gates = torch.empty_like(plain), torch.empty_like(pgates)
    kept = (2 * hc + 1) * d
    codes = torch.empty(T, kept, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, kept // 32, dtype=torch.uint8, device="cuda")
    eg.engram_gate_checkpoint(s.ctx, 0, kv.cuda(), eg.KV_F32, win.cuda(), T, h.cuda(), out, gates, codes, scales)
    ws = ws_of(eg.engram_gate_backward_workspace_bytes(s.ctx, T))
    dh = torch.empty(T, hc, d, dtype=torch.bfloat16, device="cuda")
    dkv = torch.empty(T, (hc + 1) * d, dtype=torch.bfloat16, device="cuda")
    dwq, dwk = (torch.empty(hc, d, device="cuda") for _ in range(2))
    eg.engram_gate_backward(s.ctx, 0, kv.cuda(), eg.KV_F32, h.cuda(), win.cuda(), T, dy.cuda(), dh, dkv, dwq, dwk,
                            ws)
    eg.engram_sync(s.ctx)
    half = {1 / (1 + math.exp(-1e-3)), 1 / (1 + math.exp(1e-3))}  # a NaN has either sign
    for t, b in ((1, 0), (2, 1)):
        for g in (float(gates[t, b]), float(pgates[t, b])):
            assert min(abs(g - x) for x in half) <= 1e-6
        dk = dkv[t, b * d:(b + 1) * d].cpu()
        assert not dk.isfinite().any()
    ok = torch.ones(T, hc, dtype=torch.bool)
    ok[1, 0] = ok[2, 1] = False
    assert (gates.cpu()[ok] - pgates.cpu()[ok]).abs().max() <= 1e-5
    assert dh.cpu()[ok].isfinite().all() and dkv.cpu()[:, :hc * d].reshape(T, hc, d)[ok].isfinite().all()
    assert dkv[:, hc * d:].isfinite().all()
    s.close()


def test_gate_calls_refuse_misaligned_pointers():
    s = make_layer()
    A = 1 << 20  # an aligned address that no refused call touches
    good = dict(kv=A, windows=A, hidden=A, out=A, gates=A, codes=A, scales=A)
    for name in good:
        a = {**good, name: A + 2}
        with pytest.raises(eg.EngramError) as e:
            eg.engram_gate_checkpoint(s.ctx, 0, a["kv"], eg.KV_F32, a["windows"], 1, a["hidden"], a["out"],
                                      a["gates"], a["codes"], a["scales"])
        assert e.value.status == eg.EINVAL
    names = ("windows", "dout", "dhidden", "dkv", "dwq", "dwk", "ws")
    good = dict.fromkeys(("first", "second") + names, A)
    for name in good:
        a = {**good, name: A + 8}
        last = (a["windows"], 1, a["dout"], a["dhidden"], a["dkv"], a["dwq"], a["dwk"], a["ws"])
        for f, args in ((eg.engram_gate_backward, (a["first"], eg.KV_BF16, a["second"])),
                        (eg.engram_gate_backward_checkpoint, (a["first"], a["second"]))):
            with pytest.raises(eg.EngramError) as e:
                f(s.ctx, 0, *args, *last)
            assert e.value.status == eg.EINVAL
    s.close()


def test_gate_checkpoint_of_infinities_and_nans():
    T, hc, d = 1, 1, 256
    h, kv, win, wq, wk = gate_problem(T, hc, d, 5, image=())
    kv[0, 3], kv[0, 40], h[0, 0, 70] = float("inf"), float("nan"), float("-inf")
    s = make_layer(hc, d)
    codes = torch.zeros(1, 3 * d, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, 3 * d // 32, dtype=torch.uint8, device="cuda")
    out = torch.empty(1, 1, d, dtype=torch.bfloat16, device="cuda")
    eg.engram_gate_checkpoint(s.ctx, 0, kv.cuda(), eg.KV_F32, win.cuda(), 1, h.cuda(), out, None,
                              codes, scales)
    eg.engram_sync(s.ctx)
    bad = torch.zeros(3 * d // 32, dtype=torch.bool)
    bad[[2, d // 32, d // 32 + 1]] = True
    assert torch.equal(scales.cpu()[0] == 255, bad)
    s.close()


def backward_ref(h, kv, on, wq, wk, dy):
    leaves = [x.to(F).clone().requires_grad_() for x in (h, kv, wq, wk)]
    out, _, _ = gate_ref(leaves[0], leaves[1], on, leaves[2], leaves[3])
    return torch.autograd.grad(out, leaves, dy.to(F))


def check_backward(got, ref, h, kv, dy, on, hc, d):
    dh, dkv, dwq, dwk = [x.cpu().to(F) for x in got]
    T = dh.shape[0]
    scale = dy.to(F).abs().amax() * (1 + kv.to(F).abs().amax())
    assert ((dh - ref[0]).abs() <= 2.0 ** -8 * ref[0].abs() + 2.0 ** -12 * scale).all()
    assert ((dkv - ref[1]).abs() <= 2.0 ** -8 * ref[1].abs() + 2.0 ** -12 * scale).all()
    for a, b in ((dwq, ref[2]), (dwk, ref[3])):
        assert ((a - b).abs() <= 2.0 ** -14 * (b.abs() + b.abs().mean()) + 1e-12).all()
    off = (on == 0).reshape(T)
    assert torch.equal(dh[off], dy.to(F)[off]) and not dkv[off].any()


@pytest.mark.parametrize("saved", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T,hc,d", GATE)
def test_gate_backward(T, hc, d, saved):
    h, kv, win, wq, wk = gate_problem(T, hc, d, 20 * T + hc)
    dy = rnd(3, T, hc, d)
    on = (win[:, 0] != -1).to(F).reshape(T, 1, 1)
    s = make_layer(hc, d, wq=wq, wk=wk)
    ws = ws_of(eg.engram_gate_backward_workspace_bytes(s.ctx, T))
    dh = torch.full((T, hc, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    dkv = torch.full((T, (hc + 1) * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    dwq = torch.full((hc, d), float("nan"), device="cuda")
    dwk = torch.full((hc, d), float("nan"), device="cuda")
    if saved == "mxfp8":
        codes, exps = pack_ref(torch.cat([h.float().reshape(T, hc * d), kv], 1))
        both = unpack_ref(codes, exps)
        h, kv = both[:, :hc * d].reshape(T, hc, d), both[:, hc * d:]
        eg.engram_gate_backward_checkpoint(s.ctx, 0, codes.cuda().view(torch.uint8), exps.cuda(),
                                           win.cuda(), T, dy.cuda(), dh, dkv, dwq, dwk, ws)
    else:
        if saved == "bf16":
            kv = kv.bfloat16()
        fmt = eg.KV_F32 if saved == "f32" else eg.KV_BF16
        inplace = dy.cuda()
        eg.engram_gate_backward(s.ctx, 0, kv.cuda(), fmt, h.cuda(), win.cuda(), T, inplace, inplace,
                                dkv, None, None, ws)
        dkv.fill_(float("nan"))
        eg.engram_gate_backward(s.ctx, 0, kv.cuda(), fmt, h.cuda(), win.cuda(), T, dy.cuda(), dh,
                                dkv, dwq, dwk, ws)
        assert torch.equal(inplace, dh)
    eg.engram_sync(s.ctx)
    ref = backward_ref(h.to(F), kv.to(F), on, wq, wk, dy)
    check_backward((dh, dkv, dwq, dwk), ref, h, kv, dy, on, hc, d)
    s.close()


@pytest.mark.parametrize("saved", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T,hc,d", [(700, 2, 256), (320, 4, 5120), (3, 8, 9216), (2, 1, 20_736)])
def test_gate_backward_of_many_and_of_wide_tokens(T, hc, d, saved):
    test_gate_backward(T, hc, d, saved)


GRADIENTS = [(7, 1, 256), (9, 2, 512), (5, 4, 1024), (8, 3, 1280), (6, 8, 256), (9, 5, 2816), (12, 4, 5120),
             (320, 4, 5120), (600, 2, 256), (11, 7, 1280), (7, 1, 20_480), (3, 8, 9216), (7, 1, 20_736)]


@pytest.mark.parametrize("saved", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("T,hc,d", GRADIENTS)
def test_gate_backward_term_by_term(T, hc, d, saved):
    """Every gradient to its BF16 rounding and the error of the sums behind it (gate_reference.py):
    no term of dh or dk could be missing, at any width, from dots of 2e-3 to 30."""
    h, kv, win, wq, wk, dy, on = gate_inputs(T, hc, d, T)
    s = make_layer(hc, d, wq=wq, wk=wk)
    ws = ws_of(eg.engram_gate_backward_workspace_bytes(s.ctx, T))
    dh = torch.full((T, hc, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    dkv = torch.full((T, (hc + 1) * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    dwq, dwk = (torch.full((hc, d), float("nan"), device="cuda") for _ in range(2))
    to = (win.cuda(), T, dy.cuda(), dh, dkv, dwq, dwk, ws)
    if saved == "mxfp8":
        codes, exps = pack_ref(torch.cat([h.float().reshape(T, hc * d), kv], 1))
        both = unpack_ref(codes, exps)
        h, kv = both[:, :hc * d].reshape(T, hc, d), both[:, hc * d:]
        eg.engram_gate_backward_checkpoint(s.ctx, 0, codes.cuda().view(torch.uint8), exps.cuda(), *to)
    else:
        kv = kv if saved == "f32" else kv.bfloat16()
        eg.engram_gate_backward(s.ctx, 0, kv.cuda(), eg.KV_F32 if saved == "f32" else eg.KV_BF16, h.cuda(), *to)
    eg.engram_sync(s.ctx)
    ref = GateGradients(h, kv, on, wq, wk, dy)
    assert ref.misses(dh.cpu(), dkv.cpu()) == []
    # the weights' sums over the tokens: each term dS h k w as dS, and the additions of up to T
    # terms, one after the other at the most
    dS = ref.rho * (ref.first["dh"] * h.to(F)).abs() / wq.to(F).abs()  # (first["dh"] = dS wq wk k)
    add = T * 2.0 ** -24 * (ref.first["dh"] * h.to(F)).abs() / wq.to(F).abs()
    tol = (dS + add).sum(0)
    assert ((dwq.cpu().to(F) - ref.dwq).abs() <= tol).all()
    assert ((dwk.cpu().to(F) - ref.dwk).abs() <= tol * (wq / wk).abs().to(F)).all()
    s.close()


def test_gate_backward_against_differences():
    """The kernel's gradient against central differences of the step in 64 bits."""
    T, hc, d = 2, 2, 256
    h, kv, win, wq, wk = gate_problem(T, hc, d, 77, image=())
    dy = rnd(4, T, hc, d)
    s = make_layer(hc, d, wq=wq, wk=wk)
    ws = ws_of(eg.engram_gate_backward_workspace_bytes(s.ctx, T))
    dh = torch.empty(T, hc, d, dtype=torch.bfloat16, device="cuda")
    dkv = torch.empty(T, (hc + 1) * d, dtype=torch.bfloat16, device="cuda")
    dwq, dwk = (torch.empty(hc, d, device="cuda") for _ in range(2))
    eg.engram_gate_backward(s.ctx, 0, kv.cuda(), eg.KV_F32, h.cuda(), win.cuda(), T, dy.cuda(), dh,
                            dkv, dwq, dwk, ws)
    eg.engram_sync(s.ctx)
    on = torch.ones(T, 1, 1, dtype=F)
    base = [h.to(F), kv.to(F), wq.to(F), wk.to(F)]
    value = lambda x: (gate_ref(x[0], x[1], on, x[2], x[3])[0] * dy.to(F)).sum()  # noqa: E731
    step = 1e-5
    for which, got in enumerate((dh, dkv, dwq, dwk)):
        got = got.cpu().to(F).reshape(-1)
        for i in range(0, got.numel(), 61):
            lo, hi = [x.clone() for x in base], [x.clone() for x in base]
            lo[which].view(-1)[i] -= step
            hi[which].view(-1)[i] += step
            ref = float((value(hi) - value(lo)) / (2 * step))
            assert abs(got[i] - ref) <= 2.0 ** -8 * abs(ref) + 2e-3, (which, i)
    s.close()


@pytest.mark.parametrize("where", ["zero_key", "zero_hidden", "zero_dot"])
def test_gate_backward_at_a_dot_of_zero(where):
    """|dot| <= 1e-6: the root is constant there, so only dy and dv = g dy pass."""
    T, hc, d = 2, 1, 256
    h, kv, win, wq, wk = gate_problem(T, hc, d, 8, image=())
    if where == "zero_key":
        kv[:, :d] = 0
    elif where == "zero_hidden":
        h.zero_()
    else:  # h and k never meet
        h[:, :, ::2] = 0
        kv[:, 1:d:2] = 0
    dy = rnd(9, T, hc, d)
    s = make_layer(hc, d)
    ws = ws_of(eg.engram_gate_backward_workspace_bytes(s.ctx, T))
    dh = torch.empty(T, hc, d, dtype=torch.bfloat16, device="cuda")
    dkv = torch.empty(T, 2 * d, dtype=torch.bfloat16, device="cuda")
    dwq, dwk = (torch.empty(hc, d, device="cuda") for _ in range(2))
    eg.engram_gate_backward(s.ctx, 0, kv.cuda(), eg.KV_F32, h.cuda(), win.cuda(), T, dy.cuda(), dh,
                            dkv, dwq, dwk, ws)
    eg.engram_sync(s.ctx)
    assert torch.equal(dh.cpu(), dy) and not dkv[:, :d].any() and not dwq.any() and not dwk.any()
    g = 1 / (1 + math.exp(-1e-3))
    ref = g * dy[:, 0].to(F)
    assert ((dkv[:, d:].cpu().to(F) - ref).abs() <= 2.0 ** -8 * ref.abs()).all()
    s.close()


# ---- projection backward ---------------------------------------------------------------------

@pytest.mark.parametrize("want", ["both", "demb", "dwkv"])
@pytest.mark.parametrize("T,hc,d,heads,row_dim", [(1, 1, 256, 2, 32), (63, 1, 256, 2, 32),
                                                  (64, 2, 256, 1, 64), (130, 1, 512, 3, 128),
                                                  (257, 3, 256, 8, 64), (700, 1, 256, 5, 256),
                                                  (333, 2, 512, 4, 128), (1037, 1, 256, 2, 64),
                                                  (20, 4, 1280, 2, 128)])
def test_project_backward(T, hc, d, heads, row_dim, want):
    N, K = (hc + 1) * d, 3 * heads * row_dim
    wkv, emb, dkv = rnd(1, N, K), rnd(T, T, K), rnd(T + 1, T, N)
    s = make_layer(hc, d, heads, row_dim, wkv=wkv)
    ws = ws_of(eg.engram_project_backward_workspace_bytes(s.ctx, T))
    demb = torch.full((T, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dwkv = torch.full((N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    eg.engram_project_backward(s.ctx, 0, emb.cuda() if want != "demb" else None, dkv.cuda(), T,
                               demb if want != "dwkv" else None, dwkv if want != "demb" else None,
                               ws)
    eg.engram_sync(s.ctx)
    for got, a, b, n, on in ((demb, dkv, wkv, N, want != "dwkv"), (dwkv, dkv.T, emb, T, want != "demb")):
        if not on:
            assert got.isnan().all()
            continue
        ref, mag = a.to(F) @ b.to(F), a.to(F).abs() @ b.to(F).abs()
        assert ((got.cpu().to(F) - ref).abs() <= 2.0 ** -8 * ref.abs() + n * 2.0 ** -23 * mag).all()
    s.close()


def test_project_backward_of_no_tokens():
    s = make_layer(1, 256)
    dwkv = torch.ones(512, 192, dtype=torch.bfloat16, device="cuda")
    eg.engram_project_backward(s.ctx, 0, None, None, 0, None, dwkv, None)
    eg.engram_sync(s.ctx)
    assert not dwkv.any()
    s.close()


# ---- loss --------------------------------------------------------------------------------------

LOSS = [(1, 1, 8), (1, 257, 64), (2, 1000, 40), (129, 511, 72), (300, 3001, 264), (513, 777, 1032),
        (64, 40_000, 128), (7, 129_280, 64), (16, 31, 1032), (17, 4897, 2056), (33, 130, 200),
        (64, 6001, 4104), (65, 6001, 136)]


def loss_problem(T, V, dim):
    x, head = rnd(T, T, dim), rnd(V, V, dim, sigma=2 / math.sqrt(dim))
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T)).int()
    y[0] = V - 1
    if T > 1:
        y[1] = -1
    if T > 6:
        y[5] = -100
    return x, head, y


def loss_ref(x, head, y):
    z = x.to(F) @ head.to(F).T
    lse = torch.logsumexp(z, 1)
    at = z.gather(1, y.clamp_min(0).long().unsqueeze(1)).squeeze(1)
    return z, lse, torch.where(y >= 0, lse - at, torch.zeros_like(lse))


@pytest.mark.parametrize("T,V,dim", LOSS)
def test_loss(plain_ctx, T, V, dim):
    x, head, y = loss_problem(T, V, dim)
    loss, lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    ws = ws_of(eg.engram_loss_workspace_bytes(T, V, dim))
    eg.engram_loss(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, loss, lse, ws)
    eg.engram_sync(plain_ctx)
    _, rlse, rloss = loss_ref(x, head, y)
    mag = (x.to(F).abs() @ head.to(F).abs().T).amax(1)
    tol = dim * 2.0 ** -23 * mag + 2.0 ** -20 * (1 + rlse.abs())
    assert ((lse.cpu().to(F) - rlse).abs() <= tol).all()
    assert ((loss.cpu().to(F) - rloss).abs() <= 2 * tol).all()
    assert (loss.cpu()[y < 0] == 0).all()


@pytest.mark.parametrize("want", ["both", "dx", "dhead"])
@pytest.mark.parametrize("T,V,dim", LOSS)
def test_loss_backward(plain_ctx, T, V, dim, want):
    x, head, y = loss_problem(T, V, dim)
    z, lse, _ = loss_ref(x, head, y)
    dloss = rnd(9, T, dtype=torch.float32)
    dx = torch.full((T, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    dhead = torch.full((V, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    own_lse = torch.empty(T, device="cuda")  # (the operator takes engram_loss's lse)
    ws = ws_of(eg.engram_loss_workspace_bytes(T, V, dim))
    eg.engram_loss(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, None, own_lse, ws)
    ws = ws_of(eg.engram_loss_backward_workspace_bytes(T, V, dim))
    eg.engram_loss_backward(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, own_lse,
                            dloss.cuda(), dx if want != "dhead" else None,
                            dhead if want != "dx" else None, ws)
    eg.engram_sync(plain_ctx)
    dz = torch.exp(z - lse.unsqueeze(1))
    dz[torch.arange(T), y.clamp_min(0).long()] -= 1
    dz *= torch.where(y >= 0, dloss.to(F), torch.zeros(T, dtype=F)).unsqueeze(1)
    for got, a, b, n, on in ((dx, dz, head, V, want != "dhead"), (dhead, dz.T, x, T, want != "dx")):
        if not on:
            assert got.isnan().all()
            continue
        ref, mag = a @ b.to(F), a.abs() @ b.to(F).abs()
        tol = 2.0 ** -8 * (ref.abs() + mag) + n * 2.0 ** -23 * mag
        assert ((got.cpu().to(F) - ref).abs() <= tol).all()


@pytest.mark.parametrize("T", [3, 60, 300, 700])
def test_loss_backward_of_equal_weights_is_not_scaled(plain_ctx, T):
    """With weights of 1 / T for a T that is no power of two, BF16 rounding of dz must not scale
    the gradient: its projection on the exact one is 1 to within what independent roundings of
    at most 2^-8 give over its elements (2^-8 / sqrt(T)), and the probabilities' size."""
    V, dim = 3000, 128
    x, head, y = loss_problem(T, V, dim)
    y = y.clamp_min(0)
    dloss = torch.full((T,), 1.0 / T)
    lse = torch.empty(T, device="cuda")
    ws = ws_of(max(eg.engram_loss_workspace_bytes(T, V, dim),
                   eg.engram_loss_backward_workspace_bytes(T, V, dim)))
    dev = [t.cuda() for t in (x, head, y, dloss)]
    eg.engram_loss(plain_ctx, dev[0], dev[1], V, dim, dev[2], T, None, lse, ws)
    dx = torch.empty(T, dim, dtype=torch.bfloat16, device="cuda")
    dhead = torch.empty(V, dim, dtype=torch.bfloat16, device="cuda")
    eg.engram_loss_backward(plain_ctx, dev[0], dev[1], V, dim, dev[2], T, lse, dev[3], dx, dhead, ws)
    eg.engram_sync(plain_ctx)
    z, rlse, _ = loss_ref(x, head, y)
    dz = torch.exp(z - rlse.unsqueeze(1))
    p = dz[torch.arange(T), y.long()].clone()
    dz[torch.arange(T), y.long()] -= 1
    dz *= dloss.to(F).unsqueeze(1)
    for got, ref in ((dx, dz @ head.to(F)), (dhead, dz.T @ x.to(F))):
        along = float((got.cpu().to(F) * ref).sum() / (ref * ref).sum())
        assert abs(along - 1) <= 2.0 ** -8 / math.sqrt(T) + float(p.mean()), along


def test_loss_backward_against_differences(plain_ctx):
    T, V, dim = 5, 70, 16
    x, head, y = loss_problem(T, V, dim)
    dloss = rnd(9, T, dtype=torch.float32)
    loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
    ws = ws_of(eg.engram_loss_workspace_bytes(T, V, dim))
    eg.engram_loss(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, loss, lse, ws)
    dx = torch.empty(T, dim, dtype=torch.bfloat16, device="cuda")
    dhead = torch.empty(V, dim, dtype=torch.bfloat16, device="cuda")
    ws = ws_of(eg.engram_loss_backward_workspace_bytes(T, V, dim))
    eg.engram_loss_backward(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, lse,
                            dloss.cuda(), dx, dhead, ws)
    eg.engram_sync(plain_ctx)
    value = lambda a, b: (loss_ref(a, b, y)[2] * dloss.to(F)).sum()  # noqa: E731
    step = 1e-5
    for which, got in ((0, dx), (1, dhead)):
        got = got.cpu().to(F).reshape(-1)
        for i in range(0, got.numel(), 7):
            a, b = [x.to(F), head.to(F)], [x.to(F), head.to(F)]
            a[which].view(-1)[i] += step
            b[which].view(-1)[i] -= step
            ref = float((value(*a) - value(*b)) / (2 * step))
            # dz in BF16: 2^-8 of at most sum |dz| |x| <= 2 sum |dloss| max |x|
            assert abs(got[i] - ref) <= 2.0 ** -7 * abs(ref) + 2.0 ** -8 * 2, (which, i)


def test_loss_with_no_label_counted_and_with_labels_outside(plain_ctx):
    T, V, dim = 40, 300, 64
    x, head, y = loss_problem(T, V, dim)
    y[:] = -1
    y[3] = V  # outside: ignored, reported
    loss, lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    ws = ws_of(max(eg.engram_loss_workspace_bytes(T, V, dim),
                   eg.engram_loss_backward_workspace_bytes(T, V, dim)))
    eg.engram_loss(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, loss, lse, ws)
    with pytest.raises(eg.EngramError) as e:
        eg.engram_sync(plain_ctx)
    assert e.value.status == eg.EBOUNDS and not loss.any() and lse.isfinite().all()
    dx = torch.ones(T, dim, dtype=torch.bfloat16, device="cuda")
    dhead = torch.ones(V, dim, dtype=torch.bfloat16, device="cuda")
    eg.engram_loss_backward(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, lse,
                            torch.full((T,), float("inf"), device="cuda"), dx, dhead, ws)
    eg.engram_sync(plain_ctx)
    assert not dx.any() and not dhead.any()


def test_loss_of_large_logits(plain_ctx):
    """Logits of several thousand: the running maximum keeps the sums finite."""
    T, V, dim = 20, 700, 64
    x, head, y = loss_problem(T, V, dim)
    x = (x.float() * 300).bfloat16()
    loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
    ws = ws_of(eg.engram_loss_workspace_bytes(T, V, dim))
    eg.engram_loss(plain_ctx, x.cuda(), head.cuda(), V, dim, y.cuda(), T, loss, lse, ws)
    eg.engram_sync(plain_ctx)
    _, rlse, rloss = loss_ref(x, head, y)
    mag = (x.to(F).abs() @ head.to(F).abs().T).amax(1)
    tol = dim * 2.0 ** -23 * mag + 2.0 ** -20 * (1 + rlse.abs())
    assert ((lse.cpu().to(F) - rlse).abs() <= tol).all()
    assert ((loss.cpu().to(F) - rloss).abs() <= 2 * tol).all()


# ---- one workspace for every batch ------------------------------------------------------------

def guarded(need):
    """A workspace of `need` bytes between guards, and the test that they are whole."""
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    return ws[256:], lambda: bool((ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all())


@pytest.mark.parametrize("copies", [1, 3, 8])
def test_embed_grad_of_smaller_batches_in_the_workspace_of_the_largest(plain_ctx, copies):
    rows, dim = 900, 5120
    most = 7300  # (three copies' rows: 3,644 ids make 1,822 chunks of two places, 3,700 make 740 of five)
    ws, whole = guarded(eg.engram_embed_grad_workspace_bytes(most, rows, dim))
    for n in (1, 700, 1867, 3500, 3644, 3700, most):
        ids, dout = ids_like("zipf", n, rows, n).cuda(), rnd(n, n, 1, dim).cuda().expand(n, copies, dim).contiguous()
        out = []
        for w in (ws, ws_of(eg.engram_embed_grad_workspace_bytes(1 << 20, rows, dim))):
            grad = torch.zeros(rows, dim, device="cuda")
            eg.engram_embed_grad(plain_ctx, rows, dim, ids, n, 1.0, copies, dout, None, None, grad, 0, w)
            out.append(grad)
        eg.engram_sync(plain_ctx)
        assert torch.equal(*out) and whole(), n


@pytest.mark.parametrize("hc,d,heads,row_dim,sizes", [(4, 5120, 8, 256, (100, 256, 400, 1024, 1500)),
                                                      (2, 1280, 4, 128, (64, 300, 1500, 3000))])
def test_project_backward_of_smaller_batches_in_the_workspace_of_the_largest(hc, d, heads, row_dim, sizes):
    N, K = (hc + 1) * d, 3 * heads * row_dim
    s = make_layer(hc, d, heads, row_dim, wkv=rnd(1, N, K))
    ws, whole = guarded(eg.engram_project_backward_workspace_bytes(s.ctx, sizes[-1]))
    plenty = ws_of(1 << 28)
    for T in sizes:
        emb, dkv = rnd(T, T, K).cuda(), rnd(T + 1, T, N).cuda()
        for want_dwkv in (True, False):
            out = []
            for w in (ws, plenty):
                demb = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
                dwkv = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda") if want_dwkv else None
                eg.engram_project_backward(s.ctx, 0, emb, dkv, T, demb, dwkv, w)
                out.append(demb)
            eg.engram_sync(s.ctx)
            assert torch.equal(*out) and whole(), T
    s.close()


@pytest.mark.parametrize("V,dim,sizes", [(1000, 64, (1, 16, 17, 31)), (32_000, 2048, (16, 300, 1280, 1500))])
def test_loss_of_smaller_batches_in_the_workspace_of_the_largest(plain_ctx, V, dim, sizes):
    head = rnd(V, V, dim, sigma=2 / math.sqrt(dim)).cuda()
    ws, whole = guarded(eg.engram_loss_workspace_bytes(sizes[-1], V, dim))
    back, back_whole = guarded(eg.engram_loss_backward_workspace_bytes(sizes[-1], V, dim))
    plenty = ws_of(1 << 28)
    for T in sizes:
        x, _, y = loss_problem(T, 2, dim)
        x, y, dloss = x.cuda(), y.cuda(), torch.ones(T, device="cuda")
        out = []
        for w, wb in ((ws, back), (plenty, plenty)):
            loss, lse = (torch.zeros(T, device="cuda") for _ in range(2))
            dx, dhead = torch.zeros_like(x), torch.zeros_like(head)
            eg.engram_loss(plain_ctx, x, head, V, dim, y, T, loss, lse, w)
            eg.engram_loss_backward(plain_ctx, x, head, V, dim, y, T, lse, dloss, dx, dhead, wb)
            only = torch.zeros_like(x)
            eg.engram_loss_backward(plain_ctx, x, head, V, dim, y, T, lse, dloss, only, None, wb)
            out.append((loss, lse, dx, dhead, only))
        eg.engram_sync(plain_ctx)
        assert all(torch.equal(a, b) for a, b in zip(*out)) and whole() and back_whole(), T


# ---- streams ---------------------------------------------------------------------------------------

def test_operators_run_on_their_own_stream(plain_ctx):
    """Inputs made on a side stream, the call on it, nothing on the default stream."""
    st = torch.cuda.Stream()
    T, V, dim = 100, 2000, 256
    x, head, y = loss_problem(T, V, dim)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        big = torch.randn(1 << 24, device="cuda")
        for _ in range(20):
            big = big * 1.0001
        dx, dh, dy = x.cuda(non_blocking=True), head.cuda(non_blocking=True), y.cuda(non_blocking=True)
        loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
        ws = ws_of(eg.engram_loss_workspace_bytes(T, V, dim))
        eg.engram_loss(plain_ctx, dx, dh, V, dim, dy, T, loss, lse, ws, st)
    eg.engram_sync(plain_ctx, st)
    _, rlse, _ = loss_ref(x, head, y)
    assert (lse.cpu().to(F) - rlse).abs().max() <= 1e-3


def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable():
    s = make_layer()
    V, dim = 2000, 256
    try:
        for T in (10, 100):
            x, head, y = (t.cuda() for t in loss_problem(T, V, dim))
            loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
            ws = ws_of(eg.engram_loss_workspace_bytes(T, V, dim))
            eg.engram_ctx_set_wait_limit(s.ctx, 20_000_000)
            eg.engram_debug_starve_operand(s.ctx, True)
            eg.engram_loss(s.ctx, x, head, V, dim, y, T, loss, lse, ws)
            with pytest.raises(eg.EngramError) as e:
                eg.engram_sync(s.ctx)
            assert e.value.status == eg.ETIMEOUT
            eg.engram_debug_starve_operand(s.ctx, False)
            eg.engram_ctx_set_wait_limit(s.ctx, 4_000_000_000)
            eg.engram_loss(s.ctx, x, head, V, dim, y, T, loss, lse, ws)
            eg.engram_sync(s.ctx)
            _, rlse, _ = loss_ref(x.cpu(), head.cpu(), y.cpu())
            assert (lse.cpu().to(F) - rlse).abs().max() <= 1e-3
    finally:
        s.close()


@pytest.mark.parametrize("form", ["sparse", "dense", "accumulate"])
def test_a_sort_whose_wait_runs_out_writes_no_gradient(form):
    """The sums behind an unfinished sort touch nothing: neither the outputs nor what lies beside
    them and the workspace, whatever the workspace held (here words that are no place or row)."""
    n, rows, dim = 40_000, 3000, 16
    dense, accumulate = form != "sparse", int(form == "accumulate")
    ids, dout = ids_like("zipf", n, rows, 3), rnd(4, n, 1, dim)
    need = eg.engram_embed_grad_workspace_bytes(n, rows, dim)
    out_rows = rows if dense else n
    s = make_layer()
    try:
        def call(grad, unique, ws):
            eg.engram_embed_grad(s.ctx, rows, dim, ids.cuda(), n, 1.0, 1, dout.cuda(),
                                 None if dense else unique[64:], torch.zeros(1, dtype=torch.int32, device="cuda"),
                                 grad[4:], accumulate, ws[256:])

        def buffers():
            return (torch.full((out_rows + 8, dim), 7.0, device="cuda"),
                    torch.full((n + 128,), -5, dtype=torch.int32, device="cuda"),
                    torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda"))

        grad, unique, ws = buffers()
        eg.engram_ctx_set_wait_limit(s.ctx, 20_000_000)
        eg.engram_debug_starve_operand(s.ctx, True)
        call(grad, unique, ws)
        with pytest.raises(eg.EngramError) as e:
            eg.engram_sync(s.ctx)
        assert e.value.status == eg.ETIMEOUT
        left = 0.0 if form == "dense" else 7.0
        assert (grad[4:-4] == left).all() and (grad[:4] == 7.0).all() and (grad[-4:] == 7.0).all()
        assert (unique[:64] == -5).all() and (unique[-64:] == -5).all()
        assert (ws[:256] == 0xA5).all() and (ws[-256:] == 0xA5).all()
        eg.engram_debug_starve_operand(s.ctx, False)
        eg.engram_ctx_set_wait_limit(s.ctx, 4_000_000_000)
        grad, unique, _ = buffers()
        call(grad, unique, ws)  # on what the broken-off call left
        eg.engram_sync(s.ctx)
        u, ref, tol = grad_reference(ids.long(), dout, rows, 1.0)
        got = grad[4:-4].cpu().to(F)
        if accumulate:
            ref, tol = ref + 7.0, tol + 2.0 ** -23 * (ref.abs() + 14.0)
        assert ((got[u if dense else slice(0, u.numel())] - ref).abs() <= tol).all()
        assert (grad[:4] == 7.0).all() and (grad[-4:] == 7.0).all()
        assert (ws[:256] == 0xA5).all() and (ws[-256:] == 0xA5).all()
    finally:
        s.close()


def test_operators_in_a_captured_graph(plain_ctx):
    """Captured once, replayed on new inputs in the same buffers."""
    n, rows, dim, T, V = 20_000, 3000, 64, 100, 1500
    ids, dout = ids_like("zipf", n, rows, 1).cuda(), rnd(2, n, 1, dim).cuda()
    x, head, y = (t.cuda() for t in loss_problem(T, V, dim))
    grad = torch.zeros(rows, dim, device="cuda")
    loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
    dx, dhead = torch.empty_like(x), torch.empty_like(head)
    dloss = torch.ones(T, device="cuda")
    ws1 = ws_of(eg.engram_embed_grad_workspace_bytes(n, rows, dim))
    ws2 = ws_of(max(eg.engram_loss_workspace_bytes(T, V, dim),
                    eg.engram_loss_backward_workspace_bytes(T, V, dim)))

    def calls(st):
        eg.engram_embed_grad(plain_ctx, rows, dim, ids, n, 1.0, 1, dout, None, None, grad, 0, ws1, st)
        eg.engram_loss(plain_ctx, x, head, V, dim, y, T, loss, lse, ws2, st)
        eg.engram_loss_backward(plain_ctx, x, head, V, dim, y, T, lse, dloss, dx, dhead, ws2, st)

    calls(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(torch.cuda.current_stream())
    for k in (3, 4):
        ids.copy_(ids_like("zipf", n, rows, k))
        dout.copy_(rnd(k, n, 1, dim))
        x.copy_(rnd(k, T, dim))
        graph.replay()
        eg.engram_sync(plain_ctx, torch.cuda.current_stream())
        got = [t.clone() for t in (grad, loss, lse, dx, dhead)]
        calls(None)
        torch.cuda.synchronize()
        for a, b in zip(got, (grad, loss, lse, dx, dhead)):
            assert torch.equal(a, b)


# ---- the step -----------------------------------------------------------------------------------

VOCAB, D = 500, 256


def step_model(hc=2, seed=0):
    """A small model around one layer with a BF16 table, as the example's."""
    s = EngramLayerSet(VOCAB, 400, np.arange(VOCAB, dtype=np.uint32) % 400, [3], [200], heads=2,
                       row_dim=32, hc=hc, d=D)
    g = torch.Generator().manual_seed(seed)
    new = lambda *shape, sigma=1.0: torch.randn(*shape, generator=g) * sigma  # noqa: E731
    kept = s.bind(0, 11, new((hc + 1) * D, 192, sigma=192 ** -0.5).bfloat16().cuda().view(torch.int16),
                  1 + new(hc, D, sigma=0.1), 1 + new(hc, D, sigma=0.1), flags=eg.BIND_TABLE_BF16)
    embedding, head = new(VOCAB, D, sigma=D ** -0.5), new(VOCAB, D, sigma=2 * D ** -0.5)
    return s, kept, embedding.bfloat16().cuda(), head.bfloat16().cuda()


def step_inputs(s, T, seed):
    tokens = np.random.default_rng(seed).integers(0, VOCAB, T + 1).astype(np.int32)
    session = eg.engram_session_create(s.ctx)
    image = np.zeros(T, np.uint8)
    image[T // 3] = 1
    windows = eg.engram_session_append(session, tokens[:-1], image)
    eg.engram_session_destroy(session)
    labels = tokens[1:].copy()
    labels[T // 2] = -1
    dloss = rnd(seed, T, dtype=torch.float32).abs() + 0.5
    return [torch.from_numpy(a).cuda() for a in (tokens[:-1].copy(), windows.view(np.int32), labels)] + [dloss.cuda()]


def step_outputs(step, loss):
    n, r = int(step.token_count), int(step.row_count)
    return [loss.clone(), step.dhead.clone(), step.dwq.clone(), step.dwk.clone(), step.dwkv.clone(),
            step.token_ids[:n].clone(), step.token_grad[:n].clone(), step.row_ids[:r].clone(),
            step.row_grad[:r].clone()]


def run_step(step, inputs, stream=None):
    loss = step.forward(*inputs[:3], stream)
    step.backward(*inputs, stream)
    return loss


def test_a_step_of_fewer_tokens_is_that_of_buffers_of_their_size():
    s, _, embedding, head = step_model()
    big = TrainStep(s, 0, embedding, head, 300)
    run_step(big, step_inputs(s, 300, 1))  # what the buffers hold past a shorter step
    for T in (1, 2, 16, 17, 129, 299, 300):
        inputs = step_inputs(s, T, T)
        loss = run_step(big, inputs)
        own = TrainStep(s, 0, embedding, head, T)
        own_loss = run_step(own, inputs)
        eg.engram_sync(s.ctx)
        assert loss.shape == (T,)
        for a, b in zip(step_outputs(big, loss), step_outputs(own, own_loss)):
            assert torch.equal(a, b), T
    s.close()


@pytest.mark.parametrize("given", ["none", "stream", "handle"])
def test_a_step_runs_on_its_stream(given):
    """All of a step is on one stream: the current one where none is given, else the given one,
    whatever the current one is.  The stream's work before it (a wait of some ten milliseconds,
    then the copy of the inputs) is done first, and nothing of the step runs before that."""
    T = 120
    s, _, embedding, head = step_model()
    inputs = step_inputs(s, T, 5)
    step = TrainStep(s, 0, embedding, head, T)
    loss = run_step(step, inputs)
    eg.engram_sync(s.ctx)
    want = step_outputs(step, loss)
    step = TrainStep(s, 0, embedding, head, T)
    for x in vars(step).values():  # what a step that runs too early would find
        if isinstance(x, torch.Tensor) and x is not embedding and x is not head:
            x.zero_()
    late = [torch.zeros_like(x) for x in inputs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        for a, b in zip(late, inputs):
            a.copy_(b)
    if given == "none":
        with torch.cuda.stream(side):
            loss = run_step(step, late)
    else:
        loss = run_step(step, late, side if given == "stream" else side.cuda_stream)
    eg.engram_sync(s.ctx, side)
    for a, b in zip(step_outputs(step, loss), want):
        assert torch.equal(a, b)
    s.close()


@pytest.mark.parametrize("T,hc,kv_format", [(130, 2, eg.KV_BF16), (13, 2, eg.KV_F32), (61, 1, eg.KV_BF16)])
def test_every_gradient_of_a_step(T, hc, kv_format):
    """Each part of a step against its formula in 64 bits on what the step's part before it left:
    the scales of the embedding and the rows, the mean's gradient, which buffer goes where."""
    s, kept, embedding, head = step_model(hc)
    ids, win, labels, dloss = inputs = step_inputs(s, T, 3)
    step = TrainStep(s, 0, embedding, head, T + 5, kv_format=kv_format, scale=3.0)
    loss = run_step(step, inputs)
    eg.engram_sync(s.ctx)
    c = lambda x, n=T: x[:n].cpu().to(F)  # noqa: E731
    K, N, kept_n = s.K, s.N, (2 * hc + 1) * D
    on = (win.cpu()[:, 0] != -1).to(F).reshape(T, 1, 1)
    table = kept["table"].view(torch.bfloat16)[:s.rows(0) * 32].view(-1, 32).cpu().to(F)
    wkv = kept["wkv"].view(torch.bfloat16).view(N, K).cpu().to(F)
    wq, wk = (kept[n].view(hc, D).cpu().to(F) for n in ("wq", "wk"))

    def near(got, ref, mag, n, roundings=1):
        assert ((got - ref).abs() <= roundings * 2.0 ** -8 * ref.abs() + n * 2.0 ** -23 * mag).all()

    # forward
    ref = embedding.cpu().to(F)[ids.cpu().long()] * 3.0
    near(c(step.hidden), ref.unsqueeze(1).expand(-1, hc, -1), ref.unsqueeze(1).abs(), 1)
    rows = step.rows[:T].cpu().reshape(-1)
    emb = table[rows.clamp_min(0).long()] * (rows >= 0).unsqueeze(1)
    assert torch.equal(c(step.emb), emb.reshape(T, K))
    text = on.reshape(T) == 1
    ref = c(step.emb) @ wkv.T
    near(c(step.kv)[text], ref[text], (c(step.emb).abs() @ wkv.T.abs())[text], K)
    saved = unpack_ref(step.codes[:T].cpu().view(torch.float8_e4m3fn), step.scales[:T].cpu())
    near(c(step.x), c(step.out).mean(1), c(step.out).abs().mean(1), hc)
    z = c(step.x) @ head.cpu().to(F).T
    lse, y = torch.logsumexp(z, 1), labels.cpu().long()
    again = torch.empty_like(loss)  # (the loss itself has tests of its own)
    eg.engram_loss(s.ctx, step.x, head, VOCAB, D, labels, T, again, None,
                   ws_of(eg.engram_loss_workspace_bytes(T, VOCAB, D)))
    eg.engram_sync(s.ctx)
    assert torch.equal(loss, again)
    # backward
    dz = torch.exp(z - lse.unsqueeze(1))
    dz[torch.arange(T), y.clamp_min(0)] -= 1
    dz *= (dloss.cpu().to(F) * (y >= 0)).unsqueeze(1)
    for got, a, b, n in ((c(step.dx), dz, head.cpu().to(F), VOCAB), (step.dhead.cpu().to(F), dz.T, c(step.x), T)):
        mag = a.abs() @ b.abs()
        assert ((got - a @ b).abs() <= 2.0 ** -8 * ((a @ b).abs() + mag) + n * 2.0 ** -23 * mag).all()
    dout = (step.dx[:T].float() / hc).bfloat16().cpu().unsqueeze(1).expand(-1, hc, -1)
    gate = GateGradients(saved[:, :hc * D].reshape(T, hc, D), saved[:, hc * D:], on, wq, wk, dout)
    assert gate.misses(step.dhidden[:T].cpu(), step.dkv[:T].cpu()) == []
    for got, ref in ((step.dwq, gate.dwq), (step.dwk, gate.dwk)):
        tol = ((gate.rho + T * 2.0 ** -24) * (gate.first["dh"] * saved[:, :hc * D].reshape(T, hc, D)).abs()).sum(0)
        assert ((got.cpu().to(F) - ref).abs() <= 4 * tol).all()  # (wq and wk are between 0.5 and 2)
    dkv = c(step.dkv)
    near(c(step.demb), dkv @ wkv, dkv.abs() @ wkv.abs(), N)
    near(step.dwkv.cpu().to(F), dkv.T @ c(step.emb), dkv.T.abs() @ c(step.emb).abs(), T)
    for ids_, dout, n, scale, unique, count, grad in (
            (ids.cpu(), step.dhidden[:T].cpu(), VOCAB, 3.0, step.token_ids, step.token_count, step.token_grad),
            (rows, step.demb[:T].cpu().reshape(-1, 1, 32), s.rows(0), 1.0, step.row_ids, step.row_count, step.row_grad)):
        u, ref, tol = grad_reference(ids_.long(), dout, n, scale)
        assert int(count) == u.numel() and torch.equal(unique[:u.numel()].cpu().long(), u)
        assert ((grad[:u.numel()].cpu().to(F) - ref).abs() <= tol).all()
    s.close()


def test_training_example_learns():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_engram.py")
    spec = importlib.util.spec_from_file_location("train_engram", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.run(steps=20)
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < losses[0] - 0.5
