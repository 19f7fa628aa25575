"""Layer norm, forward and backward, against the definition in 64 bits.

Tolerances. A row's sum runs over at most 32 elements in order and 10 halvings, so its error is
below 48 steps of 2^-24 of the sum of magnitudes; with the few operations around it every fp32
quantity here is within K = 2^-18 (64 steps) of the magnitudes that it is summed from. The
stored type adds half a step: finfo(t).eps / 2 of the value.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_guard import Carved

pytestmark = pytest.mark.gpu

K = 2.0 ** -18
BF, F32 = torch.bfloat16, torch.float32


def half_step(t):
    return torch.finfo(t).eps / 2


def make(shape, xt, yt, affine, seed, wt=F32, level=1.0):
    g = torch.Generator().manual_seed(seed)
    C = shape[-1]
    x = (torch.randn(shape, generator=g) * (0.25 + 4 * torch.rand(shape[:-1] + (1,), generator=g))
         + level * torch.randn(shape[:-1] + (1,), generator=g)).to(xt)
    dy = torch.randn(shape, generator=g).to(yt)
    w = b = None
    if affine != "none":
        ws = (C,) if affine == "shared" else (shape[0], C)
        w, b = (torch.randn(ws, generator=g).to(wt) for _ in range(2))
    return x, dy, w, b


def oracle(x, dy, w, b, eps, off):
    """y, mean, rstd, dx, dw, db in float64, and the magnitudes that their errors scale with."""
    x, dy = x.double(), dy.double()
    C = x.shape[-1]
    view = (lambda t: t.double().view((t.shape[0],) + (1,) * (x.dim() - 2) + (C,)) if t.dim() == 2 else t.double())
    W = torch.ones(C, dtype=torch.float64) if w is None else view(w) + off
    Bb = torch.zeros(C, dtype=torch.float64) if b is None else view(b)
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    h = (x - mean) * rstd
    y = h * W + Bb
    eh = h.abs() + x.abs().amax(-1, keepdim=True) * rstd          # error scale of h
    ey = eh * W.abs() + Bb.abs()
    g = dy * W
    m = lambda t: t.mean(-1, keepdim=True)
    dx = rstd * (g - m(g) - h * m(g * h))
    ex = rstd * (g.abs() + m(g.abs()) + eh * m(g.abs() * eh) * 3)
    if w is None:
        return y, mean, rstd, dx, None, None, ey, ex, None, None
    axes = tuple(range(1 if w.dim() == 2 else 0, x.dim() - 1))
    s = (lambda t: t.sum(axes) if axes else t)
    return y, mean, rstd, dx, s(dy * h), s(dy), ey, ex, s(dy.abs() * eh), s(dy.abs())


def near(got, want, scale, what, step=0.0):
    got = got.double().cpu()
    lim = K * scale + step * want.abs() * (1 + K) + 1e-30
    bad = ((got - want).abs() / lim).max().item()
    assert torch.isfinite(got).all(), what
    assert bad <= 1.0, f"{what}: {bad:.3f} of its bound"


def check(shape, xt=BF, yt=BF, affine="shared", seed=0, wt=F32, eps=1e-6, off=0.0, level=1.0, mis=0):
    import block_sparse_attention_major_b200 as bsa
    x, dy, w, b = make(shape, xt, yt, affine, seed, wt, level)
    y0, mean0, rstd0, dx0, dw0, db0, ey, ex, ew, eb = oracle(x, dy, w, b, eps, off)

    def dev(t):
        if t is None or not mis:
            return None if t is None else t.cuda()
        buf = torch.zeros(t.numel() + mis, dtype=t.dtype, device="cuda")
        buf[mis:] = t.flatten().cuda()
        return buf[mis:].view(t.shape)

    xd, dyd, wd, bd = dev(x), dev(dy), dev(w), dev(b)
    y, mean, rstd = bsa.layer_norm_fwd(xd, wd, bd, eps=eps, weight_offset=off, out_dtype=yt)
    assert y.dtype == yt and y.shape == x.shape
    near(y, y0, ey, "y", half_step(yt))
    near(mean, mean0[..., 0], x.double().abs().amax(-1), "mean")
    near(rstd, rstd0[..., 0], rstd0[..., 0] * (1 + x.double().abs().amax(-1) * rstd0[..., 0]), "rstd")
    dx, dw, db = bsa.layer_norm_bwd(xd, dyd, mean, rstd, wd, weight_offset=off)
    assert dx.dtype == xt
    near(dx, dx0, ex, "dx", half_step(xt))
    if w is None:
        assert dw is None and db is None
    else:
        assert dw.shape == w.shape and dw.dtype == F32
        near(dw, dw0, ew, "dweight")
        near(db, db0, eb, "dbias")


SHAPES = [(1, 1536), (1, 1), (3, 7), (5, 64), (33, 128), (2, 9, 12, 128), (17, 200), (9, 257), (40, 256), (11, 1001),
          (6, 5120), (3, 5128), (5, 5121), (2, 10240), (2, 10248), (3, 16384), (2, 16383), (700, 96), (1500, 520),
          # even widths that are not multiples of 8: below a warp, one and two slots a thread, and wide
          (33, 10), (40, 250), (12, 258), (9, 514), (7, 1002), (5, 4098), (3, 5446), (3, 9002), (2, 16382)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("types", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)], ids=["bb", "fb", "ff", "bf"])
def test_shapes_and_types(shape, types):
    check(shape, *types, seed=len(shape) + shape[-1])


@pytest.mark.parametrize("shape", [(3, 5, 128), (2, 301, 1536), (5, 1, 64), (1, 77, 200), (4, 33, 1001), (300, 2, 8),
                                   (700, 1, 520)], ids=str)
@pytest.mark.parametrize("affine", ["none", "shared", "item"])
def test_affine_forms(shape, affine):
    check(shape, affine=affine, off=1.0, seed=3)
    check(shape, xt=F32, affine=affine, wt=BF, seed=4)


def test_rows_far_from_zero():
    # the variance is that of the distances from the mean: no cancellation at 1000 times the spread
    check((64, 1536), xt=F32, yt=F32, level=1000.0, seed=5)


def test_unaligned_addresses():
    for mis in (1, 3, 4):
        check((7, 264), mis=mis, seed=6)
        check((7, 1024), xt=F32, yt=F32, mis=mis, seed=7)


def test_constant_row_and_one_column():
    import block_sparse_attention_major_b200 as bsa
    x = torch.full((3, 512), 2.5, device="cuda")
    y, mean, rstd = bsa.layer_norm_fwd(x, eps=1e-6)
    assert torch.equal(y, torch.zeros_like(y)) and torch.equal(mean, x[:, 0])
    assert (rstd - 1e3).abs().max() < 1e3 * K
    x = torch.randn((5, 1), device="cuda")
    y, mean, rstd = bsa.layer_norm_fwd(x)
    dx, _, _ = bsa.layer_norm_bwd(x, torch.randn_like(x), mean, rstd)
    assert not y.any() and not dx.any()


def test_nan_and_infinity_stay_in_their_row():
    import block_sparse_attention_major_b200 as bsa
    for C in (128, 1001, 5120):
        x = torch.randn((9, C), device="cuda").bfloat16()
        clean, _, _ = bsa.layer_norm_fwd(x)
        x[4, 3] = math.nan
        x[6, 5] = math.inf
        y, mean, rstd = bsa.layer_norm_fwd(x)
        keep = [0, 1, 2, 3, 5, 7, 8]
        assert torch.equal(y[keep], clean[keep])
        assert y[4].isnan().all() and y[6].isnan().all()
        dx, _, _ = bsa.layer_norm_bwd(x, torch.ones_like(x), mean, rstd)
        assert torch.isfinite(dx[keep]).all() and dx[4].isnan().all()


def test_gradients_against_differences():
    import block_sparse_attention_major_b200 as bsa
    g = torch.Generator().manual_seed(8)
    x, dy = (torch.randn((4, 48), generator=g) for _ in range(2))
    w, b = (torch.randn((48,), generator=g) for _ in range(2))
    y, mean, rstd = bsa.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    dx, dw, db = (t.double().cpu() for t in bsa.layer_norm_bwd(x.cuda(), dy.cuda(), mean, rstd, w.cuda()))

    def loss(x, w, b):
        x = x.double()
        h = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, correction=0, keepdim=True) + 1e-6)
        return ((h * w.double() + b.double()) * dy.double()).sum()

    # central differences: error h^2 / 6 of the third derivative, about 1e-8 here at h = 1e-4
    for t, grad, at in ((0, dx, (2, 5)), (0, dx, (0, 47)), (1, dw, (7,)), (2, db, (40,))):
        args = [x.double(), w.double(), b.double()]
        up, down = ([a.clone() for a in args] for _ in range(2))
        up[t][at] += 1e-4
        down[t][at] -= 1e-4
        want = (loss(*up) - loss(*down)) / 2e-4
        assert abs(grad[at] - want) <= 1e-5 * (1 + abs(want))


@pytest.mark.parametrize("shape", [(2, 37, 128), (3, 11, 1001), (2, 6, 5120), (40, 1, 64)], ids=str)
def test_no_writes_outside_and_same_bits_again(shape):
    import block_sparse_attention_major_b200 as bsa
    x, dy, w, b = make(shape, BF, BF, "item", 9)
    rows = shape[:-1]
    n = bsa.layer_norm_workspace_bytes(x.cuda(), w.cuda())
    c = Carved([(shape, BF)] * 4 + [(rows, F32)] * 2 + [(w.shape, F32)] * 2 + [((n,), torch.uint8)])
    xd, dyd, y, dx, mean, rstd, dw, db, ws = c.views
    xd.copy_(x), dyd.copy_(dy)
    seen = []
    for fill in (0, 255):
        ws.fill_(fill)
        bsa.layer_norm_fwd(xd, w.cuda(), b.cuda(), y=y, mean=mean, rstd=rstd)
        bsa.layer_norm_bwd(xd, dyd, mean, rstd, w.cuda(), dx=dx, dweight=dw, dbias=db, ws=ws)
        torch.cuda.synchronize()
        seen.append([t.clone() for t in (y, mean, rstd, dx, dw, db)])
    assert c.guards_intact()
    assert all(torch.equal(p, q) for p, q in zip(*seen))


def test_in_place_streams_and_graph():
    import block_sparse_attention_major_b200 as bsa
    x, dy, w, b = (t.cuda() for t in make((3, 50, 1536), BF, BF, "shared", 10))
    y0, mean, rstd = bsa.layer_norm_fwd(x, w, b)
    dx0, dw0, db0 = bsa.layer_norm_bwd(x, dy, mean, rstd, w)
    own = x.clone()
    bsa.layer_norm_fwd(own, w, b, y=own)
    g = dy.clone()
    bsa.layer_norm_bwd(x, g, mean, rstd, w, dx=g)
    assert torch.equal(own, y0) and torch.equal(g, dx0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, m1, r1 = bsa.layer_norm_fwd(x, w, b, stream=side)
    dx1, dw1, db1 = bsa.layer_norm_bwd(x, dy, m1, r1, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y1, y0) and torch.equal(dx1, dx0) and torch.equal(dw1, dw0) and torch.equal(db1, db0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, m2, r2 = bsa.layer_norm_fwd(x, w, b)
        dx2, dw2, db2 = bsa.layer_norm_bwd(x, dy, m2, r2, w)
    x.mul_(-1.5)
    graph.replay()
    want = bsa.layer_norm_fwd(x, w, b)
    want += bsa.layer_norm_bwd(x, dy, want[1], want[2], w)
    for got, w_ in zip((y2, m2, r2, dx2, dw2, db2), want):
        assert torch.equal(got, w_)


def test_parts_not_wanted():
    import block_sparse_attention_major_b200 as bsa
    x, dy, w, b = (t.cuda() for t in make((4, 128), BF, BF, "shared", 11))
    y, mean, rstd = bsa.layer_norm_fwd(x, w, want_stats=False)
    assert mean is None and rstd is None
    _, mean, rstd = bsa.layer_norm_fwd(x, w)
    full = bsa.layer_norm_bwd(x, dy, mean, rstd, w)
    n0 = bsa.launch_count()
    dx, dw, db = bsa.layer_norm_bwd(x, dy, mean, rstd, w, want_weight=False, want_bias=False)
    assert bsa.launch_count() - n0 == 1 and dw is None and db is None and torch.equal(dx, full[0])
    dx, dw, db = bsa.layer_norm_bwd(x, dy, mean, rstd, w, want_bias=False)
    assert db is None and torch.equal(dw, full[1])


def test_refusals():
    import block_sparse_attention_major_b200 as bsa
    x = torch.zeros((4, 6, 32), device="cuda", dtype=BF)
    w = torch.zeros((32,), device="cuda")
    st = torch.zeros((4, 6), device="cuda")
    for bad in (lambda: bsa.layer_norm_fwd(x.half()), lambda: bsa.layer_norm_fwd(x[:, ::2]),
                lambda: bsa.layer_norm_fwd(x, w[:16]), lambda: bsa.layer_norm_fwd(x, w, w[None].expand(4, 32)),
                lambda: bsa.layer_norm_fwd(x, w[None].expand(4, 32)), lambda: bsa.layer_norm_fwd(x, None, w),
                lambda: bsa.layer_norm_fwd(x[:0]), lambda: bsa.layer_norm_fwd(x.cpu()),
                lambda: bsa.layer_norm_fwd(x, w.cpu()), lambda: bsa.layer_norm_fwd(x, w, y=torch.zeros_like(x)[:2]),
                lambda: bsa.layer_norm_fwd(x, mean=st[:2]), lambda: bsa.layer_norm_fwd(x, w.half()),
                lambda: bsa.layer_norm_bwd(x, x, st, st[:2], w), lambda: bsa.layer_norm_bwd(x, x[:2], st, st, w),
                lambda: bsa.layer_norm_bwd(x, x, st, st, None, dweight=w)):
        with pytest.raises(ValueError):
            bad()
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(bsa.BsaError) as e:
        bsa.layer_norm_bwd(x, x, st, st, w, ws=small[:128])
    assert e.value.status == 2
    with pytest.raises(bsa.BsaError):
        bsa.layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(bsa.BsaError):
        bsa.layer_norm_fwd(torch.zeros((1, 16385), device="cuda"))


def test_offsets_past_32_bits():
    import block_sparse_attention_major_b200 as bsa
    rows, C = 1 << 20, 2100
    x = torch.zeros((rows, C), dtype=BF, device="cuda")
    x[-50:] = torch.randn((50, C), generator=torch.Generator().manual_seed(12)).to(BF).cuda()
    y, mean, rstd = bsa.layer_norm_fwd(x)
    want = bsa.layer_norm_fwd(x[-50:].clone())
    for got, w in zip((y, mean, rstd), want):
        assert torch.equal(got[-50:], w)
    assert not y[:-50].any()
    dx, _, _ = bsa.layer_norm_bwd(x, x, mean, rstd, dx=y)
    assert torch.equal(dx[-50:], bsa.layer_norm_bwd(x[-50:].clone(), x[-50:].clone(), want[1], want[2])[0])


@pytest.mark.parametrize("C", [40, 128, 258, 1536, 5120])
def test_many_items_a_block(C):
    # a block's range meets several items: each item's rows are those of a call on it alone
    import block_sparse_attention_major_b200 as bsa
    B, N = 3000, 3
    for xt in (BF, F32):
        x, dy, w, b = (t.cuda() for t in make((B, N, C), xt, BF, "item", 60 + C))
        for _ in range(3):
            y, mean, rstd = bsa.layer_norm_fwd(x, w, b, out_dtype=BF)
            dx, dw, db = bsa.layer_norm_bwd(x, dy, mean, rstd, w)
            for i in (0, 1, 7, 501, 1500, 1501, 2222, B - 1):
                y1, m1, r1 = bsa.layer_norm_fwd(x[i], w[i], b[i], out_dtype=BF)
                dx1, _, _ = bsa.layer_norm_bwd(x[i], dy[i], m1, r1, w[i])
                assert torch.equal(y[i], y1) and torch.equal(mean[i], m1) and torch.equal(dx[i], dx1)
            h = (x.double() - mean.double()[..., None]) * rstd.double()[..., None]
            near(dw, (dy.double() * h).sum(1).cpu(), (dy.double() * h).abs().sum(1).cpu(), "dweight")
            near(db, dy.double().sum(1).cpu(), dy.double().abs().sum(1).cpu(), "dbias")


@pytest.mark.parametrize("C", [4, 32, 520, 1032, 33, 30])
def test_places_past_a_row_of_large_equal_values(C):
    # mean 2^118 and rstd 2^10: (0 - mean) rstd is past fp32, and only places past the row's end see it.
    # h is 0 in the row, so dx = rstd (g - mean g), dw = 0 and db = dy.
    import block_sparse_attention_major_b200 as bsa
    eps = 2.0 ** -20
    x = torch.full((3, C), 2.0 ** 118, device="cuda")
    dy = torch.randn((3, C), generator=torch.Generator().manual_seed(70)).cuda()
    w = torch.ones(C, device="cuda")
    mean, rstd = torch.full((3,), 2.0 ** 118, device="cuda"), torch.full((3,), eps ** -0.5, device="cuda")
    dx, dw, db = bsa.layer_norm_bwd(x, dy, mean, rstd, w)
    g = dy.double().cpu()
    near(dx, 2.0 ** 10 * (g - g.mean(1, keepdim=True)), 2.0 ** 10 * (g.abs() + g.abs().mean(1, keepdim=True)), "dx", half_step(F32))
    assert not dw.any()
    near(db, g.sum(0), g.abs().sum(0), "dbias")
