"""The norm, the self-attention path and the attention to an encoder's states together, as a block
of a video diffusion transformer runs them, forward and backward."""
import math

import pytest
import torch

import _cases as C
from test_cross_gpu import BF, F64, R, near, oracle, randn, valid_keys

pytestmark = pytest.mark.gpu


def plain_norm(x, w, b, eps=1e-6):
    x = x.to(F64)
    h = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, correction=0, keepdim=True) + eps)
    return h * w.to(F64) + b.to(F64)


def test_forward_with_qk_norm_is_the_forward_of_the_normalised():
    import block_sparse_attention_major_b200 as bsa
    for name in ("ragged128", "token128", "tiny_ragged"):
        w, q, k, v, diff = C.inputs(name)
        g, p = C.geometry(w), C.params(w)
        q, k, v, diff = (t.cuda() for t in (q, k, v, diff))
        gen = torch.Generator().manual_seed(1)
        qw, qb, kw, kb = (torch.randn((w.d,), generator=gen).cuda() for _ in range(4))
        norm = bsa.QKNorm(qw, qb, kw, kb)
        n0 = bsa.launch_count()
        got = bsa.forward(g, p, q, k, v, diff, qk_norm=norm)
        assert bsa.launch_count() - n0 == bsa.launches_per_forward(p, qk_norm=True)
        qn, kn = bsa.layer_norm_fwd(q, qw, qb)[0], bsa.layer_norm_fwd(k, kw, kb)[0]
        want = bsa.forward(g, p, qn, kn, v, diff)
        torch.cuda.synchronize()
        assert bsa.read_error(got.ws) == 0
        assert torch.equal(got.mask, want.mask) and torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
        again = bsa.forward(g, p, q, k, v, diff, bufs=got, rebuild_mask=False, qk_norm=norm)
        torch.cuda.synchronize()
        assert torch.equal(again.out, want.out)


def test_cross_forward_with_qk_norm():
    import block_sparse_attention_major_b200 as bsa
    g = bsa.CrossGeometry(2, 6, 2, 128, 300, 90)
    q, k, v = randn((2, 300, 6, 128), 10), randn((2, 90, 2, 128), 11), randn((2, 90, 2, 128), 12)
    n = torch.tensor([90, 33], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(13)
    qw, qb, kw, kb = (torch.randn((128,), generator=gen).to(BF).cuda() for _ in range(4))
    b = bsa.cross_forward(g, q, k, v, kv_len=n, qk_norm=bsa.QKNorm(qw, qb, kw, kb))
    torch.cuda.synchronize()
    assert bsa.read_error(b.ws) == 0
    for got, x, wt, bi in ((b.qn, q, qw, qb), (b.kn, k, kw, kb)):
        want = plain_norm(x, wt, bi)
        assert ((got.to(F64) - want).abs() <= R * want.abs() + 1e-4).all()
    want = oracle(b.qn, b.kn, v, valid_keys(2, 90, n, None), 128 ** -0.5)
    near(b.out, want["out"], "out")
    near(b.lse, want["lse"], "lse")
    with pytest.raises(ValueError):
        bsa.cross_forward(g, q, k, v, qk_norm=bsa.QKNorm(qw, qb, kw, kb), bufs=bsa.CrossBuffers(g))


def test_block_with_its_gradients_in_one_graph():
    """x -> modulated norm -> heads -> norm of q per head -> attention to the prompt; then all the
    way back, eager and captured, against the gradients of the same in 64 bits."""
    import block_sparse_attention_major_b200 as bsa
    B, N, M, H, d = 2, 200, 77, 2, 64
    Cw = H * d
    g = bsa.CrossGeometry(B, H, H, d, N, M)
    gen = torch.Generator().manual_seed(20)
    x = torch.randn((B, N, Cw), generator=gen).cuda()
    scale, shift = (0.3 * torch.randn((B, Cw), generator=gen).cuda() for _ in range(2))
    qw, qb = (torch.randn((d,), generator=gen).cuda() for _ in range(2))
    k, v, do = randn((B, M, H, d), 21), randn((B, M, H, d), 22), randn((B, N, H, d), 23)
    n = torch.tensor([77, 20], dtype=torch.int32, device="cuda")
    ws = bsa.alloc_cross_workspace(g)

    def step():
        h, m0, r0 = bsa.layer_norm_fwd(x, scale, shift, weight_offset=1.0, out_dtype=BF)
        h = h.view(B, N, H, d)
        q, m1, r1 = bsa.layer_norm_fwd(h, qw, qb)
        out, lse = bsa.cross_attn_fwd(g, q, k, v, n, ws=ws)
        dq, dk, dv = bsa.cross_attn_bwd(g, q, k, v, out, lse, do, n, ws=ws)
        dh, dqw, dqb = bsa.layer_norm_bwd(h, dq, m1, r1, qw)
        dx, dscale, dshift = bsa.layer_norm_bwd(x, dh.view(B, N, Cw), m0, r0, scale, weight_offset=1.0)
        return out, dx, dscale, dshift, dqw, dqb, dk, dv

    got = step()
    torch.cuda.synchronize()
    assert bsa.read_error(ws) == 0
    leaves = [t.to(F64).requires_grad_() for t in (x, scale, shift, qw, qb, k, v)]
    X, S, T, QW, QB, K, V = leaves
    h = plain_norm(X, torch.ones(Cw, device="cuda"), torch.zeros(Cw, device="cuda")) * (1 + S[:, None]) + T[:, None]
    hh = h.view(B, N, H, d)
    q = (hh - hh.mean(-1, keepdim=True)) / torch.sqrt(hh.var(-1, correction=0, keepdim=True) + 1e-6) * QW + QB
    s = torch.einsum("bnhd,bmhd->bhnm", q, K) / math.sqrt(d)
    s = s.masked_fill(~valid_keys(B, M, n, None)[:, None, None], -math.inf)
    out = torch.einsum("bhnm,bmhd->bnhd", torch.softmax(s, -1), V)
    grads = torch.autograd.grad(out, leaves, do.to(F64))
    # five roundings to bf16 on the way (h, q, P, dS or its like, the result), each at most R and
    # independent of the others: sqrt(5) R of the norm, times 2 for the parts that cancel
    for a, b, name in zip(got, (out,) + grads, ("out", "dx", "dscale", "dshift", "dqw", "dqb", "dk", "dv")):
        b = b.detach()
        assert (a.to(F64) - b).norm() <= 2 * math.sqrt(5) * R * b.norm(), name

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.mul_(0.7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_forward_with_qk_norm_of_an_earlier_output():
    import block_sparse_attention_major_b200 as bsa
    for name in ("ragged128", "token128"):
        w, q, k, v, diff = C.inputs(name)
        g, p = C.geometry(w), C.params(w)
        q, k, v, diff = (t.cuda() for t in (q, k, v, diff))
        gen = torch.Generator().manual_seed(2)
        norm = bsa.QKNorm(*(torch.randn((w.d,), generator=gen).cuda() for _ in range(4)))
        for i in range(3):
            bufs = bsa.forward(g, p, q, k, v, diff)
            x = [q, k, v]
            x[i] = bufs.out.clone()
            want = bsa.forward(g, p, *x, diff, qk_norm=norm)
            x[i] = bufs.out
            got = bsa.forward(g, p, *x, diff, bufs=bufs, qk_norm=norm)
            torch.cuda.synchronize()
            assert bsa.read_error(got.ws) == 0
            assert torch.equal(got.mask, want.mask) and torch.equal(got.out, want.out), "qkv"[i]
