"""Attention to an encoder's states of another length, forward and backward, against the
definition in 64 bits.

Tolerances, element by element. R = 2^-8 is half a step of bf16 relative to the value. The
probabilities enter the P V product in bf16 and the output is stored in bf16; everything else
is fp32, whose part (scores of d terms, exponentials, sums) is put at E = 2^-11 of the
magnitudes, eight times below R:
    out   (R + E) sum_j w_j |v_j|  +  R |out|                                       =: e_out
    lse   2^-18 (1 + |lse| + max_j scale sum_c |q_c k_c|)
    dv    (R + E) sum_i p |do|  +  R |dv|
    ds    (R + E) |ds| + p (e_D + E |do|.|v|),  e_D = |do|.e_out, since D is taken from the stored output
    dq    scale sum_j e_ds |k_j| + R |dq|,  dk  scale sum_i e_ds |q_i| + R |dk|
"""
import math

import pytest
import torch

from test_gpu_guard import Carved

pytestmark = pytest.mark.gpu

R, E = 2.0 ** -8, 2.0 ** -11
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF).cuda()


def oracle(q, k, v, valid, scale, dout=None):
    """Everything in float64 with its error bounds; valid: bool [B, M]."""
    B, N, H, d = q.shape
    M, Hkv = k.shape[1:3]
    out = torch.zeros((B, N, H, d), dtype=F64, device="cuda")
    lse = torch.full((B, H, N), -math.inf, dtype=F64, device="cuda")
    r = {"out": (out, torch.zeros_like(out)), "lse": (lse, torch.full_like(lse, 2.0 ** -18))}
    if dout is not None:
        r["dq"] = (torch.zeros_like(out), torch.zeros_like(out))
        for n in ("dk", "dv"):
            z = torch.zeros((B, M, Hkv, d), dtype=F64, device="cuda")
            r[n] = (z, torch.zeros_like(z))
    for b in range(B):
        js = valid[b].nonzero()[:, 0]
        if js.numel() == 0:
            continue
        for h in range(H):
            c = h // (H // Hkv)
            Q, K, V = q[b, :, h].to(F64), k[b, js, c].to(F64), v[b, js, c].to(F64)
            s = scale * Q @ K.T
            L = torch.logsumexp(s, 1)
            p = torch.exp(s - L[:, None])
            o = p @ V
            eo = (R + E) * (p @ V.abs()) + R * o.abs()
            r["out"][0][b, :, h], r["out"][1][b, :, h] = o, eo
            r["lse"][0][b, h] = L
            r["lse"][1][b, h] = 2.0 ** -18 * (1 + L.abs() + (scale * Q.abs() @ K.abs().T).amax(1))
            if dout is None:
                continue
            G = dout[b, :, h].to(F64)
            t = G @ V.T
            ds = p * (t - (p * t).sum(1, keepdim=True))
            eD = (G.abs() * eo).sum(1, keepdim=True)
            eds = (R + E) * ds.abs() + p * (eD + E * (G.abs() @ V.abs().T))
            if js.numel() == 1:
                ds, eds = torch.zeros_like(ds), torch.zeros_like(ds)      # the weight is 1: exactly nothing
            dq = scale * ds @ K
            r["dq"][0][b, :, h] = dq
            r["dq"][1][b, :, h] = scale * eds @ K.abs() + R * dq.abs()
            r["dk"][0][b, js, c] += scale * ds.T @ Q
            r["dk"][1][b, js, c] += scale * eds.T @ Q.abs()
            r["dv"][0][b, js, c] += p.T @ G
            r["dv"][1][b, js, c] += (R + E) * (p.T @ G.abs())
    if dout is not None:
        for n in ("dk", "dv"):
            r[n][1].add_(R * r[n][0].abs())
    return r


def near(got, want, what):
    want, lim = want
    got = got.to(F64)
    none = torch.isinf(want)
    same, nans = torch.equal(none, torch.isinf(got)), int(got.isnan().sum())
    assert same and nans == 0, f"{what}: {nans} NaN of {got.numel()}"
    err = (got - want)[~none].abs()
    worst = (err / (lim[~none] + 1e-30)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of its bound, max error {err.max().item():.3e}"


def valid_keys(B, M, kv_len, key_mask):
    ok = torch.ones((B, M), dtype=torch.bool, device="cuda")
    if kv_len is not None:
        ok &= torch.arange(M, device="cuda")[None] < kv_len[:, None]
    if key_mask is not None:
        ok &= key_mask
    return ok


def check(B, N, M, H, Hkv, d, kv_len=None, key_mask=None, seed=0, train=True, scale=None, q=None, k=None, v=None,
          poison=False):
    import block_sparse_attention_major_b200 as bsa
    g = bsa.CrossGeometry(B, H, Hkv, d, N, M)
    q = randn((B, N, H, d), seed) if q is None else q
    k = randn((B, M, Hkv, d), seed + 1) if k is None else k
    v = randn((B, M, Hkv, d), seed + 2) if v is None else v
    if kv_len is not None:
        kv_len = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    if key_mask is not None:
        key_mask = torch.as_tensor(key_mask, dtype=torch.bool).cuda()
    ok = valid_keys(B, M, kv_len, key_mask)
    if poison:
        bad = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(BF).max], device="cuda").to(BF)
        fill = bad[torch.arange(M, device="cuda") % 4][None, :, None, None]
        k, v = (torch.where(ok[:, :, None, None], t, fill) for t in (k, v))
    ws = bsa.alloc_cross_workspace(g)
    ws[256:] = 255                                        # nothing but the error word needs a value
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    out, lse = bsa.cross_attn_fwd(g, q, k, v, kv_len, key_mask, scale=scale, ws=ws)
    torch.cuda.synchronize()
    assert bsa.read_error(ws) == 0
    dout = randn((B, N, H, d), seed + 3) if train else None
    want = oracle(q, k, v, ok, sc, dout)
    near(out, want["out"], "out")
    near(lse, want["lse"], "lse")
    empty = bool(out[~ok.any(1)].any())
    assert not empty
    if not train:
        return
    ws[256:] = 255
    dq, dk, dv = bsa.cross_attn_bwd(g, q, k, v, out, lse, dout, kv_len, key_mask, scale=scale, ws=ws)
    torch.cuda.synchronize()
    assert bsa.read_error(ws) == 0
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        near(t, want[n], n)
    masked = bool(dk[~ok].any() or dv[~ok].any())
    assert not masked


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,M", [(1, 1), (1, 512), (3, 2), (127, 127), (128, 128), (129, 129), (255, 300), (256, 64),
                                 (257, 513), (1000, 77), (5, 1000)])
def test_lengths(N, M, d):
    check(1, N, M, 2, 2, d, seed=N + M)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 2), (10, 2), (8, 1), (24, 1), (40, 1), (128, 1), (65, 1), (14, 2)])
def test_head_layouts(H, Hkv):
    # groups of 3, 5, 7, 24, 40 and 65 heads leave rows of a 128-row tile empty
    check(2, 67, 150, H, Hkv, 64, seed=H)
    check(1, 31, 200, H, Hkv, 128, kv_len=[133], seed=H + 1)


@pytest.mark.parametrize("d", [64, 128])
def test_lengths_per_item(d):
    check(6, 140, 300, 2, 2, d, kv_len=[0, 1, 128, 129, 300, 299], seed=20)
    check(3, 33, 257, 4, 2, d, kv_len=[-5, 1000, 256], seed=21)          # clamped to [0, M]
    check(2, 33, 130, 2, 1, d, kv_len=[0, 0], seed=22)


@pytest.mark.parametrize("d", [64, 128])
def test_masks(d):
    g = torch.Generator().manual_seed(30)
    m = torch.rand((5, 391), generator=g) < 0.7
    m[1] = False
    m[2] = False
    m[2, 390] = True                      # one key, the last
    m[3, 128:256] = False                 # a whole tile
    m[4, :300] = False                    # padded on the left
    check(5, 150, 391, 4, 2, d, key_mask=m, seed=31)
    check(5, 150, 391, 4, 2, d, key_mask=m, kv_len=[391, 5, 390, 200, 310], seed=32)


@pytest.mark.parametrize("d", [64, 128])
def test_what_masked_keys_hold_does_not_matter(d):
    g = torch.Generator().manual_seed(40)
    m = torch.rand((3, 333), generator=g) < 0.6
    check(3, 200, 333, 2, 2, d, key_mask=m, seed=41, poison=True)
    check(3, 200, 333, 4, 2, d, kv_len=[0, 130, 256], seed=42, poison=True)
    check(2, 4, 1300, 4, 2, d, kv_len=[700, 1], seed=43, poison=True)    # few queries: split keys


def test_few_queries_split_over_the_keys():
    check(1, 1, 5000, 4, 4, 128, seed=50, train=False)
    check(2, 16, 3001, 24, 8, 128, kv_len=[3001, 100], seed=51)
    check(2, 7, 2048, 6, 2, 64, key_mask=(torch.arange(2048)[None] % 700 < torch.tensor([[0], [3]])), seed=52)


def test_many_units():
    check(2, 9001, 200, 4, 4, 128, kv_len=[200, 77], seed=60)
    check(1, 20000, 300, 4, 2, 64, seed=61)


def test_growing_scores_rescale_the_output():
    # keys grow along the sequence, so the running maximum moves by far more than 2^8 a tile
    B, N, M, H, d = 1, 130, 700, 2, 128
    k = (randn((B, M, H, d), 70).float() * torch.linspace(0.1, 6, M, device="cuda")[None, :, None, None]).to(BF)
    check(B, N, M, H, H, d, seed=71, k=k)
    check(B, N, M, H, H, d, seed=72, k=k.flip(1).contiguous())
    check(B, N, M, H, H, d, seed=73, scale=1.0)


def test_one_valid_key():
    import block_sparse_attention_major_b200 as bsa
    for kw in (dict(M=1), dict(M=200, kv_len=[1]), dict(M=200, key_mask=torch.arange(200)[None] == 150)):
        check(1, 300, kw["M"], 2, 2, 128, seed=80, **{n: x for n, x in kw.items() if n != "M"})
    g = bsa.CrossGeometry(1, 2, 2, 128, 300, 1)
    q, k, v, do = randn((1, 300, 2, 128), 81), randn((1, 1, 2, 128), 82), randn((1, 1, 2, 128), 83), randn((1, 300, 2, 128), 84)
    out, lse = bsa.cross_attn_fwd(g, q, k, v)
    assert torch.equal(out, v.expand_as(out))             # a weight of 1 returns the value itself
    dq, dk, _ = bsa.cross_attn_bwd(g, q, k, v, out, lse, do)
    assert not dq.any() and not dk.any()


@pytest.mark.parametrize("M", [2, 3, 5, 17, 128])
def test_gradients_of_few_keys_keep_two_roundings(M):
    # dq and dk carry the rounding of dS and that of the result, each uniform within R of the value at
    # most: R / sqrt(3) each, sqrt(2 / 3) R together. D taken from the rounded output would add as
    # much again where few keys share a row.
    import block_sparse_attention_major_b200 as bsa
    B, N, H, d = 2, 700, 4, 128
    g = bsa.CrossGeometry(B, H, H, d, N, M)
    q, k, v, do = randn((B, N, H, d), 160), randn((B, M, H, d), 161), randn((B, M, H, d), 162), randn((B, N, H, d), 163)
    out, lse = bsa.cross_attn_fwd(g, q, k, v)
    dq, dk, _ = bsa.cross_attn_bwd(g, q, k, v, out, lse, do)
    want = oracle(q, k, v, torch.ones((B, M), dtype=torch.bool, device="cuda"), d ** -0.5, do)
    for name, got in (("dq", dq), ("dk", dk)):
        w = want[name][0]
        rel = ((got.to(F64) - w).norm() / w.norm()).item()
        assert rel <= math.sqrt(2 / 3) * R, (name, rel)


def test_strided_and_shared_inputs():
    B, N, M, H, Hkv, d = 3, 150, 140, 4, 2, 64
    qkv = randn((B, N, 3, H, d), 90)
    kv = randn((B, M, 2, Hkv, d), 91)
    check(B, N, M, H, Hkv, d, q=qkv[:, :, 1], k=kv[:, :, 0], v=kv[:, :, 1], seed=92)
    # heads ahead of tokens; padded rows; every item the same keys and queries
    qh = randn((B, H, N, d), 93).transpose(1, 2)
    wide = randn((B, M, Hkv, d + 8), 94)[..., :d]
    check(B, N, M, H, Hkv, d, q=qh, k=wide, v=wide, seed=95)
    one = randn((1, M, Hkv, d), 96).expand(B, M, Hkv, d)
    check(B, N, M, H, Hkv, d, q=randn((1, N, H, d), 97).expand(B, N, H, d), k=one, v=one, kv_len=[140, 3, 0], seed=98)
    # an axis of one index may have any stride
    odd = torch.as_strided(randn((B * M * d,), 99), (B, M, 1, d), (M * d, d, 3, 1))
    check(B, N, M, 2, 1, d, k=odd, v=odd, seed=100)


def test_constants_and_values_of_one():
    import block_sparse_attention_major_b200 as bsa
    g = bsa.CrossGeometry(1, 2, 2, 128, 200, 300)
    z = torch.zeros((1, 200, 2, 128), dtype=BF, device="cuda")
    k, v = randn((1, 300, 2, 128), 101), torch.ones((1, 300, 2, 128), dtype=BF, device="cuda")
    out, lse = bsa.cross_attn_fwd(g, z, k, v)
    assert (out.float() - 1).abs().max() <= 2 * R and (lse - math.log(300)).abs().max() < 1e-5


def test_gradients_against_differences():
    import block_sparse_attention_major_b200 as bsa
    B, N, M, H, Hkv, d = 1, 9, 21, 2, 1, 64
    g = bsa.CrossGeometry(B, H, Hkv, d, N, M)
    q, k, v, do = randn((B, N, H, d), 110), randn((B, M, Hkv, d), 111), randn((B, M, Hkv, d), 112), randn((B, N, H, d), 113)
    out, lse = bsa.cross_attn_fwd(g, q, k, v)
    grads = bsa.cross_attn_bwd(g, q, k, v, out, lse, do)
    bound = oracle(q, k, v, torch.ones((B, M), dtype=torch.bool, device="cuda"), d ** -0.5, do)

    def loss(q, k, v):
        k, v = (t.repeat_interleave(H // Hkv, 2) for t in (k, v))
        s = torch.einsum("bnhd,bmhd->bhnm", q, k) * d ** -0.5
        return (torch.einsum("bhnm,bmhd->bnhd", torch.softmax(s, -1), v) * do.double()).sum()

    for i, (name, at) in enumerate((("dq", (0, 3, 1, 7)), ("dk", (0, 20, 0, 63)), ("dv", (0, 0, 0, 5)))):
        up, down = ([t.double().clone() for t in (q, k, v)] for _ in range(2))
        up[i][at] += 1e-5
        down[i][at] -= 1e-5
        want = (loss(*up) - loss(*down)) / 2e-5           # off by about 1e-9
        assert (grads[i][at].double() - want).abs() <= bound[name][1][at] + 1e-6


@pytest.mark.parametrize("case", [(2, 130, 200, 6, 2, 64), (1, 257, 129, 2, 2, 128), (2, 3, 1500, 4, 2, 128)], ids=str)
def test_no_writes_outside_and_same_bits_again(case):
    import block_sparse_attention_major_b200 as bsa
    B, N, M, H, Hkv, d = case
    g = bsa.CrossGeometry(B, H, Hkv, d, N, M)
    qs, ks = (B, N, H, d), (B, M, Hkv, d)
    q, k, v, do = randn(qs, 120), randn(ks, 121), randn(ks, 122), randn(qs, 123)
    mask = torch.rand((B, M), generator=torch.Generator().manual_seed(124)).cuda() < 0.8
    c = Carved([(qs, BF)] * 2 + [(ks, BF)] * 2 + [((B, H, N), F32), ((bsa.cross_workspace_bytes(g),), torch.uint8)])
    out, dq, dk, dv, lse, ws = c.views
    seen = []
    for fill in (0, 255):
        ws.fill_(fill)
        bsa.clear_error(ws)
        bsa.cross_attn_fwd(g, q, k, v, None, mask, out=out, lse=lse, ws=ws)
        bsa.cross_attn_bwd(g, q, k, v, out, lse, do, None, mask, dq=dq, dk=dk, dv=dv, ws=ws)
        torch.cuda.synchronize()
        assert bsa.read_error(ws) == 0
        seen.append([t.clone() for t in (out, lse, dq, dk, dv)])
    assert c.guards_intact()
    assert all(torch.equal(p, r) for p, r in zip(*seen))


def test_streams_and_graph():
    import block_sparse_attention_major_b200 as bsa
    B, N, M, H, d = 2, 300, 200, 4, 128
    g = bsa.CrossGeometry(B, H, H, d, N, M)
    q, k, v, do = randn((B, N, H, d), 130), randn((B, M, H, d), 131), randn((B, M, H, d), 132), randn((B, N, H, d), 133)
    n = torch.tensor([150, 200], dtype=torch.int32, device="cuda")

    def both(stream=None):
        out, lse = bsa.cross_attn_fwd(g, q, k, v, n, stream=stream)
        return (out, lse) + bsa.cross_attn_bwd(g, q, k, v, out, lse, do, n, stream=stream)

    want = both()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in sides:                                        # two calls at once, each with a workspace of its own
        s.wait_stream(torch.cuda.current_stream())
        got.append(both(s))
    for s, r in zip(sides, got):
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(x, y) for x, y in zip(r, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    q.mul_(-0.5)
    n.copy_(torch.tensor([7, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, both()))


def test_without_lse_and_launches():
    import block_sparse_attention_major_b200 as bsa
    g = bsa.CrossGeometry(1, 40, 40, 64, 1024, 100)
    q, k, v = randn((1, 1024, 40, 64), 140), randn((1, 100, 40, 64), 141), randn((1, 100, 40, 64), 142)
    out, lse = bsa.cross_attn_fwd(g, q, k, v)
    n0 = bsa.launch_count()
    alone, none = bsa.cross_attn_fwd(g, q, k, v, want_lse=False)
    assert bsa.launch_count() - n0 == 1 and none is None and torch.equal(alone, out)


def test_refusals():
    import block_sparse_attention_major_b200 as bsa
    g = bsa.CrossGeometry(2, 4, 2, 64, 10, 12)
    q, k = randn((2, 10, 4, 64), 150), randn((2, 12, 2, 64), 151)
    out, lse = bsa.cross_attn_fwd(g, q, k, k)
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: bsa.cross_attn_fwd(g, q.half(), k, k), lambda: bsa.cross_attn_fwd(g, q[:, :5], k, k),
                lambda: bsa.cross_attn_fwd(g, q, k.cpu(), k), lambda: bsa.cross_attn_fwd(g, q, k, k, i32.long()),
                lambda: bsa.cross_attn_fwd(g, q, k, k, i32[:1]),
                lambda: bsa.cross_attn_fwd(g, q, k, k, key_mask=torch.ones((2, 12), device="cuda")),
                lambda: bsa.cross_attn_fwd(g, q, k, k, lse=lse[:1]),
                lambda: bsa.cross_attn_fwd(g, q, k, randn((2, 12, 64, 2), 1).transpose(2, 3)),
                lambda: bsa.cross_attn_bwd(g, q, k, k, out, lse, q.transpose(0, 1)),
                lambda: bsa.cross_attn_bwd(g, q, k, k, out, lse.double(), q)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros((2, 12, 2, 68), dtype=BF, device="cuda")[..., :64]          # rows 136 bytes apart
    off = torch.zeros(2 * 12 * 2 * 64 + 4, dtype=BF, device="cuda")[4:].view(2, 12, 2, 64)
    heads = randn((2, 12, 1, 64), 152).expand(2, 12, 2, 64)                       # heads at stride 0
    for bad in (lambda: bsa.cross_attn_fwd(g, q, odd, k), lambda: bsa.cross_attn_fwd(g, q, k, off),
                lambda: bsa.cross_attn_fwd(g, q, heads, k), lambda: bsa.cross_attn_fwd(g, q, k, k, scale=0.0),
                lambda: bsa.cross_attn_fwd(g, q, k, k, scale=math.inf),
                lambda: bsa.cross_attn_fwd(g, q, k, k, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(bsa.BsaError):
            bad()
    assert bsa.cross_workspace_bytes(bsa.CrossGeometry(1, 4, 3, 64, 1, 1)) == 0


def test_offsets_past_32_bits():
    # 2.3e9 elements of q and out: the last tokens are those of a call on them alone
    import block_sparse_attention_major_b200 as bsa
    N, H, d, M = 140000, 128, 128, 5
    k, v = randn((1, M, 16, d), 170), randn((1, M, 16, d), 171)
    q = torch.zeros((1, N, H, d), dtype=BF, device="cuda")
    q[:, -300:] = randn((1, 300, H, d), 172)
    out, lse = bsa.cross_attn_fwd(bsa.CrossGeometry(1, H, 16, d, N, M), q, k, v)
    last, last_lse = bsa.cross_attn_fwd(bsa.CrossGeometry(1, H, 16, d, 300, M), q[:, -300:], k, v)
    assert torch.equal(out[:, -300:], last) and torch.equal(lse[:, :, -300:], last_lse)
    assert torch.equal(out[:, 7], out[:, N - 301])


@pytest.mark.parametrize("d", [64, 128])
def test_items_without_keys_between_many_units(d):
    # one key tile, five items of which two are empty, several units of each a block: every item's
    # rows are those of a call on it alone, and the same again
    import block_sparse_attention_major_b200 as bsa
    B, N, M, H = 5, 9000, 100, 12
    q, k, v = randn((B, N, H, d), 180), randn((B, M, H, d), 181), randn((B, M, H, d), 182)
    lens = [M, 0, M, 0, 77]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g, one = bsa.CrossGeometry(B, H, H, d, N, M), bsa.CrossGeometry(1, H, H, d, N, M)
    ws = bsa.alloc_cross_workspace(g)
    want = [bsa.cross_attn_fwd(one, q[b:b + 1], k[b:b + 1], v[b:b + 1], n[b:b + 1]) for b in range(B)]
    for _ in range(4):
        out, lse = bsa.cross_attn_fwd(g, q, k, v, n, ws=ws)
        torch.cuda.synchronize()
        assert bsa.read_error(ws) == 0
        for b in range(B):
            assert torch.equal(out[b:b + 1], want[b][0]) and torch.equal(lse[b:b + 1], want[b][1])
            assert lens[b] or not out[b].any()
