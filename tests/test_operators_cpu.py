"""Cross attention and layer norm without a GPU: what the library refuses on the host, its
workspace sizes, and what the binding passes on."""
import contextlib
import ctypes

import pytest
import torch

P = 0x10000          # a pointer that no refused call follows


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_major_b200 import _build
    import block_sparse_attention_major_b200 as bsa
    _build.build()
    return bsa.load_library()


def cross(lib, geom=(2, 4, 2, 64, 10, 12), st=None, q=P, k=P, v=P, kv_len=None, mask=None, scale=0.125, out=P, lse=P,
          ws=P, ws_bytes=1 << 40, bwd=False, dout=P, dq=P, dk=P, dv=P):
    import block_sparse_attention_major_b200 as bsa
    g = bsa.bsa_cross_geom(*geom)
    s = None if st is None else ctypes.byref(bsa.bsa_cross_strides(*((ctypes.c_longlong * 3)(*x) for x in st)))
    if bwd:
        return lib.bsa_cross_attn_bwd(ctypes.byref(g), s, q, k, v, out, lse, dout, kv_len, mask, scale, dq, dk, dv, ws,
                                      ws_bytes, None)
    return lib.bsa_cross_attn_fwd(ctypes.byref(g), s, q, k, v, kv_len, mask, scale, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("geom", [(0, 4, 2, 64, 10, 12), (2, 0, 2, 64, 10, 12), (2, 4, 0, 64, 10, 12), (2, 4, 3, 64, 10, 12),
                                  (2, 4, 2, 96, 10, 12), (2, 4, 2, 64, 0, 12), (2, 4, 2, 64, 10, 0), (2, 4, 2, 64, -1, 12),
                                  (1, 129, 1, 64, 10, 12), (65536, 1, 1, 64, 1, 1), (1, 32768, 32768, 64, 1 << 17, 12),
                                  (1, 32768, 32768, 64, 10, 1 << 17), (1, 1, 1, 64, 10, 2147483647),
                                  (1, 1, 1, 64, 10, (1 << 22) + 1)], ids=str)
def test_cross_geometry_refused(lib, geom):
    import block_sparse_attention_major_b200 as bsa
    assert lib.bsa_cross_workspace_bytes(ctypes.byref(bsa.bsa_cross_geom(*geom))) == 0
    assert cross(lib, geom) == 1 and cross(lib, geom, bwd=True) == 1


def test_cross_arguments_refused(lib):
    for bwd in (False, True):
        for name in ("q", "k", "v", "out") + (("dout", "dq", "dk", "dv") if bwd else ()):
            for bad in (None, P + 8, P + 2):
                assert cross(lib, bwd=bwd, **{name: bad}) == 1, (name, bad)
        assert cross(lib, bwd=bwd, lse=P + 2) == 1
        assert cross(lib, bwd=bwd, kv_len=P + 2) == 1
        for scale in (0.0, -1.0, float("inf"), float("nan")):
            assert cross(lib, bwd=bwd, scale=scale) == 1
        assert cross(lib, bwd=bwd, ws=None) == 2 and cross(lib, bwd=bwd, ws=P + 128) == 2
        assert cross(lib, bwd=bwd, ws_bytes=256) == 2
    assert cross(lib, bwd=True, lse=None) == 1


def test_cross_strides_refused(lib):
    dense = [(10 * 4 * 64, 4 * 64, 64), (12 * 2 * 64, 2 * 64, 64), (12 * 2 * 64, 2 * 64, 64)]
    for i in range(3):
        for axis in range(3):
            for bad in (4, 65, -64, 1 << 38, 0):
                if axis == 0 and bad == 0:
                    continue                            # one tensor for every item is allowed
                st = [list(x) for x in dense]
                st[i][axis] = bad
                assert cross(lib, st=st) == 1, (i, axis, bad)
                assert cross(lib, st=st, bwd=True) == 1


def test_cross_workspace_sizes(lib):
    import block_sparse_attention_major_b200 as bsa
    size = lambda *g: bsa.cross_workspace_bytes(bsa.CrossGeometry(*g))
    # the parts of cut dk, dv units: two for each of 148 blocks, dk and dv of 128 keys in fp32
    cut = 148 * 2 * 2 * 128 * 128 * 4
    n = size(1, 12, 12, 128, 32760, 512)
    assert cut + 12 * 32760 * 8 <= n <= cut + 12 * 32760 * 8 + 8192
    # one query over 512 keys: 12 units, so the keys are split 4 ways; these parts are smaller
    assert size(1, 12, 12, 128, 1, 512) <= cut + 8192
    assert n % 256 == 0


def norm(lib, rows=4, C=32, items=1, per=0, xt=0, yt=0, wt=1, eps=1e-6, off=0.0, bwd=False, **kw):
    import block_sparse_attention_major_b200 as bsa
    f = bsa.bsa_norm_shape(rows, C, items, per, xt, yt, wt, eps, off)
    a = dict(x=P, w=P, b=P, y=P, mean=P, rstd=P, dy=P, dx=P, dw=P, db=P, ws=P, n=1 << 40) | kw
    if bwd:
        return lib.bsa_layer_norm_bwd(ctypes.byref(f), a["x"], a["dy"], a["mean"], a["rstd"], a["w"], a["dx"], a["dw"],
                                      a["db"], a["ws"], a["n"], None)
    return lib.bsa_layer_norm_fwd(ctypes.byref(f), a["x"], a["w"], a["b"], a["y"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("bad", [dict(rows=0), dict(rows=-1), dict(rows=1 << 40), dict(C=0), dict(C=16385), dict(xt=2),
                                 dict(yt=-1), dict(wt=3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                 dict(off=float("nan")), dict(per=1, items=0), dict(per=1, items=3),
                                 dict(per=1, items=65536, rows=65536), dict(x=None), dict(x=P + 1), dict(w=P + 2)], ids=str)
def test_norm_refused(lib, bad):
    assert norm(lib, **bad) == 1
    assert norm(lib, bwd=True, **bad) == 1


def test_norm_outputs_refused(lib):
    assert norm(lib, y=None) == 1 and norm(lib, yt=1, y=P + 2) == 1 and norm(lib, mean=P + 2) == 1
    for name in ("dy", "mean", "rstd", "dx"):
        assert norm(lib, bwd=True, **{name: None}) == 1, name
    assert norm(lib, bwd=True, dw=P + 2) == 1
    assert norm(lib, bwd=True, ws=None) == 2 and norm(lib, bwd=True, n=256) == 2 and norm(lib, bwd=True, ws=P + 8) == 2


def test_norm_workspace_holds_a_partial_row_for_every_block_and_item(lib):
    import block_sparse_attention_major_b200 as bsa
    for C in (1, 64, 128, 250, 520, 1001, 1536, 5120, 5128, 9000, 16384):
        for xt in (0, 1):
            f = bsa.bsa_norm_shape(10 ** 6, C, 5, 1, xt, 0, 1, 1e-6, 0.0)
            n = lib.bsa_layer_norm_workspace_bytes(ctypes.byref(f))
            assert n >= (148 + 5) * C * 8 and n % 256 == 0
    f = bsa.bsa_norm_shape(1, 512, 1, 0, 0, 0, 1, 1e-6, 0.0)
    assert lib.bsa_layer_norm_workspace_bytes(ctypes.byref(f)) == 2 * 512 * 8


class FakeStream:
    device = torch.device("cpu")
    cuda_stream = 0x5000


def fake(monkeypatch, bsa, calls):
    class FakeLib:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or 0

    monkeypatch.setattr(bsa, "load_library", lambda path=None: FakeLib())
    monkeypatch.setattr(bsa, "_need", lambda *a: None)
    monkeypatch.setattr(bsa, "_need_strided", lambda *a: None)
    monkeypatch.setattr(bsa, "_need_ws", lambda ws: None)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream())


def test_binding_passes_cross_attention_on(monkeypatch):
    import block_sparse_attention_major_b200 as bsa
    calls = []
    fake(monkeypatch, bsa, calls)
    g = bsa.CrossGeometry(2, 4, 2, 64, 10, 11)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    q, k, v, out, do = bf(2, 10, 4, 64), bf(2, 11, 2, 64), bf(2, 11, 2, 64), bf(2, 10, 4, 64), bf(2, 10, 4, 64)
    lse, ws, n = torch.zeros(2, 4, 10), torch.zeros(4096, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    m = torch.ones(2, 11, dtype=torch.bool)
    bsa.cross_attn_fwd(g, q, k, v, n, m, 0.5, out, lse, ws)
    name, a = calls[-1]
    assert name == "bsa_cross_attn_fwd" and a[1] is None
    assert a[2:] == (q.data_ptr(), k.data_ptr(), v.data_ptr(), n.data_ptr(), m.data_ptr(), 0.5, out.data_ptr(),
                     lse.data_ptr(), ws.data_ptr(), 4096, 0x5000)
    dq, dk, dv = bf(2, 10, 4, 64), bf(2, 11, 2, 64), bf(2, 11, 2, 64)
    kv = bf(2, 11, 2, 2, 64)
    bsa.cross_attn_bwd(g, q, kv[:, :, 0], kv[:, :, 1], out, lse, do, None, None, None, dq, dk, dv, ws)
    name, a = calls[-1]
    st = a[1]._obj
    assert list(st.q) == [2560, 256, 64] and list(st.k) == [2816, 256, 64] and list(st.v) == [2816, 256, 64]
    assert name == "bsa_cross_attn_bwd" and a[2:8] == (q.data_ptr(), kv.data_ptr(), kv.data_ptr() + 256, out.data_ptr(),
                                                      lse.data_ptr(), do.data_ptr())
    assert a[8:] == (None, None, 0.125, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), 4096, 0x5000)
    with pytest.raises(ValueError, match="share one device"):
        bsa.cross_attn_fwd(g, q, k, v.to("meta"), n, m, 0.5, out, lse, ws)
    assert len(calls) == 2


def test_forward_norms_through_the_output_buffer(monkeypatch):
    import types
    import block_sparse_attention_major_b200 as bsa
    calls = []
    fake(monkeypatch, bsa, calls)
    monkeypatch.setattr(bsa, "_norm_shape", lambda *a: bsa.bsa_norm_shape(1, 64, 1, 0, 0, 0, 1, 1e-6, 0.0))
    g, p = bsa.Geometry(1, 2, 64, 4, 8, 8), bsa.MaskParams(1, 1)
    x = torch.zeros(g.B, g.N, g.H, g.d, dtype=torch.bfloat16)
    b = types.SimpleNamespace(**{n: torch.zeros(8) for n in ("qt", "kt", "vt", "qbar", "kbar", "mask", "kv_count", "lse")},
                              out=torch.zeros_like(x), ws=torch.zeros(4096, dtype=torch.uint8))
    w = torch.ones(64)
    bsa.forward(g, p, x, x, x, torch.zeros(1, g.NT), bufs=b, qk_norm=bsa.QKNorm(w, w, w, w))
    names = [c[0] for c in calls]
    assert names == ["bsa_layer_norm_fwd", "bsa_reorder_pool"] * 2 + ["bsa_reorder", "bsa_build_mask_pooled",
                                                                      "bsa_sparse_attn_fwd"]
    assert calls[0][1][4] == b.out.data_ptr() and calls[1][1][1].value == b.out.data_ptr()


@pytest.mark.parametrize("C,blocks", [(2049, 2), (2305, 2), (2559, 2), (4097, 1), (8200, 1), (9000, 1), (10240, 1), (16384, 1)])
def test_norm_grid_is_what_is_resident(lib, C, blocks):
    # a partial row for each block and one more: wide rows are read by kernels built for 512 or 640
    # threads, one block an SM or, with half the threads, two
    import block_sparse_attention_major_b200 as bsa
    for xt in (0, 1):
        f = bsa.bsa_norm_shape(10 ** 6, C, 1, 0, xt, xt, 1, 1e-6, 0.0)
        n = (148 * blocks + 1) * C * 8
        assert lib.bsa_layer_norm_workspace_bytes(ctypes.byref(f)) == (n + 255) // 256 * 256


@pytest.mark.parametrize("which", range(3))
def test_forward_with_norms_leaves_inputs_in_the_output_buffer_alone(monkeypatch, which):
    import types
    import block_sparse_attention_major_b200 as bsa
    calls = []
    fake(monkeypatch, bsa, calls)
    monkeypatch.setattr(bsa, "_norm_shape", lambda *a: bsa.bsa_norm_shape(1, 64, 1, 0, 0, 0, 1, 1e-6, 0.0))
    g, p = bsa.Geometry(1, 2, 64, 5, 6, 7), bsa.MaskParams(1, 1)
    x = [torch.zeros(g.B, g.N, g.H, g.d, dtype=torch.bfloat16) for _ in range(3)]
    tiled = lambda: torch.zeros(g.B, g.H, g.NT, 64, g.d, dtype=torch.bfloat16)
    b = types.SimpleNamespace(**{n: torch.zeros(8) for n in ("qbar", "kbar", "mask", "kv_count", "lse")}, qt=tiled(),
                              kt=tiled(), vt=tiled(), out=x[which], ws=torch.zeros(4096, dtype=torch.uint8))
    w = torch.ones(64)
    bsa.forward(g, p, *x, torch.zeros(1, g.NT), bufs=b, qk_norm=bsa.QKNorm(w, w, w, w))
    norms = [c[1] for c in calls if c[0] == "bsa_layer_norm_fwd"]
    pools = [c[1] for c in calls if c[0] == "bsa_reorder_pool"]
    assert [n[1] for n in norms] == [x[0].data_ptr(), x[1].data_ptr()]
    # Q through the place of the tiled K, K through that of V, each before it is filled
    assert [n[4] for n in norms] == [b.kt.data_ptr(), b.vt.data_ptr()] == [q[1].value for q in pools]
    assert [q[2].value for q in pools] == [b.qt.data_ptr(), b.kt.data_ptr()]


def test_cross_wait_selftest_arguments_refused(lib):
    assert lib.bsa_selftest_cross_wait(None, None) == 1
    assert lib.bsa_selftest_cross_wait(ctypes.c_void_p(P + 2), None) == 1
