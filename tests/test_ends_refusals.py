"""What the embedding and linear-layer calls refuse, on the host (no GPU work:
every call below returns or raises before any CUDA call)."""
import ctypes

import pytest
import torch

from atomistic_mlip_b200 import build as build_mod
from atomistic_mlip_b200 import e2f


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return e2f.lib()


D64 = ctypes.c_void_p(64)


def test_embed_abi(lib):
    f, b = lib.e2f_embed_forward, lib.e2f_embed_backward
    d, inf = D64, float("inf")

    def fwd(ids=d, it=2, N=4, table=d, dt=0, V=9, D=8, scale=1.0, Q=1, out=d, ot=0):
        return f(ids, it, N, table, dt, V, D, scale, Q, out, ot, None)

    def bwd(ids=d, it=2, N=4, g=d, dt=0, V=9, D=8, scale=1.0, Q=1, grad=d, acc=0):
        return b(ids, it, N, g, dt, V, D, scale, Q, grad, acc, None)

    for call in (fwd, bwd):
        assert call(N=-1) == 1 and call(V=0) == 1 and call(D=0) == 1 and call(Q=0) == 1
        assert call(N=1 << 31) == 1 and call(V=(1 << 31) - 1) == 1
        assert call(scale=inf) == 1 and call(scale=float("nan")) == 1
        assert call(it=0) == 4 and call(dt=2) == 4 and call(D=(1 << 20) + 1) == 4 and call(D=1 << 20, Q=2048) == 4
        assert call(ids=None) == 1
        assert call(ids=ctypes.c_void_p(66)) == 1 and call(it=3, ids=ctypes.c_void_p(68)) == 1
    assert fwd(table=None) == 1 and fwd(out=None) == 1 and fwd(ot=3) == 4
    assert fwd(table=ctypes.c_void_p(66)) == 1 and fwd(out=ctypes.c_void_p(65), ot=1) == 1
    assert bwd(g=None) == 1 and bwd(grad=None) == 1 and bwd(acc=2) == 1 and bwd(grad=ctypes.c_void_p(66)) == 1
    assert fwd(N=0, ids=None, table=None, out=None) == 0


def test_embed_binding():
    ids, table = torch.zeros(4, dtype=torch.int64), torch.zeros(5, 6)
    for bad in (lambda: e2f.embed_forward(ids.float(), table),                 # id type
                lambda: e2f.embed_forward(ids[None], table),                   # shape
                lambda: e2f.embed_forward(torch.zeros(8, dtype=torch.int64)[::2], table),
                lambda: e2f.embed_forward(ids, table.double()),
                lambda: e2f.embed_forward(ids, table.t()),
                lambda: e2f.embed_forward(ids, table, out=torch.zeros(4, 2, 6)),
                lambda: e2f.embed_forward(ids, table, out=torch.zeros(4, 1, 6), out_dtype=torch.bfloat16),
                lambda: e2f.embed_forward(ids, table),                         # not on a GPU
                lambda: e2f.embed_backward(ids, torch.zeros(3, 6), 5),
                lambda: e2f.embed_backward(ids, torch.zeros(4, 12)[:, ::2], 5),
                lambda: e2f.embed_backward(ids, torch.zeros(4, 6).half(), 5),
                lambda: e2f.embed_backward(ids, torch.zeros(4, 6), 5, accumulate=True),
                lambda: e2f.embed_backward(ids, torch.zeros(4, 6), 5, grad_table=torch.zeros(6, 6)),
                lambda: e2f.embed_backward(ids, torch.zeros(4, 6), 5)):
        with pytest.raises(ValueError):
            bad()


def _lin(dtype=0, act=1, M=4, K=8, N=6, x=64, ldx=8, W=128, ldw=8, bias=None):
    return ctypes.byref(e2f.Linear(dtype, act, M, K, N, x, ldx, W, ldw, bias))


def test_linear_abi(lib):
    f, b = lib.e2f_linear_forward, lib.e2f_linear_backward
    o = ctypes.c_void_p(1024)

    def fwd(p=None, r=None, ldr=6, out=o, ldo=6, ot=0):
        return f(p or _lin(), r, ldr, out, ldo, ot, None)

    def bwd(p=None, dy=ctypes.c_void_p(512), ldg=6, ot=0, gx=o, ldgx=8, gw=ctypes.c_void_p(2048), ldgw=8, gb=None):
        return b(p or _lin(), dy, ldg, ot, gx, ldgx, gw, ldgw, gb, None)

    assert f(None, None, 6, o, 6, 0, None) == 1
    for call in (fwd, bwd):
        assert call(p=_lin(dtype=2)) == 4 and call(p=_lin(act=3)) == 4 and call(ot=2) == 4
        assert call(p=_lin(M=-1)) == 1 and call(p=_lin(M=1 << 31)) == 1
        assert call(p=_lin(K=0)) == 1 and call(p=_lin(N=0)) == 1
        assert call(p=_lin(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21)) == 4
        assert call(p=_lin(ldx=7)) == 1 and call(p=_lin(ldw=7)) == 1 and call(p=_lin(ldx=1 << 40)) == 1
        assert call(p=_lin(x=None)) == 1 and call(p=_lin(W=None)) == 1
        assert call(p=_lin(x=66)) == 1 and call(p=_lin(dtype=1, W=65)) == 1 and call(p=_lin(bias=66)) == 1
    assert fwd(out=None) == 1 and fwd(ldo=5) == 1 and fwd(r=ctypes.c_void_p(4096), ldr=5) == 1
    assert fwd(out=ctypes.c_void_p(64)) == 1 and fwd(out=ctypes.c_void_p(128)) == 1      # x, W as the output
    assert fwd(r=o, ldr=7) == 1                                                          # in place, other stride
    assert fwd(out=ctypes.c_void_p(1026)) == 1 and fwd(r=ctypes.c_void_p(4098)) == 1
    assert fwd(p=_lin(M=0, x=None, W=None), out=None) == 0
    assert bwd(dy=None) == 1 and bwd(ldg=5) == 1 and bwd(ldgx=7) == 1 and bwd(ldgw=7) == 1
    assert bwd(gx=ctypes.c_void_p(512)) == 1 and bwd(gw=ctypes.c_void_p(128)) == 1
    assert bwd(gx=ctypes.c_void_p(1026)) == 1 and bwd(gb=ctypes.c_void_p(1026)) == 1


def test_linear_binding():
    x, W, dy = torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(4, 6)
    f, b = e2f.linear_forward, e2f.linear_backward
    for bad in (lambda: f(x, W),                                             # not on a GPU
                lambda: f(x.double(), W.double()), lambda: f(x, W.bfloat16()), lambda: f(x, torch.zeros(6, 9)),
                lambda: f(x[None], W), lambda: f(x, W, act="relu"), lambda: f(x, W, bias=torch.zeros(5)),
                lambda: f(x, W, bias=torch.zeros(6).bfloat16()), lambda: f(torch.zeros(8, 4).t(), W),
                lambda: f(torch.zeros(1, 8).expand(4, 8), W), lambda: f(x, W, residual=torch.zeros(4, 5)),
                lambda: f(x, W, residual=torch.zeros(4, 6).bfloat16()), lambda: f(x, W, out=torch.zeros(3, 6)),
                lambda: f(x, W, out=torch.zeros(4, 6), out_dtype=torch.bfloat16), lambda: f(x, W, out_dtype=torch.half),
                lambda: b(x, W, dy), lambda: b(x, W, torch.zeros(4, 5)), lambda: b(x, W, dy.double()),
                lambda: b(x, W, dy, grad_x=torch.zeros(4, 9)), lambda: b(x, W, dy, grad_W=torch.zeros(6, 8).bfloat16())):
        with pytest.raises(ValueError):
            bad()


def test_limits_and_aliases(lib):
    """More rows than E2F_MAX_ROWS (tile counts are formed as rows + tile - 1 in
    32 bits), outputs that are an input or another output."""
    top = (1 << 31) - 4096
    d, o = D64, ctypes.c_void_p(4096)
    ef = lambda N=4, V=9, out=o: lib.e2f_embed_forward(d, 2, N, ctypes.c_void_p(128), 0, V, 8, 1.0, 1, out, 0, None)
    eb = lambda N=4, V=9, out=o: lib.e2f_embed_backward(d, 2, N, ctypes.c_void_p(128), 0, V, 8, 1.0, 1, out, 0, None)
    for call in (ef, eb):
        assert call(N=top + 1) == 1 and call(V=top + 1) == 1
        assert call(out=d) == 1 and call(out=ctypes.c_void_p(128)) == 1
    assert lib.e2f_linear_forward(_lin(M=top + 1), None, 6, o, 6, 0, None) == 1
    assert lib.e2f_linear_forward(_lin(bias=4096), None, 6, o, 6, 0, None) == 1
    b = lambda p, gx, gw, gb: lib.e2f_linear_backward(p, ctypes.c_void_p(512), 6, 0, gx, 8, gw, 8, gb, None)
    assert b(_lin(M=top + 1), o, None, None) == 1
    assert b(_lin(), o, o, None) == 1 and b(_lin(), o, None, o) == 1 and b(_lin(), None, o, o) == 1


def test_stream_is_a_keyword():
    """The calls make `stream` current while they allocate: it must reach them by name."""
    ids, table, x, W = torch.zeros(4, dtype=torch.int64), torch.zeros(5, 6), torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(TypeError):
        e2f.embed_forward(ids, table, 1.0, 1, None, None, None)
    with pytest.raises(TypeError):
        e2f.linear_forward(x, W, None, None, "none", None, None, None)
