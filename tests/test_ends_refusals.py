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
