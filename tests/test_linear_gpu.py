"""Linear layers (bias, activation, residual) and their gradient against the
definition in 64 bits.

Tolerances count roundings.  A contraction of K products in fp32 on the tensor
cores: each product, and each partial sum of 16, loses at most one unit in the
last place (2^-23, truncation) of the sum of magnitudes S; fp32 operands in
three bf16 terms leave out less than 4 * 2^-24 of each product:
    acc(K) = (K + ceil(K / 16) + 8) 2^-23 S.
Activations: |act'| <= 1.13, |act''| <= 0.8, their fp32 evaluation is good to
16 * 2^-24 (1 + |z|).  bf16 values are rounded to 2^-8, fp32 ones to 2^-24.
Integers whose sums stay below 2^24 must come out exactly."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E23, E24, EB = 2.0 ** -23, 2.0 ** -24, 2.0 ** -8


def _acc(K):
    return (K + math.ceil(K / 16) + 8) * E23


def _act(z, act):
    import torch
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def _make(M, K, N, Q, dt, seed, integers=False):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if integers:   # |x w| <= 7 * 1023, sums of up to 2000 below 2^24; exact in bf16 up to 8 bits
        top = 1024 if dt == torch.float32 else 129
        x = torch.randint(-top + 1, top, (M, Q, K), generator=g, device="cuda").to(dt)
        W = torch.randint(-7, 8, (N, K), generator=g, device="cuda").to(dt)
        b = torch.randint(-9, 10, (N,), generator=g, device="cuda").float()
    else:
        x = torch.randn(M, Q, K, generator=g, device="cuda").to(dt)
        W = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).to(dt)
        b = torch.randn(N, generator=g, device="cuda") * 0.3
    return x[:, 0, :], W, b, g


SHAPES = [  # M, K, N, Q
    (0, 5, 7, 1), (1, 1, 1, 1), (1, 1024, 512, 1), (2, 77, 300, 1), (3, 5, 7, 4), (128, 64, 128, 1), (129, 65, 130, 1),
    (127, 63, 17, 1), (1000, 1, 33, 9), (17, 300, 1, 1), (300, 129, 8, 1), (64, 2000, 64, 1), (5, 1999, 260, 1),
    (3000, 128, 64, 25), (2051, 104, 205, 1), (700, 136, 520, 1), (257, 264, 1000, 9), (4099, 8, 24, 1),
    (33, 640, 1280, 1), (1, 4096, 9, 1), (40000, 24, 16, 1), (19000, 128, 512, 1), (16, 513, 129, 1),
    (2500, 2056, 1288, 1), (20001, 64, 264, 1), (5000, 1160, 640, 1), (128, 8, 8, 1),
    (1, 5000, 130, 1), (2, 4104, 70, 1), (50003, 64, 2, 1), (50003, 7, 1, 9), (9000, 4200, 2, 1), (3, 1000, 999, 1), (8, 2048, 600, 1),
    (2000, 72, 4, 1), (513, 40, 40, 1), (40, 513, 40, 1), (512, 30, 512, 25),
]
TYPES = [("float32", "float32"), ("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "bfloat16")]


def _fwd_ref(x, W, b, act):
    z = x.double() @ W.double().t()
    S = x.double().abs() @ W.double().abs().t()
    if b is not None:
        z, S = z + b.double(), S + b.double().abs()
    return z, S


def _check_forward(out, x, W, b, r, act):
    import torch
    K = x.shape[1]
    z, S = _fwd_ref(x, W, b, act)
    y, _ = _act(z, act)
    tol = 1.13 * _acc(K) * S + 16 * E24 * (1 + z.abs()) * (act != "none")
    if r is not None:
        y = y + r.double()
    tol = tol + (E24 + (EB if out.dtype == torch.bfloat16 else 0)) * 1.01 * (y.abs() + tol)
    assert out.shape == y.shape
    assert bool(((out.double() - y).abs() <= tol).all())


def _check_backward(gx, gw, gb, x, W, b, dy, act):
    import torch
    (M, K), N = x.shape, W.shape[0]
    z, S = _fwd_ref(x, W, b, act)
    _, d = _act(z, act)
    dz = dy.double() * d
    edz = dy.double().abs() * (0.8 * _acc(K) * S + 16 * E24 * (1 + z.abs())) if act != "none" else dz.abs() * 0
    tb = edz.sum(0) + (M + 2) * E24 * dz.abs().sum(0)     # the bias sums fp32 values
    round_out = E24
    if x.dtype == torch.bfloat16:
        edz = edz + EB * (dz.abs() + edz)                  # dz as a bf16 operand
        round_out = EB + E24
    x8, W8 = x.double(), W.double()
    rx, rw = dz @ W8, dz.t() @ x8
    mag = dz.abs() + edz
    tx = edz @ W8.abs() + _acc(N) * (mag @ W8.abs())
    tw = edz.t() @ x8.abs() + _acc(M) * (mag.t() @ x8.abs())
    assert gx.dtype == x.dtype and gw.dtype == x.dtype and gb.dtype == torch.float32
    assert bool(((gx.double() - rx).abs() <= tx + round_out * 1.01 * (rx.abs() + tx)).all())
    assert bool(((gw.double() - rw).abs() <= tw + round_out * 1.01 * (rw.abs() + tw)).all())
    assert bool(((gb.double() - dz.sum(0)).abs() <= tb).all())


@pytest.mark.parametrize("M,K,N,Q", SHAPES)
@pytest.mark.parametrize("dt,ot", TYPES)
def test_forward(cuda_ok, M, K, N, Q, dt, ot):
    import torch
    from atomistic_mlip_b200 import e2f
    dt, ot = getattr(torch, dt), getattr(torch, ot)
    x, W, b, g = _make(M, K, N, Q, dt, M + 3 * K + N)
    for act, bias, resid in (("silu", b, False), ("gelu", None, True), ("none", b, True)):
        r = torch.randn(M, N, generator=g, device="cuda").to(ot) if resid else None
        out = e2f.linear_forward(x, W, bias=bias, residual=r, act=act, out_dtype=ot)
        assert e2f.stream_status() == 0 and out.dtype == ot
        _check_forward(out, x, W, bias, r, act)


@pytest.mark.parametrize("M,K,N,Q", SHAPES)
@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
def test_backward(cuda_ok, M, K, N, Q, dt, gt, act):
    import torch
    from atomistic_mlip_b200 import e2f
    dt, gt = getattr(torch, dt), getattr(torch, gt)
    x, W, b, g = _make(M, K, N, Q, dt, 5 * M + 3 * K + N)
    dy = torch.randn(M, N, generator=g, device="cuda").to(gt)
    grads = e2f.linear_backward(x, W, dy, bias=b, act=act)
    assert e2f.stream_status() == 0
    _check_backward(*grads, x, W, b, dy, act)
    again = e2f.linear_backward(x, W, dy, bias=b, act=act)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))   # bit for bit


@pytest.mark.parametrize("M,K,N,Q", [(129, 65, 130, 1), (300, 200, 257, 9), (1, 640, 333, 1), (700, 1999, 40, 1),
                                     (260, 256, 512, 1), (1999, 72, 100, 1), (515, 130, 2, 1), (6, 100, 300, 1)])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_integers_are_exact(cuda_ok, M, K, N, Q, dt):
    """Every sum is an integer below 2^24 in magnitude: no rounding anywhere."""
    import torch
    from atomistic_mlip_b200 import e2f
    dt = getattr(torch, dt)
    x, W, b, g = _make(M, K, N, Q, dt, M + K + N, integers=True)
    r = torch.randint(-50, 51, (M, N), generator=g, device="cuda").float()
    out = e2f.linear_forward(x, W, bias=b, residual=r, out_dtype=torch.float32)
    want = x.double() @ W.double().t() + b.double() + r.double()
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(out.double(), want)
    dy = torch.randint(-5, 6, (M, N), generator=g, device="cuda").to(dt)
    gx, gw, gb = e2f.linear_backward(x, W, dy, bias=b)
    wx, ww = dy.double() @ W.double(), dy.double().t() @ x.double()
    assert float(ww.abs().max()) < 2 ** 24
    if dt == torch.bfloat16:   # one rounding of an exact integer
        assert torch.equal(gx, wx.float().to(dt)) and torch.equal(gw, ww.float().to(dt))
    else:
        assert torch.equal(gx.double(), wx) and torch.equal(gw.double(), ww)
    assert torch.equal(gb.double(), dy.double().sum(0))


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_strides_alignment_and_neighbours(cuda_ok, dt):
    """Operands and results inside larger buffers at odd offsets and strides;
    what lies between the rows and around them stays as it was.  (Layouts take
    different kernels, whose sums have different orders: each result is held to
    the 64-bit definition.)"""
    import torch
    from atomistic_mlip_b200 import e2f
    dt = getattr(torch, dt)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def rows(r, c, ld, off, fill=None):
        buf = torch.randn(off + (r + 1) * ld, generator=g, device="cuda").to(dt)
        if fill is not None:
            buf.fill_(fill)
        return buf, torch.as_strided(buf, (r, c), (ld, 1), off)

    for M, K, N in ((150, 70, 90), (1, 40, 33), (5, 264, 136), (300, 128, 128)):
        for pad, off in ((0, 0), (1, 1), (8, 0), (5, 3), (16, 8)):
            _, x = rows(M, K, K + pad, off)
            _, W = rows(N, K, K + pad, off)
            _, r = rows(M, N, N + pad, off)
            ob, out = rows(M, N, N + pad + 1, off, 7.0)
            e2f.linear_forward(x, W, residual=r, act="silu", out=out)
            _check_forward(out, x, W, None, r, "silu")
            out.fill_(7.0)
            assert bool((ob == 7).all())
            # in place on the residual
            r2 = r.clone(memory_format=torch.contiguous_format)
            e2f.linear_forward(x, W, residual=r2, act="silu", out=r2)
            _check_forward(r2, x, W, None, r, "silu")
            _, dy = rows(M, N, N + pad, off)
            xb, gx = rows(M, K, K + pad + 3, off, 7.0)
            wb, gw = rows(N, K, K + pad + 3, off, 7.0)
            got = e2f.linear_backward(x, W, dy, act="gelu", need_bias=True, grad_x=gx, grad_W=gw)
            _check_backward(*got, x, W, None, dy, "gelu")
            gx.fill_(7.0), gw.fill_(7.0)
            assert bool((xb == 7).all()) and bool((wb == 7).all())
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_parts_of_the_gradient(cuda_ok, dt):
    """Any subset of the gradients equals the same ones computed together."""
    import torch
    from atomistic_mlip_b200 import e2f
    x, W, b, g = _make(300, 72, 96, 1, getattr(torch, dt), 4)
    for act in ("silu", "none"):
        dy = torch.randn(300, 96, generator=g, device="cuda")
        full = e2f.linear_backward(x, W, dy, bias=b, act=act)
        for nx, nw, nb in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 0, 0)):
            part = e2f.linear_backward(x, W, dy, bias=b, act=act, need_x=bool(nx), need_W=bool(nw), need_bias=bool(nb))
            for p, q, n in zip(part, full, (nx, nw, nb)):
                assert torch.equal(p, q) if n else p is None


def test_gradient_against_differences(cuda_ok):
    """Directional derivatives of the 64-bit forward by central differences
    (step 1e-4: truncation below 1e-7 of the derivative's scale)."""
    import torch
    from atomistic_mlip_b200 import e2f
    for act in ("silu", "gelu"):
        x, W, b, g = _make(60, 45, 37, 1, torch.float32, 11)
        dy = torch.randn(60, 37, generator=g, device="cuda")
        grads = e2f.linear_backward(x, W, dy, bias=b, act=act)
        pt = [x.double(), W.double(), b.double()]

        def L(q):
            return float((_act(q[0] @ q[1].t() + q[2], act)[0] * dy.double()).sum())

        for i in range(3):
            d = torch.randn(pt[i].shape, generator=g, device="cuda").double()
            h = 1e-4
            num = (L([p + h * d if j == i else p for j, p in enumerate(pt)]) -
                   L([p - h * d if j == i else p for j, p in enumerate(pt)])) / (2 * h)
            ana = float((grads[i].double() * d).sum())
            scale = float((grads[i].double() * d).abs().sum())
            assert abs(num - ana) <= (1e-6 + _acc(60)) * scale


def test_infinities_and_nan(cuda_ok):
    """An infinity or NaN reaches the outputs that an fp32 multiply-add gives
    it, and no others."""
    import torch
    from atomistic_mlip_b200 import e2f
    for dt in (torch.float32, torch.bfloat16):
        for M, K, N in ((200, 100, 150), (3, 100, 150), (40, 2000, 30)):
            x, W, b, _ = _make(M, K, N, 1, dt, 21)
            x = x.clone()
            W = W.abs() + 0.5
            x[1, 3], x[2, 7] = float("inf"), float("nan")
            out = e2f.linear_forward(x, W, bias=b)
            ref = x.double() @ W.double().t() + b.double()
            assert torch.equal(torch.isnan(out), torch.isnan(ref)) and torch.equal(torch.isinf(out), torch.isinf(ref))
            assert bool((out[1] == float("inf")).all())
            # the largest finite values, and subnormals, pass through a unit matrix
            eye = torch.eye(K, device="cuda").to(dt)
            big = torch.full((M, K), torch.finfo(dt).max, device="cuda", dtype=dt)
            assert torch.equal(e2f.linear_forward(big, eye), big)


def test_offsets_beyond_32_bits(cuda_ok):
    """Rows of x and of the output that start behind 2^32 bytes, and behind
    2^31 elements."""
    import torch
    from atomistic_mlip_b200 import e2f
    M, K, N, ld = 70_000, 24, 40, 32_768
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    buf = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (M, K), (ld, 1), 0)
    x.copy_(torch.randn(M, K, generator=g, device="cuda"))
    W = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    obuf = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(obuf, (M, N), (ld, 1), 0)
    e2f.linear_forward(x, W, out=out)
    _check_forward(out, x, W, None, None, "none")
    gx = torch.as_strided(obuf, (M, K), (ld, 1), 64)
    got = e2f.linear_backward(x, W, out, act="silu", grad_x=gx, need_bias=True)
    _check_backward(*got, x, W, None, out, "silu")


def test_streams_and_graphs(cuda_ok):
    """On two side streams at once; captured twice and replayed, interleaved,
    with other inputs in the same buffers."""
    import torch
    from atomistic_mlip_b200 import e2f
    for dt in (torch.float32, torch.bfloat16):
        x, W, b, g = _make(500, 600, 72, 1, dt, 31)
        dy = torch.randn(500, 72, generator=g, device="cuda")

        def both():
            return (e2f.linear_forward(x, W, bias=b, act="silu"), *e2f.linear_backward(x, W, dy, bias=b, act="silu"))

        want = both()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for s in streams:
            with torch.cuda.stream(s):
                got.append(both())
        torch.cuda.synchronize()
        for o in got:
            assert all(torch.equal(p, q) for p, q in zip(o, want))
        graphs = []
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                o = both()
            graphs.append((gr, o))
        for seed in range(3):
            x.copy_(torch.randn(500, 600, generator=g, device="cuda"))
            dy.copy_(torch.randn(500, 72, generator=g, device="cuda"))
            for gr, _ in graphs:
                gr.replay()
            want = both()
            for _, o in graphs:
                assert all(torch.equal(p, q) for p, q in zip(o, want))
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("dt,ot", TYPES)
def test_extreme_preactivations(cuda_ok, dt, ot):
    """Pre-activations from -3e4 to 3e4 and +-infinity side by side (pairs share
    a reciprocal): every output as in 64 bits, NaN exactly where silu(-inf) and
    the products of infinities with zero give it."""
    import torch
    from atomistic_mlip_b200 import e2f
    dt, ot = getattr(torch, dt), getattr(torch, ot)
    N = 264
    for M in (3, 200):
        vals = torch.tensor([0.0, 1.0, -1.0, 20.0, -20.0, 60.0, -60.0, 90.0, -90.0, 700.0, -700.0, 3e4, -3e4, 1e-30, -1e-30, 0.5])
        x = vals.repeat(M, 1).to("cuda", dt)
        sel = torch.arange(N) % 16
        W = torch.zeros(N, 16)
        W[torch.arange(N), sel] = 1.0
        W = W.to("cuda", dt)
        dy = torch.ones(M, N, device="cuda", dtype=ot)
        for act in ("silu", "gelu"):
            out = e2f.linear_forward(x, W, act=act, out_dtype=ot)
            _check_forward(out, x, W, None, None, act)
            _check_backward(*e2f.linear_backward(x, W, dy, act=act, need_bias=True), x, W, None, dy, act)
            b = torch.zeros(N, device="cuda")
            b[5], b[6], b[8] = float("inf"), float("-inf"), float("nan")
            out = e2f.linear_forward(x, W, bias=b, act=act, out_dtype=ot)
            keep = torch.ones(N, dtype=torch.bool, device="cuda")
            keep[torch.tensor([5, 6, 8])] = False
            _check_forward(out[:, keep], x, W[keep], None, None, act)
            assert bool((out[:, 5] == float("inf")).all()) and bool(torch.isnan(out[:, 6]).all())
            assert bool(torch.isnan(out[:, 8]).all())


@pytest.mark.parametrize("M,K,N", [(20000, 1, 37), (20011, 2, 96), (4000, 4, 513), (3001, 5, 2000), (2500, 8, 300),
                                   (33000, 13, 132), (700, 16, 1030), (129, 16, 20000)])
@pytest.mark.parametrize("dt,ot", TYPES)
def test_few_inputs(cuda_ok, M, K, N, dt, ot):
    """Up to 16 inputs and many results: rows that are and are not whole 16-byte
    pieces, more blocks of rows than CTAs, and the same inside wider buffers."""
    import torch
    from atomistic_mlip_b200 import e2f
    dt, ot = getattr(torch, dt), getattr(torch, ot)
    x, W, b, g = _make(M, K, N, 1, dt, M + 3 * K + N)
    r = torch.randn(M, N, generator=g, device="cuda").to(ot)
    for pad in (0, 3):
        if pad:
            wide = lambda t: torch.nn.functional.pad(t, (pad, 2))[:, pad:-2]
            x, W, r = wide(x), wide(W), wide(r)
        for act, resid in (("silu", None), ("gelu", r)):
            out = torch.full((M + 1, N + pad), 7.0, device="cuda", dtype=ot)
            e2f.linear_forward(x, W, bias=b, residual=resid, act=act, out=out[:M, :N])
            _check_forward(out[:M, :N], x, W, b, resid, act)
            assert bool((out[M] == 7).all()) and bool((out[:, N:] == 7).all())
        grads = e2f.linear_backward(x, W, r, bias=b, act="silu")
        _check_backward(*grads, x, W, b, r, "silu")
    assert e2f.stream_status() == 0
