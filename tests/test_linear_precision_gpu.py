"""What the linear layers' kernels do for their precision, each at a size where its
loss would show: three terms of an fp32 operand, chains of MMAs that end, two terms
of dz in the bf16 backward.

Three terms: an fp32 value times one, plus zeros, is itself.
Chains: the tensor core's accumulation truncates, by measurement about 1e-8 of the
sum per MMA of 16 products, all in one direction where the products have one sign.
A chain ends after 1,024 products (64 MMAs: 6.4e-7; twice that is allowed), and the
K / 1,024 pieces are added with a rounding each (2^-24).  One chain over 16,384
products would be off by 1e-5, five times the bound."""
import pytest

from .test_linear_gpu import E24, EB, SHAPES, _acc, _act, _check_backward, _check_forward, _fwd_ref, _make

pytestmark = pytest.mark.gpu

K = 16384
CHAIN = 2 * 64 * 1e-8 + K / 1024 * 2.0 ** -24


def _full_mantissas(r, c, g):
    """Values whose 24 bits all matter, over some 40 powers of two."""
    import torch
    m = torch.randint(1 << 23, 1 << 24, (r, c), generator=g, device="cuda").float() + 0.0
    m = m * torch.exp2(torch.randint(-43, -3, (r, c), generator=g, device="cuda").float())
    return m * (torch.randint(0, 2, (r, c), generator=g, device="cuda") * 2 - 1)


# short and split contractions, a chain of several pieces; rows that are and are not
# whole 16-byte pieces
@pytest.mark.parametrize("M,K,pad", [(600, 600, 0), (300, 1200, 0), (1600, 1160, 0), (1601, 1163, 0), (600, 515, 3)])
def test_fp32_operands_keep_every_bit(cuda_ok, M, K, pad):
    """Through permutations, from either operand of all three products."""
    import torch
    from atomistic_mlip_b200 import e2f
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    wide = lambda t: torch.nn.functional.pad(t, (0, pad))[:, :t.shape[1]]
    x, perm = _full_mantissas(M, K, g), torch.randperm(K, generator=g, device="cuda")
    P = torch.eye(K, device="cuda")[perm]                       # P x = x[perm], x P^T = x[:, perm]
    xw, Pw = wide(x), wide(P)
    assert torch.equal(e2f.linear_forward(xw, Pw), x[:, perm])
    assert torch.equal(e2f.linear_forward(Pw, xw), x[:, perm].t())
    dy = _full_mantissas(M, K, g)
    gx, _, _ = e2f.linear_backward(torch.zeros(M, K, device="cuda"), Pw, dy, need_W=False)   # dy P
    assert torch.equal(gx, dy[:, torch.argsort(perm)])
    W = _full_mantissas(K, M, g)
    gx, _, _ = e2f.linear_backward(torch.zeros(K, M, device="cuda"), wide(W), P, need_W=False)   # P W
    assert torch.equal(gx, W[perm])
    _, gw, _ = e2f.linear_backward(wide(W), torch.zeros(K, M, device="cuda"), P, need_x=False)   # P^T W
    assert torch.equal(gw, W[torch.argsort(perm)])
    D = _full_mantissas(K, M, g)
    _, gw, _ = e2f.linear_backward(Pw, torch.zeros(M, K, device="cuda"), D, need_x=False)        # D^T P
    assert torch.equal(gw, D.t()[:, torch.argsort(perm)])
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_long_sums_of_one_sign(cuda_ok, dt):
    """144 tiles: contractions that are not split, so that only the ends of the chains
    keep the error down."""
    import torch
    from atomistic_mlip_b200 import e2f
    M = 1536
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    dt = getattr(torch, dt)
    x = (torch.rand(M, K, generator=g, device="cuda") * 0.5 + 0.5).to(dt)
    W = (torch.rand(M, K, generator=g, device="cuda") * 0.5 + 0.5).to(dt)
    want = x.double() @ W.double().t()
    out = e2f.linear_forward(x, W, out_dtype=torch.float32)
    assert float(((out.double() - want) / want).abs().max()) <= CHAIN
    r = torch.rand(M, M, generator=g, device="cuda")
    out = e2f.linear_forward(x, W, bias=r[0].contiguous(), residual=r, out_dtype=torch.float32)
    full = want + r[0].double() + r.double()
    assert float(((out.double() - full) / full).abs().max()) <= CHAIN + 2.0 ** -23
    if dt == torch.float32:
        a, b = x.t().contiguous(), W.t().contiguous()          # [K, M]
        _, gw, _ = e2f.linear_backward(b, torch.zeros(M, M, device="cuda"), a, need_x=False)   # a^T b
        assert float(((gw.double() - want) / want).abs().max()) <= CHAIN
        gx, _, _ = e2f.linear_backward(torch.zeros(M, M, device="cuda"), b, x, need_W=False)   # x b
        assert float(((gx.double() - want) / want).abs().max()) <= CHAIN
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("M,C,N", [(10513, 1427, 9), (9473, 1025, 40), (18945, 1088, 3), (6000, 2051, 130), (200, 4099, 300)])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_split_contractions_of_tall_products(cuda_ok, M, C, N, dt):
    """Tiles that leave a wave of SMs uneven, so that contractions through registers
    are split into several parts (rows off 16-byte boundaries for bf16), forward, in
    place on the residual, and backward."""
    import torch
    from atomistic_mlip_b200 import e2f
    x, W, b, g = _make(M, C + 1, N, 1, getattr(torch, dt), M + N)
    x, W = x[:, 1:], W[:, 1:]
    r = torch.randn(M, N, generator=g, device="cuda")
    _check_forward(e2f.linear_forward(x, W, bias=b, act="silu", out_dtype=torch.float32), x, W, b, None, "silu")
    out = r.clone()
    e2f.linear_forward(x, W, bias=b, residual=out, out=out, act="gelu")
    _check_forward(out, x, W, b, r, "gelu")
    _check_backward(*e2f.linear_backward(x, W, r, bias=b, act="silu"), x, W, b, r, "silu")
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("M,K,N,Q", [s for s in SHAPES if s[0]] + [(3000, 128, 514, 1), (900, 77, 130, 1), (10304, 128, 512, 1),
                                                                   (3001, 8, 100, 1), (2, 300, 70, 1), (4099, 1000, 2050, 1)])
@pytest.mark.parametrize("gt,act", [("bfloat16", "silu"), ("float32", "gelu"), ("float32", "none"), ("bfloat16", "none")])
def test_bf16_gradients_are_rounded_once(cuda_ok, M, K, N, Q, gt, act):
    """dz enters the products of bf16 layers in two bf16 terms: each bf16 result is off
    by its own rounding, 2^-16 of dz (2^-8 of what the first term leaves, which is at
    most 2^-8 where it is rounded; 2^-16 where it is cut) and what the fp32 sums of
    twice as many products lose.  One term would add 2^-8 of dz."""
    import torch
    from atomistic_mlip_b200 import e2f
    x, W, b, g = _make(M, K, N, Q, torch.bfloat16, 7 * M + K + N)
    dy = torch.randn(M, N, generator=g, device="cuda").to(getattr(torch, gt))
    gx, gw, _ = e2f.linear_backward(x, W, dy, bias=b, act=act)
    assert e2f.stream_status() == 0
    z, S = _fwd_ref(x, W, b, act)
    _, d = _act(z, act)
    dz = dy.double() * d
    edz = dy.double().abs() * (0.8 * _acc(K) * S + 16 * E24 * (1 + z.abs())) if act != "none" else dz.abs() * 0
    edz = edz + 1.01 * 2.0 ** -16 * (dz.abs() + edz)
    mag = dz.abs() + edz
    for got, a, e, m, o in ((gx, dz, edz, mag, W.double()), (gw, dz.t(), edz.t(), mag.t(), x.double())):
        r = a @ o
        t = e @ o.abs() + _acc(2 * a.shape[1]) * (m @ o.abs())
        assert bool(((got.double() - r).abs() <= t + (EB + E24) * 1.01 * (r.abs() + t)).all())


@pytest.mark.parametrize("M,K,N", [(300, 72, 96), (900, 77, 130), (3000, 128, 512), (2000, 600, 520)])
def test_bf16_gradients_beside_infinities(cuda_ok, M, K, N):
    """An infinity of dL/dout, W or x meets both terms of dz as it meets dz."""
    import torch
    from atomistic_mlip_b200 import e2f
    inf, nan = float("inf"), float("nan")
    x, W, _, g = _make(M, K, N, 1, torch.bfloat16, M)
    x = x.contiguous()
    dy = torch.randn(M, N, generator=g, device="cuda")
    dy[::2] = dy[::2].bfloat16().float()             # nothing left for the second term
    dy[0] = 0.0
    x[2, 3], x[3, 5], W[4, 6], W[7, 8] = inf, -inf, -inf, nan
    for planted in (False, True):
        if planted:
            dy[5, 2], dy[6, 9], dy[11, 11] = inf, -inf, torch.finfo(torch.float32).max
        gx, gw, _ = e2f.linear_backward(x, W, dy)
        d8, x8, W8 = dy.double(), x.double(), W.double()
        if planted:                                  # (bf16 results: FLT_MAX itself is one step above their largest)
            d8 = d8.clone()
            d8[11, 11] = float(torch.finfo(torch.bfloat16).max)
        for got, ref in ((gx, d8 @ W8), (gw, d8.t() @ x8)):
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            for s in (inf, -inf):
                near = (ref == s) | (ref * (1 if s > 0 else -1) > 3e38)
                assert bool((got == s)[ref == s].all()) and not bool(((got == s) & ~near).any())
    assert e2f.stream_status() == 0
