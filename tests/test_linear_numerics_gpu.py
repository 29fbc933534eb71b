"""Linear layers where their kernels' number formats end: infinities and NaN, the
largest and the smallest fp32 values; and which bits may depend on what."""
import math

import pytest

from .test_linear_gpu import TYPES, _acc, _make

pytestmark = pytest.mark.gpu

# fp32 products of tiles on the tensor cores, in all three operand orders: short
# contractions, split ones, and chains of more than 1,024
TILED = [(600, 300, 520), (40, 2000, 150), (1600, 1200, 1100)]


def _same(got, ref, tol):
    """NaN, +inf and -inf where ref has them; elsewhere within tol."""
    import torch
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got == float("inf"), ref == float("inf"))
    assert torch.equal(got == float("-inf"), ref == float("-inf"))
    assert bool(((got.double() - ref).abs() <= tol)[fine].all())


def _plant(t, rows):
    inf, nan = float("inf"), float("nan")
    t[rows[0], 3] = inf
    t[rows[1], 7] = nan
    t[rows[2], 0], t[rows[2], t.shape[1] - 1] = -inf, inf
    t[rows[3], 11] = -inf


@pytest.mark.parametrize("M,K,N", TILED)
def test_infinities_and_nan_of_both_operands(cuda_ok, M, K, N):
    """They reach the outputs that an fp32 multiply-add gives them, and no others."""
    import torch
    from atomistic_mlip_b200 import e2f
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda")
    W = torch.randn(N, K, generator=g, device="cuda")
    dy = torch.randn(M, N, generator=g, device="cuda")
    r = torch.randn(M, N, generator=g, device="cuda")
    W[5, 3] = dy[1, 4] = 0.0                 # inf * 0
    _plant(x, (1, 2, 17, M - 1))
    _plant(W, (N - 1, 20, 33, 64))
    x8, W8, dy8 = x.double(), W.double(), dy.double()
    _same(e2f.linear_forward(x, W), x8 @ W8.t(), 1.01 * _acc(K) * (x8.abs() @ W8.abs().t()))
    S = x8.abs() @ W8.abs().t() + r.double().abs()
    _same(e2f.linear_forward(x, W, residual=r), x8 @ W8.t() + r.double(), 1.01 * _acc(K) * S)
    _plant(dy, (0, 19, 30, M - 2))
    dy8 = dy.double()
    gx, gw, gb = e2f.linear_backward(x, W, dy, need_bias=True)
    _same(gx, dy8 @ W8, 1.01 * _acc(N) * (dy8.abs() @ W8.abs()))
    _same(gw, dy8.t() @ x8, 1.01 * _acc(M) * (dy8.abs().t() @ x8.abs()))
    _same(gb, dy8.sum(0), 1.01 * _acc(M) * dy8.abs().sum(0))
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("M,K", [(600, 600), (1600, 1200)])
def test_values_beyond_the_bf16_range(cuda_ok, M, K):
    """fp32 values that round to a bf16 infinity pass through a unit matrix as they
    are, from either operand; products beyond the fp32 range are infinities."""
    import torch
    from atomistic_mlip_b200 import e2f
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    top = 0x7f7fffff                          # the largest finite value's bits
    bits = torch.randint(0x7f7f0000, top + 1, (M, K), generator=g, device="cuda", dtype=torch.int32)
    x = bits.view(torch.float32) * (torch.randint(0, 2, (M, K), generator=g, device="cuda") * 2 - 1)
    x[0] = torch.finfo(torch.float32).max
    x[1] = -x[0]
    eye = torch.eye(K, device="cuda")
    assert torch.equal(e2f.linear_forward(x, eye), x)
    assert torch.equal(e2f.linear_forward(eye, x), x.t())
    gx, gw, _ = e2f.linear_backward(eye, x, torch.eye(K, M, device="cuda"))       # dy W, dy^T x
    assert torch.equal(gx, torch.nn.functional.pad(x, (0, 0, 0, max(0, K - M)))[:K])
    assert torch.equal(gw, torch.eye(M, K, device="cuda"))
    big = torch.full((M, K), 1e30, device="cuda")
    out = e2f.linear_forward(big, torch.full((K, K), 1.1e20, device="cuda"))
    assert bool((out == float("inf")).all())
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("M,K", [(600, 512), (1600, 1200)])
def test_fp32_operands_of_small_magnitude(cuda_ok, M, K):
    """Operands are held to 2^-133: from 2^-109 on that is half of their last bit, and
    below it the error stays there, whatever the other operand.  By arithmetic: half
    of the operand is rounded to fp32 (whose least step is 2^-149: off by 2^-150, so
    by 2^-149 of the operand), its terms to bf16 (least step 2^-133: off by 2^-134, so
    by 2^-133); results are rounded to fp32 (2^-24, or 2^-150 where they are below its
    normal range, times four after the halving)."""
    import torch
    from atomistic_mlip_b200 import e2f
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    for w in (1.0, 2.0 ** 60, 2.0 ** 100):
        eye = torch.eye(K, device="cuda") * w
        for e in (-90, -108, -112, -120, -126, -130, -140, -149):
            x = (torch.rand(M, K, generator=g, device="cuda", dtype=torch.float64) + 1).mul(2.0 ** e).float()
            want = x.double() * w
            tol = (2.0 ** -133 + 2.0 ** -149) * w + 2.0 ** -24 * want.abs() + 2.0 ** -148
            assert bool(((e2f.linear_forward(x, eye).double() - want).abs() <= tol).all())
            assert bool(((e2f.linear_forward(eye, x).double() - want.t()).abs() <= tol.t()).all())
            if e >= -108:
                assert torch.equal(e2f.linear_forward(x, eye).double(), want.float().double())
    assert e2f.stream_status() == 0


def test_nan_costs_nothing(cuda_ok):
    """A diverged step takes no longer than another one (medians of device times; the
    factor of three leaves room for a clock that changes between them)."""
    import torch
    from atomistic_mlip_b200 import e2f
    x, W = torch.randn(1024, 1024, device="cuda"), torch.randn(512, 1024, device="cuda")
    one, dy = x.clone(), torch.randn(1024, 512, device="cuda")
    one[3, 5] = float("nan")
    nan = torch.full_like(x, float("nan"))

    def us(x, dy):
        t = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            out = e2f.linear_forward(x, W)
            gw = e2f.linear_backward(x, W, dy, need_x=False)[1]
            b.record()
            b.synchronize()
            t.append(a.elapsed_time(b) * 1e3)
        return sorted(t)[4], out, gw

    usual, _, _ = us(x, dy)
    t, out, gw = us(one, dy)
    assert bool(torch.isnan(out[3]).all()) and int(torch.isnan(out).sum()) == 512
    assert bool(torch.isnan(gw[:, 5]).all()) and int(torch.isnan(gw).sum()) == 512
    assert t <= 3 * usual
    t, out, gw = us(nan, dy)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(gw).all()) and t <= 3 * usual
    assert e2f.stream_status() == 0


@pytest.mark.parametrize("M,K,N", [(700, 136, 520), (3000, 128, 512), (2500, 2056, 1288), (5000, 1160, 640), (1600, 1200, 1100),
                                   (257, 2056, 130), (3000, 128, 514), (2500, 2056, 1290), (3001, 8, 100), (2, 300, 70), (130, 40, 2), (120, 72, 96), (900, 77, 130)])
@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
def test_any_subset_of_the_gradients_has_the_same_bits(cuda_ok, M, K, N, dt, gt, act):
    import torch
    from atomistic_mlip_b200 import e2f
    dt, gt = getattr(torch, dt), getattr(torch, gt)
    x, W, b, g = _make(M, K, N, 1, dt, M + K + N)
    dy = torch.randn(M, N, generator=g, device="cuda").to(gt)
    full = e2f.linear_backward(x, W, dy, bias=b, act=act)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)):
        part = e2f.linear_backward(x, W, dy, bias=b, act=act, need_x=bool(need[0]), need_W=bool(need[1]),
                                   need_bias=bool(need[2]))
        for p, q, n in zip(part, full, need):
            assert torch.equal(p, q) if n else p is None
    assert e2f.stream_status() == 0


def _through(act, z, K, M, dt, dy=None):
    """act (or its gradient) of the values z [K], repeated in M rows, through a unit matrix."""
    import torch
    from atomistic_mlip_b200 import e2f
    x = z.to(dt).repeat(M, 1)
    eye = torch.eye(K, device="cuda").to(dt)
    if dy is None:
        return e2f.linear_forward(x, eye, act=act, out_dtype=torch.float32)
    ones = torch.full((M, K), dy, device="cuda")
    return e2f.linear_backward(x, eye, ones, act=act, need_x=False, need_W=False, need_bias=True)[2] / M


# M, K, type: streamed rows, few inputs, the CUDA cores, fp32 and unaligned tiles, tiles by TMA
KERNELS = [(2, 512, "float32"), (64, 16, "float32"), (64, 128, "float32"), (1024, 512, "float32"), (2048, 1280, "float32"),
           (1024, 515, "bfloat16"), (1024, 512, "bfloat16"), (256, 1280, "bfloat16"), (2048, 1280, "bfloat16")]


def _phi_by_formula(z):
    """Abramowitz and Stegun 7.1.26 in 64 bits, for z < 0."""
    import torch
    t = 1 / (1 + 0.3275911 * z.abs() / math.sqrt(2))
    q = 0.254829592 + t * (-0.284496736 + t * (1.421413741 + t * (-1.453152027 + t * 1.061405429)))
    return 0.5 * t * q * torch.exp(-0.5 * z * z)


@pytest.mark.parametrize("M,K,dt", KERNELS)
def test_gelu_in_its_lower_tail(cuda_ok, M, K, dt):
    """Relative to the formula that the kernels evaluate: its exponent z^2 / 2 is off by
    3 roundings, exponential and reciprocal by 2^-22 each, the polynomial (whose terms
    are at most 3.3 times their sum) and the products by 3.3 * 16 roundings.  Relative
    to Phi: the formula's own 0.4 %."""
    import torch
    dt = getattr(torch, dt)
    z = torch.linspace(-6.0, -3.0, K, device="cuda").to(dt).double()
    tol = (3 * z * z / 2 + 8 + 53) * 2.0 ** -24 * 1.01
    y = _through("gelu", z, K, M, dt)
    assert torch.equal(y, y[:1].expand_as(y))
    want = z * _phi_by_formula(z)
    assert bool(((y[0].double() - want).abs() <= tol * want.abs()).all())
    exact = 0.5 * z * torch.erfc(-z / math.sqrt(2))
    assert bool(((y[0].double() - exact).abs() <= (4e-3 + tol) * exact.abs()).all())
    # the gradient Phi + z phi: the column sums of dz = 1 act'(z), M equal terms
    g = _through("gelu", z, K, M, dt, 1.0).double()
    pdf = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    want = _phi_by_formula(z) + z * pdf
    mag = _phi_by_formula(z) + z.abs() * pdf
    assert bool(((g - want).abs() <= tol * mag + (M + 2) * 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_pre_activation_gives_the_same_bits_in_every_kernel(cuda_ok, act):
    import torch
    for dt in ("float32", "bfloat16"):
        z = torch.cat([torch.linspace(-14, 14, 497), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 88.0, -88.0, 1e4, -1e4,
                                                                   2.0 ** -20, -2.0 ** -20, 3.0, -3.0, 1.0])]).cuda()
        z = z.to(getattr(torch, dt)).float()
        seen = None
        for M, K, kd in KERNELS:
            if kd != dt and not (dt == "bfloat16" and kd == "float32"):
                continue
            out = torch.cat([_through(act, torch.nn.functional.pad(zz, (0, K - zz.numel())), K, M, getattr(torch, kd))[M - 1, :zz.numel()]
                             for zz in z.split(K)])
            if seen is None:
                seen = out
            assert torch.equal(out, seen), (M, K, kd)
