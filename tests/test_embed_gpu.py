"""The embedding lookup and its gradient against the definition in 64 bits.

Tolerances count roundings.  Lookup: the product scale * table is rounded to
fp32 (2^-24 relative) and, for bfloat16 outputs, once more (2^-8).  Gradient:
a sum of n fp32 terms in any order is off by at most (n - 1) 2^-24 times the
sum of the terms' magnitudes, the product with scale and the addition to an
accumulated table by one rounding more each; (n + 2) 2^-24 (1 + 2^-10) covers
the second order for every n used here (n 2^-24 < 2^-8 for n < 65,536)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _ids(rng, N, V, kind):
    if kind == "one":
        ids = np.full(N, V // 2)
    elif kind == "species":
        ids = np.where(rng.random(N) < 0.66, min(1, V - 1), rng.integers(0, V, N))
    elif kind == "sorted":
        ids = np.sort(rng.integers(0, V, N))
    elif kind == "padded":
        ids = np.where(rng.random(N) < 0.3, -1, rng.integers(0, V, N))
    elif kind == "all_padded":
        ids = np.full(N, -1)
    else:
        ids = rng.integers(0, V, N)
    return ids


FWD = [  # N, V, D, Q, kind
    (0, 5, 8, 9, "uniform"), (1, 1, 1, 1, "one"), (24, 119, 8, 9, "species"), (7, 3, 3, 4, "padded"),
    (300, 1000, 130, 1, "uniform"), (33, 70000, 770, 1, "uniform"), (1025, 119, 128, 25, "padded"),
    (513, 17, 1, 1, "uniform"), (40, 9, 1023, 2, "uniform"), (9, 4, 64, 49, "all_padded"), (300, 6, 12, 1, "uniform"),
    (130, 50, 516, 1, "padded"), (17, 50, 2056, 1, "uniform"), (1001, 3, 65, 1, "padded"),
]


@pytest.mark.parametrize("N,V,D,Q,kind", FWD)
@pytest.mark.parametrize("tt,ot,it", [("float32", "float32", "int32"), ("bfloat16", "float32", "int64"),
                                      ("float32", "bfloat16", "int64"), ("bfloat16", "bfloat16", "int32")])
def test_lookup(cuda_ok, N, V, D, Q, kind, tt, ot, it):
    import torch
    from atomistic_mlip_b200 import e2f
    rng = np.random.default_rng(N * 7 + V + D)
    ids = _ids(rng, N, V, kind)
    scale = 1.7
    table = torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)).to("cuda", getattr(torch, tt))
    idt = torch.from_numpy(ids).to("cuda", getattr(torch, it))
    out = e2f.embed_forward(idt, table, scale=scale, Q=Q, out_dtype=getattr(torch, ot))
    assert e2f.stream_status() == 0
    ref = np.zeros((N, Q, D))
    live = ids >= 0
    ref[live, 0] = np.float64(np.float32(scale)) * table.double().cpu().numpy()[ids[live]]
    tol = 2.0 ** -24 if ot == "float32" else 2.0 ** -8 + 2.0 ** -23
    got = out.double().cpu().numpy()
    assert out.shape == (N, Q, D)
    assert np.all(np.abs(got - ref) <= tol * np.abs(ref))


BWD = [  # N, V, D, Q, kind
    (0, 5, 8, 9, "uniform"), (1, 1, 1, 1, "one"), (1, 300, 4, 1, "uniform"), (24, 119, 8, 9, "species"),
    (31, 2, 3, 4, "uniform"), (255, 255, 130, 1, "uniform"), (256, 256, 32, 1, "sorted"), (257, 257, 128, 1, "one"),
    (1025, 119, 128, 25, "species"), (2049, 65536, 6, 1, "uniform"), (5000, 119, 64, 9, "padded"),
    (4097, 70001, 257, 1, "uniform"), (20001, 7, 1, 1, "sorted"), (20001, 1, 1, 1, "one"), (20001, 2, 16, 1, "species"),
    (9000, 40, 768, 1, "species"), (300, 119, 128, 9, "all_padded"), (60000, 119, 128, 1, "one"),
    (30011, 1000, 24, 1, "padded"), (12000, 3, 1000, 1, "uniform"),
    (4096, 3, 130, 1, "species"), (3000, 119, 128, 25, "species"), (4096, 60000, 40, 1, "uniform"),
    (4097, 5, 12, 1, "padded"), (1024, 119, 128, 25, "species"), (1023, 3, 770, 1, "padded"), (1000, 60000, 12, 1, "uniform"), (200000, 2, 8, 1, "species"), (70000, 66000, 16, 1, "one"),
]


def _ref_grad(ids, g, V, scale):
    s64 = np.float64(np.float32(scale))
    D = g.shape[1]
    ref, mag, cnt = np.zeros((V, D)), np.zeros((V, D)), np.zeros((V, 1))
    live = (ids >= 0) & (ids < V)
    np.add.at(ref, ids[live], g[live])
    np.add.at(mag, ids[live], np.abs(g[live]))
    np.add.at(cnt, ids[live], 1.0)
    return s64 * ref, abs(s64) * mag, cnt


@pytest.mark.parametrize("N,V,D,Q,kind", BWD)
@pytest.mark.parametrize("gt,it", [("float32", "int32"), ("bfloat16", "int64")])
def test_gradient(cuda_ok, N, V, D, Q, kind, gt, it):
    import torch
    from atomistic_mlip_b200 import e2f
    rng = np.random.default_rng(N * 5 + V + D)
    ids = _ids(rng, N, V, kind)
    scale = 0.3
    g = torch.from_numpy(rng.standard_normal((N, Q, D)).astype(np.float32)).to("cuda", getattr(torch, gt))
    idt = torch.from_numpy(ids).to("cuda", getattr(torch, it))
    ref, mag, cnt = _ref_grad(ids, g[:, 0].double().cpu().numpy(), V, scale)
    tol = (cnt + 2) * 2.0 ** -24 * (1 + 2.0 ** -10) * mag
    got = e2f.embed_backward(idt, g, V, scale=scale)
    assert e2f.stream_status() == 0
    assert got.dtype == torch.float32 and got.shape == (V, D)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
    assert torch.equal(got, e2f.embed_backward(idt, g, V, scale=scale))   # bit for bit
    # added to a table that holds something
    old = torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)).cuda()
    acc = old.clone()
    e2f.embed_backward(idt, g, V, scale=scale, grad_table=acc, accumulate=True)
    want = old.double().cpu().numpy() + ref
    assert np.all(np.abs(acc.double().cpu().numpy() - want) <= tol + 2.0 ** -24 * (np.abs(want) + tol))


@pytest.mark.parametrize("off", [1, 2, 3])
def test_unaligned_views(cuda_ok, off):
    """Tables, outputs and gradients that start off a 16-byte boundary."""
    import torch
    from atomistic_mlip_b200 import e2f
    rng = np.random.default_rng(off)
    N, V, D = 700, 50, 64
    idt = torch.from_numpy(rng.integers(0, V, N)).cuda()
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.randn(V * D + off, device="cuda").to(dt)
        table = buf[off:].view(V, D)
        out = torch.full((N * D + off + 5,), 7.0, device="cuda", dtype=dt)
        e2f.embed_forward(idt, table, out=out[off:off + N * D].view(N, 1, D))
        assert torch.equal(out[off:off + N * D].view(N, D), table[idt])
        assert bool((out[:off] == 7).all()) and bool((out[off + N * D:] == 7).all())
        g = torch.randn(N * D + off, device="cuda").to(dt)[off:].view(N, D)
        gt = torch.full((V * D + off + 5,), 7.0, device="cuda")
        e2f.embed_backward(idt, g, V, grad_table=gt[off:off + V * D].view(V, D))
        assert torch.equal(gt[off:off + V * D].view(V, D), e2f.embed_backward(idt, g.clone(), V))
        assert bool((gt[:off] == 7).all()) and bool((gt[off + V * D:] == 7).all())


def test_ids_outside_the_table(cuda_ok):
    import torch
    from atomistic_mlip_b200 import e2f
    table = torch.randn(5, 8, device="cuda")
    ids = torch.tensor([0, 5, -1, 4, -2, 1 << 40], device="cuda")
    out = e2f.embed_forward(ids, table)
    assert e2f.stream_status() == 7
    ok = torch.tensor([0, 3], device="cuda")
    assert torch.equal(out[ok, 0], table[ids[ok]])
    assert bool((out[torch.tensor([1, 2, 4, 5], device="cuda")] == 0).all())
    g = torch.randn(6, 8, device="cuda")
    gt = e2f.embed_backward(ids, g, 5)
    assert e2f.stream_status() == 7
    want = torch.zeros(5, 8, device="cuda")
    want[0], want[4] = g[0], g[3]
    assert torch.equal(gt, want)
    e2f.embed_forward(torch.tensor([0, -1], device="cuda"), table)
    assert e2f.stream_status() == 0


def test_nonfinite_rows_stay_in_their_ids(cuda_ok):
    import torch
    from atomistic_mlip_b200 import e2f
    g = torch.randn(1000, 36, device="cuda")
    ids = torch.arange(1000, device="cuda") % 7
    g[ids == 3] = float("inf")
    g[12, :] = float("nan")          # id 5
    ids[100] = -1
    g[100] = float("nan")            # takes no part
    gt = e2f.embed_backward(ids, g, 9)
    assert bool(torch.isinf(gt[3]).all()) and bool(torch.isnan(gt[5]).all())
    rest = torch.tensor([0, 1, 2, 4, 6, 7, 8], device="cuda")
    assert bool(torch.isfinite(gt[rest]).all())


def test_offsets_beyond_32_bits(cuda_ok):
    """2.2e9 output elements, and a gradient read at such offsets."""
    import torch
    from atomistic_mlip_b200 import e2f
    N, V, D, Q = 700_001, 90, 128, 25
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.randn(V, D, generator=g, device="cuda").to(torch.bfloat16)
    out = e2f.embed_forward(ids, table, Q=Q, out_dtype=torch.bfloat16)
    assert torch.equal(out[:, 0], table[ids.long()])
    assert int(torch.count_nonzero(out[-50_000:, 1:])) == 0
    gt = e2f.embed_backward(ids, out, V)     # counts * table
    cnt = torch.bincount(ids.long(), minlength=V).double()[:, None]
    want = cnt * table.double()
    # equal terms: the partial sums are below n |t|, each of the n - 1 additions off by 2^-24 of that
    assert bool(((gt.double() - want).abs() <= (cnt + 2) * 2.0 ** -24 * 1.01 * want.abs()).all())


def test_streams_and_graphs(cuda_ok):
    """On a side stream; captured twice (two graphs with their own scratch) and
    replayed with other inputs in the same buffers, interleaved."""
    import torch
    from atomistic_mlip_b200 import e2f
    N, V, D = 5000, 300, 48
    ids = torch.randint(0, V, (N,), device="cuda")
    tab, g = torch.randn(V, D, device="cuda"), torch.randn(N, D, device="cuda")
    want = (e2f.embed_forward(ids, tab), e2f.embed_backward(ids, g, V))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = (e2f.embed_forward(ids, tab), e2f.embed_backward(ids, g, V))
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = (e2f.embed_forward(ids, tab), e2f.embed_backward(ids, g, V))
        graphs.append((gr, o))
    for seed in range(3):
        torch.manual_seed(seed)
        ids.copy_(torch.randint(0, V, (N,), device="cuda"))
        g.copy_(torch.randn(N, D, device="cuda"))
        for gr, _ in graphs:
            gr.replay()
        want = (e2f.embed_forward(ids, tab), e2f.embed_backward(ids, g, V))
        for _, o in graphs:
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    assert e2f.stream_status() == 0
