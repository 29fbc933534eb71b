"""The two ends together with what lies between them: species -> scaled
embedding -> attention or blocks -> readout -> structure sums, and the way back
to forces and weight gradients, against the fp64 oracles.

Bounds: the attention and its backward are held to 1e-4 of the largest entry
in fp32 elsewhere in this suite, the block to 1e-4 as well; the readout and the
sums add fp32 roundings of a few 1e-7.  Energies are sums of at most 24 atoms'
terms of order one, so 1e-4 of the largest is kept for all quantities here,
against sums of magnitudes where terms cancel."""
import numpy as np
import pytest

from atomistic_mlip_b200 import workloads as wlmod
from tests import helpers

pytestmark = pytest.mark.gpu


def _silu(z):
    s = 1 / (1 + np.exp(-z))
    return z * s, s * (1 + z * (1 - s))


def _system(L=2, C=16, H=2, seed=70):
    """Two copies of the 24-atom cluster 60 apart (two structures) and one
    lone atom that belongs to none."""
    base = wlmod.make_workload(0)
    pos = np.concatenate([base.pos, base.pos + np.float32(60), [[300, 0, 0]]]).astype(np.float32)
    rng = np.random.default_rng(seed)
    species = rng.choice([1, 6, 8], size=49)
    species[48] = -1
    structure = np.concatenate([np.zeros(24), np.ones(24), [-1]]).astype(np.int32)
    wl = wlmod.make_custom(pos, None, base.r_c, L=L, C=C, H=H, precision="fp32", seed=seed)
    table = rng.standard_normal((9, C)).astype(np.float32)
    head = [rng.standard_normal((12, C)).astype(np.float32) / np.float32(C ** 0.5), rng.standard_normal(12).astype(np.float32),
            rng.standard_normal((1, 12)).astype(np.float32), rng.standard_normal(1).astype(np.float32)]
    return wl, species, structure, table, head


def _features(species, table, Q, scale):
    x = np.zeros((len(species), Q, table.shape[1]))
    live = species >= 0
    x[live, 0] = np.float64(np.float32(scale)) * table[species[live]]
    return x


def _dev(*arrays):
    import torch
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def test_energy_forces_and_gradients(cuda_ok):
    from atomistic_mlip_b200 import e2f
    from oracle import attention as oa
    from oracle import attention_grad as ag
    from oracle import neighbors as nb
    wl, species, structure, table, head = _system()
    scale, Q = 0.7, (wl.L + 1) ** 2
    gE = np.array([1.0, -0.5], np.float32)
    pos, sp, st, tab, ge = _dev(wl.pos, species, structure, table, gE)
    dw = e2f.DeviceWeights.from_workload(wl, "cuda", "fp32")
    dh = e2f.DeviceReadout(*_dev(*head))
    nl = e2f.build_neighbors(pos, None, wl.r_c)
    E, F, g = e2f.attention_energy_forces(sp, pos, nl, tab, dw, dh, st, 2, scale=scale, grad_energy=ge)
    assert e2f.stream_status() == 0

    csr = nb.neighbors(wl.pos, None, wl.r_c)
    x = _features(species, table, Q, scale)
    wl.x = x
    o = oa.attention_workload(wl, csr=csr)
    W1, b1, W2, b2 = (np.asarray(h, np.float64) for h in head)
    z = o[:, 0] @ W1.T + b1
    h, dh_ = _silu(z)
    e = (h @ W2.T + b2)[:, 0]
    live = structure >= 0
    Er = np.array([e[structure == k].sum() for k in range(2)])
    assert np.max(np.abs(E.double().cpu().numpy() - Er)) <= 1e-4 * max(np.abs(e[structure == k]).sum() for k in range(2))
    ga = np.where(live, np.float64(gE)[structure], 0.0)          # dL/de
    gz = ga[:, None] * W2 * dh_
    G = np.zeros_like(o)
    G[:, 0] = gz @ W1
    ref = ag.gradients(wl, csr, G, x=x)
    assert helpers.rel_err(F.double().cpu().numpy(), -ref["pos"]) <= 1e-4
    want = dict(W1=gz.T @ o[:, 0], b1=gz.sum(0), W2=(ga[:, None] * h).sum(0)[None], b2=np.array([ga.sum()]))
    gt = np.zeros(table.shape)
    ok = species >= 0
    np.add.at(gt, species[ok], np.float64(np.float32(scale)) * ref["x"][ok, 0])
    want["table"] = gt
    for k, r in want.items():
        assert helpers.rel_err(g[k].double().cpu().numpy(), r) <= 1e-4, k
    # the lone atom of no structure feels nothing and moves nothing
    assert np.all(F[48].cpu().numpy() == 0)


def test_forces_against_differences(cuda_ok):
    """Central differences of the oracle's energy along a random direction
    (step 1e-5 in fp64; the library's forces are good to 1e-4 of the largest)."""
    from atomistic_mlip_b200 import e2f
    from oracle import attention as oa
    from oracle import neighbors as nb
    wl, species, structure, table, head = _system(seed=71)
    x = _features(species, table, (wl.L + 1) ** 2, 1.0)
    wl.x = x
    csr = nb.neighbors(wl.pos, None, wl.r_c)
    pos, sp, st, tab = _dev(wl.pos, species, structure, table)
    nl = e2f.build_neighbors(pos, None, wl.r_c)
    _, F, _ = e2f.attention_energy_forces(sp, pos, nl, tab, e2f.DeviceWeights.from_workload(wl, "cuda", "fp32"),
                                          e2f.DeviceReadout(*_dev(*head)), st, 2)
    W1, b1, W2, b2 = (np.asarray(h, np.float64) for h in head)
    p0 = np.float64(wl.pos)

    def energy(p):
        wl.pos = p
        o = oa.attention_workload(wl, csr=csr)
        return float(((_silu(o[:, 0] @ W1.T + b1)[0] @ W2.T + b2)[:, 0] * (structure >= 0)).sum())

    d = np.random.default_rng(5).standard_normal(p0.shape)
    num = (energy(p0 + 1e-5 * d) - energy(p0 - 1e-5 * d)) / 2e-5
    Fn = F.double().cpu().numpy()
    assert abs(num + float((Fn * d).sum())) <= 2e-4 * np.max(np.abs(Fn)) * np.abs(d).sum()


def test_blocks_between_the_ends(cuda_ok):
    """model_energy through one block against the block oracle."""
    from atomistic_mlip_b200 import e2f
    from oracle import block as ob
    from oracle import neighbors as nb
    wl, species, structure, table, head = _system(seed=72)
    lw = wlmod.make_layer_weights(wl.L, wl.C, wl.H, "fp32", 73)
    pos, sp, st, tab = _dev(wl.pos, species, structure, table)
    nl = e2f.build_neighbors(pos, None, wl.r_c)
    dh = e2f.DeviceReadout(*_dev(*head))
    E = e2f.model_energy(sp, pos, nl, tab, [e2f.DeviceBlockWeights.from_layer(lw)], dh, st, 2, scale=0.9)
    csr = nb.neighbors(wl.pos, None, wl.r_c)
    y = ob.block_forward(wl.pos, None, wl.r_c, csr, _features(species, table, (wl.L + 1) ** 2, 0.9), lw)
    W1, b1, W2, b2 = (np.asarray(h, np.float64) for h in head)
    e = (_silu(y[:, 0] @ W1.T + b1)[0] @ W2.T + b2)[:, 0]
    Er = np.array([e[structure == k].sum() for k in range(2)])
    tol = 1e-4 * max(np.abs(e[structure == k]).sum() + 1 for k in range(2))
    assert np.max(np.abs(E.double().cpu().numpy() - Er)) <= tol


def test_given_stream(cuda_ok):
    """stream=s with another stream current: the results of the same call on the
    current stream, in memory that belongs to s (so that neither pending work of
    other streams nor their later allocations meet it), and so the intermediates:
    nothing is allocated for the current stream."""
    import torch
    from atomistic_mlip_b200 import e2f
    wl, species, structure, table, head = _system()
    pos, sp, st, tab = _dev(wl.pos, species, structure, table)
    dw = e2f.DeviceWeights.from_workload(wl, "cuda", "fp32")
    dh = e2f.DeviceReadout(*_dev(*head))
    nl = e2f.build_neighbors(pos, None, wl.r_c)
    ids, tb = torch.arange(3000, device="cuda") % 50, torch.randn(50, 64, device="cuda")
    go = torch.randn(3000, 64, device="cuda")

    def run(stream):
        E, F, g = e2f.attention_energy_forces(sp, pos, nl, tab, dw, dh, st, 2, stream=stream)
        y = e2f.embed_forward(ids, tb, stream=stream)[:, 0]
        gt = e2f.embed_backward(ids, go, 50, stream=stream)
        z = e2f.linear_forward(y, tb, act="gelu", stream=stream)
        return [E, F, gt, z, *e2f.linear_backward(y, tb, z, act="gelu", stream=stream)[:2], *(g[k] for k in sorted(g))]

    want = run(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    here = torch.cuda.current_stream().cuda_stream

    def held(stream):   # bytes of the blocks handed out for a stream
        return sum(seg["allocated_size"] for seg in torch.cuda.memory_snapshot() if seg["stream"] == stream)

    before = held(here)
    got = run(s)
    assert held(here) == before
    s.synchronize()
    for w, t in zip(want, got):
        assert torch.equal(w, t) or bool(((w - t).abs() <= 1e-4 * w.abs().max()).all())   # (forces: the attention's bound)
        own = [seg for seg in torch.cuda.memory_snapshot() if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]]
        assert len(own) == 1 and own[0]["stream"] == s.cuda_stream
    assert e2f.stream_status() == 0


def test_tall_column_sums(cuda_ok):
    """70 million rows of one value: more blocks of rows than a grid has in y."""
    import torch
    from atomistic_mlip_b200 import e2f
    M = 70_000_001
    x = torch.ones(M, 1, device="cuda", dtype=torch.bfloat16)
    W = torch.full((3, 1), 0.5, device="cuda", dtype=torch.bfloat16)
    dy = torch.ones(M, 3, device="cuda", dtype=torch.bfloat16)
    _, _, gb = e2f.linear_backward(x, W, dy, need_x=False, need_W=False, need_bias=True)
    # ones: a CTA's 1,024 are exact, as are partial sums below 2^24; the last steps add at most 70 terms
    # of 2^20, each rounded by at most 2^-24 of a sum below 2^27: 70 * 2^3
    assert bool(((gb.double() - M).abs() <= 560).all())
    assert e2f.stream_status() == 0
