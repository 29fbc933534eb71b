"""The operators at the two ends of a model, as they are timed: the scaled embedding lookup that makes the
node features (species or token ids -> rows) with its gradient, and the linear layer of a readout (matrix
product, bias, activation, residual) with its gradient.

``own`` chooses between the plain form (elementary torch operations) and the library's entry points.
"""
import math

import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
_SZ = {"fp32": 4, "bf16": 2}
_IT = {"i32": torch.int32, "i64": torch.int64}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # the 24-atom cluster of the test configurations (L = 2, C = 8): launch latency
        dict(name="embed_cluster", op="embed_fwd", N=24, V=119, D=8, Q=9, dtype="fp32", out="fp32", ids="species",
             itype="i32", scale=1.0),
        # the residual stream of the 100,002-atom water box (L = 4, C = 128) from its atomic numbers
        dict(name="embed_water100k", op="embed_fwd", N=100002, V=119, D=128, Q=25, dtype="fp32", out="fp32",
             ids="species", itype="i32", scale=0.5),
        # a token batch of a ragged length and an odd width
        dict(name="embed_tokens", op="embed_fwd", N=16381, V=50021, D=770, Q=1, dtype="bf16", out="bf16", ids="zipf",
             itype="i64", scale=math.sqrt(770.0)),
        # the gradient of the 100,002-atom box's species table: two long segments, strided l = 0 rows
        dict(name="embed_grad_water100k", op="embed_bwd", N=100002, V=119, D=128, Q=25, dtype="fp32", ids="species",
             itype="i32", scale=0.5),
        # the gradient of a vocabulary: many short segments, a few long ones
        dict(name="embed_grad_tokens", op="embed_bwd", N=32771, V=50021, D=768, Q=1, dtype="bf16", ids="zipf",
             itype="i64", scale=math.sqrt(768.0)),
        # one row through a layer, as a serving step does
        dict(name="linear_one_row", op="linear_fwd", M=1, K=1024, N=4096, Q=1, dtype="bf16", out="bf16", act="silu",
             bias=True, residual=False),
        # the readout's first layer on the 3,000-atom box: l = 0 rows of the fp32 stream (L = 4, C = 128)
        dict(name="linear_head_3k", op="linear_fwd", M=3000, K=128, N=64, Q=25, dtype="fp32", out="fp32", act="silu",
             bias=True, residual=False),
        # the block's feed-forward width on every atom of the 100,002-atom box
        dict(name="linear_ffn_100k", op="linear_fwd", M=100002, K=128, N=512, Q=1, dtype="bf16", out="bf16",
             act="silu", bias=True, residual=False),
        # a wide layer added into an fp32 residual stream
        dict(name="linear_wide", op="linear_fwd", M=8192, K=4096, N=4096, Q=1, dtype="bf16", out="fp32", act="gelu",
             bias=True, residual=True),
        # the readout's gradient on the 10,304-atom molecule batch, fp32, strided l = 0 rows
        dict(name="linear_grad_head_10k", op="linear_bwd", M=10304, K=128, N=128, Q=25, dtype="fp32", out="fp32",
             act="silu", bias=True),
        # the gradient of the feed-forward width at 100,002 atoms
        dict(name="linear_grad_ffn_100k", op="linear_bwd", M=100002, K=128, N=512, Q=1, dtype="bf16", out="bf16",
             act="silu", bias=True),
        # the gradient of a wide layer of ragged sizes
        dict(name="linear_grad_wide", op="linear_bwd", M=4099, K=1000, N=2050, Q=1, dtype="bf16", out="fp32",
             act="gelu", bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the same ranges: 1 to 131,072 rows, widths 1 to 4,096 (lookups: 1 to 1,024 over up to
    65,536 rows of the table), fp32 and bf16, plain and strided rows."""
    op = rng.choice(["embed_fwd", "embed_bwd", "linear_fwd", "linear_bwd"])
    dtype = rng.choice(["fp32", "bf16"])
    if op.startswith("embed"):
        while True:
            N, V, D = _log(rng, 1, 131072), _log(rng, 1, 65536), _log(rng, 1, 1024)
            Q = rng.choice([1, 1, 1, 9, 25])
            if N * Q * D <= 100002 * 25 * 128 and V * D <= 50021 * 770:
                break
        c = dict(op=op, N=N, V=V, D=D, Q=Q, dtype=dtype, ids=rng.choice(["species", "zipf", "uniform"]),
                 itype=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, 0.5, math.sqrt(D)]))
        if op == "embed_fwd":
            c["out"] = rng.choice(["fp32", "bf16"])
        return c
    # products bounded so that no drawn pass costs more than the widest listed one
    cap = 8192 * 4096 * 4096 // (1 if op == "linear_fwd" else 4)
    if dtype == "fp32":
        cap //= 4
    while True:
        M, K, N = _log(rng, 1, 131072), _log(rng, 1, 4096), _log(rng, 1, 4096)
        Q = rng.choice([1, 1, 1, 9, 25])
        if M * K * N <= cap and M * K * Q <= 1 << 28 and M * N <= 1 << 27:
            break
    c = dict(op=op, M=M, K=K, N=N, Q=Q, dtype=dtype, out=dtype if dtype == "fp32" else rng.choice(["fp32", "bf16"]),
             act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.8)
    if op == "linear_fwd":
        c["residual"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _ids(case, g):
    N, V = case["N"], case["V"]
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    if case["ids"] == "species":      # two hydrogens to an oxygen, a few other species among them
        ids = torch.where(u < 0.66, 1, torch.where(u < 0.99, 8, (u * 1e6).long() % 90))
    elif case["ids"] == "zipf":       # frequency ~ 1 / rank
        ids = torch.exp(u * math.log(V + 1.0)).long() - 1
        ids = (ids * 7919) % V        # ranks scattered over the table
    else:
        ids = (u * V).long()
    return (ids % V).to(_IT[case["itype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    dt = _DT[case["dtype"]]
    st = dict(case=case)
    if case["op"].startswith("embed"):
        st["ids"] = _ids(case, g)
        if case["op"] == "embed_fwd":
            st["table"] = randn(case["V"], case["D"], dtype=dt)
        else:
            st["grad_out"] = randn(case["N"], case["Q"], case["D"], dtype=dt)
        return st
    M, K, N, Q = case["M"], case["K"], case["N"], case["Q"]
    st["x"] = randn(M, Q, K, dtype=dt)[:, 0, :]     # the l = 0 rows of a feature tensor when Q > 1
    st["W"] = randn(N, K, dtype=dt, std=1.0 / math.sqrt(K))
    st["bias"] = randn(N, dtype=torch.float32, std=0.1) if case["bias"] else None
    if case["op"] == "linear_fwd":
        st["residual"] = randn(M, N, dtype=_DT[case["out"]]) if case["residual"] else None
    else:
        st["grad_out"] = randn(M, N, dtype=_DT[case["out"]])
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from atomistic_mlip_b200 import e2f
    c = st["case"]
    if c["op"] == "embed_fwd":
        return e2f.embed_forward(st["ids"], st["table"], scale=c["scale"], Q=c["Q"], out_dtype=_DT[c["out"]])
    if c["op"] == "embed_bwd":
        return e2f.embed_backward(st["ids"], st["grad_out"], c["V"], scale=c["scale"])
    if c["op"] == "linear_fwd":
        return e2f.linear_forward(st["x"], st["W"], bias=st["bias"], residual=st["residual"], act=c["act"],
                                  out_dtype=_DT[c["out"]])
    gx, gw, gb = e2f.linear_backward(st["x"], st["W"], st["grad_out"], bias=st["bias"], act=c["act"])
    return (gx, gw, gb) if st["bias"] is not None else (gx, gw)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _run_plain(st):
    c = st["case"]
    if c["op"] == "embed_fwd":
        rows = st["table"][st["ids"].long()].float() * c["scale"]
        out = torch.zeros(c["N"], c["Q"], c["D"], dtype=_DT[c["out"]], device="cuda")
        out[:, 0, :] = rows.to(out.dtype)
        return out
    if c["op"] == "embed_bwd":      # sums of up to N terms: 64 bits
        acc = torch.zeros(c["V"], c["D"], dtype=torch.float64, device="cuda")
        acc.index_add_(0, st["ids"].long(), st["grad_out"][:, 0, :].double())
        return (acc * c["scale"]).float()
    x, W, b = st["x"].float(), st["W"].float(), st["bias"]
    if c["op"] == "linear_fwd":
        z = x @ W.t()
        if b is not None:
            z = z + b
        y = _act(z, c["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return y.to(_DT[c["out"]])
    dz = st["grad_out"].float()
    if c["act"] != "none":
        z = x @ W.t()
        if b is not None:
            z = z + b
        dz = dz * _act_grad(z, c["act"])
    gx = (dz @ W).to(st["x"].dtype)
    gw = (dz.t() @ x).to(st["W"].dtype)
    if b is None:
        return gx, gw
    return gx, gw, dz.double().sum(0).float()


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    if case["op"].startswith("embed"):
        N, V, D, Q = case["N"], case["V"], case["D"], case["Q"]
        ib = N * (4 if case["itype"] == "i32" else 8)
        if case["op"] == "embed_fwd":
            return {"bytes": ib + min(N, V) * D * _SZ[case["dtype"]] + N * Q * D * _SZ[case["out"]], "flops": N * D}
        return {"bytes": ib + N * D * _SZ[case["dtype"]] + V * D * 4, "flops": N * D}
    M, K, N = case["M"], case["K"], case["N"]
    s, o = _SZ[case["dtype"]], _SZ[case["out"]]
    b = 4 * N if case["bias"] else 0
    if case["op"] == "linear_fwd":
        return {"bytes": (M * K + N * K) * s + b + M * N * o * (2 if case["residual"] else 1), "flops": 2 * M * N * K}
    products = 2 if case["act"] == "none" else 3
    return {"bytes": 2 * (M * K + N * K) * s + 2 * b + M * N * o, "flops": 2 * products * M * N * K}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "embed_fwd":
        N, V, D, Q = case["N"], case["V"], case["D"], case["Q"]
        full = torch.zeros(V, Q * D, dtype=f8, device="cuda") if V * Q * D <= 1 << 27 else None
        if full is not None:
            full[:, :D] = st["table"].to(f8)
            return torch.index_select(full, 0, st["ids"].long()).mul_(case["scale"]).view(N, Q, D)
        out = torch.zeros(N, Q * D, dtype=f8, device="cuda")
        out[:, :D] = torch.index_select(st["table"].to(f8), 0, st["ids"].long()).mul_(case["scale"])
        return out.view(N, Q, D)
    if case["op"] == "embed_bwd":
        # per id the difference of running sums over the rows in the order of their ids
        ids, order = torch.sort(st["ids"].long(), stable=True)
        out = torch.empty(case["V"], case["D"], dtype=f8, device="cuda")
        ends = torch.searchsorted(ids, torch.arange(case["V"], device="cuda"), right=True)
        starts = torch.searchsorted(ids, torch.arange(case["V"], device="cuda"), right=False)
        for c0 in range(0, case["D"], 256):
            rows = st["grad_out"][:, 0, c0:c0 + 256].to(f8)[order]
            run_sum = torch.cat([torch.zeros_like(rows[:1]), torch.cumsum(rows, 0)])
            out[:, c0:c0 + 256] = (run_sum[ends] - run_sum[starts]) * case["scale"]
        return out
    x, W = st["x"].to(f8), st["W"].to(f8)
    b = torch.zeros(case["N"], dtype=f8, device="cuda") if st["bias"] is None else st["bias"].to(f8)
    z = torch.addmm(b, x, W.T)
    if case["act"] == "silu":
        s = torch.sigmoid(z)
        y, dy = z * s, s + z * s * (1 - s)
    elif case["act"] == "gelu":
        p = 0.5 * torch.special.erfc(-z / 2 ** 0.5)
        y, dy = z * p, p + z * torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5
    else:
        y, dy = z, torch.ones_like(z)
    if case["op"] == "linear_fwd":
        return y if st["residual"] is None else y + st["residual"].to(f8)
    dz = st["grad_out"].to(f8) * dy
    gx, gw = dz.matmul(W), dz.T.matmul(x)
    return (gx, gw) if st["bias"] is None else (gx, gw, dz.sum(dim=0))
