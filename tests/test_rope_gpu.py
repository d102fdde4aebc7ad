"""Rotary positions on the GPU against the formula in 64 bits: layouts, part of the head,
scalings, far and negative positions, strides, in place, gradients, streams and graphs."""
import numpy as np
import pytest
import torch

import paged_ref as R
from exact_io_aware_60_b200 import fa
from exact_io_aware_60_b200 import workloads as W
from parity import oracle_full, rel_l2

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def randn(g, *shape, dtype):
    return torch.randn(shape, generator=g).to(dtype)


CASES = [
    # B, H, Hk, N, d, rot, layout, scaling, dtype, positions
    (1, 1, 1, 1, 64, 64, "half", "none", torch.bfloat16, None),
    (2, 3, 1, 37, 64, 32, "half", "linear", torch.float16, None),
    (3, 5, 5, 130, 128, 128, "half", "yarn", torch.bfloat16, "batch"),
    (2, 4, 2, 33, 128, 48, "interleaved", "ntk", torch.float16, "shared"),
    (1, 9, 3, 257, 128, 96, "half", "none", torch.float16, "far"),
    (2, 2, 2, 65, 64, 16, "interleaved", "none", torch.bfloat16, "far"),
    (1, 40, 8, 5000, 64, 64, "interleaved", "yarn", torch.bfloat16, None),
]


def setup(case, seed=3):
    B, H, Hk, N, d, rot, layout, scaling, dtype, kind = case
    g = torch.Generator().manual_seed(seed)
    q, k = randn(g, B, H, N, d, dtype=dtype), randn(g, B, Hk, N, d, dtype=dtype)
    pos = {None: None, "batch": torch.randint(0, 100000, (B, N), generator=g),
           "shared": torch.randint(-50, 50, (N,), generator=g),
           "far": torch.randint(-2**31, 2**31, (B, N), generator=g)}[kind]
    pos = None if pos is None else pos.to(torch.int32)
    f, mag = R.inv_freq(rot, 10000.0, scaling, 8.0, 4096)
    plan = fa.rope_plan(rot, layout=layout, scaling=scaling, factor=8.0, original_length=4096)
    full = torch.arange(N)[None].expand(B, N) if pos is None else pos.expand(B, N)
    return q, k, pos, full, f, mag, plan


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("direction", ["fwd", "bwd"])
def test_matches_the_formula(case, direction):
    B, H, Hk, N, d, rot, layout, scaling, dtype, kind = case
    q, k, pos, full, f, mag, plan = setup(case)
    sign = 1.0 if direction == "fwd" else -1.0
    p = None if pos is None else pos.to(DEV)
    if direction == "fwd":
        out = fa.rope(q.to(DEV), plan, k=k.to(DEV), positions=p)
    else:
        out = fa.rope_backward(q.to(DEV), plan, dk_rot=k.to(DEV), positions=p)
    # at positions near 2^31 the 64-bit reference's own angle is off by up to 2^31 2^-52
    far = 2.0 ** -20 if kind == "far" else 0.0
    for name, x, y in (("q", q, out[0]), ("k", k, out[1])):
        want, e = R.rope(x, full, rot, layout, f, mag, sign)
        R.check(name, y, want, (1 + far * 1e6) * e + R.rounding(want, dtype))
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


def test_strided_views_and_in_place():
    """q and k as views of one fused projection [B, N, H + 2 Hk, d], outputs in place."""
    B, H, Hk, N, d = 2, 6, 2, 77, 64
    g = torch.Generator().manual_seed(5)
    fused = randn(g, B, N, H + 2 * Hk, d, dtype=torch.bfloat16)
    plan = fa.rope_plan(32, layout="half")
    f, mag = R.inv_freq(32)
    x = fused.to(DEV)
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    fa.fa_rope(q, q, plan, k=k, k_out=k)
    full = torch.arange(N)[None].expand(B, N)
    want, e = R.rope(fused[:, :, :H + Hk].transpose(1, 2), full, 32, "half", f, mag)
    R.check("in place", x[:, :, :H + Hk].transpose(1, 2), want, e + R.rounding(want, torch.bfloat16))
    assert torch.equal(x[:, :, H + Hk:].cpu(), fused[:, :, H + Hk:])


def test_broadcast_input():
    g = torch.Generator().manual_seed(6)
    one = randn(g, 1, 1, 19, 128, dtype=torch.float16)
    plan = fa.rope_plan(128)
    a = fa.rope(one.to(DEV).expand(3, 4, 19, 128), plan)
    b = fa.rope(one.to(DEV), plan)
    assert torch.equal(a, b.expand(3, 4, 19, 128))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_backward_is_the_transpose_and_agrees_with_differences(layout):
    """<R x, y> = <x, R^T y> in fp16 roundings, and R^T y against central differences of the
    64-bit formula's <R x, y>."""
    g = torch.Generator().manual_seed(7)
    x, y = randn(g, 1, 2, 9, 64, dtype=torch.float16), randn(g, 1, 2, 9, 64, dtype=torch.float16)
    plan = fa.rope_plan(48, layout=layout, scaling="yarn", factor=4.0, original_length=64)
    f, mag = R.inv_freq(48, 10000.0, "yarn", 4.0, 64)
    full = torch.arange(9)[None]
    dx = fa.rope_backward(y.to(DEV), plan).double().cpu().numpy()
    h = 2.0 ** -6
    x64, y64 = x.double(), y.double().numpy()
    for idx in [(0, 0, 1, 0), (0, 1, 8, 23), (0, 0, 5, 24), (0, 1, 3, 47), (0, 0, 2, 60)]:
        up, dn = x64.clone(), x64.clone()
        up[idx] += h
        dn[idx] -= h
        num = ((R.rope(up, full, 48, layout, f, mag)[0] - R.rope(dn, full, 48, layout, f, mag)[0])
               * y64).sum() / (2 * h)
        # the map is linear: differences are exact up to 64-bit rounding
        assert abs(dx[idx] - num) <= R.half_step(torch.float16) * abs(num) + 1e-5, idx
    rx = fa.rope(x.to(DEV), plan).double().cpu().numpy()
    lhs, rhs = (rx * y64).sum(), (x64.numpy() * dx).sum()
    slack = R.half_step(torch.float16) * (np.abs(rx * y64).sum() + np.abs(x64.numpy() * dx).sum())
    assert abs(lhs - rhs) <= slack + 1e-5 * np.abs(rx * y64).sum()


def test_relative_positions_only():
    """Scores of rotated vectors depend on the distance alone, at far positions too."""
    g = torch.Generator().manual_seed(8)
    q, k = randn(g, 1, 1, 1, 128, dtype=torch.float16), randn(g, 1, 1, 1, 128, dtype=torch.float16)
    plan = fa.rope_plan(128)

    def score(i, j):
        a = fa.rope(q.to(DEV), plan, positions=torch.tensor([i], dtype=torch.int32, device=DEV))
        b = fa.rope(k.to(DEV), plan, positions=torch.tensor([j], dtype=torch.int32, device=DEV))
        return float((a.double() * b.double()).sum())

    # each of the 128 products carries two roundings
    slack = 2 * 2 * R.half_step(torch.float16) * float((q.double().abs().norm() * k.double().abs().norm()))
    assert abs(score(1000007, 1000000) - score(7, 0)) <= slack


def test_other_stream_and_graph():
    case = CASES[2]
    q, k, pos, full, f, mag, plan = setup(case)
    qd, kd, pd = q.to(DEV), k.to(DEV), pos.to(DEV)
    torch.cuda.synchronize()
    want = fa.rope(qd, plan, k=kd, positions=pd)
    side = torch.cuda.Stream()
    got = fa.rope(qd, plan, k=kd, positions=pd, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qo, ko = torch.empty_like(qd), torch.empty_like(kd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(qd, qo, plan, k=kd, k_out=ko, positions=pd)
    pd.add_(11)
    graph.replay()
    torch.cuda.synchronize()
    want = fa.rope(qd, plan, k=kd, positions=pd)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_training_step_with_rotation():
    """forward_rope / backward_rope against the oracle: attention of the rotated inputs, its
    dq and dk turned back."""
    w = W.custom("rope", B=2, H=3, N=200, d=64, dtype=torch.bfloat16, causal=True)
    inp = W.make_inputs(w, seed=21)
    plan = fa.rope_plan(64)
    f, mag = R.inv_freq(64)
    q, k, v, do = (inp[n].to(DEV) for n in ("q", "k", "v", "do"))
    o, lse, qr, kr = fa.forward_rope(q, k, v, plan, scale=w.scale, causal=True)
    dq, dk, dv = fa.backward_rope(qr, kr, v, o, do, lse, plan, scale=w.scale, causal=True)
    ref = oracle_full({**inp, "q": qr.cpu(), "k": kr.cpu()}, w.scale, True)
    full = torch.arange(w.N)[None].expand(w.B, w.N)
    assert rel_l2(o.double().cpu().numpy(), ref["o"]) <= 1e-2
    for got, name in ((dq, "dq"), (dk, "dk")):
        want, _ = R.rope(torch.from_numpy(ref[name]), full, 64, "half", f, mag, -1.0)
        assert rel_l2(got.double().cpu().numpy(), want) <= 2e-2, name
    assert rel_l2(dv.double().cpu().numpy(), ref["dv"]) <= 2e-2
