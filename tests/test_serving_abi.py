"""Refusals of the rotary and paged-cache entry points, on the host alone: C status codes with
addresses that are never dereferenced, the binding's own checks, and the frequency plans."""
import math
from fractions import Fraction

import pytest
import torch

import paged_ref as R
from exact_io_aware_60_b200 import fa

P = 4096      # fake, aligned, non-null "device" address: never dereferenced
S3 = fa._I3
BAD, NO = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


def rope(fn="fa_rope", **over):
    a = dict(q=P, qo=P, k=P, ko=P, B=2, H=4, Hk=2, N=8, d=64, qs=None, qos=None, ks=None, kos=None,
             pos=None, per=0, turns=P, rot=32, inter=0, mag=1.0, dt=0)
    a.update(over)
    return getattr(fa.lib(), fn)(*[a[n] for n in (
        "q", "qo", "k", "ko", "B", "H", "Hk", "N", "d", "qs", "qos", "ks", "kos", "pos", "per",
        "turns", "rot", "inter", "mag", "dt")], None)


@pytest.mark.parametrize("fn", ["fa_rope", "fa_rope_bwd"])
@pytest.mark.parametrize("over,code", [
    (dict(q=None), BAD), (dict(qo=P + 8), BAD), (dict(k=None), BAD), (dict(ko=None), BAD),
    (dict(B=0), BAD), (dict(N=0), BAD), (dict(H=0), BAD), (dict(Hk=0), BAD), (dict(dt=2), BAD),
    (dict(pos=P + 2), BAD), (dict(per=2), BAD), (dict(turns=None), BAD), (dict(turns=P + 4), BAD),
    (dict(rot=0), BAD), (dict(rot=80), BAD), (dict(inter=3), BAD), (dict(mag=float("nan")), BAD),
    (dict(mag=0.0), BAD), (dict(qs=S3(2048, 512, 63)), BAD), (dict(qos=S3(2048, 0, 64)), BAD),
    (dict(ks=S3(-1024, 512, 64)), BAD), (dict(kos=S3(1024, 511, 64)), BAD),
    (dict(rot=24), NO), (dict(d=96), NO), (dict(B=1 << 16, N=1 << 15), NO), (dict(H=65534), NO),
])
def test_rope_refusals(fn, over, code):
    assert rope(fn, **over) == code


def append(**over):
    a = dict(k=P, v=P, kc=P, vc=P, q=P, qo=P, B=2, H=4, Hk=2, T=3, d=64, ks=None, vs=None, qs=None,
             qos=None, kcs=None, vcs=None, pages=9, page=16, table=P, blocks=4, held=P, new=None,
             pos=None, turns=P, rot=64, inter=0, mag=1.0, dt=0)
    a.update(over)
    return fa.lib().fa_kv_append(*[a[n] for n in (
        "k", "v", "kc", "vc", "q", "qo", "B", "H", "Hk", "T", "d", "ks", "vs", "qs", "qos", "kcs",
        "vcs", "pages", "page", "table", "blocks", "held", "new", "pos", "turns", "rot", "inter",
        "mag", "dt")], None)


@pytest.mark.parametrize("over,code", [
    (dict(k=None), BAD), (dict(v=P + 2), BAD), (dict(kc=None), BAD), (dict(vc=P + 8), BAD),
    (dict(q=None), BAD), (dict(qo=None), BAD), (dict(T=0), BAD), (dict(Hk=0), BAD), (dict(H=0), BAD),
    (dict(pages=0), BAD), (dict(page=0), BAD), (dict(table=None), BAD), (dict(table=P + 1), BAD),
    (dict(blocks=0), BAD), (dict(held=None), BAD), (dict(held=P + 2), BAD), (dict(new=P + 2), BAD),
    (dict(pos=P + 3), BAD), (dict(rot=128), BAD), (dict(mag=-1.0), BAD), (dict(dt=9), BAD),
    (dict(kcs=S3(0, 1024, 64)), BAD), (dict(vcs=S3(4096, 1024, 4)), BAD),
    (dict(page=4), NO), (dict(page=24), NO), (dict(rot=8), NO), (dict(d=80), NO),
    (dict(blocks=1 << 28), NO),
])
def test_append_refusals(over, code):
    assert append(**over) == code


def paged(**over):
    a = dict(q=P, kc=P, vc=P, o=P, lse=P, B=2, H=4, Hk=2, T=3, d=64, qs=None, os=None, kcs=None,
             vcs=None, pages=9, page=16, table=P, blocks=4, held=P, new=None, tree=None, per=0,
             scale=0.125, dt=0, ws=P, wsb=1 << 40)
    a.update(over)
    return fa.lib().fa_fwd_paged(*[a[n] for n in (
        "q", "kc", "vc", "o", "lse", "B", "H", "Hk", "T", "d", "qs", "os", "kcs", "vcs", "pages",
        "page", "table", "blocks", "held", "new", "tree", "per", "scale", "dt", "ws", "wsb")], None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), BAD), (dict(kc=P + 8), BAD), (dict(vc=None), BAD), (dict(o=None), BAD),
    (dict(lse=None), BAD), (dict(lse=P + 2), BAD), (dict(H=5), BAD), (dict(Hk=0), BAD),
    (dict(B=0), BAD), (dict(T=-1), BAD), (dict(per=2), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(dt=3), BAD), (dict(table=None), BAD),
    (dict(held=None), BAD), (dict(pages=0), BAD), (dict(os=S3(0, 192, 64)), BAD),
    (dict(kcs=S3(2048, 0, 64)), BAD), (dict(page=12), NO), (dict(d=256), NO),
    (dict(blocks=1 << 27), NO), (dict(H=65536, Hk=65536), NO),
])
def test_paged_refusals(over, code):
    assert paged(**over) == code


def test_paged_workspace_size():
    L = fa.lib()
    assert L.fa_fwd_paged_workspace_bytes(0, 4, 2, 1, 64) == 0
    assert L.fa_fwd_paged_workspace_bytes(1, 5, 2, 1, 64) == 0
    assert L.fa_fwd_paged_workspace_bytes(1, 4, 2, 1, 96) == 0
    one, many = (L.fa_fwd_paged_workspace_bytes(1, 4, 2, t, 64) for t in (1, 4000))
    assert 0 < one < many
    # the shares are fixed by the device: neither batch nor length enters
    assert one == L.fa_fwd_paged_workspace_bytes(99, 4, 2, 1, 64)


def test_status_text():
    assert fa.lib().fa_strerror(fa.FA_ERR_BAD_PAGE).decode() == fa.fa_strerror(fa.FA_ERR_BAD_PAGE)
    assert "page" in fa.fa_strerror(fa.FA_ERR_BAD_PAGE)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_frequencies(scaling, rot):
    f, mag = fa.rope_frequencies(rot, scaling=scaling, factor=8.0, original_length=4096)
    want, wmag = R.inv_freq(rot, 10000.0, scaling, 8.0, 4096)
    assert mag == pytest.approx(wmag, rel=1e-15)
    assert all(abs(a - b) <= 4e-16 * 8 * b for a, b in zip(f, want))


def test_ntk_scales_the_slowest_pair_by_the_factor():
    a, _ = fa.rope_frequencies(64)
    b, _ = fa.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert b[0] == a[0] and b[-1] == pytest.approx(a[-1] / 8.0, rel=1e-12)


def test_plan_holds_fractions_of_a_turn():
    plan = fa.rope_plan(32, device="cpu")
    f, _ = fa.rope_frequencies(32)
    for bits, x in zip(plan.turns.tolist(), f):
        for pos in (1, 1000003, -77):
            frac = ((pos * bits) % 2 ** 64) / 2 ** 64
            turn = pos * x / (2 * math.pi)
            assert abs((frac - turn + 0.5) % 1.0 - 0.5) < 1e-9
    custom = fa.rope_plan(16, frequencies=[2 * math.pi * 3.25] * 8, magnitude=0.5, device="cpu")
    # 3.25 turns in 64 bits after three roundings: off by at most 3.25 * 3 * 2^-53 turns
    assert all(abs(t - (1 << 62)) <= 3.25 * 3 * 2 ** 11 for t in custom.turns.tolist())
    assert custom.magnitude == 0.5


@pytest.mark.parametrize("kw", [
    dict(rot_dim=20), dict(rot_dim=0), dict(rot_dim=32, layout="pairs"),
    dict(rot_dim=32, scaling="other"), dict(rot_dim=32, factor=0.5),
    dict(rot_dim=32, scaling="yarn", factor=2.0), dict(rot_dim=32, frequencies=[1.0]),
    dict(rot_dim=32, frequencies=[float("nan")] * 16), dict(rot_dim=32, magnitude=0.0),
    dict(rot_dim=32, base=-1.0),
])
def test_plan_refusals(kw):
    with pytest.raises(fa.FAError):
        fa.rope_plan(device="cpu", **kw)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((1, 2, 4, 64), dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    plan = fa.rope_plan(64, device="cpu")
    with pytest.raises(fa.FAError):
        fa.fa_rope(x, x, plan)
    with pytest.raises(fa.FAError):
        fa.fa_kv_append(x, x, x, x, i[None], i)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_paged(x, x, x, i[None], i, x, x[..., 0].float(), scale=1.0,
                        workspace=torch.zeros(8, dtype=torch.uint8))


def test_quick_binding_leaves_other_calls_alone():
    """What is not a plain call gets None, with nothing called (the address is null)."""
    assert fa._quick is not None
    x = torch.zeros((1, 2, 4, 64), dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    turns = torch.zeros(32, dtype=torch.int64)
    assert fa._quick.rope(0, x, x, None, None, None, turns, 64, False, 1.0, None) is None
    assert fa._quick.rope(0, None, x, None, None, None, turns, 64, False, 1.0, None) is None
    assert fa._quick.rope(0) is None
    assert fa._quick.append(0, x, x, x, x, i[None], i, None, None, None, None, None, 0, False, 1.0,
                            None) is None
    assert fa._quick.paged(0, x, x, x, i[None], i, None, x, x, None, x, "scale", None) is None


@pytest.mark.parametrize("x", [1e308, -1e308, 1e290, 3e18, -0.75, 5e-324, 0.0])
def test_plan_takes_any_finite_angle(x):
    bits = fa.rope_plan(16, frequencies=[x] * 8, device="cpu").turns.tolist()
    turn = Fraction(x / (2.0 * math.pi))
    want = (turn * 2 ** 64) % 2 ** 64
    off = (bits[0] - want + 2 ** 63) % 2 ** 64 - 2 ** 63
    assert bits == bits[:1] * 8 and abs(off) <= Fraction(1, 2)


@pytest.mark.parametrize("kw", [dict(factor=1e300), dict(factor=1e200, base=1e100)])
def test_an_ntk_base_that_overflows_is_refused(kw):
    with pytest.raises(fa.FAError):
        fa.rope_plan(16, scaling="ntk", device="cpu", **kw)


def test_paged_refuses_batches_that_outlast_a_wait():
    assert paged(B=(1 << 24) + 1, H=1, Hk=1, T=1, blocks=100) == NO
