"""The paged cache on the GPU: append with rotation and attention of one token, chains and
drafted trees, against plain implementations in 64 bits (bounds in paged_ref.py)."""
import numpy as np
import pytest
import torch

import paged_ref as R
from exact_io_aware_60_b200 import fa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF, FP = torch.bfloat16, torch.float16


def tree_rows(g, B, T, reach=6):
    """Ancestors-or-self of random trees [B, T, T] and depths [B, T]."""
    rows, depth = torch.zeros((B, T, T), dtype=torch.uint8), torch.zeros((B, T), dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            rows[b, t, t] = 1
            if t:
                up = int(torch.randint(max(0, t - reach), t, (1,), generator=g))
                rows[b, t] |= rows[b, up]
                depth[b, t] = depth[b, up] + 1
    return rows, depth


def problem(B, Hk, G, T, d, page, lens, dtype, *, new=None, tree=False, seed=0, garbage=float("nan"),
            spare=2):
    """CPU tensors; slots that no sequence holds are `garbage`."""
    g = torch.Generator().manual_seed(seed)
    blocks = max(-(-(max(lens) + T) // page), 1)
    P = B * blocks + spare
    table = torch.randperm(P, generator=g)[:B * blocks].reshape(B, blocks).to(torch.int32)
    kc = torch.full((P, Hk, page, d), garbage, dtype=dtype)
    vc = torch.full((P, Hk, page, d), garbage, dtype=dtype)
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32)
    for b in range(B):
        n = lens[b] + (T if new is None else new[b])
        s = torch.arange(n)
        pages = table[b][s // page].long()
        kc[pages, :, s % page] = torch.randn((n, Hk, d), generator=g).to(dtype)
        vc[pages, :, s % page] = torch.randn((n, Hk, d), generator=g).to(dtype)
    q = torch.randn((B, Hk * G, T, d), generator=g).to(dtype)
    rows = tree_rows(g, B, T)[0] if tree else None
    return dict(q=q, kc=kc, vc=vc, table=table, cache_len=torch.tensor(lens, dtype=torch.int32),
                new_len=new_t, tree=rows)


def on_gpu(c):
    return {n: None if t is None else t.to(DEV) for n, t in c.items()}


def run(c, **over):
    x = on_gpu(c)
    x.update(over)
    o, lse = fa.forward_paged(x["q"], x["kc"], x["vc"], x["table"], x["cache_len"],
                              new_len=x["new_len"], tree_mask=x["tree"])
    return o, lse


def against_reference(c, **over):
    o, lse = run(c, **over)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    scale = c["q"].shape[-1] ** -0.5
    wo, wl, ob, lb = R.paged(c["q"], c["kc"], c["vc"], c["table"], c["cache_len"], c["new_len"],
                             c["tree"], scale)
    R.check("o", o, wo, ob + R.rounding(wo, c["q"].dtype))
    R.check("lse", lse, wl, lb)
    return o, lse


CASES = [
    # B, Hk, G, T, d, page, lens, dtype, new, tree
    (1, 1, 1, 1, 64, 8, [0], FP, None, False),            # one key in all
    (1, 1, 1, 1, 128, 16, [1], BF, None, False),
    (2, 2, 4, 1, 64, 16, [126, 127], FP, None, False),     # the tile's edge
    (3, 1, 8, 1, 128, 64, [128, 500, 255], BF, None, False),
    (2, 2, 1, 5, 128, 32, [300, 40], FP, [5, 2], False),   # short chains
    (3, 2, 3, 7, 64, 16, [0, 200, 77], BF, [7, 1, 4], True),
    (2, 1, 2, 33, 64, 8, [130, 600], FP, [33, 20], True),  # rows in two copies
    (1, 2, 5, 16, 128, 128, [900], BF, None, True),
    (2, 1, 16, 9, 64, 16, [250, 3], BF, [9, 0], True),     # more than one row tile, none new
    (1, 1, 7, 61, 128, 32, [513], FP, None, True),
    (1, 2, 2, 200, 64, 64, [0], BF, None, False),          # a prompt
    (1, 1, 1, 300, 128, 256, [333], FP, None, False),      # a page of two tiles
    (2, 1, 3, 150, 128, 16, [700, 20], BF, [150, 131], False),
    (40, 2, 2, 1, 64, 16, [(37 * i) % 300 for i in range(40)], FP, None, False),  # many short
    (1, 1, 4, 1, 128, 64, [20000], BF, None, False),       # one long: cut into many pieces
    (1, 1, 1, 64, 64, 32, [9000], FP, None, True),
    (2, 2, 5, 20, 128, 32, [90, 256], FP, [20, 11], True), # one row tile, not repeated
    (3, 2, 5, 20, 64, 32, [0, 256, 700], FP, [20, 1, 17], True),
    (1, 1, 1, 100, 64, 64, [0], BF, None, False),
    (1, 1, 1, 129, 64, 16, [77], BF, None, True),          # masks of more than 128 columns
    (2, 1, 2, 200, 128, 32, [0, 500], FP, [200, 170], True),
    (1, 1, 130, 2, 64, 16, [140], BF, None, True),         # a token's heads in two row tiles
    (2, 1, 300, 1, 128, 64, [10, 200], FP, None, False),
    (1, 2, 128, 3, 64, 32, [50], FP, None, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_matches_the_definition(case):
    B, Hk, G, T, d, page, lens, dtype, new, tree = case
    against_reference(problem(B, Hk, G, T, d, page, lens, dtype, new=new, tree=tree, seed=len(lens) + T))


LONG = [
    # Every CTA's share wraps its ring of tiles several times and crosses items.
    (6, 8, 2, 16, 64, 16, [6000, 11, 4097, 300, 0, 5555], FP, [16, 3, 16, 1, 9, 2], True),
    (5, 8, 4, 12, 128, 32, [5000, 3000, 129, 7000, 900], BF, None, True),
    (4, 8, 8, 13, 64, 64, [4000, 6100, 77, 2049], FP, None, False),
    (4, 8, 8, 20, 128, 16, [3500, 6000, 1, 4444], BF, [20, 17, 20, 4], True),
    (3, 8, 4, 70, 64, 128, [7000, 2500, 4100], BF, None, False),
    (7, 8, 3, 33, 64, 16, [130, 6000, 0, 127, 2000, 90, 4000], BF, [33, 5, 1, 33, 20, 30, 33], True),
    (90, 4, 5, 17, 64, 32, [(61 * i) % 400 for i in range(90)], FP, None, True),
    (8, 4, 4, 1, 128, 64, [16000] * 8, BF, None, False),   # tiles come in slower than they are used
    (8, 4, 4, 1, 64, 64, [20000] * 8, FP, None, False),
    (600, 4, 3, 1, 64, 16, [(97 * i) % 520 for i in range(600)], FP, None, False),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_long_shares(case):
    B, Hk, G, T, d, page, lens, dtype, new, tree = case
    c = problem(B, Hk, G, T, d, page, lens, dtype, new=new, tree=tree, seed=B)
    o, lse = run(c)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    heads = [0, Hk * G // 2 + 1, Hk * G - 1]
    wo, wl, ob, lb = R.paged(c["q"], c["kc"], c["vc"], c["table"], c["cache_len"], c["new_len"],
                             c["tree"], d ** -0.5, heads)
    R.check("o", o[:, heads], wo[:, heads], (ob + R.rounding(wo, dtype))[:, heads])
    R.check("lse", lse[:, heads], wl[:, heads], lb[:, heads])
    assert torch.isfinite(o.float()).all()


def against_heads(c, heads):
    """against_reference for some of the heads (long problems)."""
    o, lse = run(c)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    wo, wl, ob, lb = R.paged(c["q"], c["kc"], c["vc"], c["table"], c["cache_len"], c["new_len"],
                             c["tree"], c["q"].shape[-1] ** -0.5, heads)
    R.check("o", o[:, heads], wo[:, heads], (ob + R.rounding(wo, c["q"].dtype))[:, heads])
    R.check("lse", lse[:, heads], wl[:, heads], lb[:, heads])
    assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("case", [
    (1, 2, 4, 2500, 128, 64, [0], BF, None),
    (2, 2, 2, 2100, 64, 16, [300, 0], FP, [2100, 1777]),
    (1, 4, 1, 3333, 128, 128, [500], FP, None),
    (3, 1, 5, 1031, 64, 32, [0, 127, 1], BF, [1031, 900, 1]),
], ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_prompts_over_an_empty_or_short_cache(case):
    B, Hk, G, T, d, page, lens, dtype, new = case
    c = problem(B, Hk, G, T, d, page, lens, dtype, new=new, seed=T)
    against_heads(c, [0, Hk * G - 1])


@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("wide", [False, True], ids=["tight", "wide"])
@pytest.mark.parametrize("T,G,d,news", [
    # new tokens on both sides of a copy's, a warp's, a row tile's and an item's end
    (8, 4, 64, [8, 7, 1, 2]), (8, 4, 128, [7, 8, 3, 1]), (16, 4, 128, [8, 9, 16, 1]), (15, 4, 64, [8, 7, 15, 2]),
    (25, 5, 64, [6, 7, 12, 13, 25]), (25, 5, 128, [6, 7, 13, 19, 25]),
    (61, 3, 64, [42, 43, 61, 41]), (61, 3, 128, [42, 43, 61, 11]),
    (100, 3, 64, [84, 85, 42, 100, 43]), (100, 3, 128, [85, 84, 43, 100, 42]),
])
def test_new_tokens_end_about_a_row_tile(T, G, d, news, wide, tree):
    """Ragged new tokens in cut items of every form."""
    B, dtype = len(news), FP if d == 64 else BF
    c = problem(B, 2, G, T, d, 32, [3000 + 517 * i for i in range(B)], dtype, new=news, tree=tree, seed=T + d)
    if wide:
        c = widen(c, 800)
    against_heads(c, [0, G, 2 * G - 1])
    o, lse = run(c)
    for b, n in enumerate(news):
        assert torch.all(o[b, :, n:] == 0) and torch.all(torch.isneginf(lse[b, :, n:]))


def widen(c, tiles):
    """The same problem in a table with room for `tiles` tiles of 128 keys; the entries behind the
    sequences' are no pages at all.  (The room decides between one and two softmax groups, and
    whether items are cut.)"""
    B, blocks = c["table"].shape
    room = -(-tiles * 128 // c["kc"].shape[2])
    assert room >= blocks
    c["table"] = torch.cat([c["table"], torch.full((B, room - blocks), -1, dtype=torch.int32)], 1)
    return c


@pytest.mark.parametrize("case", [
    (3, 2, 5, 20, 64, 32, [0, 256, 700], FP, [20, 1, 17], True),
    (1, 1, 1, 100, 64, 64, [0], BF, None, False),          # one tile, the second group has none
    (2, 1, 3, 40, 64, 16, [100, 128], BF, None, False),    # two tiles, the last short
    (2, 2, 4, 32, 64, 8, [125, 383], FP, [0, 32], True),
    (1, 2, 128, 1, 64, 32, [1500], BF, None, False),
    (1, 1, 13, 9, 64, 128, [5000], FP, None, True),
], ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_more_room_than_keys(case):
    B, Hk, G, T, d, page, lens, dtype, new, tree = case
    c = problem(B, Hk, G, T, d, page, lens, dtype, new=new, tree=tree, seed=len(lens) + T)
    tight, tight_lse = against_reference(c)
    o, lse = against_reference(widen(c, 800))
    assert torch.equal(torch.isneginf(lse), torch.isneginf(tight_lse))
    empty = torch.isneginf(lse)
    assert torch.all(o[empty] == 0) and torch.all(tight[empty] == 0)


def test_many_short_in_a_wide_table():
    B = 90
    c = problem(B, 4, 5, 17, 64, 32, [(61 * i) % 400 for i in range(B)], FP, tree=True, seed=B)
    against_reference(widen(c, 12))


@pytest.mark.parametrize("B,Hk,lens,every", [
    (256, 2, [60], 2),
    (256, 8, [60], 2),
    (200, 4, [(37 * i) % 108 for i in range(200)], 3),
], ids=lambda c: str(len(c)) if isinstance(c, list) else str(c))
def test_short_sequences_next_to_finished_ones(B, Hk, lens, every):
    """Two softmax groups: pieces of one tile, written by the group that worked on them, and
    pieces of sequences without a new token, of no tile, behind one another in one CTA."""
    T, G = 20, 5
    new = [T if i % every == 0 else 0 for i in range(B)]
    c = widen(problem(B, Hk, G, T, 64, 16, [lens[i % len(lens)] for i in range(B)], BF, new=new, seed=B + Hk), 8)
    o, lse = against_reference(c)
    x = on_gpu(c)
    ws = fa.paged_workspace_for(x["q"], Hk)
    for _ in range(50):
        again, lse_again = fa.forward_paged(x["q"], x["kc"], x["vc"], x["table"], x["cache_len"],
                                            new_len=x["new_len"], workspace=ws)
        assert torch.equal(again, o) and torch.equal(lse_again, lse)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_hidden_keys_in_a_wide_table(value):
    c = widen(problem(1, 1, 5, 20, 64, 16, [250], FP, tree=True, seed=6), 800)
    s = 250 + 5
    page, row = int(c["table"][0, s // 16]), s % 16
    clean, _ = against_reference(c)
    c["vc"][page, 0, row, 7] = value
    c["kc"][page, 0, row] = float("nan")
    sees = c["tree"][0, :, 5] != 0
    o, lse = run(c)
    assert sees.any() and (~sees).any()
    assert torch.equal(o[0, :, ~sees], clean[0, :, ~sees])
    assert torch.isnan(o[0, :, sees]).all() and torch.isnan(lse[0, :, sees]).all()


def test_rows_that_see_nothing_in_a_wide_table():
    c = widen(problem(3, 1, 3, 40, 64, 16, [0, 5, 200], FP, tree=True, seed=4), 400)
    c["tree"][0] = 0
    c["tree"][1, 20] = 0
    o, lse = against_reference(c)
    assert torch.all(o[0] == 0) and torch.all(torch.isneginf(lse[0]))


@pytest.mark.parametrize("T", [1, 3, 40])
def test_rows_that_see_nothing(T):
    c = problem(3, 1, 3, T, 64, 16, [0, 5, 200], FP, tree=True, seed=4)
    c["tree"][0] = 0                       # no held key, no visible new one
    c["tree"][1, T // 2] = 0               # held keys only
    o, lse = against_reference(c)
    assert torch.all(o[0] == 0) and torch.all(torch.isneginf(lse[0]))


def test_new_rows_behind_the_last_are_empty():
    c = problem(2, 2, 2, 70, 128, 16, [90, 0], BF, new=[3, 0], seed=5)
    c["q"][0, :, 3:] = float("nan")
    o, lse = against_reference(c)
    assert torch.all(o[0, :, 3:] == 0) and torch.all(torch.isneginf(lse[0, :, 3:]))
    assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T,G", [(12, 2), (12, 5), (20, 5), (50, 4)])
def test_not_finite_values_in_hidden_keys(value, T, G):
    """A drafted token's K and V that are not finite reach the rows that see it, and no other."""
    c = problem(1, 1, G, T, 64, 16, [100], FP, tree=True, seed=6)
    x = 5
    s = 100 + x
    page, row = int(c["table"][0, s // 16]), s % 16
    clean = {n: None if t is None else t.clone() for n, t in c.items()}
    c["vc"][page, 0, row, 7] = value
    c["vc"][page, 0, row, 40] = -value
    c["kc"][page, 0, row] = float("nan")
    sees = c["tree"][0, :, x] != 0
    o, lse = run(c)
    wo, wl = run(clean)
    hidden = ~sees
    assert hidden.any() and sees.any()
    assert torch.equal(o[0, :, hidden], wo[0, :, hidden]) and torch.equal(lse[0, :, hidden], wl[0, :, hidden])
    assert torch.isnan(o[0, :, sees]).all() and torch.isnan(lse[0, :, sees]).all()
    c["kc"] = clean["kc"]                  # V alone
    o, lse = run(c)
    assert torch.equal(o[0, :, hidden], wo[0, :, hidden]) and torch.equal(lse, wl)
    touched = torch.tensor([7, 40])
    rest = torch.tensor([i for i in range(64) if i not in (7, 40)])
    assert torch.equal(o[0][:, :, rest], wo[0][:, :, rest])
    bad = o[0, :, sees][:, :, touched].float().cpu()
    if value == value:
        assert torch.all(bad[..., 0] == value) and torch.all(bad[..., 1] == -value)
    else:
        assert torch.isnan(bad).all()


FORMS = [(5, 4, 64), (5, 4, 128), (12, 5, 64), (12, 5, 128), (20, 5, 64), (20, 5, 128), (50, 4, 64), (50, 4, 128)]


def spiked(c, slot):
    """One key that every row puts all its weight on (some 400 nats above the others)."""
    page = c["kc"].shape[2]
    c["q"][..., 0] = 4.0
    c["kc"][int(c["table"][0, slot // page]), :, slot % page, 0] = 100.0 * c["q"].shape[-1] ** 0.5
    return c


def against_infinite(c, marks):
    """Sequence 0 of the problem with values that are not finite: marks = [(slot, column, value)],
    all key/value heads.  A row that sees such a key has their sum in the column, however small the
    key's weight (in 64 bits all are above 0); everything else is as with finite values there."""
    page, past = c["kc"].shape[2], int(c["cache_len"][0])
    wo, wl, ob, lb = R.paged(c["q"], c["kc"], c["vc"], c["table"], c["cache_len"], c["new_len"],
                             c["tree"], c["q"].shape[-1] ** -0.5)
    ob = ob + R.rounding(wo, c["q"].dtype)
    c = dict(c, vc=c["vc"].clone())
    n = c["q"].shape[2] if c["new_len"] is None else int(c["new_len"][0])
    hit = np.zeros(wo.shape)
    for slot, col, value in marks:
        c["vc"][int(c["table"][0, slot // page]), :, slot % page, col] = value
        x = slot - past
        with np.errstate(all="ignore"):
            for t in range(n):
                if x < 0 or (x <= t if c["tree"] is None else bool(c["tree"][0, t, x])):
                    hit[0, :, t, col] += value
    assert (hit != 0).any()
    o, lse = run(c)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    R.check("o", o, np.where(hit != 0, hit, wo), ob)
    R.check("lse", lse, wl, lb)
    return o, hit


@pytest.mark.parametrize("spike", [None, 10], ids=["even", "spiked"])
@pytest.mark.parametrize("T,G,d", FORMS)
@pytest.mark.parametrize("wide", [False, True], ids=["tight", "wide"])
def test_infinite_values_of_new_keys_in_cut_items(T, G, d, wide, spike):
    """An infinite V in a drafted token of an item in many pieces: that infinity in the rows that
    see it, however small its weight, nothing in the others."""
    past = 5000
    c = problem(1, 1, G, T, d, 16, [past], BF if T == 12 else FP, tree=True, seed=T + d)
    if wide:
        c = widen(c, 800)
    if spike is not None:
        c = spiked(c, spike)
    _, hit = against_infinite(c, [(past + T // 2, 7, float("inf")), (past + T // 2, d - 1, float("-inf"))])
    assert (hit[0, 0, :, 7] == 0).any()


@pytest.mark.parametrize("past", [90, 5000])
@pytest.mark.parametrize("spike", [None, "low", "high"])
@pytest.mark.parametrize("T,G,d", [(1, 1, 64), (1, 8, 128), *FORMS])
@pytest.mark.parametrize("wide", [False, True], ids=["tight", "wide"])
def test_infinite_values_of_held_keys(T, G, d, wide, spike, past):
    """Infinite values of keys that every row sees, in an uncut and a cut item: held ones in
    different places of a tile, and a single new token's own.  low, high: the weight of all other
    keys rounds to 0, first or last key."""
    dtype = BF if (T + d) % 3 == 0 else FP
    c = problem(1, 2, G, T, d, 16, [past], dtype, seed=T + d + past)
    if wide:
        c = widen(c, 800)
    if spike is not None:
        c = spiked(c, 3 if spike == "low" else past - 1)
    inf = float("inf")
    marks = [(past // 2, 0, inf), (past // 2 + 33, 9, -inf), (past - 2, 31, inf), (1, 32, -inf),
             (past // 2, 40, inf), (past // 2 + 1, 40, inf), (past - 2, 41, inf), (2, 41, -inf),
             (past, d - 1, inf), (past // 3, d - 2, float("nan"))]
    against_infinite(c, marks)


def test_weights_that_are_not_finite_stay_so():
    """A visible key whose score is NaN makes its rows NaN, infinite values or not; a row that sees
    nothing stays empty."""
    for T, G, d in FORMS:
        c = problem(1, 1, G, T, d, 16, [200], BF, tree=True, seed=T)
        c["tree"][0] = torch.tril(torch.ones((T, T), dtype=torch.uint8))
        page, row = int(c["table"][0, 201 // 16]), 201 % 16
        c["kc"][page, 0, row] = float("nan")
        c["vc"][int(c["table"][0, 3]), 0, 0, 5] = float("inf")
        o, lse = run(c)
        assert torch.isnan(o[0, :, 1:]).all() and torch.isnan(lse[0, :, 1:]).all()
        assert torch.all(o[0, :, 0, 5] == float("inf")) and torch.isfinite(lse[0, :, 0]).all()
        c = problem(1, 1, G, T, d, 16, [0], BF, tree=True, seed=T)
        c["tree"][0, 0] = 0
        c["vc"][int(c["table"][0, 0]), 0, 1, 5] = float("inf")
        o, lse = run(c)
        assert torch.all(o[0, :, 0] == 0) and torch.all(torch.isneginf(lse[0, :, 0]))
        assert torch.all(o[0, :, 1, 5] == float("inf"))


def test_not_finite_values_in_a_chain():
    c = problem(1, 2, 2, 140, 128, 32, [60], BF, seed=7)
    clean = {n: None if t is None else t.clone() for n, t in c.items()}
    s = 60 + 100
    c["vc"][int(c["table"][0, s // 32]), :, s % 32, 3] = float("nan")
    o, lse = run(c)
    wo, wl = run(clean)
    assert torch.equal(o[:, :, :100], wo[:, :, :100]) and torch.equal(lse, wl)
    assert torch.isnan(o[:, :, 100:, 3]).all()


def test_shared_tree_and_strided_tensors():
    """One mask for all sequences; q, o as [B, T, H, d] views, caches as [P, page, Hk, d] views
    of one buffer."""
    c = problem(3, 2, 2, 9, 64, 16, [40, 300, 128], BF, tree=True, seed=8)
    c["tree"] = c["tree"][1].clone()
    P, Hk, page, d = c["kc"].shape
    both = torch.empty((P, 2, page, Hk, d), dtype=BF)
    both[:, 0], both[:, 1] = c["kc"].transpose(1, 2), c["vc"].transpose(1, 2)
    both = both.to(DEV)
    x = on_gpu(c)
    q = x["q"].transpose(1, 2).contiguous().transpose(1, 2)
    o = torch.empty_like(x["q"].transpose(1, 2).contiguous()).transpose(1, 2)
    lse = torch.empty(q.shape[:3], device=DEV)
    ws = fa.paged_workspace_for(q, Hk)
    fa.fa_fwd_paged(q, both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2), x["table"],
                    x["cache_len"], o, lse, scale=d ** -0.5, tree_mask=x["tree"], workspace=ws)
    wo, wl = against_reference(c)
    assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_bad_pages_and_lengths_are_reported_and_hidden():
    """Page numbers outside the cache hide their keys; the rest of the row is as if they were
    masked.  Lengths beyond the table are clamped."""
    c = problem(2, 1, 2, 1, 64, 16, [160, 90], FP, seed=9)
    dead = {n: None if t is None else t.clone() for n, t in c.items()}
    c["table"][0, 3] = -5
    c["table"][0, 7] = 1 << 20
    o, lse = run(c)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    assert fa.fa_get_device_status() == fa.FA_OK
    keep = [s for s in range(161) if s // 16 not in (3, 7)]
    k = R.gather(dead["kc"], dead["table"][0], torch.arange(161))[0][keep].double().numpy()
    v = R.gather(dead["vc"], dead["table"][0], torch.arange(161))[0][keep].double().numpy()
    z = dead["q"][0, :, 0].double().numpy() @ k.T / 8
    w = np.exp(z - z.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    bound = 2 * R.half_step(FP) * (w @ np.abs(v)) + 1e-4
    assert np.all(np.abs(o[0, :, 0].double().cpu().numpy() - w @ v) <= bound)
    full = torch.tensor([1 << 30, -3], dtype=torch.int32)
    x = dict(dead, cache_len=full)
    o, lse = run(x)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    assert torch.all(o[0] == 0)            # the table is full: no room for the new token


def test_workspace_contents_do_not_matter_and_results_repeat():
    c = problem(2, 1, 4, 6, 128, 32, [5000, 777], BF, tree=True, seed=10)
    x = on_gpu(c)
    outs = []
    for fill in (0, 255, 127):
        ws = fa.paged_workspace_for(x["q"], 1)
        ws.fill_(fill)
        outs.append(fa.forward_paged(x["q"], x["kc"], x["vc"], x["table"], x["cache_len"],
                                     tree_mask=x["tree"], workspace=ws))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_two_streams_with_their_own_workspaces():
    cs = [problem(2, 2, 2, 4, 64, 16, [3000, 50], FP, tree=True, seed=s) for s in (11, 12)]
    want = [run(c) for c in cs]
    xs = [on_gpu(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(5):
        for x, st in zip(xs, streams):
            got.append(fa.forward_paged(x["q"], x["kc"], x["vc"], x["table"], x["cache_len"],
                                        tree_mask=x["tree"], stream=st))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_two_graphs_share_a_workspace():
    """Captured calls replayed one after the other on a stream, lengths advancing between."""
    c = problem(2, 2, 4, 1, 128, 16, [700, 30], BF, seed=13)
    c2 = problem(1, 2, 4, 1, 128, 16, [4000], BF, seed=14)
    x, y = on_gpu(c), on_gpu(c2)
    ws = fa.paged_workspace_for(x["q"], 2)
    outs, graphs = [], []
    for z in (x, y):
        o = torch.empty_like(z["q"])
        lse = torch.empty(z["q"].shape[:3], device=DEV)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fa.fa_fwd_paged(z["q"], z["kc"], z["vc"], z["table"], z["cache_len"], o, lse,
                            scale=128 ** -0.5, workspace=ws)
        graphs.append(gr)
        outs.append((o, lse))
    for step in range(3):
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for z, got, cpu in ((x, outs[0], c), (y, outs[1], c2)):
            now = dict(cpu, cache_len=z["cache_len"].cpu())
            want = run(now)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        x["cache_len"].sub_(9)
        y["cache_len"].sub_(500)


# ------------------------------------------------------------------------------ append

APPENDS = [
    # B, H, Hk, T, d, page, lens, dtype, new, rot, layout, tree
    (1, 4, 1, 1, 64, 8, [0], FP, None, 64, "half", False),
    (3, 6, 2, 5, 128, 16, [14, 0, 31], BF, [5, 0, 3], 32, "interleaved", True),
    (2, 0, 3, 40, 64, 32, [100, 7], FP, [40, 13], 16, "half", False),
    (2, 8, 8, 129, 128, 128, [120, 0], BF, None, 128, "half", False),
    (70, 16, 4, 1, 128, 64, [(53 * i) % 200 for i in range(70)], FP, None, 64, "interleaved", False),
    (2, 4, 4, 3, 64, 16, [10, 20], BF, None, None, "half", False),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_append(case):
    B, H, Hk, T, d, page, lens, dtype, new, rot, layout, tree = case
    c = problem(B, Hk, 1, T, d, page, lens, dtype, new=new, seed=T, garbage=7.0)
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn((B, Hk, T, d), generator=g).to(dtype), torch.randn((B, Hk, T, d), generator=g).to(dtype)
    q = torch.randn((B, H, T, d), generator=g).to(dtype) if H else None
    pos = None
    full = c["cache_len"][:, None] + torch.arange(T)
    if tree:
        pos = (c["cache_len"][:, None] + tree_rows(g, B, T)[1]).to(torch.int32)
        full = pos
    plan = f = None
    if rot:
        plan = fa.rope_plan(rot, layout=layout, scaling="yarn", factor=4.0, original_length=512)
        f, mag = R.inv_freq(rot, 10000.0, "yarn", 4.0, 512)
    x = on_gpu(c)
    q_out = torch.full_like(q, 3.0).to(DEV) if H else None
    fa.fa_kv_append(k.to(DEV), v.to(DEV), x["kc"], x["vc"], x["table"], x["cache_len"],
                    new_len=x["new_len"], rope=plan, positions=None if pos is None else pos.to(DEV),
                    q=None if q is None else q.to(DEV), q_out=q_out)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    wk, ek = R.rope(k, full, rot, layout, f, mag) if rot else (k.double().numpy(), 0.0)
    ek = ek + R.rounding(wk, dtype) * (1 if rot else 0)
    kc, ke, vc = c["kc"].double().numpy(), np.zeros(c["kc"].shape), c["vc"].clone()
    for b in range(B):
        n = T if new is None else new[b]
        for t in range(n):
            s = lens[b] + t
            p, r = int(c["table"][b, s // page]), s % page
            kc[p, :, r] = wk[b, :, t]
            ke[p, :, r] = ek[b, :, t] if rot else 0.0
            vc[p, :, r] = v[b, :, t]
    R.check("k", x["kc"], kc, ke)
    assert torch.equal(x["vc"].cpu(), vc)
    if H:
        wq, eq = R.rope(q, full, rot, layout, f, mag) if rot else (q.double().numpy(), np.zeros(q.shape))
        eq = eq + R.rounding(wq, dtype)
        for b in range(B):
            n = T if new is None else new[b]
            wq[b, :, n:], eq[b, :, n:] = 3.0, 0.0
        R.check("q", q_out, wq, eq)


def test_append_refuses_slots_outside_the_cache():
    c = problem(2, 1, 1, 4, 64, 8, [0, 3], FP, seed=2, garbage=7.0)
    c["table"][0, 0] = c["kc"].shape[0]
    k = torch.ones((2, 1, 4, 64), dtype=FP, device=DEV)
    x = on_gpu(c)
    before_k, before_v = x["kc"].clone(), x["vc"].clone()
    fa.fa_kv_append(k, k, x["kc"], x["vc"], x["table"], torch.tensor([0, 1 << 30], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    # nothing was written: sequence 0's page and sequence 1's slots lie outside
    assert torch.equal(x["kc"].view(torch.int16), before_k.view(torch.int16))
    assert torch.equal(x["vc"].view(torch.int16), before_v.view(torch.int16))


def test_offsets_beyond_32_bits():
    """Pages at the end of caches of more than 2^32 bytes and 2^31 elements."""
    P, Hk, page, d, T = 35000, 4, 128, 128, 3
    kc = torch.zeros((P, Hk, page, d), dtype=BF, device=DEV)
    vc = torch.zeros((P, Hk, page, d), dtype=BF, device=DEV)
    assert kc.numel() > 2 ** 31
    small = problem(1, Hk, 2, T, d, page, [300], BF, seed=15)
    n = small["table"].shape[1]
    far = torch.arange(P - n, P, dtype=torch.int32)[None]
    kc[far[0].long()] = small["kc"][small["table"][0].long()].to(DEV)
    vc[far[0].long()] = small["vc"][small["table"][0].long()].to(DEV)
    g = torch.Generator().manual_seed(16)
    k = torch.randn((1, Hk, T, d), generator=g).to(BF)
    want = run(dict(small, **{}))
    x = on_gpu(small)
    o, lse = fa.forward_paged(x["q"], kc, vc, far.to(DEV), x["cache_len"])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    fa.fa_kv_append(k.to(DEV), k.to(DEV), kc, vc, far.to(DEV), x["cache_len"])
    s = torch.arange(300, 303)
    assert torch.equal(kc[far[0].long()[s // page], :, s % page].cpu(), k[0].transpose(0, 1))


def test_drafted_step_against_one_token_at_a_time():
    """The operators together: a tree is appended and attended at once; each of its paths,
    decoded token by token in a cache of its own, gives the same outputs."""
    B, H, Hk, T, d, page, past = 1, 4, 2, 7, 64, 16, 45
    g = torch.Generator().manual_seed(17)
    plan = fa.rope_plan(d, layout="interleaved")
    rows, depth = tree_rows(g, B, T, reach=3)
    q, k, v = (torch.randn((B, h, T, d), generator=g).to(FP).to(DEV) for h in (H, Hk, Hk))
    pk, pv = (torch.randn((B, Hk, past, d), generator=g).to(FP).to(DEV) for _ in range(2))
    table = torch.randperm(8, generator=g)[:4].to(torch.int32).to(DEV)[None]
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)

    def cache():
        kc = torch.full((8, Hk, page, d), float("nan"), dtype=FP, device=DEV)
        vc = torch.full_like(kc, float("nan"))
        fa.fa_kv_append(pk, pv, kc, vc, table, zero, rope=plan)
        return kc, vc

    kc, vc = cache()
    held = torch.tensor([past], dtype=torch.int32, device=DEV)
    o, lse = fa.step_paged(q, k, v, kc, vc, table, held, rope=plan, positions=(held.cpu()[:, None] + depth).to(torch.int32).to(DEV),
                           tree_mask=rows.to(DEV))
    for leaf in range(T):
        path = [t for t in range(T) if rows[0, leaf, t]]
        kc, vc = cache()
        for i, t in enumerate(path):
            at = torch.tensor([past + i], dtype=torch.int32, device=DEV)
            one, l1 = fa.step_paged(q[:, :, t:t + 1], k[:, :, t:t + 1], v[:, :, t:t + 1], kc, vc,
                                    table, at, rope=plan)
        # the same keys in another order of sums: both within u of the exact weights' output
        tol = 4 * R.half_step(FP) * float(v.abs().max())
        assert (one[:, :, 0] - o[:, :, leaf]).abs().max() <= tol
        assert (l1[:, :, 0] - lse[:, :, leaf]).abs().max() <= 2e-5
    assert fa.fa_get_device_status() == fa.FA_OK


def test_prompt_then_decode_agrees_with_dense_attention():
    """A prompt appended and attended in two chunks gives fa_fwd's rows."""
    B, H, N, d, page = 2, 3, 333, 128, 32
    g = torch.Generator().manual_seed(18)
    q, k, v = (torch.randn((B, H, N, d), generator=g).to(BF).to(DEV) for _ in range(3))
    plan = fa.rope_plan(64)
    o, lse, _, _ = fa.forward_rope(q, k, v, plan, causal=True)
    blocks = -(-N // page)
    table = torch.randperm(B * blocks, generator=g).reshape(B, blocks).to(torch.int32).to(DEV)
    kc = torch.empty((B * blocks, H, page, d), dtype=BF, device=DEV)
    vc = torch.empty_like(kc)
    for lo, hi in ((0, 200), (200, 332), (332, 333)):
        held = torch.full((B,), lo, dtype=torch.int32, device=DEV)
        oo, ll = fa.step_paged(q[:, :, lo:hi], k[:, :, lo:hi], v[:, :, lo:hi], kc, vc, table, held,
                               rope=plan)
        tol = 4 * R.half_step(BF) * float(v.abs().max())
        assert (oo.float() - o[:, :, lo:hi].float()).abs().max() <= tol
        assert (ll - lse[:, :, lo:hi]).abs().max() <= 1e-4


@pytest.mark.parametrize("quick", [True, False], ids=["quick", "ctypes"])
def test_both_bindings_make_the_same_call(quick, monkeypatch):
    """The compiled binding and ctypes: strided and contiguous tensors, every optional argument."""
    assert fa._quick is not None
    if not quick:
        monkeypatch.setattr(fa, "_quick", None)
    c = problem(2, 2, 2, 5, 64, 16, [40, 300], BF, new=[5, 3], tree=True, seed=20)
    against_reference(c)
    g = torch.Generator().manual_seed(21)
    x = on_gpu(c)
    fused = torch.randn((2, 5, 8, 64), generator=g).to(BF).to(DEV)
    q, k, v = fused[:, :, :4].transpose(1, 2), fused[:, :, 4:6].transpose(1, 2), fused[:, :, 6:].transpose(1, 2)
    plan = fa.rope_plan(32)
    pos = torch.arange(10, dtype=torch.int32, device=DEV).reshape(2, 5)
    outs = []
    for args in ((q, k, v), tuple(t.contiguous() for t in (q, k, v))):
        kc, vc, qo = x["kc"].clone(), x["vc"].clone(), torch.zeros((2, 4, 5, 64), dtype=BF, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        fa.fa_kv_append(args[1], args[2], kc, vc, x["table"], x["cache_len"], new_len=x["new_len"],
                        rope=plan, positions=pos, q=args[0], q_out=qo, stream=side)
        side.synchronize()
        outs.append((qo, kc, vc))
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    got = fa.rope(q, plan, k=k, positions=pos[0])
    want = fa.rope(q.contiguous(), plan, k=k.contiguous(), positions=pos[:1].expand(2, 5).contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def wrong_calls():
    z = lambda *s, dtype=FP: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    q, kc, lens = z(2, 4, 3, 64), z(9, 2, 16, 64), z(2, dtype=torch.int32)
    table, lse, ws = z(2, 4, dtype=torch.int32), z(2, 4, 3, dtype=torch.float32), z(1 << 22, dtype=torch.uint8)
    k, plan = z(2, 2, 3, 64), fa.rope_plan(32)
    paged = dict(q=q, k_cache=kc, v_cache=kc, block_table=table, cache_len=lens, o=z(2, 4, 3, 64), lse=lse,
                 scale=0.125, workspace=ws)
    for over in (dict(q=q.float()), dict(q=q.cpu()), dict(k_cache=kc.bfloat16()), dict(v_cache=kc[:8]),
                 dict(k_cache=z(9, 3, 16, 64), v_cache=z(9, 3, 16, 64)), dict(block_table=table.long()),
                 dict(block_table=table[:1]), dict(cache_len=lens[:1]), dict(new_len=lens.cpu()),
                 dict(o=z(2, 4, 2, 64)), dict(lse=lse.half()), dict(tree_mask=z(3, 4, dtype=torch.uint8)),
                 dict(tree_mask=z(3, 3)), dict(scale=0.0), dict(scale=float("nan")), dict(workspace=ws[:64]),
                 dict(workspace=ws.view(torch.int8)), dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)),
                 dict(o=z(1, 4, 3, 64).expand(2, 4, 3, 64)), dict(k_cache=z(9, 2, 12, 64), v_cache=z(9, 2, 12, 64))):
        yield "fa_fwd_paged", {**paged, **over}
    app = dict(k=k, v=k, k_cache=kc, v_cache=kc.clone(), block_table=table, cache_len=lens, rope=plan, q=q, q_out=z(2, 4, 3, 64))
    for over in (dict(k=k[:, :1]), dict(v=k.bfloat16()), dict(q=None), dict(q_out=None), dict(q=z(2, 4, 2, 64)),
                 dict(positions=lens), dict(rope=object()), dict(new_len=table), dict(q_out=q[..., :32])):
        yield "fa_kv_append", {**app, **over}
    rot = dict(q=q, q_out=z(2, 4, 3, 64), plan=plan, k=k, k_out=z(2, 2, 3, 64))
    for over in (dict(q_out=z(2, 4, 3, 32)), dict(k_out=None), dict(k=None), dict(k=z(1, 2, 3, 64)),
                 dict(positions=table), dict(plan=None), dict(q=q.double()), dict(plan=fa.rope_plan(128))):
        yield "fa_rope", {**rot, **over}


@pytest.mark.parametrize("quick", [True, False], ids=["quick", "ctypes"])
def test_wrong_arguments_are_refused(quick, monkeypatch):
    if not quick:
        monkeypatch.setattr(fa, "_quick", None)
    for name, kw in wrong_calls():
        with pytest.raises(fa.FAError):
            getattr(fa, name)(**kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


def test_two_host_threads():
    """Calls of two host threads at once, each on its own stream with its own workspace."""
    import threading

    cs = [problem(2, 2, 4, 3, 128, 32, [2000, 60], BF, tree=True, seed=30),
          problem(1, 2, 2, 150, 64, 64, [700], FP, seed=31)]
    want = [run(c) for c in cs]
    xs = [on_gpu(c) for c in cs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        st, x = torch.cuda.Stream(), xs[i]
        for _ in range(20):
            o, lse = fa.forward_paged(x["q"], x["kc"], x["vc"], x["table"], x["cache_len"],
                                      tree_mask=x["tree"], stream=st)
            st.synchronize()
            if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and fa.fa_get_device_status() == fa.FA_OK


def test_many_rows_captured_and_replayed():
    """A chunk with two row tiles and its merge in a graph, lengths changing between replays."""
    c = problem(2, 2, 2, 180, 128, 64, [3000, 400], BF, seed=32)
    x = on_gpu(c)
    o, lse = torch.empty_like(x["q"]), torch.empty(x["q"].shape[:3], device=DEV)
    ws = fa.paged_workspace_for(x["q"], 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd_paged(x["q"], x["kc"], x["vc"], x["table"], x["cache_len"], o, lse,
                        scale=128 ** -0.5, workspace=ws)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = run(dict(c, cache_len=x["cache_len"].cpu()))
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        x["cache_len"].sub_(130)
