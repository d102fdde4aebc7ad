"""The serving and position operators: cases, inputs, plain forms and definitions in 64 bits.

Three operators, which a program that serves or trains a language model with this library
uses next to its attention calls:

* ``rope``: rotary positions applied to queries and keys (forward) and to their gradients
  (backward): half and interleaved pair layouts, part of the head, frequencies scaled for
  long contexts.
* ``append``: a step's new keys and values written into a paged cache, queries and keys
  rotated on the way.
* ``paged``: attention of the step's new tokens (one token, a chain, or a tree of drafted
  tokens) over the paged cache, with key/value heads shared by groups of query heads.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits,
angles in 64) or, with ``own`` set, through the library's entry points.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_TWO_PI = 2.0 * math.pi


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # One sequence decoding its next token at a far position: the smallest call of the
        # rotation, nothing but latency.
        dict(name="rope_token", op="rope", dir="fwd", B=1, H=16, Hk=4, N=1, d=128, rot=128,
             layout="half", scaling="none", dtype="fp16", start=32767),
        # Queries and keys of the GPT-2-small training shape, whole head.
        dict(name="rope_gpt2", op="rope", dir="fwd", B=8, H=12, Hk=12, N=1024, d=64, rot=64,
             layout="half", scaling="none", dtype="bf16", start=0),
        # Gradients of a ragged batch whose sequences start at different positions; half of
        # the head rotated, adjacent pairs.
        dict(name="rope_part_grad", op="rope", dir="bwd", B=5, H=16, Hk=2, N=1537, d=128, rot=64,
             layout="interleaved", scaling="linear", dtype="fp16", start=-1),
        # Gradients of the very long causal training shape, frequencies scaled by parts: the
        # largest call of the rotation.
        dict(name="rope_64k_grad", op="rope", dir="bwd", B=1, H=16, Hk=16, N=65536, d=128,
             rot=128, layout="half", scaling="yarn", dtype="bf16", start=0),
        # One new token for each of eight sequences in a long cache: a decoding step.
        dict(name="append_decode", op="append", B=8, H=16, Hk=4, T=1, d=128, page=64, L=32000,
             ragged=True, tree=False, rot=128, layout="half", scaling="yarn", dtype="bf16"),
        # Drafted trees of up to 24 tokens, positions by depth, small pages, ragged.
        dict(name="append_tree", op="append", B=48, H=32, Hk=8, T=24, d=64, page=16, L=2000,
             ragged=True, tree=True, rot=32, layout="interleaved", scaling="none", dtype="fp16"),
        # A long prompt's chunk for two sequences: bandwidth.
        dict(name="append_prompt", op="append", B=2, H=32, Hk=8, T=4096, d=128, page=128, L=8192,
             ragged=False, tree=False, rot=128, layout="half", scaling="none", dtype="bf16"),
        # One token of one short sequence: the smallest attention call, latency.
        dict(name="paged_token", op="paged", B=1, H=8, Hk=2, T=1, d=64, page=16, L=300,
             ragged=False, tree=False, dtype="fp16"),
        # Decoding against 32K keys: the cache's bytes.
        dict(name="paged_decode32k", op="paged", B=8, H=16, Hk=4, T=1, d=128, page=64, L=32768,
             ragged=False, tree=False, dtype="bf16"),
        # Sixteen sequences of very different lengths, each with a drafted tree.
        dict(name="paged_tree", op="paged", B=16, H=32, Hk=8, T=16, d=128, page=16, L=8000,
             ragged=True, tree=True, dtype="bf16"),
        # Large trees at d = 64, odd group size.
        dict(name="paged_tree64", op="paged", B=6, H=15, Hk=5, T=61, d=64, page=32, L=10000,
             ragged=True, tree=True, dtype="fp16"),
        # A prompt chunk of 512 tokens against 16384 keys: the products.
        dict(name="paged_chunk16k", op="paged", B=1, H=16, Hk=16, T=512, d=128, page=128,
             L=15872, ragged=False, tree=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "paged", "paged"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    rot = rng.choice([16, 32, 48, 64] if d == 64 else [16, 32, 64, 96, 128])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    Hk = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    G = rng.choice([1, 1, 2, 3, 4, 5, 8])
    while Hk * G > 64:
        G = max(1, G // 2)
    H = Hk * G
    if op == "rope":
        B = _log(rng, 1, 16)
        most = max(1, (1 << 27) // (B * (H + Hk) * d))
        N = _log(rng, 1, min(65536, most))
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), B=B, H=H, Hk=Hk, N=N, d=d, rot=rot,
                    layout=layout, scaling=scaling, dtype=dtype,
                    start=rng.choice([-1, 0, _log(rng, 1, 500000)]))
    page = rng.choice([16, 32, 64, 128])
    tree = rng.random() < 0.5
    if op == "append":
        B = _log(rng, 1, 64)
        most = max(1, (1 << 25) // (B * (H + 2 * Hk) * d))
        T = _log(rng, 1, min(64 if tree else 4096, most))
        room = (1 << 27) // (2 * B * Hk * d)  # keeps the cache itself small
        return dict(op=op, B=B, H=H, Hk=Hk, T=T, d=d, page=page, L=_log(rng, 1, max(2, room)),
                    ragged=rng.random() < 0.7, tree=tree, rot=rot, layout=layout,
                    scaling=scaling, dtype=dtype)
    B = _log(rng, 1, 32)
    T = _log(rng, 1, 128) if tree else rng.choice([1, _log(rng, 1, 512)])
    by_bytes = (1 << 27) // (B * Hk * d)               # the decode32k case's keys
    by_flops = (1 << 27) // (B * H * T) * 128 // d     # the chunk16k case's pairs
    L = _log(rng, 1, max(2, min(32768, by_bytes, by_flops)))
    return dict(op=op, B=B, H=H, Hk=Hk, T=T, d=d, page=page, L=L, ragged=rng.random() < 0.7,
                tree=tree, dtype=dtype)


def _lengths(case, seed):
    """(cache_len, new_len) of a case's sequences, from the seed: ragged batches spread over
    [0, L] and [1, T]."""
    r = random.Random(seed * 7919 + 13)
    B, T, L = case["B"], case["T"], case["L"]
    if not case["ragged"]:
        return [L] * B, [T] * B
    return [r.randint(0, L) for _ in range(B)], [r.randint(1, T) for _ in range(B)]


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["B"] * (case["H"] + case["Hk"]) * case["N"]
        return {"bytes": 4 * n * d, "flops": 3 * n * case["rot"]}
    # of ragged lengths, the mean (they follow from the seed)
    B, T, L, H, Hk = case["B"], case["T"], case["L"], case["H"], case["Hk"]
    t = (1 + T) / 2 if case["ragged"] else T
    past = L / 2 if case["ragged"] else L
    if case["op"] == "append":
        return {"bytes": 4 * B * t * (H + 2 * Hk) * d, "flops": 3 * B * t * (H + Hk) * case["rot"]}
    pairs = t * past + t * (t + 1) / 2
    return {"bytes": 4 * B * (past + t) * Hk * d + 4 * B * t * H * d, "flops": 4 * B * H * d * pairs}


# ------------------------------------------------------------------------------ inputs

def _inverse_frequencies(rot, scaling):
    """(angle per position of each pair, magnitude) in 64 bits; factor 8 over 4096 positions."""
    base, s, length = 10000.0, 8.0, 4096
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / s, 1.0
    if scaling == "yarn":
        gamma = ((length * f / _TWO_PI - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return (1.0 - gamma) * f / s + gamma * f, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _plan(case):
    """The rotation plan that a program keeps."""
    from exact_io_aware_60_b200 import fa
    return fa.rope_plan(case["rot"], layout=case["layout"], base=10000.0,
                        scaling=case["scaling"], factor=8.0, original_length=4096,
                        device="cuda")


def _trees(case, seed, new_len):
    """Random drafted trees: ([B, T, T] ancestors-or-self, [B, T] depths)."""
    r = random.Random(seed * 104729 + 7)
    B, T = case["B"], case["T"]
    rows, depth = torch.zeros((B, T, T), dtype=torch.uint8), torch.zeros((B, T), dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            rows[b, t, t] = 1
            if t > 0:
                up = r.randint(max(0, t - 8), t - 1)
                rows[b, t] |= rows[b, up]
                depth[b, t] = depth[b, up] + 1
    return rows, depth


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]
    B, H, Hk, d = case["B"], case["H"], case["Hk"], case["d"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    s = {"case": case}
    if case["op"] == "rope":
        N = case["N"]
        s["q"], s["k"] = randn(B, H, N, d), randn(B, Hk, N, d)
        if case["start"] == 0:
            s["positions"] = None
        else:
            r = random.Random(seed * 31 + 5)
            first = [r.randint(0, 100000) if case["start"] < 0 else case["start"] for _ in range(B)]
            first = torch.tensor(first, dtype=torch.int32, device=dev)
            s["positions"] = (first[:, None] + torch.arange(N, dtype=torch.int32, device=dev)).contiguous()
        s["plan"] = _plan(case) if own else None
        if own:
            s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        return s

    T, L, page = case["T"], case["L"], case["page"]
    past, new = _lengths(case, seed)
    blocks = -(-(L + T) // page)
    pages = B * blocks + 3
    s["k_cache"], s["v_cache"] = randn(pages, Hk, page, d), randn(pages, Hk, page, d)
    order = torch.randperm(pages, generator=g, device=dev)[:B * blocks]
    s["table"] = order.to(torch.int32).reshape(B, blocks).contiguous()
    s["cache_len"] = torch.tensor(past, dtype=torch.int32, device=dev)
    s["new_len"] = torch.tensor(new, dtype=torch.int32, device=dev) if case["ragged"] else None
    s["q"] = randn(B, H, T, d)
    if case["tree"]:
        rows, depth = _trees(case, seed, new)
        s["tree"] = rows.to(dev)
        s["positions"] = s["cache_len"][:, None] + depth.to(dev)
    else:
        s["tree"] = s["positions"] = None
    if case["op"] == "append":
        s["k"], s["v"] = randn(B, Hk, T, d), randn(B, Hk, T, d)
        # rows behind a sequence's last new token stay as they are in every form
        s["q_out"] = torch.zeros_like(s["q"])
        s["plan"] = _plan(case) if own else None
        return s
    if own:
        from exact_io_aware_60_b200 import fa
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, H, T), dtype=torch.float32, device=dev)
        n = fa.fa_fwd_paged_workspace_bytes(B, H, Hk, T, d)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "paged": _own_paged}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "paged": _plain_paged}[op](state)


def _own_rope(s):
    from exact_io_aware_60_b200 import fa
    call = fa.fa_rope if s["case"]["dir"] == "fwd" else fa.fa_rope_bwd
    call(s["q"], s["q_out"], s["plan"], k=s["k"], k_out=s["k_out"], positions=s["positions"])
    return s["q_out"], s["k_out"]


def _own_append(s):
    from exact_io_aware_60_b200 import fa
    fa.fa_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cache_len"],
                    new_len=s["new_len"], rope=s["plan"], positions=s["positions"], q=s["q"],
                    q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_paged(s):
    from exact_io_aware_60_b200 import fa
    fa.fa_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cache_len"], s["o"],
                    s["lse"], scale=s["case"]["d"] ** -0.5, new_len=s["new_len"],
                    tree_mask=s["tree"], workspace=s["workspace"])
    return s["o"], s["lse"]


def _rotated(x, positions, case, sign):
    """x [B, heads, N, d] rotated by positions [B or 1, N]: angles in 64 bits, the rest in 32."""
    rot = case["rot"]
    f, mag = _inverse_frequencies(rot, case["scaling"])
    angle = positions.to(torch.float64)[:, None, :, None] * f.to(x.device)
    cos, sin = (angle.cos() * mag).float(), (angle.sin() * (mag * sign)).float()
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((turned.to(x.dtype), x[..., rot:]), dim=-1)


def _plain_rope(s):
    c = s["case"]
    p = s["positions"]
    if p is None:
        p = torch.arange(c["N"], device=s["q"].device)[None]
    sign = 1.0 if c["dir"] == "fwd" else -1.0
    return _rotated(s["q"], p, c, sign), _rotated(s["k"], p, c, sign)


def _plain_append(s):
    c = s["case"]
    t = torch.arange(c["T"], device=s["q"].device)
    p = s["positions"]
    if p is None:
        p = s["cache_len"][:, None] + t
    q, k = _rotated(s["q"], p, c, 1.0), _rotated(s["k"], p, c, 1.0)
    slot = (s["cache_len"][:, None] + t).long()
    where = torch.gather(s["table"].long(), 1, (slot // c["page"]))
    row = slot % c["page"]
    if s["new_len"] is None:
        s["k_cache"][where, :, row] = k.transpose(1, 2)
        s["v_cache"][where, :, row] = s["v"].transpose(1, 2)
        return q, s["k_cache"], s["v_cache"]
    real = t < s["new_len"][:, None]
    s["k_cache"][where[real], :, row[real]] = k.transpose(1, 2)[real]
    s["v_cache"][where[real], :, row[real]] = s["v"].transpose(1, 2)[real]
    q = torch.where(real[:, None, :, None], q, s["q_out"])
    return q, s["k_cache"], s["v_cache"]


def _plain_paged(s):
    c = s["case"]
    B, H, Hk, T, d, page = (c[n] for n in ("B", "H", "Hk", "T", "d", "page"))
    keys = s["table"].shape[1] * page

    def gathered(cache):
        return cache[s["table"].long()].transpose(1, 2).reshape(B, Hk, keys, d).float()

    q = s["q"].float().reshape(B, Hk, (H // Hk) * T, d)
    scores = (q @ gathered(s["k_cache"]).transpose(-1, -2)) * d ** -0.5
    past = s["cache_len"].long()[:, None, None]
    new = s["new_len"].long() if s["new_len"] is not None else torch.full((B,), T, device=q.device)
    j = torch.arange(keys, device=q.device)[None, None, :] - past      # [B, 1, keys]
    t = torch.arange(T, device=q.device)[None, :, None]
    if s["tree"] is None:
        seen = j <= t
    else:
        at = j.clamp(0, T - 1).expand(B, T, keys)
        seen = (torch.gather(s["tree"], 2, at) != 0) | (j < 0)
    seen = seen & (j < new[:, None, None]) & (t < new[:, None, None])   # [B, T, keys]
    scores = scores.view(B, H, T, keys).masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True).clamp_min(-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.view(B, Hk, (H // Hk) * T, keys) @ gathered(s["v_cache"])).view(B, H, T, d)
    o = o / total.clamp_min(1e-30)
    lse = (top + total.log()).squeeze(-1)
    return o.to(s["q"].dtype), torch.where(total.squeeze(-1) > 0, lse, -math.inf)


# ------------------------------------------------------------------ definitions, 64 bits

def _turn64(x, angles, mag, layout):
    """Tokens [..., tokens, d] turned by `angles` [tokens, rot / 2]."""
    n = angles.shape[-1]
    x = x.double()
    out = x.clone()
    turn = torch.polar(torch.full_like(angles, mag), angles)
    if layout == "half":
        z = torch.complex(x[..., :n], x[..., n:2 * n]) * turn
        out[..., :n], out[..., n:2 * n] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :2 * n].reshape(*x.shape[:-1], n, 2).contiguous()) * turn
        out[..., :2 * n] = torch.view_as_real(z).flatten(-2)
    return out


def _angles64(case, positions):
    f, mag = _inverse_frequencies(case["rot"], case["scaling"])
    return positions.double()[..., None] * f.to(positions.device), mag


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "paged": _exact_paged}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    out = []
    for x in (s["q"], s["k"]):
        y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for b in range(c["B"]):
            p = torch.arange(c["N"], device=x.device) if s["positions"] is None else s["positions"][b]
            a, mag = _angles64(c, p)
            for h in range(x.shape[1]):
                y[b, h] = _turn64(x[b, h], a if c["dir"] == "fwd" else -a, mag, c["layout"])
        out.append(y)
    return tuple(out)


def _exact_append(s):
    c = s["case"]
    q, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    for b in range(c["B"]):
        past = int(s["cache_len"][b])
        n = c["T"] if s["new_len"] is None else int(s["new_len"][b])
        slots = torch.arange(past, past + n, device=q.device)
        p = slots if s["positions"] is None else s["positions"][b, :n]
        a, mag = _angles64(c, p)
        q[b, :, :n] = _turn64(s["q"][b, :, :n], a, mag, c["layout"])
        k = _turn64(s["k"][b, :, :n], a, mag, c["layout"])
        pages, rows = s["table"][b].long()[slots // c["page"]], slots % c["page"]
        for h in range(c["Hk"]):
            kc[pages, h, rows] = k[h]
            vc[pages, h, rows] = s["v"][b, h, :n].double()
    return q, kc, vc


def _exact_paged(s):
    c = s["case"]
    B, H, Hk, T, d = (c[n] for n in ("B", "H", "Hk", "T", "d"))
    dev = s["q"].device
    o = torch.zeros((B, H, T, d), dtype=torch.float64, device=dev)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        past = int(s["cache_len"][b])
        n = T if s["new_len"] is None else int(s["new_len"][b])
        slots = torch.arange(past + n, device=dev)
        pages, rows = s["table"][b].long()[slots // c["page"]], slots % c["page"]
        seen = torch.ones((n, past + n), dtype=torch.bool, device=dev)
        seen[:, past:] = (torch.ones((n, n), device=dev).tril() if s["tree"] is None
                          else s["tree"][b, :n, :n]) != 0
        for h in range(H):
            kv = h // (H // Hk)
            k, v = s["k_cache"][pages, kv, rows].double(), s["v_cache"][pages, kv, rows].double()
            z = (s["q"][b, h, :n].double() @ k.T) / math.sqrt(d)
            z = torch.where(seen, z, -math.inf)
            lse[b, h, :n] = torch.logsumexp(z, dim=-1)
            w = torch.softmax(z, dim=-1)
            o[b, h, :n] = torch.where(seen.any(-1, keepdim=True), w, 0.0) @ v
    return o, lse
