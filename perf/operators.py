"""Cases of the paged-cache operators: appending rotated keys to a paged cache, decode attention over it with a
sliding window and a few first tokens that stay visible, and decode attention for a batch with a shared prefix.

Three kinds of call, in the order a serving step makes them:

* ``append``  new tokens' key rows go to their places in the pages, the position rotation applied on the way, and
  the same tokens' queries are rotated (latent cache in bf16 or E4M3, or keys and values of grouped kv heads);
* ``window``  every query token attends to the keys of its sequence at positions up to its own, within the window
  or among the first tokens (window 0: all of them), read through a block table (the same three caches);
* ``prefix``  all sequences of the batch attend to one shared prefix and each to its own further keys.

``run`` computes them with elementary torch operations in 32 bits where ``own`` is false and makes the calls of
this repository's package where it is true; ``exact`` gives the same results in 64 bits.
"""
import math
import random

import torch

own = False

D_QK, D_V, D_ROPE, D_HEAD = 576, 512, 64, 128
MAX_POSITIONS = 40960


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a busy server: one new token a sequence, 128 query heads to rotate
        {"name": "append, one token for each of 64", "op": "append", "kind": "mla", "B": 64, "new": 1, "spread": 1,
         "H": 128, "Hkv": 1, "past": 4096, "page": 64, "interleaved": True},
        # a prefill batch of prompts of very different lengths, the first ones after cached turns
        {"name": "append, ragged prompts", "op": "append", "kind": "mla", "B": 9, "new": 3600, "spread": 30, "H": 16,
         "Hkv": 1, "past": 1500, "page": 64, "interleaved": True},
        # chunked prefill into a cache of E4M3 codes, small pages
        {"name": "append, E4M3 chunks", "op": "append", "kind": "mla_fp8", "B": 8, "new": 1021, "spread": 1, "H": 16,
         "Hkv": 1, "past": 900, "page": 16, "interleaved": False},
        # grouped kv heads: keys rotated, values copied, mixed chunks and single tokens
        {"name": "append, keys and values", "op": "append", "kind": "mha", "B": 33, "new": 250, "spread": 50, "H": 32,
         "Hkv": 8, "past": 1200, "page": 16, "interleaved": False},
        # the smallest call, where latency counts
        {"name": "window, one short sequence", "op": "window", "kind": "mla", "B": 1, "Sq": 1, "H": 16, "Hkv": 1,
         "L_lo": 700, "L_hi": 700, "page": 16, "window": 128, "first": 4, "sinks": False},
        # long chats, a window of 4096 and 4 first tokens
        {"name": "window, 64 long sequences", "op": "window", "kind": "mla", "B": 64, "Sq": 1, "H": 128, "Hkv": 1,
         "L_lo": 1000, "L_hi": 32768, "page": 64, "window": 4096, "first": 4, "sinks": False},
        # E4M3 pages, two query tokens a sequence (a drafted one), few heads a GPU
        {"name": "window, E4M3, two tokens", "op": "window", "kind": "mla_fp8", "B": 132, "Sq": 2, "H": 16, "Hkv": 1,
         "L_lo": 1, "L_hi": 8192, "page": 64, "window": 2048, "first": 16, "sinks": True},
        # grouped kv heads with sink logits
        {"name": "window, grouped heads", "op": "window", "kind": "mha", "B": 64, "Sq": 1, "H": 32, "Hkv": 8,
         "L_lo": 1000, "L_hi": 8192, "page": 32, "window": 4095, "first": 100, "sinks": True},
        # no window: the whole paged cache of a mixed batch
        {"name": "window 0, mixed lengths", "op": "window", "kind": "mla", "B": 64, "Sq": 1, "H": 128, "Hkv": 1,
         "L_lo": 1024, "L_hi": 8192, "page": 64, "window": 0, "first": 0, "sinks": False},
        # a few agents on one system prompt
        {"name": "prefix, 8 short sequences", "op": "prefix", "kind": "mla", "B": 8, "Sq": 1, "H": 16, "Hkv": 1,
         "P": 2000, "L_lo": 1, "L_hi": 300, "page": 64, "sinks": False},
        # many samples of one prompt
        {"name": "prefix, 64 sequences", "op": "prefix", "kind": "mla", "B": 64, "Sq": 1, "H": 128, "Hkv": 1,
         "P": 8192, "L_lo": 1, "L_hi": 1024, "page": 64, "sinks": False},
        # a long document, two query tokens a sequence, few heads a GPU
        {"name": "prefix, long document, 16 heads", "op": "prefix", "kind": "mla", "B": 132, "Sq": 2, "H": 16,
         "Hkv": 1, "P": 16384, "L_lo": 2, "L_hi": 2048, "page": 128, "sinks": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["append", "window", "window", "prefix"])
    page = rng.choice([16, 32, 64, 64, 128, 192, 256])
    if op == "append":
        kind = rng.choice(["mla", "mla_fp8", "mha"])
        H, Hkv = (rng.choice([16, 32, 64, 128]), 1) if kind != "mha" else rng.choice([(8, 8), (16, 2), (32, 8), (7, 7)])
        tokens = _spread(rng, 1, 4000)
        B = min(tokens, _spread(rng, 1, 128))
        return {"op": op, "kind": kind, "B": B, "new": max(1, tokens // B), "spread": rng.choice([1, 10]), "H": H,
                "Hkv": Hkv, "past": _spread(rng, 1, 2000), "page": page, "interleaved": rng.random() < 0.5}
    if op == "window":
        kind = rng.choice(["mla", "mla", "mla_fp8", "mha"])
        if kind != "mha":
            H, Hkv, Sq = rng.choice([16, 32, 64, 128]), 1, rng.choice([1, 1, 2, 3])
        else:
            (H, Hkv), Sq = rng.choice([(8, 8), (16, 2), (32, 8), (24, 3)]), rng.choice([1, 1, 2])
        B, window, L = _spread(rng, 1, 96), rng.choice([0, _spread(rng, 1, 4096)]), _spread(rng, 1, 16384)
        if window == 0:  # the whole cache: a cost below the largest listed case's
            L = max(1, min(L, 200000 // (B * Sq)))
        return {"op": op, "kind": kind, "B": B, "Sq": Sq, "H": H, "Hkv": Hkv, "L_lo": rng.randint(0, L), "L_hi": L,
                "page": page, "window": window, "first": rng.choice([0, 1, 4, 77]) if window else 0,
                "sinks": rng.random() < 0.5}
    H, Sq, B = rng.choice([16, 32, 64, 128]), rng.choice([1, 1, 2]), _spread(rng, 1, 96)
    P = max(1, min(_spread(rng, 1, 16384), 60000000 // (B * Sq * H)))
    L = max(1, min(_spread(rng, 1, 2000), 60000 // (B * Sq)))
    return {"op": op, "kind": "mla", "B": B, "Sq": Sq, "H": H, "Hkv": 1, "P": P, "L_lo": rng.randint(0, L),
            "L_hi": L, "page": page, "sinks": rng.random() < 0.5}


def _plan_lengths(case):
    """Lengths are part of the case: the same for every seed.  (lengths, new tokens of each sequence)"""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] != "append":
        lengths = [rng.randint(case["L_lo"], case["L_hi"]) for _ in range(case["B"] - 1)]
        return [case["L_hi"], *lengths], [case["Sq"]] * case["B"]  # one sequence is as long as the plan allows
    new = [max(1, _spread(rng, max(1, case["new"] // case["spread"]), case["new"])) for _ in range(case["B"])]
    return [rng.randint(0, case["past"]) + n for n in new], new


# ---------------------------------------------------------------- inputs

def _table(lengths, page, gen, spare=3):
    """Pages in random order: (block table [B, most], number of pages).  Entries past a sequence's pages are -1."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def _rotation(dim, base=10000.0):
    """cos and sin of every position's angles, in 64 bits before they are rounded: [positions, dim / 2 + dim / 2]."""
    inv = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    angle = torch.arange(MAX_POSITIONS, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    lengths, new = _plan_lengths(case)
    B, H, Hkv, page = case["B"], case["H"], case["Hkv"], case["page"]

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    def cache(pages):
        if case["kind"] == "mha":
            return {"k_pages": normal(pages, page, Hkv, D_HEAD), "v_pages": normal(pages, page, Hkv, D_HEAD)}
        kv = normal(pages, page, D_QK)
        return {"kv_pages": kv.float().mul_(60.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
                if case["kind"] == "mla_fp8" else kv}

    s = {"case": case, "seqlens": torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    if case["op"] == "append":
        T = sum(new)
        s["table"], pages = _table(lengths, page, gen)
        s.update(cache(pages))
        s["cu_tokens"] = torch.tensor([0] + [sum(new[:i + 1]) for i in range(B)], dtype=torch.int32, device="cuda")
        if case["kind"] == "mha":
            s["rotation"] = _rotation(D_HEAD)
            s.update(k=normal(T, Hkv, D_HEAD), v=normal(T, Hkv, D_HEAD), q_in=normal(T, H, D_HEAD),
                     q=torch.empty(T, H, D_HEAD, dtype=torch.bfloat16, device="cuda"))
        else:
            s["rotation"] = _rotation(D_ROPE)
            # the latent and the key's rotated part are two slices of one projection's rows
            row = normal(T, D_QK)
            s.update(latent=row[:, :D_V], k_rope=row[:, D_V:], q_rope=normal(T, H, D_ROPE), q=normal(T, H, D_QK),
                     kv_scale=1.0 / 60.0)
        return s

    Sq, D = case["Sq"], D_HEAD if case["kind"] == "mha" else D_QK
    s["table"], pages = _table(lengths, page, gen)
    if case["op"] == "prefix":
        at = -(-case["P"] // page)
        s["prefix_table"] = torch.arange(pages, pages + at, dtype=torch.int32, device="cuda").flip(0).contiguous()
        s["prefix_len"] = torch.tensor([case["P"]], dtype=torch.int32, device="cuda")
        pages += at
    s.update(cache(pages))
    if case["kind"] == "mla_fp8":
        s["kv_scale"] = float(torch.tensor(1.0 / 60.0, dtype=torch.float32))
    s["q"] = normal(B, Sq, H, D)
    s["scale"] = float(torch.tensor(D ** -0.5, dtype=torch.float32))
    s["sinks"] = normal(H, dtype=torch.float32) if case["sinks"] else None
    s["out"] = torch.empty(B, Sq, H, D_HEAD if case["kind"] == "mha" else D_V, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(B, Sq, H, dtype=torch.float32, device="cuda")
    if own:
        import mla_decode_attention_11_b200 as M
        L_max = max(1, case["L_hi"])
        if case["op"] == "prefix":
            s["plan"] = M.mla_decode_plan_prefix(B, Sq, H, L_max, case["P"], page)
        elif case["kind"] == "mha":
            s["plan"] = M.mha_decode_plan_paged(B, Sq, H, Hkv, L_max, page, window=case["window"],
                                                first_tokens=case["first"])
        else:
            make = M.mla_decode_plan_paged_fp8 if case["kind"] == "mla_fp8" else M.mla_decode_plan_paged
            s["plan"] = make(B, Sq, H, L_max, page, window=case["window"], first_tokens=case["first"])
        s["workspace"] = M.alloc_workspace(s["plan"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    return _append(s) if op == "append" else _window(s) if op == "window" else _prefix(s)


def _run_own(s):
    import mla_decode_attention_11_b200 as M
    case = s["case"]
    if case["op"] == "append" and case["kind"] == "mha":
        M.mha_cache_append(s["k"], s["v"], s["rotation"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"],
                           cu_tokens=s["cu_tokens"], q_in=s["q_in"], q_out=s["q"], interleaved=case["interleaved"])
        return s["k_pages"], s["v_pages"], s["q"]
    if case["op"] == "append":
        M.mla_cache_append(s["latent"], s["k_rope"], s["rotation"], s["kv_pages"], s["table"], s["seqlens"],
                           cu_tokens=s["cu_tokens"], q_rope=s["q_rope"], q=s["q"],
                           kv_scale=s["kv_scale"] if case["kind"] == "mla_fp8" else None,
                           interleaved=case["interleaved"])
        return s["kv_pages"], s["q"]
    if case["op"] == "prefix":
        M.mla_decode_run_prefix(s["plan"], s["q"], s["kv_pages"], s["prefix_table"], s["prefix_len"], s["table"],
                                s["seqlens"], s["scale"], s["out"], s["lse"], s["workspace"], sinks=s["sinks"])
    elif case["kind"] == "mha":
        M.mha_decode_run_paged(s["plan"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"], s["scale"],
                               s["out"], s["lse"], s["workspace"], sinks=s["sinks"])
    elif case["kind"] == "mla_fp8":
        M.mla_decode_run_paged_fp8(s["plan"], s["q"], s["kv_pages"], s["kv_scale"], s["table"], s["seqlens"], s["scale"],
                                   s["out"], s["lse"], s["workspace"], sinks=s["sinks"])
    else:
        M.mla_decode_run_paged(s["plan"], s["q"], s["kv_pages"], s["table"], s["seqlens"], s["scale"], s["out"],
                               s["lse"], s["workspace"], sinks=s["sinks"])
    return s["out"], s["lse"]


def _rotated(x, cos, sin, interleaved):
    """x [..., 2 n] in 32 bits turned by the angles of cos, sin [..., n]."""
    n = cos.shape[-1]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _append(s):
    case, page = s["case"], s["case"]["page"]
    token = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu_tokens"][1:].long(), token, right=True)
    pos = s["seqlens"].long()[seq] - s["cu_tokens"].long()[seq + 1] + token
    place = s["table"].long()[seq, pos // page] * page + pos % page
    cos, sin = s["rotation"][pos].chunk(2, dim=1)
    turn = (cos[:, None], sin[:, None], case["interleaved"])
    if case["kind"] == "mha":
        s["k_pages"].flatten(0, 1)[place] = _rotated(s["k"].float(), *turn).bfloat16()
        s["v_pages"].flatten(0, 1)[place] = s["v"]
        s["q"].copy_(_rotated(s["q_in"].float(), *turn).bfloat16())
        return s["k_pages"], s["v_pages"], s["q"]
    row = torch.cat([s["latent"].float(), _rotated(s["k_rope"].float(), cos, sin, case["interleaved"])], dim=1)
    if case["kind"] == "mla_fp8":
        scale = torch.tensor(s["kv_scale"], dtype=torch.float32, device="cuda")
        codes = (row / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["kv_pages"].view(torch.uint8).flatten(0, 1)[place] = codes.view(torch.uint8)
    else:
        s["kv_pages"].flatten(0, 1)[place] = row.bfloat16()
    s["q"][..., D_V:] = _rotated(s["q_rope"].float(), *turn).bfloat16()
    return s["kv_pages"], s["q"]


def _attend(scores, values, sinks):
    """Softmax over the last axis of masked scores [B, Hkv, rows, keys] (and a sink logit a row), times values
    [B, Hkv, keys, D], and the scores' log-sum-exp; a row with nothing to see gives 0 and its sink (-inf: none)."""
    top = scores.amax(-1, keepdim=True)
    if sinks is not None:
        top = torch.maximum(top, sinks)
    base = torch.where(top == -math.inf, 0.0, top)
    weight = torch.exp(scores - base)
    total = weight.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - base)
    o = torch.matmul(weight, values) / torch.where(total == 0, 1.0, total)
    return o, (base + torch.log(total)).squeeze(-1)


def _sequence_rows(s, pos):
    """fp32 keys and values [B, Hkv, n, D] of the positions pos [B, n] (any, where they are not of the sequence)."""
    case, page = s["case"], s["case"]["page"]
    p = pos.clamp(0, s["table"].shape[1] * page - 1)
    place = torch.gather(s["table"].long(), 1, p // page).clamp_min(0) * page + p % page
    if case["kind"] == "mha":
        return (s["k_pages"].flatten(0, 1)[place].transpose(1, 2).float(),
                s["v_pages"].flatten(0, 1)[place].transpose(1, 2).float())
    if case["kind"] == "mla_fp8":
        codes = s["kv_pages"].view(torch.uint8).flatten(0, 1)[place]
        kv = (codes.view(torch.float8_e4m3fn).float() * s["kv_scale"])[:, None]
    else:
        kv = s["kv_pages"].flatten(0, 1)[place].float()[:, None]
    return kv, kv[..., :D_V]


def _rows(s):
    """Queries as [B, Hkv, rows of the kv head, D] in 32 bits, and each row's token."""
    B, Sq, H, D = s["q"].shape
    Hkv = s["case"]["Hkv"]
    q = s["q"].float().view(B, Sq, Hkv, H // Hkv, D).transpose(1, 2).reshape(B, Hkv, Sq * (H // Hkv), D)
    return q, torch.arange(Sq, device="cuda").repeat_interleave(H // Hkv)


def _sink_rows(s):
    B, Sq, H, _ = s["q"].shape
    Hkv = s["case"]["Hkv"]
    return None if s["sinks"] is None else s["sinks"].view(1, Hkv, 1, H // Hkv).expand(B, Hkv, Sq, H // Hkv).reshape(
        B, Hkv, Sq * (H // Hkv), 1)


def _written(s, o, lse):
    B, Sq, H, _ = s["q"].shape
    Hkv = s["case"]["Hkv"]
    s["out"].copy_(o.view(B, Hkv, Sq, H // Hkv, -1).transpose(1, 2).reshape(s["out"].shape))
    s["lse"].copy_(lse.view(B, Hkv, Sq, H // Hkv).transpose(1, 2).reshape(s["lse"].shape))
    return s["out"], s["lse"]


def _window(s):
    case = s["case"]
    Sq, window, first = case["Sq"], case["window"], case["first"]
    L = s["seqlens"].long()[:, None]
    if window and first + window + Sq - 1 < case["L_hi"]:
        # only the positions that some token can see: the first ones, then the last window + Sq - 1
        at = torch.arange(window + Sq - 1, device="cuda")[None] + L - (window + Sq - 1)
        lead = torch.arange(first, device="cuda")[None].expand(L.shape[0], first)
        pos = torch.cat([torch.where(lead < L, lead, -1), torch.where(at >= first, at, -1)], dim=1)
    else:
        pos = torch.arange(max(1, case["L_hi"]), device="cuda")[None].expand(L.shape[0], -1)
    k, v = _sequence_rows(s, pos)
    q, token = _rows(s)
    own_pos = (L - Sq)[:, :, None] + token[None, :, None]
    j = pos[:, None, :]
    sees = (j >= 0) & (j <= own_pos)
    if window:
        sees = sees & ((j > own_pos - window) | (j < first))
    scores = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    scores = torch.where(sees[:, None], scores, -math.inf)
    used = sees.any(1)[:, None, :, None]
    return _written(s, *_attend(scores, torch.where(used, v, 0.0), _sink_rows(s)))


def _prefix(s):
    case, page, P = s["case"], s["case"]["page"], s["case"]["P"]
    at = torch.arange(P, device="cuda")
    shared = s["kv_pages"].flatten(0, 1)[s["prefix_table"].long()[at // page] * page + at % page].float()
    L = s["seqlens"].long()[:, None]
    pos = torch.arange(max(1, case["L_hi"]), device="cuda")[None].expand(L.shape[0], -1)
    k, v = _sequence_rows(s, pos)
    q, token = _rows(s)
    sees = pos[:, None, :] <= (L - case["Sq"])[:, :, None] + token[None, :, None]
    mine = torch.where(sees[:, None], torch.matmul(q, k.transpose(-1, -2)) * s["scale"], -math.inf)
    v = torch.where(sees.any(1)[:, None, :, None], v, 0.0)
    theirs = torch.matmul(q, shared.t()) * s["scale"]
    sinks = _sink_rows(s)
    top = torch.maximum(theirs.amax(-1, keepdim=True), mine.amax(-1, keepdim=True))
    if sinks is not None:
        top = torch.maximum(top, sinks)
    a, b = torch.exp(theirs - top), torch.exp(mine - top)
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - top)
    o = (torch.matmul(a, shared[:, :D_V]) + torch.matmul(b, v)) / total
    return _written(s, o, (top + torch.log(total)).squeeze(-1))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    lengths, new = _plan_lengths(case)
    B, H, Hkv = case["B"], case["H"], case["Hkv"]
    if case["op"] == "append":
        T = sum(new)
        if case["kind"] == "mha":
            return {"bytes": T * (Hkv * D_HEAD * 8 + H * D_HEAD * 4 + 4 * D_HEAD) + 12 * B,
                    "flops": T * (H + Hkv) * D_HEAD * 3}
        out = D_QK * (1 if case["kind"] == "mla_fp8" else 2)
        return {"bytes": T * (D_QK * 2 + out + H * D_ROPE * 4 + 4 * D_ROPE) + 12 * B, "flops": T * (H + 1) * D_ROPE * 3}
    Sq = case["Sq"]
    window, first = case.get("window", 0), case.get("first", 0)
    keys = pairs = 0
    for L in lengths:
        lo = max(0, L - Sq + 1 - window) if window else 0
        keys += L - lo + min(first, lo, L) if L else 0
        for t in range(Sq):
            p = L - Sq + t
            if p >= 0:
                lo = max(0, p + 1 - window) if window else 0
                pairs += p + 1 - lo + min(first, lo)
    if case["op"] == "prefix":
        keys += case["P"]
        pairs += B * Sq * case["P"]
    rows, pages = B * Sq * H, keys // case["page"] + B
    key, value = ((Hkv * D_HEAD * 4, D_HEAD) if case["kind"] == "mha" else
                  (D_QK if case["kind"] == "mla_fp8" else D_QK * 2, D_V))
    width = D_HEAD if case["kind"] == "mha" else D_QK
    return {"bytes": keys * key + rows * (2 * width + 2 * value + 4) + 4 * pages + 4 * B,
            "flops": pairs * H * 2 * (width + value)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lengths, new = _plan_lengths(case)
    page, table = case["page"], s["table"].tolist()

    def turned(x, p):
        """x [..., 2 n] as n complex numbers times exp(i angle) of position p."""
        x = x.double()
        c = s["rotation"][p].double()
        n = c.shape[0] // 2
        z = torch.complex(x[..., 0::2], x[..., 1::2]) if case["interleaved"] else torch.complex(x[..., :n], x[..., n:])
        z = torch.view_as_real(z * torch.complex(c[:n], c[n:]))
        return z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)

    if case["op"] == "append":
        if sum(new) > 20000:
            return None  # one token at a time takes too long
        names = ("k_pages", "v_pages") if case["kind"] == "mha" else ("kv_pages",)
        caches = [s[n].double() for n in names]
        q = s["q"].double()
        i = 0
        for b, n in enumerate(new):
            for p in range(lengths[b] - n, lengths[b]):
                at = (table[b][p // page], p % page)
                if case["kind"] == "mha":
                    caches[0][at], caches[1][at] = turned(s["k"][i], p), s["v"][i].double()
                    q[i] = turned(s["q_in"][i], p)
                else:
                    row = torch.cat([s["latent"][i].double(), turned(s["k_rope"][i], p)])
                    caches[0][at] = row / s["kv_scale"] if case["kind"] == "mla_fp8" else row
                    q[i, :, D_V:] = turned(s["q_rope"][i], p)
                i += 1
        if case["kind"] == "mla_fp8":
            caches[0].clamp_(-448, 448)
        return (*caches, q)

    B, Sq, H, _ = s["q"].shape
    Hkv = case["Hkv"]
    outs = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lses = torch.empty(B, Sq, H, dtype=torch.float64, device="cuda")
    keys = [s[n].flatten(0, 1) for n in (("k_pages", "v_pages") if case["kind"] == "mha" else ("kv_pages", "kv_pages"))]
    at = [e * page + r for e in s["prefix_table"].tolist() for r in range(page)][:case["P"]] if "P" in case else []
    shared = None if case["op"] != "prefix" else keys[0][torch.tensor(at, dtype=torch.long, device="cuda")].double()
    for b, L in enumerate(lengths):
        rows = [table[b][p // page] * page + p % page for p in range(L)]
        rows = torch.tensor(rows, dtype=torch.long, device="cuda")
        if case["kind"] == "mla_fp8":
            k = v = keys[0].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double() * s["kv_scale"]
        else:
            k, v = (x[rows].double() for x in keys)
        if case["kind"] != "mha":
            k, v = k[:, None], v[:, None, :D_V]
            if case["op"] == "prefix":
                k, v = torch.cat([shared[:, None], k]), torch.cat([shared[:, None, :D_V], v])
        for t in range(Sq):
            p, w = L - Sq + t, case.get("window", 0)
            sees = set(range(max(0, p + 1 - w) if w else 0, p + 1)) | set(range(min(case.get("first", 0), p + 1)))
            see = torch.tensor([*range(len(at)), *(len(at) + j for j in sorted(sees))], dtype=torch.long, device="cuda")
            for g in range(Hkv):
                heads = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
                x = s["q"][b, t, heads].double() @ k[see, g].t() * s["scale"]
                if s["sinks"] is not None:
                    x = torch.cat([x, s["sinks"][heads].double()[:, None]], dim=1)
                if x.shape[1] == 0:
                    lses[b, t, heads] = -math.inf
                    continue
                lses[b, t, heads] = torch.logsumexp(x, dim=1)
                outs[b, t, heads] = torch.softmax(x, dim=1)[:, :len(see)] @ v[see, g]
    return outs, lses
