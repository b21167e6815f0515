"""The paged key/value cache's operators, as measured: rotary positions written
into the cache, attention of new tokens over it, and the page bookkeeping.

Three operators, each in a plain form (elementary torch operations in 32 bits)
and through the library's public binding:

  attn   w4v.paged_attn: every new token attends, causally, to its sequence's
         cached tokens (grouped heads, ragged batches, optional window);
  rope   w4v.rope_append: the new tokens' q and k are rotated by their
         positions, k and v written into the cache's pages;
  pages  w4v.kv_extend / kv_truncate / kv_fork / kv_compact: pages handed out,
         given back after rejected drafts, shared between sequences, moved down.
"""
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------- cases
def listed():
    """The listed cases; head layouts 20 x 128 are those of the 2560-wide target."""
    return [
        # one sequence, one new token, a short context: the smallest call, latency
        {"name": "attn_decode_b1", "op": "attn", "B": 1, "T": 1, "ragged": False, "ctx": 1000, "Hq": 20, "Hkv": 4,
         "D": 128, "page": 16, "window": 0, "lse": False},
        # the verify block of one sequence (K = 15) over a long context
        {"name": "attn_verify_b1_32k", "op": "attn", "B": 1, "T": 16, "ragged": False, "ctx": 32781, "Hq": 16,
         "Hkv": 4, "D": 256, "page": 16, "window": 0, "lse": False},
        # eight sequences' verify blocks (K = 20), contexts of 1/16 to all of 9000 tokens, full heads
        {"name": "attn_verify_b8", "op": "attn", "B": 8, "T": 21, "ragged": False, "ctx": 9000, "Hq": 20, "Hkv": 20,
         "D": 128, "page": 64, "window": 0, "lse": True},
        # many short requests with narrow heads, some without a new token, a sliding window
        {"name": "attn_window_b32", "op": "attn", "B": 32, "T": 40, "ragged": True, "ctx": 4001, "Hq": 20, "Hkv": 4,
         "D": 64, "page": 8, "window": 1000, "lse": False},
        # prompts taken in chunks of up to 1500 tokens over what is cached already
        {"name": "attn_chunk_b4", "op": "attn", "B": 4, "T": 1500, "ragged": True, "ctx": 12000, "Hq": 16, "Hkv": 4,
         "D": 256, "page": 128, "window": 0, "lse": False},
        # the long prompt in one piece: the largest
        {"name": "attn_prefill_8k", "op": "attn", "B": 1, "T": 8192, "ragged": False, "ctx": 8192, "Hq": 20,
         "Hkv": 20, "D": 128, "page": 64, "window": 0, "lse": False},
        # one verify block: latency
        {"name": "rope_verify_b1", "op": "rope", "B": 1, "T": 16, "ragged": False, "ctx": 5000, "Hq": 20, "Hkv": 4,
         "D": 128, "rot": 128, "page": 16, "inter": False, "scaling": "none", "fused": True},
        # interleaved pairs over part of the head, ragged batch of verify blocks
        {"name": "rope_inter_b37", "op": "rope", "B": 37, "T": 33, "ragged": True, "ctx": 3000, "Hq": 20, "Hkv": 20,
         "D": 128, "rot": 96, "page": 8, "inter": True, "scaling": "linear", "fused": False},
        # a long prompt's rows out of the fused projection, positions scaled for long contexts
        {"name": "rope_prefill_8k", "op": "rope", "B": 1, "T": 8192, "ragged": False, "ctx": 100000, "Hq": 16,
         "Hkv": 4, "D": 256, "rot": 64, "page": 64, "inter": False, "scaling": "yarn", "fused": True},
        # the bookkeeping of one verify step: pages for K + 1 tokens, the rejected ones given back
        {"name": "pages_step_b8", "op": "pages", "kind": "step", "B": 8, "ctx": 2000, "T": 16, "page": 16,
         "n_pages": 2048, "planes": 2, "Hkv": 4, "D": 128},
        # eight continuations of each of four prompts dropped and forked anew
        {"name": "pages_refork_4x8", "op": "pages", "kind": "refork", "B": 4, "C": 8, "ctx": 3000, "page": 64,
         "n_pages": 1024, "planes": 16, "Hkv": 4, "D": 128},
        # half of a fragmented cache's pages live: the upper ones moved down
        {"name": "pages_compact_4k", "op": "pages", "kind": "compact", "B": 64, "ctx": 700, "page": 16,
         "n_pages": 4096, "planes": 16, "Hkv": 4, "D": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "pages"])
    Hkv = rng.choice([1, 2, 4, 5, 8, 20])
    if op == "attn":
        g = rng.choice([1, 2, 3, 4, 5, 7, 8]) if Hkv < 20 else 1
        c = {"op": op, "B": _log(rng, 1, 32), "T": _log(rng, 1, 4096), "ragged": rng.random() < 0.5,
             "Hq": Hkv * g, "Hkv": Hkv, "D": rng.choice([64, 128, 256]), "page": rng.choice([8, 16, 32, 64, 128, 256]),
             "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)]), "lse": rng.random() < 0.3}
        c["ctx"] = c["T"] + _log(rng, 1, 32768)
        while c["B"] * c["Hq"] * c["T"] * c["ctx"] * c["D"] > 20 * 8192 * 8192 * 128 // 2 and c["T"] > 1:
            c["T"] = max(1, c["T"] // 2)
        while c["B"] * c["ctx"] * Hkv * c["D"] > 32 * 9000 * 4 * 256 and c["ctx"] > 2 * c["T"]:
            c["ctx"] = max(c["T"] + 1, c["ctx"] * 2 // 3)
        return c
    if op == "rope":
        D = rng.choice([64, 128, 256])
        c = {"op": op, "B": _log(rng, 1, 64), "T": _log(rng, 1, 8192), "ragged": rng.random() < 0.5,
             "Hq": Hkv * rng.choice([1, 2, 4, 7]) if Hkv < 20 else 20, "Hkv": Hkv, "D": D,
             "rot": rng.choice([D, D, D // 2, D // 4, D - 14]), "page": rng.choice([8, 16, 64, 256]),
             "inter": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
             "fused": rng.random() < 0.5}
        while c["B"] * c["T"] * (c["Hq"] + 2 * Hkv) * D > 8192 * 24 * 256:
            if c["B"] > c["T"]:
                c["B"] = max(1, c["B"] // 2)
            else:
                c["T"] = max(1, c["T"] // 2)
        c["ctx"] = c["T"] + _log(rng, 1, 100000 // c["B"])
        return c
    kind = rng.choice(["step", "refork", "compact"])
    page = rng.choice([8, 16, 32, 64])
    c = {"op": op, "kind": kind, "page": page, "planes": rng.choice([2, 4, 16]), "Hkv": rng.choice([1, 2, 4]), "D": 128}
    if kind == "step":
        c |= {"B": _log(rng, 1, 256), "T": rng.randint(1, 21), "ctx": _log(rng, 10, 4000)}
        c["n_pages"] = c["B"] * (-(-(c["ctx"] + c["T"]) // page) + 1) + rng.randint(1, 500)
    elif kind == "refork":
        c |= {"B": _log(rng, 1, 8), "C": rng.randint(1, 8), "ctx": _log(rng, 10, 4000)}
        c["n_pages"] = c["B"] * (-(-c["ctx"] // page) + c["C"]) + rng.randint(1, 300)
    else:
        c |= {"B": _log(rng, 2, 200), "ctx": _log(rng, 10, 2000)}
        c["n_pages"] = c["B"] * -(-c["ctx"] // page) + rng.randint(0, 300)
    while c["n_pages"] * page > 65536:
        c["B"], c["n_pages"] = max(1, c["B"] // 2), max(c["n_pages"] // 2, 1)
        if c["B"] == 1:
            c["ctx"] = max(10, c["ctx"] // 2)
    c["n_pages"] = max(c["n_pages"], c["B"] * (-(-(c["ctx"] + c.get("T", 0)) // page) + c.get("C", 1)) + 1)
    return c


# -------------------------------------------------------------------- inputs
def _batch(case):
    """New tokens and lengths (with the new tokens) of every sequence: from the
    case alone, so that the sizes do not change with the seed."""
    B, T, ctx = case["B"], case["T"], case["ctx"]
    r = np.random.default_rng([B, T, ctx])
    n = r.integers(0, T + 1, B) if case["ragged"] else np.full(B, T)
    n[0] = T
    full = np.full(B, ctx)
    if B > 1:
        full[1:] = np.round(ctx * 2.0 ** -r.uniform(0, 4, B - 1)).astype(np.int64)
    return n.astype(np.int64), np.maximum(full, n).astype(np.int64)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _half(shape, g, mul=1.0):
    """N(0, mul^2) in fp16."""
    x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(generator=g)
    return x.mul_(mul) if mul != 1.0 else x


def _tables(lens, page, n_pages, g, extra=0):
    """Pages of every sequence, drawn without order from the pool; -1 past the end."""
    need = -(-np.asarray(lens, np.int64) // page)
    width = max(1, int(need.max()) + extra)
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    nd = torch.as_tensor(need).cuda()
    at = (torch.cumsum(nd, 0) - nd)[:, None] + col[None, :]
    live = col[None, :] < nd[:, None]
    return torch.where(live, perm[torch.where(live, at, torch.zeros_like(at))], torch.full_like(at, -1, dtype=torch.int32))


_SCALING = {"none": None, "linear": ("linear", 4.0), "ntk": ("ntk", 4.0), "yarn": ("yarn", 8.0, 16384),
            "banded": ("banded", 8.0, 1.0, 4.0, 8192)}


def _frequencies(rot, scaling):
    """Angle a position adds to each pair, and what cos and sin are multiplied by (64 bits)."""
    base, i = 10000.0, np.arange(rot // 2, dtype=np.float64)
    kind = scaling[0] if scaling else "none"
    if kind == "ntk":
        base *= scaling[1] ** (rot / (rot - 2.0))
    f, m = base ** (-2.0 * i / rot), 1.0
    if kind == "linear":
        f = f / scaling[1]
    elif kind == "yarn":
        s, orig = scaling[1], scaling[2]
        turn = lambda b: rot * math.log(orig / (b * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f, m = f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    elif kind == "banded":
        s, low, high, orig = scaling[1:]
        turns = orig * f / (2 * math.pi)
        smooth = np.clip((turns - low) / (high - low), 0.0, 1.0)
        f = f / s * (1 - smooth) + f * smooth
    return f, m


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, g)
    n, lens = _batch(case)
    B, D, Hq, Hkv, page = case["B"], case["D"], case["Hq"], case["Hkv"], case["page"]
    n_pages = int((-(-lens // page)).sum()) + 7
    s = {"case": case, "lens": lens, "n": n, "n_max": int(n.max()), "len_max": int(lens.max()),
         "table": _tables(lens, page, n_pages, g), "lengths": _i32(lens),
         "offsets": _i32(np.concatenate([[0], np.cumsum(n)]))}
    tokens = int(n.sum())
    s["k_cache"] = _half((n_pages, Hkv, page, D), g)
    s["v_cache"] = _half((n_pages, Hkv, page, D), g)
    if case["op"] == "attn":
        s["q"] = _half((tokens, Hq, D), g, 1.5)      # logits of deviation 1.5: neither flat nor one-hot
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((tokens, Hq), dtype=torch.float32, device="cuda") if case["lse"] else None
        if own:
            from speculative_decoding_verify_w4a16_gb300 import w4v
            s["ws"] = w4v.workspace(w4v.paged_attn_workspace_bytes(tokens, B, Hq, Hkv, D, s["table"].shape[1] * page))
        return s
    if case["fused"]:                                # one projection's rows: q | k | v side by side
        qkv = _half((tokens, (Hq + 2 * Hkv) * D), g)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        s["q"], s["k"], s["v"] = (_half((tokens, h, D), g) for h in (Hq, Hkv, Hkv))
    s["q_out"] = torch.empty((tokens, Hq, D), dtype=torch.float16, device="cuda")
    scaling = _SCALING[case["scaling"]]
    f, m = _frequencies(case["rot"], scaling)
    turns = np.array([int(round(x / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64 for x in f], np.uint64)
    s["turns"], s["mul"] = torch.as_tensor(turns.view(np.int64)).cuda(), float(m)
    if own:
        from speculative_decoding_verify_w4a16_gb300 import w4v
        s["rope"] = w4v.Rope(case["rot"], interleaved=case["inter"], scaling=scaling)
    return s


def _prepare_pages(case, g):
    B, page, n_pages, kind = case["B"], case["page"], case["n_pages"], case["kind"]
    r = np.random.default_rng([B, page, case["ctx"]])
    C = case.get("C", 0)
    lens = r.integers(max(1, case["ctx"] // 2), case["ctx"] + 1, B)
    if kind == "compact":
        lens[r.random(B) < 0.3] = 0                  # requests that have ended
    T = case.get("T", 0)
    table = _tables(lens, page, n_pages, g, extra=-(-T // page) + 1)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    s = {"case": case, "refs": refs,
         "pool": _half((case["planes"], n_pages, case["Hkv"], page, case["D"]), g)}
    if kind == "refork":
        table = torch.cat([table, torch.full((B * C, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
        s["parents"] = _i32(np.repeat(np.arange(B), C))
        s["children"] = _i32(B + np.arange(B * C))
        s["dropped"] = _i32(np.concatenate([lens, np.zeros(B * C, np.int64)]))
        lens = np.concatenate([lens, np.zeros(B * C, np.int64)])
    s["table"], s["lengths"] = table, _i32(lens)
    if kind == "step":
        s["want"] = _i32(lens + T)
        s["kept"] = _i32(lens + r.integers(1, T + 1, B))
    if kind == "compact":
        s["refs_out"], s["table_out"] = torch.empty_like(refs), torch.empty_like(table)
    if own:
        from speculative_decoding_verify_w4a16_gb300 import w4v
        s["ws"] = w4v.workspace(w4v.kv_workspace_bytes(n_pages, table.shape[0]))
        s["short"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ----------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    return _own(s) if own else _plain_attn(s) if op == "attn" else _plain_rope(s) if op == "rope" else _plain_pages(s)


def _own(s):
    from speculative_decoding_verify_w4a16_gb300 import w4v
    c = s["case"]
    if c["op"] == "attn":
        w4v.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"],
                       window=c["window"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return [s["out"], s["lse"]]
    if c["op"] == "rope":
        w4v.rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"],
                        s["rope"], q_out=s["q_out"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if c["kind"] == "step":
        w4v.kv_extend(s["pool"], s["refs"], s["table"], s["lengths"], s["want"], short=s["short"], ws=s["ws"])
        w4v.kv_truncate(s["refs"], s["table"], s["lengths"], s["kept"], c["page"])
        return [s["refs"], s["table"], s["lengths"]]
    if c["kind"] == "refork":
        w4v.kv_truncate(s["refs"], s["table"], s["lengths"], s["dropped"], c["page"])
        w4v.kv_fork(s["pool"], s["refs"], s["table"], s["lengths"], s["parents"], s["children"], short=s["short"],
                    ws=s["ws"])
        return [s["refs"], s["table"], s["lengths"], s["pool"]]
    w4v.kv_compact(s["pool"], s["refs"], s["table"], s["lengths"], refs_out=s["refs_out"],
                   table_out=s["table_out"], ws=s["ws"])
    return [s["refs_out"], s["table_out"], s["pool"]]


def _plain_attn(s):
    """The whole padded batch at once: scores, masked softmax, product, in 32 bits."""
    c, n_max = s["case"], s["n_max"]
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    g, L = Hq // Hkv, s["table"].shape[1] * page
    pages = s["table"].clamp(min=0).long()
    key = torch.arange(L, device="cuda")
    held = key < s["lengths"][:, None]                                      # [B, L]
    k = s["k_cache"][pages].transpose(1, 2).reshape(B, Hkv, L, D).float()
    v = s["v_cache"][pages].transpose(1, 2).reshape(B, Hkv, L, D).float()
    v = torch.where(held[:, None, :, None], v, torch.zeros((), device="cuda"))
    i = torch.arange(n_max, device="cuda")
    n = s["offsets"][1:] - s["offsets"][:-1]
    new = i < n[:, None]                                                    # [B, n_max]
    row = torch.where(new, s["offsets"][:-1, None] + i, 0).long()
    pos = s["lengths"][:, None] - n[:, None] + i
    q = s["q"].float()[row].reshape(B, n_max, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n_max * g, D)
    x = (q @ k.transpose(2, 3) * D ** -0.5).reshape(B, Hkv, n_max, g, L)
    seen = held[:, None, :] & (key <= pos[:, :, None])
    if c["window"]:
        seen &= key > pos[:, :, None] - c["window"]
    x = torch.where(seen[:, None, :, None, :], x, torch.full((), -math.inf, device="cuda"))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = x.sum(-1, keepdim=True)
    o = (x.reshape(B, Hkv, n_max * g, L) @ v).reshape(B, Hkv, n_max, g, D) / torch.where(total == 0, 1.0, total)
    s["out"][row[new]] = o.permute(0, 2, 1, 3, 4).reshape(B, n_max, Hq, D)[new].half()
    if s["lse"] is not None:
        lse = (top + torch.log(total))[..., 0]
        s["lse"][row[new]] = lse.permute(0, 2, 1, 3).reshape(B, n_max, Hq)[new]
    return [s["out"], s["lse"]]


def _plain_rope(s):
    c = s["case"]
    rot, page, Hkv = c["rot"], c["page"], c["Hkv"]
    token = torch.arange(s["q"].shape[0], device="cuda")
    b = (token[:, None] >= s["offsets"][None, 1:]).sum(1)
    pos = (s["lengths"][b] - s["offsets"][b + 1] + token).long()
    part = (pos[:, None] * s["turns"] >> 32).float() * (2 * math.pi / 2.0 ** 32)   # the angle past whole turns
    cos, sin = torch.cos(part)[:, None] * s["mul"], torch.sin(part)[:, None] * s["mul"]

    def turned(x):
        y = x.float()
        a, z = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        u, w = a * cos - z * sin, z * cos + a * sin
        u = torch.stack((u, w), -1).flatten(-2) if c["inter"] else torch.cat((u, w), -1)
        return torch.cat((u, y[..., rot:]), -1).half()

    s["q_out"].copy_(turned(s["q"]))
    at = s["table"][b, pos // page].long()
    s["k_cache"][at, :, pos % page] = turned(s["k"])
    s["v_cache"][at, :, pos % page] = s["v"]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _count(lengths, page):
    return torch.div(lengths + (page - 1), page, rounding_mode="floor")


def _plain_truncate(s, keep, page):
    col = torch.arange(s["table"].shape[1], device="cuda")
    have, left = _count(s["lengths"], page), _count(torch.minimum(keep, s["lengths"]), page)
    gone = (col >= left[:, None]) & (col < have[:, None])
    s["refs"].index_add_(0, s["table"][gone].long(), torch.full((), -1, dtype=torch.int32, device="cuda").expand(int(gone.sum())))
    s["table"][gone] = -1
    torch.minimum(keep, s["lengths"], out=s["lengths"])


def _plain_pages(s):
    c = s["case"]
    page = c["page"]
    col = torch.arange(s["table"].shape[1], device="cuda")
    if c["kind"] == "step":                          # no page is shared here, so nothing is copied
        fresh = (col >= _count(s["lengths"], page)[:, None]) & (col < _count(s["want"], page)[:, None])
        free = torch.nonzero(s["refs"] == 0)[:, 0][:int(fresh.sum())]
        s["table"][fresh] = free.to(torch.int32)
        s["refs"][free] = 1
        torch.maximum(s["want"], s["lengths"], out=s["lengths"])
        _plain_truncate(s, s["kept"], page)
        return [s["refs"], s["table"], s["lengths"]]
    if c["kind"] == "refork":
        _plain_truncate(s, s["dropped"], page)
        p, ch = s["parents"].long(), s["children"].long()
        lens = s["lengths"][p]
        whole, part = torch.div(lens, page, rounding_mode="floor"), lens % page != 0
        rows = torch.where(col < whole[:, None], s["table"][p], -1)
        shared = rows[rows >= 0].long()
        s["refs"].index_add_(0, shared, torch.ones((), dtype=torch.int32, device="cuda").expand(shared.numel()))
        free = torch.nonzero(s["refs"] == 0)[:, 0][:int(part.sum())]
        src = s["table"][p[part], whole[part].long()].long()
        rows[part, whole[part].long()] = free.to(torch.int32)
        s["refs"][free] = 1
        s["table"][ch] = rows
        s["lengths"][ch] = lens
        s["pool"][:, free] = s["pool"][:, src]
        return [s["refs"], s["table"], s["lengths"], s["pool"]]
    live = s["refs"] > 0
    count = int(live.sum())
    src = torch.nonzero(live[count:])[:, 0] + count
    dst = torch.nonzero(~live[:count])[:, 0]
    to = torch.arange(c["n_pages"], dtype=torch.int32, device="cuda")
    to[src] = dst.to(torch.int32)
    held = col < _count(s["lengths"], page)[:, None]
    s["table_out"].copy_(torch.where(held, to[s["table"].clamp(min=0).long()], s["table"]))
    s["refs_out"].copy_(s["refs"])
    s["refs_out"][dst] = s["refs"][src]
    s["refs_out"][src] = 0
    s["pool"][:, dst] = s["pool"][:, src]
    return [s["refs_out"], s["table_out"], s["pool"]]


# ---------------------------------------------------------------------- work
def _visible(case):
    """Per sequence: (cached tokens that any new token sees, visible pairs)."""
    n, lens = _batch(case)
    w = case["window"] or int(lens.max()) + 1
    tokens = np.where(n > 0, np.minimum(lens, w + n - 1), 0)
    pairs = [int(np.minimum(np.arange(l - m, l) + 1, w).sum()) for m, l in zip(n, lens)]
    return int(tokens.sum()), sum(pairs)


def work(case):
    if case["op"] == "attn":
        n = int(_batch(case)[0].sum())
        tokens, pairs = _visible(case)
        D, Hq = case["D"], case["Hq"]
        return {"bytes": 4 * D * (tokens * case["Hkv"] + n * Hq) + (4 * n * Hq if case["lse"] else 0),
                "flops": 4 * D * Hq * pairs}
    if case["op"] == "rope":
        n = int(_batch(case)[0].sum())
        return {"bytes": 4 * n * (case["Hq"] + 2 * case["Hkv"]) * case["D"],
                "flops": 3 * n * (case["Hq"] + case["Hkv"]) * case["rot"]}
    page = case["planes"] * case["Hkv"] * case["page"] * case["D"] * 2
    r = np.random.default_rng([case["B"], case["page"], case["ctx"]])
    lens = r.integers(max(1, case["ctx"] // 2), case["ctx"] + 1, case["B"])
    if case["kind"] == "step":
        return {"bytes": 4 * (case["n_pages"] + 6 * case["B"]), "flops": 0}
    if case["kind"] == "refork":
        copies = case["C"] * int((lens % case["page"] != 0).sum())
        shared = case["C"] * int((lens // case["page"]).sum())
        return {"bytes": 2 * copies * page + 4 * (case["n_pages"] + 4 * shared), "flops": 0}
    lens[r.random(case["B"]) < 0.3] = 0
    live = int((-(-lens // case["page"])).sum())
    moved = live * (case["n_pages"] - live) // case["n_pages"]          # pages lie without order: the expected count
    return {"bytes": 2 * moved * page + 4 * (2 * case["n_pages"] + 2 * live), "flops": 0}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"] == "pages":
        return None                                  # whole numbers and copies
    s = prepare(case, seed)
    n, lens = s["n"], s["lens"]
    D, Hq, Hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "attn":
        g, first = Hq // Hkv, 0
        out = torch.zeros((int(n.sum()), Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((int(n.sum()), Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            m, length = int(n[b]), int(lens[b])
            if m == 0:
                continue
            at = torch.arange(length, device="cuda")
            page_of = s["table"][b].long()[at // page]
            where = torch.arange(length - m, length, device="cuda")
            for h in range(Hq):
                K = s["k_cache"][page_of, h // g, at % page].double()
                V = s["v_cache"][page_of, h // g, at % page].double()
                logit = s["q"][first:first + m, h].double().mm(K.t()) / math.sqrt(D)
                hidden = at[None, :] > where[:, None]
                if case["window"]:
                    hidden |= at[None, :] <= where[:, None] - case["window"]
                logit.masked_fill_(hidden, -math.inf)
                lse[first:first + m, h] = torch.logsumexp(logit, 1)
                out[first:first + m, h] = torch.softmax(logit, 1).mm(V)
            first += m
        return [out.cpu().numpy(), lse.cpu().numpy() if case["lse"] else None]
    rot, half = case["rot"], case["rot"] // 2
    f, mul = _frequencies(rot, _SCALING[case["scaling"]])
    pos = np.concatenate([np.arange(length - m, length) for m, length in zip(n, lens)])
    seq = np.repeat(np.arange(case["B"]), n)
    angle = np.mod(pos[:, None] * f[None, :], 2 * math.pi)
    rotor = torch.as_tensor(mul * np.exp(1j * angle)).cuda()[:, None, :]

    def spin(x):
        y = x.double().clone()
        lo = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
        hi = lo + (1 if case["inter"] else half)
        z = torch.complex(y[..., lo], y[..., hi]) * rotor
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    k = s["k_cache"].double()
    pt, bt = torch.as_tensor(pos).cuda(), torch.as_tensor(seq).cuda()
    k[s["table"][bt, pt // page].long(), :, pt % page] = spin(s["k"])
    return [spin(s["q"]).cpu().numpy(), k.cpu().numpy(), None]
