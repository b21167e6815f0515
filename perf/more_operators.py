"""What several continuations of one prompt need next to the paged cache, as measured.

Four operators, each in a plain form (elementary torch operations in 32 bits) and
through the library's public binding:

  norm     w4v.norm_rope_append: every head's q and k divided by its root mean
           square and weighted, rotated by its position, k and v into the pages;
  sinks    w4v.paged_attn(window=, sinks=): a sliding window, and a few first
           tokens that stay visible;
  shared   w4v.paged_attn_shared: attention of sequences that share a long
           prefix, whose keys are read once for all of them;
  logprob  w4v.token_logprobs: log probabilities of given tokens, the rows'
           entropy and their most likely tokens.
"""
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------- cases
def listed():
    """The listed cases; 20 x 128 heads and 151936 tokens are those of the 2560-wide target."""
    return [
        # one verify block (K = 15): the smallest call, latency
        {"name": "norm_verify_b1", "op": "norm", "B": 1, "T": 16, "ragged": False, "ctx": 5000, "Hq": 20, "Hkv": 4,
         "D": 128, "rot": 128, "page": 16, "inter": False, "scaling": "none", "fused": True, "centred": False},
        # a ragged batch of verify blocks, interleaved pairs over part of the head, weights around zero
        {"name": "norm_inter_b40", "op": "norm", "B": 40, "T": 33, "ragged": True, "ctx": 3100, "Hq": 20, "Hkv": 20,
         "D": 128, "rot": 96, "page": 8, "inter": True, "scaling": "linear", "fused": False, "centred": True},
        # a long prompt's rows out of the fused projection, a quarter of each wide head rotated
        {"name": "norm_prefill_8k", "op": "norm", "B": 1, "T": 8192, "ragged": False, "ctx": 90000, "Hq": 16,
         "Hkv": 4, "D": 256, "rot": 64, "page": 64, "inter": False, "scaling": "yarn", "fused": True, "centred": True},
        # one token of one long conversation: only the window and four first tokens are read
        {"name": "sinks_decode_b1", "op": "sinks", "B": 1, "T": 1, "ragged": False, "ctx": 20000, "Hq": 20, "Hkv": 4,
         "D": 128, "page": 16, "window": 1000, "sinks": 4, "lse": False},
        # verify blocks (K = 20) of many requests over a few hundred first tokens (the system's prompt) and the window
        {"name": "sinks_verify_b24", "op": "sinks", "B": 24, "T": 21, "ragged": True, "ctx": 12000, "Hq": 16, "Hkv": 4,
         "D": 256, "page": 64, "window": 2000, "sinks": 300, "lse": True},
        # the long prompt in one piece
        {"name": "sinks_prefill_8k", "op": "sinks", "B": 1, "T": 8192, "ragged": False, "ctx": 8192, "Hq": 20,
         "Hkv": 20, "D": 128, "page": 64, "window": 1024, "sinks": 64, "lse": False},
        # eight continuations of one short prompt, a token each: latency
        {"name": "shared_decode_1x8", "op": "shared", "G": 1, "C": 8, "T": 1, "ragged": False, "prefix": 2000,
         "tail": 100, "Hq": 20, "Hkv": 4, "D": 128, "page": 16, "lse": False},
        # verify blocks (K = 15) of sixteen continuations of each of two prompts
        {"name": "shared_verify_2x16", "op": "shared", "G": 2, "C": 16, "T": 16, "ragged": True, "prefix": 8200,
         "tail": 700, "Hq": 20, "Hkv": 4, "D": 128, "page": 16, "lse": True},
        # sixty-four samples of a long document's answer
        {"name": "shared_decode_1x64", "op": "shared", "G": 1, "C": 64, "T": 1, "ragged": False, "prefix": 32781,
         "tail": 900, "Hq": 16, "Hkv": 4, "D": 256, "page": 64, "lse": False},
        # one decoded token's log probability: latency
        {"name": "logprob_row", "op": "logprob", "M": 1, "V": 151936, "half": False, "n": 1, "top": 0, "heat": 1.0,
         "masked": False},
        # candidates of a constrained batch: fp16 logits of an odd vocabulary, much of it masked, twenty alternatives
        {"name": "logprob_masked_300", "op": "logprob", "M": 300, "V": 50001, "half": True, "n": 4, "top": 20,
         "heat": 0.8, "masked": True},
        # a prompt scored token by token, five alternatives each: the largest
        {"name": "logprob_prompt_2k", "op": "logprob", "M": 2048, "V": 151936, "half": False, "n": 1, "top": 5,
         "heat": 1.0, "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "sinks", "shared", "logprob"])
    if op == "logprob":
        c = {"op": op, "M": _log(rng, 1, 2048), "V": rng.choice([_log(rng, 100, 200000), 151936, 1024, 32000]),
             "half": rng.random() < 0.5, "n": rng.choice([1, 1, 2, 16]), "top": rng.choice([0, 1, 5, 20, 32]),
             "heat": rng.choice([1.0, round(rng.uniform(0.3, 2.0), 2)]), "masked": rng.random() < 0.4}
        while c["M"] * c["V"] > 2048 * 151936:
            c["M"] //= 2
        return c
    Hkv = rng.choice([1, 2, 4, 5, 8, 20])
    if op == "norm":
        D = rng.choice([64, 128, 256])
        c = {"op": op, "B": _log(rng, 1, 64), "T": _log(rng, 1, 8192), "ragged": rng.random() < 0.5,
             "Hq": Hkv * rng.choice([1, 2, 4, 7]) if Hkv < 20 else 20, "Hkv": Hkv, "D": D,
             "rot": rng.choice([D, D, D // 2, D // 4, D - 14]), "page": rng.choice([8, 16, 64, 256]),
             "inter": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
             "fused": rng.random() < 0.5, "centred": rng.random() < 0.5}
        while c["B"] * c["T"] * (c["Hq"] + 2 * Hkv) * D > 8192 * 24 * 256:
            if c["B"] > c["T"]:
                c["B"] = max(1, c["B"] // 2)
            else:
                c["T"] = max(1, c["T"] // 2)
        c["ctx"] = c["T"] + _log(rng, 1, 100000 // c["B"])
        return c
    g = rng.choice([1, 2, 3, 4, 5, 7, 8]) if Hkv < 20 else 1
    c = {"op": op, "T": _log(rng, 1, 4096 if op == "sinks" else 64), "ragged": rng.random() < 0.5, "Hq": Hkv * g,
         "Hkv": Hkv, "D": rng.choice([64, 128, 256]), "page": rng.choice([8, 16, 32, 64, 128, 256]),
         "lse": rng.random() < 0.3}
    if op == "sinks":
        c |= {"B": _log(rng, 1, 32), "window": _log(rng, 16, 4096), "sinks": _log(rng, 1, 600)}
        c["ctx"] = c["T"] + _log(rng, 1, 32768)
        while c["B"] * c["Hq"] * c["T"] * c["ctx"] * c["D"] > 20 * 8192 * 8192 * 128 // 2 and c["T"] > 1:
            c["T"] = max(1, c["T"] // 2)
        while c["B"] * c["ctx"] * Hkv * c["D"] > 32 * 9000 * 4 * 256 and c["ctx"] > 2 * c["T"]:
            c["ctx"] = max(c["T"] + 1, c["ctx"] * 2 // 3)
        return c
    c |= {"G": _log(rng, 1, 6), "C": _log(rng, 1, 64), "prefix": _log(rng, 1, 32768), "tail": _log(rng, 1, 2000)}
    while c["G"] * c["C"] * c["T"] * c["Hq"] * c["D"] * (c["prefix"] + c["tail"]) > 64 * 16 * 256 * 33700 * 4 and c["T"] > 1:
        c["T"] //= 2
    while c["G"] * c["C"] * (c["prefix"] + c["tail"] + c["T"]) * Hkv * c["D"] > 64 * 33700 * 4 * 256:
        if c["C"] > 2:
            c["C"] //= 2
        else:
            c["prefix"] = max(1, c["prefix"] // 2)
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


def _groups(case):
    """The same of G prompts with C continuations each, and the prompts' lengths."""
    G, C, T = case["G"], case["C"], case["T"]
    r = np.random.default_rng([G, C, T, case["prefix"]])
    n = r.integers(0, T + 1, G * C) if case["ragged"] else np.full(G * C, T)
    n[0] = T
    prefix = np.full(G, case["prefix"])
    prefix[1:] = np.maximum(1, np.round(case["prefix"] * 2.0 ** -r.uniform(0, 2, G - 1)))
    lens = np.repeat(prefix, C) + r.integers(0, case["tail"] + 1, G * C) + n
    return n.astype(np.int64), lens.astype(np.int64), prefix.astype(np.int64)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _half(shape, g, mul=1.0):
    """N(0, mul^2) in fp16."""
    x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(generator=g)
    return x.mul_(mul) if mul != 1.0 else x


def _tables(lens, page, n_pages, g):
    """Pages of every sequence, drawn without order from the pool; -1 past the end."""
    need = -(-np.asarray(lens, np.int64) // page)
    perm = torch.randperm(n_pages, generator=g, device="cuda").cpu().numpy()
    table, at = np.full((len(need), max(1, int(need.max()))), -1, np.int32), 0
    for b, c in enumerate(need):
        table[b, :c] = perm[at:at + c]
        at += c
    return table


def _forked_tables(lens, prefix, C, page, n_pages, g):
    """The same where the members of a group share the whole pages of its prefix."""
    need = -(-lens // page)
    perm = torch.randperm(n_pages, generator=g, device="cuda").cpu().numpy()
    table, at = np.full((len(need), max(1, int(need.max()))), -1, np.int32), 0
    for b, c in enumerate(need):
        s = int(prefix[b // C]) // page if b % C else 0
        table[b, :s] = table[b - b % C, :s]
        table[b, s:c] = perm[at:at + c - s]
        at += c - s
    return table


_SCALING = {"none": None, "linear": ("linear", 4.0), "ntk": ("ntk", 4.0), "yarn": ("yarn", 8.0, 16384),
            "banded": ("banded", 8.0, 1.0, 4.0, 8192)}
_EPS = 1e-6


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
    if case["op"] == "logprob":
        return _prepare_logits(case, g)
    D, Hq, Hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "shared":
        n, lens, prefix = _groups(case)
        C, own_pages = case["C"], -(-lens // page)
        own_pages = own_pages - np.where(np.arange(len(n)) % C, np.repeat(prefix, C) // page, 0)
        n_pages = int(own_pages.sum()) + 7
        table = _forked_tables(lens, prefix, C, page, n_pages, g)
    else:
        n, lens = _batch(case)
        n_pages = int((-(-lens // page)).sum()) + 7
        table = _tables(lens, page, n_pages, g)
    tokens = int(n.sum())
    s = {"case": case, "lens": lens, "n": n, "n_max": int(n.max()), "host_table": table, "table": _i32(table),
         "lengths": _i32(lens), "offsets": _i32(np.concatenate([[0], np.cumsum(n)]))}
    s["k_cache"] = _half((n_pages, Hkv, page, D), g)
    s["v_cache"] = _half((n_pages, Hkv, page, D), g)
    if case["op"] == "norm":
        return _prepare_norm(case, s, tokens, g)
    if case["op"] == "shared":
        s["groups"], s["prefix"] = _i32(np.arange(case["G"] + 1) * C), _i32(prefix)
        for b in range(len(n)):                      # a prefix ends inside a page: every member has its own copy
            p = int(prefix[b // C])
            if b % C and p % page:
                for cache in (s["k_cache"], s["v_cache"]):
                    cache[int(table[b, p // page]), :, :p % page] = cache[int(table[b - b % C, p // page]), :, :p % page]
    s["q"] = _half((tokens, Hq, D), g, 1.5)          # logits of deviation 1.5: neither flat nor one-hot
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((tokens, Hq), dtype=torch.float32, device="cuda") if case["lse"] else None
    if own:
        from speculative_decoding_verify_w4a16_gb300 import w4v
        if case["op"] == "shared":
            s["ws"] = w4v.workspace(w4v.paged_attn_shared_workspace_bytes(tokens, len(n), case["G"], Hq, Hkv, D))
        else:
            s["ws"] = w4v.workspace(w4v.paged_attn_workspace_bytes(tokens, len(n), Hq, Hkv, D, table.shape[1] * page))
    return s


def _prepare_norm(case, s, tokens, g):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["fused"]:                                # one projection's rows: q | k | v side by side
        qkv = _half((tokens, (Hq + 2 * Hkv) * D), g, 2.0)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        s["q"], s["k"], s["v"] = (_half((tokens, h, D), g, 2.0) for h in (Hq, Hkv, Hkv))
    s["q_weight"], s["k_weight"] = (_half((D,), g, 0.2) + (0.0 if case["centred"] else 1.0) for _ in range(2))
    s["q_out"] = torch.empty((tokens, Hq, D), dtype=torch.float16, device="cuda")
    scaling = _SCALING[case["scaling"]]
    f, m = _frequencies(case["rot"], scaling)
    turns = np.array([int(round(x / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64 for x in f], np.uint64)
    s["turns"], s["mul"] = torch.as_tensor(turns.view(np.int64)).cuda(), float(m)
    if own:
        from speculative_decoding_verify_w4a16_gb300 import w4v
        s["rope"] = w4v.Rope(case["rot"], interleaved=case["inter"], scaling=scaling)
        s["norm"] = w4v.HeadNorm(s["q_weight"], s["k_weight"], eps=_EPS, zero_centred=case["centred"])
    return s


def _prepare_logits(case, g):
    """Logits of deviation 2, in every other row with a few tokens that stand out; where masked, what a
    grammar forbids is -inf: a third of a row, and in every fourth row all but three tokens."""
    M, V, n = case["M"], case["V"], case["n"]
    x = torch.empty((M, V), dtype=torch.float16 if case["half"] else torch.float32, device="cuda").normal_(generator=g)
    x.mul_(2.0)
    high = (torch.randint(0, V, (M, 1), generator=g, device="cuda") + torch.arange(3, device="cuda") * (V // 3)) % V
    rise = torch.tensor([9.0, 7.0, 6.0], device="cuda") * (torch.arange(M, device="cuda") % 2)[:, None]
    x.scatter_(1, high, x.gather(1, high) + rise.to(x.dtype))
    tokens = torch.randint(0, V, (M, n), generator=g, device="cuda").to(torch.int32)
    tokens[:, 0] = torch.where(torch.rand(M, generator=g, device="cuda") < 0.7, high[:, 0].to(torch.int32), tokens[:, 0])
    if n > 1:
        tokens[:, n - 1] = -1                        # the sentinel of a draft that was shorter
    if case["masked"]:
        few = (torch.arange(M, device="cuda") % 4 == 3)[:, None]
        hide = (torch.rand((M, V), generator=g, device="cuda") < 1 / 3) | few
        hide.scatter_(1, high, False)
        x.masked_fill_(hide, -math.inf)
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    return {"case": case, "x": x, "tokens": tokens,
            "out": (torch.empty((M, n), **f32), torch.empty(M, **f32), torch.empty((M, case["top"]), **i32),
                    torch.empty((M, case["top"]), **f32))}


# ----------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    return _plain_norm(s) if op == "norm" else _plain_logprobs(s) if op == "logprob" else _plain_attn(s)


def _own(s):
    from speculative_decoding_verify_w4a16_gb300 import w4v
    c = s["case"]
    if c["op"] == "norm":
        w4v.norm_rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                             s["offsets"], s["rope"], s["norm"], q_out=s["q_out"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if c["op"] == "sinks":
        w4v.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"],
                       window=c["window"], sinks=c["sinks"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return [s["out"], s["lse"]]
    if c["op"] == "shared":
        w4v.paged_attn_shared(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"],
                              s["groups"], s["prefix"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return [s["out"], s["lse"]]
    return list(w4v.token_logprobs(s["x"], s["tokens"], top=c["top"], temperature=c["heat"], out=s["out"]))


def _plain_attn(s):
    """The whole padded batch at once: scores, masked softmax, product, in 32 bits."""
    c, n_max = s["case"], s["n_max"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    B, g, L = s["table"].shape[0], Hq // Hkv, s["table"].shape[1] * page
    pages = s["table"].clamp(min=0).long()
    key = torch.arange(L, device="cuda")
    held = key < s["lengths"][:, None]                                      # [B, L]
    k = s["k_cache"][pages].transpose(1, 2).reshape(B, Hkv, L, D).float()
    v = s["v_cache"][pages].transpose(1, 2).reshape(B, Hkv, L, D).float()
    i = torch.arange(n_max, device="cuda")
    n = s["offsets"][1:] - s["offsets"][:-1]
    new = i < n[:, None]                                                    # [B, n_max]
    row = torch.where(new, s["offsets"][:-1, None] + i, 0).long()
    pos = s["lengths"][:, None] - n[:, None] + i
    q = s["q"].float()[row].reshape(B, n_max, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n_max * g, D)
    x = (q @ k.transpose(2, 3) * D ** -0.5).reshape(B, Hkv, n_max, g, L)
    seen = held[:, None, :] & (key <= pos[:, :, None])
    if c["op"] == "sinks":
        seen &= (key > pos[:, :, None] - c["window"]) | (key < c["sinks"])
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


def _plain_norm(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    token = torch.arange(s["q"].shape[0], device="cuda")
    b = (token[:, None] >= s["offsets"][None, 1:]).sum(1)
    pos = (s["lengths"][b] - s["offsets"][b + 1] + token).long()
    part = (pos[:, None] * s["turns"] >> 32).float() * (2 * math.pi / 2.0 ** 32)   # the angle past whole turns
    cos, sin = torch.cos(part)[:, None] * s["mul"], torch.sin(part)[:, None] * s["mul"]

    def turned(x, weight):
        y = x.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + _EPS) * (weight.float() + (1.0 if c["centred"] else 0.0))
        a, z = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        u, w = a * cos - z * sin, z * cos + a * sin
        u = torch.stack((u, w), -1).flatten(-2) if c["inter"] else torch.cat((u, w), -1)
        return torch.cat((u, y[..., rot:]), -1).half()

    s["q_out"].copy_(turned(s["q"], s["q_weight"]))
    at = s["table"][b, pos // page].long()
    s["k_cache"][at, :, pos % page] = turned(s["k"], s["k_weight"])
    s["v_cache"][at, :, pos % page] = s["v"]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _plain_logprobs(s):
    c = s["case"]
    z = s["x"].float()
    top = z.amax(1, keepdim=True)
    d = (z - top) / c["heat"]
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total - torch.where(e == 0, 0.0, e * d).sum(1, keepdim=True) / total
    at = s["tokens"].long()
    given = torch.where(at >= 0, d.gather(1, at.clamp(min=0)) - log_total, -math.inf)
    k = c["top"]
    ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k] if k else at[:, :0]     # ties: the lower index
    return [given, entropy[:, 0], ids.to(torch.int32), d.gather(1, ids) - log_total]


# ---------------------------------------------------------------------- work
def _visible(case):
    """Per sequence: (cached tokens that any new token sees, visible pairs) of a window with first tokens."""
    n, lens = _batch(case)
    w, s, keys, pairs = case["window"], case["sinks"], 0, 0
    for m, length in zip(n, lens):
        pos = np.arange(length - m, length)
        lo = np.maximum(pos - w + 1, 0)
        pairs += int((pos - lo + 1 + np.minimum(s, lo)).sum())
        if m:
            keys += int(length - lo[0] + min(s, lo[0]))
    return keys, pairs


def work(case):
    if case["op"] == "logprob":
        M, V = case["M"], case["V"]
        return {"bytes": M * V * (2 if case["half"] else 4) + M * (8 * case["n"] + 4 + 8 * case["top"]), "flops": 6 * M * V}
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "norm":
        n = int(_batch(case)[0].sum())
        return {"bytes": 4 * n * (Hq + 2 * Hkv) * D + 4 * D, "flops": n * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    if case["op"] == "sinks":
        n = int(_batch(case)[0].sum())
        keys, pairs = _visible(case)
    else:
        new, lens, prefix = _groups(case)
        n = int(new.sum())
        live = np.repeat(prefix, case["C"]) * (new > 0)
        keys = int(((lens - live) * (new > 0)).sum() + live.reshape(case["G"], -1).max(1).sum())
        pairs = int((new * lens - new * (new - 1) // 2).sum())
    return {"bytes": 4 * D * (keys * Hkv + n * Hq) + (4 * n * Hq if case["lse"] else 0), "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprob":
        return _exact_logprobs(case, s)
    n, lens, table = s["n"], s["lens"], s["host_table"]
    D, Hq, Hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    if case["op"] != "norm":
        first, g = 0, Hq // Hkv
        out = torch.zeros((int(n.sum()), Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((int(n.sum()), Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(len(n)):
            m, length = int(n[b]), int(lens[b])
            if m == 0:
                continue
            at = torch.arange(length, device="cuda")
            page_of = torch.as_tensor(table[b].astype(np.int64)).cuda()[at // page]
            where = torch.arange(length - m, length, device="cuda")
            hidden = at[None, :] > where[:, None]
            if case["op"] == "sinks":
                hidden |= (at[None, :] <= where[:, None] - case["window"]) & (at[None, :] >= case["sinks"])
            for h in range(Hq):
                K = s["k_cache"][page_of, h // g, at % page].double()
                V = s["v_cache"][page_of, h // g, at % page].double()
                logit = s["q"][first:first + m, h].double().mm(K.t()) / math.sqrt(D)
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

    def spin(x, weight):
        y = x.double()
        y = y * torch.rsqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / D + _EPS)
        y *= weight.double() + float(case["centred"])
        lo = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
        hi = lo + (1 if case["inter"] else half)
        z = torch.complex(y[..., lo], y[..., hi]) * rotor
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    k = s["k_cache"].double()
    pt, bt = torch.as_tensor(pos).cuda(), torch.as_tensor(seq).cuda()
    k[s["table"][bt, pt // page].long(), :, pt % page] = spin(s["k"], s["k_weight"])
    return [spin(s["q"], s["q_weight"]).cpu().numpy(), k.cpu().numpy(), None]


def _exact_logprobs(case, s):
    M, V = case["M"], case["V"]
    given, entropy, best = np.zeros((M, case["n"])), np.zeros(M), np.zeros((M, case["top"]))
    for r in range(0, M, 256):                       # some rows at a time
        p = torch.log_softmax(s["x"][r:r + 256].double() / case["heat"], 1)
        t = s["tokens"][r:r + 256].cpu().numpy()
        entropy[r:r + 256] = torch.special.entr(p.exp()).sum(1).cpu().numpy()
        at = torch.as_tensor(np.where(t < 0, 0, t).astype(np.int64)).cuda()
        given[r:r + 256] = np.where(t < 0, -np.inf, torch.take_along_dim(p, at, 1).cpu().numpy())
        if case["top"]:
            best[r:r + 256] = torch.topk(p, case["top"], 1)[0].cpu().numpy()
    return [given, entropy, None, best]
