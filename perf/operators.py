"""The cases on which the grouped-head attention operators are measured: `paged_append` (keys and values into a paged cache,
rotated on the way), `paged_decode_attn` (one new token over the paged cache) and `prompt_attn` (packed causal prompts).

`run` computes each in plain torch operations in 32 bits, or, with `own` set, by the library's calls."""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of eight sequences: the write of a single token each, where launch latency is all
        dict(name="append_b8", op="append", lens="1,1,1,1,1,1,1,1", starts="8100,4500,17,0,6143,2049,511,7777", H=32, HK=8,
             d=128, page=16, pages=512, rot=128, pairs=False, act="bf16", cache="bf16", fused=False),
        # a packed batch of prompts straight out of a fused q/k/v projection (strided rows), one of them a later chunk
        dict(name="append_8k", op="append", lens="4096,2731,1000,365", starts="0,0,4096,0", H=32, HK=8, d=128, page=16,
             pages=512, rot=128, pairs=False, act="bf16", cache="bf16", fused=True),
        # a prompt into an FP8 cache, half of the dims rotated, in neighbouring pairs
        dict(name="append_2k_fp8", op="append", lens="1531,517", starts="0,0", H=16, HK=4, d=128, page=64, pages=24, rot=64,
             pairs=True, act="bf16", cache="fp8", fused=False),
        # one user's short chat: the smallest decode, latency
        dict(name="decode_b1_1k", op="decode", lens="1001", H=32, HK=8, d=128, page=16, window=0, sink=False, act="bf16", cache="bf16"),
        # a busy server: 32 sequences of mixed length, small pages
        dict(name="decode_b32_8k", op="decode", lens=",".join(str(250 * i + 3 * i * i + 1) for i in range(1, 33)), H=32, HK=8, d=128,
             page=16, window=0, sink=False, act="bf16", cache="bf16"),
        # few long documents at this library's decode context of 131,072
        dict(name="decode_b4_128k", op="decode", lens="131072,131001,100000,65537", H=64, HK=8, d=128, page=64, window=0, sink=True,
             act="bf16", cache="bf16"),
        # long contexts in an FP8 cache
        dict(name="decode_b16_32k_fp8", op="decode", lens=",".join(str(32768 - 517 * i) for i in range(16)), H=32, HK=8, d=128, page=64,
             window=0, sink=False, act="bf16", cache="fp8"),
        # full precision, the window of 128 tokens and the sink of this library's window layer
        dict(name="decode_b8_f32", op="decode", lens="5000,4097,900,128,127,60,2,1", H=8, HK=8, d=64, page=16, window=128, sink=True,
             act="f32", cache="f32"),
        # a handful of very short prompts: latency
        dict(name="prompt_short", op="prompt", lens="1,17,64,200", H=8, HK=2, d=64, window=0, sink=False, act="bf16"),
        # a packed batch of mixed prompts with sinks, strided rows
        dict(name="prompt_mixed_8k", op="prompt", lens="37,2048,511,1,1300,96,2600,129,640,777", H=32, HK=8, d=128, window=0, sink=True, act="bf16"),
        # one long prompt: the largest
        dict(name="prompt_16k", op="prompt", lens="16384", H=32, HK=8, d=128, window=0, sink=False, act="bf16"),
        # this library's full-precision prompt: 1024 tokens, 8 heads of 64
        dict(name="prompt_1k_f32", op="prompt", lens="1024", H=8, HK=8, d=64, window=0, sink=False, act="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "prompt", "prompt", "prompt"])
    act = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 256]) if op != "prompt" or act == "bf16" else rng.choice([64, 128])
    HK = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    while HK * G > 64:
        G = rng.choice([1, 2, 3, 4])
    c = dict(op=op, H=HK * G, HK=HK, d=d, act=act)
    if op == "append":
        n = rng.randint(1, 12)
        one = rng.random() < 0.4
        lens = [1] * n if one else [_spread(rng, 1, 2000) for _ in range(n)]
        starts = [_spread(rng, 1, 6000) - 1 for _ in range(n)]
        page = rng.choice([8, 16, 32, 64])
        cache = rng.choice(["bf16", "fp8"]) if act == "bf16" else "f32"
        c.update(lens=",".join(map(str, lens)), starts=",".join(map(str, starts)), page=page,
                 pages=max(-(-(a + b) // page) for a, b in zip(lens, starts)) + rng.randint(0, 3),
                 rot=rng.choice([0, d // 2, d]), pairs=rng.random() < 0.5, cache=cache, fused=rng.random() < 0.5)
        return c
    c.update(window=rng.choice([0, 0, 0, 128, _spread(rng, 1, 5000)]), sink=rng.random() < 0.5)
    if op == "decode":
        n = _spread(rng, 1, 48)
        top = _spread(rng, 16, min(131072, 2 ** 29 // (n * HK * d) if act == "bf16" else 2 ** 25 // (n * HK * d)) + 17)
        lens = [_spread(rng, 1, top) for _ in range(n - 1)] + [top]
        c.update(lens=",".join(map(str, lens)), page=rng.choice([8, 16, 32, 64, 100]),
                 cache=rng.choice(["bf16", "fp8"]) if act == "bf16" else "f32")
        return c
    n = _spread(rng, 1, 16)
    # the scores of the padded batch stay within 2^32 values (2^29 in full precision, where the products are slow)
    top = _spread(rng, 20, int(math.sqrt(2 ** (32 if act == "bf16" else 29) / (n * HK * G))))
    lens = [_spread(rng, 1, top) for _ in range(n - 1)] + [top]
    c.update(lens=",".join(map(str, lens)))
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _visible(n, W):
    """Keys that a query with n keys up to its own sees."""
    return min(n, W) if W else n


def _row(c, fmt):
    return c["d"] * {"bf16": 2, "f32": 4, "fp8": 1}[fmt] + (c["d"] // 16 if fmt == "fp8" else 0)


def work(case):
    c = case
    lens, b = _ints(c["lens"]), 2 if c["act"] == "bf16" else 4
    H, HK, d = c["H"], c["HK"], c["d"]
    n = sum(lens)
    if c["op"] == "append":
        data = n * (2 * H + 3 * HK) * d * b + 2 * n * HK * _row(c, c["cache"])
        return {"bytes": data, "flops": 3 * n * (H + HK) * c["rot"]}
    W = c["window"]
    if c["op"] == "decode":
        seen = sum(_visible(m, W) for m in lens)
        pages = sum(-(-_visible(m, W) // c["page"]) for m in lens)
        return {"bytes": 2 * seen * HK * _row(c, c["cache"]) + 2 * len(lens) * H * d * b + 4 * pages, "flops": 4 * H * d * seen}
    pairs = sum(m * (m + 1) // 2 if not W or m <= W else W * (W + 1) // 2 + (m - W) * W for m in lens)
    return {"bytes": n * (2 * H + 2 * HK) * d * b, "flops": 4 * H * d * pairs}


def _quantize(x):
    """Rows in 64-channel groups: E4M3 codes (their bytes) and the groups' scales."""
    g = x.float().unflatten(-1, (-1, 64))
    top = g.abs().amax(-1)
    s = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return (g / s[..., None]).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8), s


def _values(codes, scales):
    return (codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 64)) * scales[..., None]).flatten(-2)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    dev, act = "cuda", TYPES[c["act"]]
    H, HK, d, lens = c["H"], c["HK"], c["d"], _ints(c["lens"])
    n, total = len(lens), sum(lens)
    s = dict(c)
    s["scale"] = d ** -0.5

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def tensor(v, t):
        return torch.tensor(v, dtype=t, device=dev)

    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    if c["op"] in ("append", "prompt"):
        if c.get("fused", True):  # q, k and v as the rows of one projection's output
            qkv = normal(total, (H + 2 * HK) * d).to(act)
            s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in qkv.split([H * d, HK * d, HK * d], 1))
        else:
            s["q"], s["k"], s["v"] = normal(total, H, d).to(act), normal(total, HK, d).to(act), normal(total, HK, d).to(act)
        s["cu"] = tensor(cu, torch.int32)
    if c["op"] == "prompt":
        s["sinks"] = normal(H) if c["sink"] else None
        s["out"] = torch.zeros(total, H, d, dtype=act, device=dev)
        s["longest"] = max(lens)
        if own:
            K, p = _params(c)
            s["p"], s["ws"] = p, torch.empty(K.gqa_workspace_size(p, K.OP_PROMPT_ATTN, n, total, 0), dtype=torch.uint8, device=dev)
        return s
    page = c["page"]
    if c["op"] == "append":
        per = c["pages"]
        s["pos0"] = tensor(_ints(c["starts"]), torch.int64)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / max(c["rot"], 1))
        s["q_out"] = torch.zeros(total, H, d, dtype=act, device=dev)
        s["k_out"] = torch.zeros(total, HK, d, dtype=act, device=dev)
    else:
        per = -(-max(lens) // page)
        s["q"] = normal(n, H, d).to(act)
        s["q_pos"] = tensor(lens, torch.int64) - 1
        s["sinks"] = normal(H) if c["sink"] else None
        s["out"] = torch.zeros(n, H, d, dtype=act, device=dev)
    held = [per if c["op"] == "append" else -(-m // page) for m in lens]
    pool = sum(held)
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((n, per), -1, dtype=torch.int32)  # pages a sequence does not hold yet
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        at += h
    s["table"] = table.to(dev)
    for name in ("k_cache", "v_cache"):
        if c["op"] == "append" and c["cache"] == "fp8":
            s[name] = torch.zeros(pool, HK, page, d, dtype=torch.uint8, device=dev)
            s[name + "_scales"] = torch.ones(pool, HK, page, d // 64, device=dev)
            continue
        x = normal(pool, HK, page, d)
        if c["cache"] == "fp8":
            s[name], s[name + "_scales"] = _quantize(x)
        else:
            s[name] = x.to(TYPES[c["cache"]])
        del x
    if own:
        K, p = _params(c)
        fmt = p.cache_fmt
        s["p"] = p
        s["stored"] = [K.Stored(fmt, s[k], s.get(k + "_scales")) for k in ("k_cache", "v_cache")]
        if c["op"] == "decode":
            s["ws"] = torch.empty(K.gqa_workspace_size(p, K.OP_PAGED_DECODE, n, n, per * page), dtype=torch.uint8, device=dev)
    return s


def _params(c):
    import compressed_sparse_attention_13_b200 as K
    fmts = {"bf16": K.BF16, "f32": K.F32, "fp8": K.FP8_S64}
    return K, K.gqa_params(c["H"], c["HK"], c["d"], c["d"] ** -0.5, page_size=c.get("page", 16), window=c.get("window", 0),
                           rot_dim=c.get("rot", 0), act_fmt=fmts[c["act"]], cache_fmt=fmts[c.get("cache", c["act"])],
                           flags=K.FLAG_ROT_PAIRS if c.get("pairs") else 0)


def run(state):
    s = state
    if s["op"] == "append":
        (_append_own if own else _append)(s)
        caches = [s["k_cache"], s["v_cache"]]
        if s["cache"] == "fp8":  # the values that the codes stand for
            caches = [_values(s[k], s[k + "_scales"]).to(torch.bfloat16) for k in ("k_cache", "v_cache")]
        return {"q": s["q_out"], "k": s["k_out"], "k_cache": caches[0], "v_cache": caches[1]}
    if own:
        import compressed_sparse_attention_13_b200 as K
        if s["op"] == "decode":
            K.paged_decode_attn(s["p"], s["q"].shape[0], s["q"], *s["stored"], s["table"], s["q_pos"], s["sinks"], s["out"], s["ws"])
        else:
            K.prompt_attn(s["p"], s["cu"].numel() - 1, s["q"], s["k"], s["v"], s["cu"], s["cu"], s["sinks"], s["out"], s["ws"])
        return s["out"]
    return _decode(s) if s["op"] == "decode" else _prompt(s)


def _append_own(s):
    import compressed_sparse_attention_13_b200 as K
    K.paged_append(s["p"], s["pos0"].numel(), s["q"].shape[0], s["cu"], s["pos0"], s["q"], s["k"], s["v"], s["inv_freq"],
                   s["q_out"], s["k_out"], *s["stored"], s["table"])


def _rotate(x, cos, sin, rot, pairs):
    if rot == 0:
        return x
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append(s):
    cu, pos0, page = s["cu"].long(), s["pos0"], s["page"]
    i = torch.arange(s["q"].shape[0], device=pos0.device)
    seq = torch.searchsorted(cu, i, right=True) - 1
    pos = pos0[seq] + i - cu[seq]
    angle = pos[:, None].double() * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _rotate(s["q"].float(), cos, sin, s["rot"], s["pairs"])
    k = _rotate(s["k"].float(), cos, sin, s["rot"], s["pairs"])
    s["q_out"].copy_(q)
    s["k_out"].copy_(k)
    at, off = s["table"][seq, pos // page].long(), pos % page
    if s["cache"] == "fp8":
        s["k_cache"][at, :, off], s["k_cache_scales"][at, :, off] = _quantize(k)
        s["v_cache"][at, :, off], s["v_cache_scales"][at, :, off] = _quantize(s["v"])
    else:
        s["k_cache"][at, :, off] = k.to(s["k_cache"].dtype)
        s["v_cache"][at, :, off] = s["v"].to(s["v_cache"].dtype)


def _softmax_(x, masked, sinks):
    """In place over the last axis; masked places 0, a sink in the denominator, a row without keys all 0."""
    x.masked_fill_(masked, -math.inf)
    top = x.amax(-1, keepdim=True)
    if sinks is not None:
        top = torch.maximum(top, sinks)
    top = torch.where(top == -math.inf, 0.0, top)
    x.sub_(top).exp_()
    den = x.sum(-1, keepdim=True)
    if sinks is not None:
        den = den + torch.exp(sinks - top)
    return x.div_(torch.where(den == 0, 1.0, den))


def _paged(s, name):
    """The sequences' cache rows as [batch][HK][rows][d] in 32 bits, in order."""
    t = s["table"].clamp(min=0).long()
    x = s[name][t]
    x = _values(x, s[name + "_scales"][t]) if s["cache"] == "fp8" else x.float()
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _decode(s):
    n, H, d, HK = s["q"].shape[0], s["H"], s["d"], s["HK"]
    k, v = _paged(s, "k_cache"), _paged(s, "v_cache")
    x = torch.matmul(s["q"].float().view(n, HK, H // HK, d), k.transpose(2, 3)).mul_(s["scale"])
    at, t = torch.arange(k.shape[2], device=k.device), s["q_pos"][:, None]
    masked = at > t
    if s["window"]:
        masked |= at <= t - s["window"]
    p = _softmax_(x, masked[:, None, None], None if s["sinks"] is None else s["sinks"].view(HK, H // HK, 1))
    return torch.matmul(p, v).view(n, H, d).to(s["q"].dtype)


def _prompt(s):
    cu, L = s["cu"].long(), s["longest"]
    n, H, d, HK = cu.numel() - 1, s["H"], s["d"], s["HK"]
    G = H // HK
    i = torch.arange(L, device=cu.device)
    lens = cu[1:] - cu[:-1]
    there = i < lens[:, None]                               # the padded batch [n][L] of the packed tokens
    at = torch.where(there, cu[:-1, None] + i, 0)
    q = s["q"][at].float().view(n, L, HK, G, d).permute(0, 2, 3, 1, 4).reshape(n, HK, G * L, d)
    k, v = (s[x][at].float().transpose(1, 2) for x in ("k", "v"))
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(n, HK, G, L, L)
    masked = i > i[:, None]
    if s["window"]:
        masked = masked | (i <= i[:, None] - s["window"])
    p = _softmax_(x, masked, None if s["sinks"] is None else s["sinks"].view(HK, G, 1, 1))
    o = torch.matmul(p.view(n, HK, G * L, L), v).view(n, HK, G, L, d).permute(0, 3, 1, 2, 4).reshape(n, L, H, d)
    return o[there].to(s["q"].dtype)


def exact(case, seed):
    """The operators' definitions in 64 bits, a sequence and a head at a time."""
    c, s = case, prepare(case, seed)
    H, HK, d, lens = c["H"], c["HK"], c["d"], _ints(c["lens"])
    if c["op"] == "append":
        return _exact_append(c, s, lens)
    W, G, rows, first = c["window"], H // HK, [], 0
    for b, m in enumerate(lens):
        if c["op"] == "prompt":
            q = s["q"][first:first + m].double()
            k, v = s["k"][first:first + m].double(), s["v"][first:first + m].double()
            t = torch.arange(m, device=q.device)
            first += m
        else:
            q = s["q"][b:b + 1].double()
            t = torch.tensor([m - 1], device=q.device)
            pages = s["table"][b, :-(-m // c["page"])].long()
            k, v = (_exact_rows(c, s, x, pages)[:m] for x in ("k_cache", "v_cache"))
        out = torch.zeros(q.shape[0], H, d, dtype=torch.float64, device=q.device)
        j = torch.arange(m, device=q.device)
        for h in range(H):
            for a in range(0, q.shape[0], 4096):
                e = slice(a, min(a + 4096, q.shape[0]))
                logits = (q[e, h] @ k[:, h // G].T) * s["scale"]
                hidden = j[None] > t[e, None]
                if W:
                    hidden |= j[None] <= t[e, None] - W
                logits[hidden] = -math.inf
                if s["sinks"] is not None:
                    logits = torch.cat([logits, s["sinks"][h].double().expand(logits.shape[0], 1)], 1)
                out[e, h] = torch.softmax(logits, 1)[:, :m] @ v[:, h // G]
        rows.append(out)
    return torch.cat(rows)


def _exact_rows(c, s, name, pages):
    x = s[name][pages]
    if c["cache"] == "fp8":
        x = x.view(torch.float8_e4m3fn).double() * s[name + "_scales"][pages].double().repeat_interleave(64, -1)
    return x.double().transpose(1, 2).reshape(-1, c["HK"], c["d"])


def _exact_append(c, s, lens):
    d, rot, page = c["d"], c["rot"], c["page"]
    pos = np.concatenate([a + np.arange(m, dtype=np.int64) for a, m in zip(_ints(c["starts"]), lens)])
    seq = np.repeat(np.arange(len(lens)), lens)
    angle = pos[:, None].astype(np.float64) * s["inv_freq"].cpu().numpy()[None]
    turn = torch.from_numpy(np.exp(1j * angle)).cuda()[:, None]

    def turned(x):
        y = x.double().clone()
        if rot:
            lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if c["pairs"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
            y[..., lo], y[..., hi] = z.real, z.imag
        return y

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double()
    where = s["table"].cpu().numpy()[seq, pos // page]
    caches = []
    for name, rows in (("k_cache", k), ("v_cache", v)):
        if c["cache"] == "fp8":
            caches.append(None)   # codes: the nearest of a few values, no value of their own in 64 bits
            continue
        x = s[name].double()
        x[torch.from_numpy(where).long().cuda(), :, torch.from_numpy(pos % page).cuda()] = rows
        caches.append(x)
    return {"q": q, "k": k, "k_cache": caches[0], "v_cache": caches[1]}
