"""The operators around the quantized KV cache, as cases that can be timed and compared.

* ``attend``: attention of one or more new tokens per sequence over the quantized cache, each token seeing the positions up to
  its own, with scores capped by a tanh, biased by the distance, limited to a window, and a prefix that every token sees;
* ``rotary``: the norms of the query and key heads and the position rotation in one pass over the projection's output, which
  leaves the rows that the cache appends and the queries that it attends with;
* ``reorder``: sequences of the cache taking over other sequences' contents (beam search, forks of a prompt).

``own`` false: elementary torch operations in 32 bits (64 for the angles); true: the calls of ``asymmetric_kv_cache_b200.kvq``.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"fp16": 2, "bf16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases
def _attend(name, kb, vb, G, d, hq, hkv, batch, lo, hi, q_lo, q_hi, dtype, cap=0.0, slopes=False, window=0, prefix=0, recent=0,
            sink=0, salt=1):
    return {"name": name, "op": "attend", "kb": kb, "vb": vb, "group": G, "d": d, "hq": hq, "hkv": hkv, "batch": batch, "lo": lo,
            "hi": hi, "q_lo": q_lo, "q_hi": q_hi, "dtype": dtype, "cap": cap, "slopes": slopes, "window": window, "prefix": prefix,
            "recent": recent, "sink": sink, "salt": salt}


def _rotary(name, d, hq, hkv, batch, lo, hi, pos_hi, dtype, out, norm, pairs, interleaved=False, axes=0, salt=1):
    return {"name": name, "op": "rotary", "d": d, "hq": hq, "hkv": hkv, "batch": batch, "lo": lo, "hi": hi, "pos_hi": pos_hi,
            "dtype": dtype, "out": out, "norm": norm, "pairs": pairs, "interleaved": interleaved, "axes": axes, "salt": salt}


def _reorder(name, kb, vb, G, d, hkv, requests, beams, lo, hi, shared, recent=0, salt=1):
    return {"name": name, "op": "reorder", "kb": kb, "vb": vb, "group": G, "d": d, "hkv": hkv, "requests": requests,
            "beams": beams, "lo": lo, "hi": hi, "shared": shared, "recent": recent, "salt": salt}


def listed():
    return [
        # one token over a 256-token, one-head cache with fp32 queries: the smallest call, all latency
        _attend("attend tiny", 4, 2, 32, 64, 1, 1, 1, 256, 256, 1, 1, "fp32", cap=20.0),
        # a decoding step of a layer with 8 sequences at 4k, scores capped
        _attend("attend step cap", 4, 2, 32, 128, 32, 8, 8, 4113, 4113, 1, 1, "fp16", cap=50.0),
        # a decoding step over one context of 128k with a distance bias: the cache's bytes are what counts
        _attend("attend step 128k bias", 2, 2, 32, 128, 32, 8, 1, 131072, 131072, 1, 1, "fp16", slopes=True),
        # a ragged batch of 64 sequences, 64 query heads, each token seeing 1024 others and the first 4
        _attend("attend step ragged window", 4, 2, 64, 128, 64, 8, 64, 1024, 8192, 1, 1, "bf16", window=1024, prefix=4),
        # five proposed tokens per sequence checked at once, fp16 recent and first tokens, smaller heads
        _attend("attend five tokens", 4, 4, 32, 64, 16, 4, 16, 500, 3000, 5, 5, "bf16", recent=64, sink=4),
        # a new turn of some hundred tokens in each of 6 conversations
        _attend("attend turn", 4, 2, 64, 128, 32, 8, 6, 1500, 5000, 90, 700, "bf16"),
        # a piece of 2048 tokens of two long prompts
        _attend("attend piece of a prompt", 4, 2, 32, 128, 32, 8, 2, 18432, 18432, 2048, 2048, "fp16", cap=50.0),
        # the projection's output of one step of 8 sequences
        _rotary("rotary step", 128, 32, 8, 8, 1, 1, 60000, "fp16", "fp16", True, 64),
        # a prompt piece of 16k rows
        _rotary("rotary prompt", 128, 32, 8, 4, 3900, 4096, 100000, "bf16", "fp16", True, 64),
        # an image's tokens between text, time, height and width on the axes, part of the head rotated, fp32
        _rotary("rotary three axes", 64, 12, 4, 3, 200, 1500, 30000, "fp32", "fp16", False, 24, axes=3),
        # four beams of 8 requests after a prompt that they share
        _reorder("reorder beams", 4, 2, 32, 128, 8, 8, 4, 4096, 4200, True),
        # 16 sequences of 8k among each other, nothing shared
        _reorder("reorder whole", 4, 2, 32, 128, 8, 4, 4, 8000, 8192, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "rotary", "reorder"])
    salt = rng.randrange(1 << 20)
    d = rng.choice([64, 128])
    G = rng.choice([32, 64])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "rotary":
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
        batch = _log(rng, 1, 32)
        hi = max(1, min(_log(rng, 1, 8192), 16000 * 48 * 128 // (batch * (hq + 2 * hkv) * d)))
        axes = rng.choice([0, 0, 1, 3])
        return {k: v for k, v in _rotary("", d, hq, hkv, batch, rng.randint(max(1, hi // 3), hi), hi, _log(rng, 10, 100000),
                                         rng.choice(list(DTYPES)), rng.choice(["fp16", "fp16", "bf16", "fp32"]), rng.random() < 0.6,
                                         rng.choice([d // 2, d // 4, 12, 24, 31]), rng.random() < 0.4, axes, salt).items()
                if k != "name"}
    kb, vb = rng.choice([2, 4]), rng.choice([2, 4])
    if op == "reorder":
        requests, beams = _log(rng, 1, 8), rng.choice([2, 3, 4, 8])
        hi = max(1, min(_log(rng, 20, 16384), 16 * 8192 * 8 // (requests * beams * hkv)))
        return {k: v for k, v in _reorder("", kb, vb, G, d, hkv, requests, beams, rng.randint(max(1, hi // 2), hi), hi,
                                          rng.random() < 0.5, rng.choice([0, 0, 32, 128]), salt).items() if k != "name"}
    hq = hkv * rng.choice([1, 2, 4, 4, 5, 8, 12])
    batch = _log(rng, 1, 64)
    hi = max(1, min(_log(rng, 1, 131072), 131072 * 8 // (batch * hkv)))
    most = int(min(hi, 2.4e9 // (batch * hq * hi), 4096))
    q_hi = 1 if rng.random() < 0.4 or most < 2 else _log(rng, 1, most)
    lo = rng.randint(max(q_hi, hi // 3), hi)
    return {k: v for k, v in _attend("", kb, vb, G, d, hq, hkv, batch, lo, hi, rng.randint(1, q_hi), q_hi, rng.choice(list(DTYPES)),
                                     cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3,
                                     window=rng.choice([0, 0, _log(rng, 1, 4096)]), prefix=rng.choice([0, 0, rng.randint(1, 100)]),
                                     recent=rng.choice([0, 0, 16, 128]), sink=rng.choice([0, 0, 4, 33]), salt=salt).items()
            if k != "name"}


def _ragged(case, n, lo, hi, what):
    r = random.Random("%d %s" % (case["salt"], what))
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    return _ragged(case, case["batch"], case["lo"], case["hi"], "lens")


def _n_q(case):
    return _ragged(case, case["batch"], case["q_lo"], case["q_hi"], "q")


def _split(case, n):
    """(tokens of the sink, quantized ones after them) of a sequence of n tokens."""
    s = min(n, case.get("sink", 0))
    return s, case["group"] * (max(0, n - s - case["recent"]) // case["group"])


def _block_bytes(case):
    G, d = case["group"], case["d"]
    return G * d * (case["kb"] + case["vb"]) // 8 + 4 * d + 4 * d


# ---------------------------------------------------------------- work
def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rotary":
        n = sum(_ragged(case, case["batch"], case["lo"], case["hi"], "rows"))
        x = n * (case["hq"] + 2 * hkv) * d
        return {"bytes": x * (SIZES[case["dtype"]] + SIZES[case["out"]]), "flops": 7 * x}
    if case["op"] == "reorder":
        moved, lens, parents, shared = 0, *_beams(case)
        for b, p in enumerate(parents):
            if b != p:
                _, N = _split(case, lens[p])
                moved += hkv * ((N // case["group"] - shared // case["group"]) * _block_bytes(case) + (lens[p] - N) * 4 * d)
        return {"bytes": 2 * moved, "flops": 0}
    total, pairs = 0, 0
    for n, m in zip(_lens(case), _n_q(case)):
        s, N = _split(case, n)
        w, pre = case["window"] or n, min(case["prefix"], n)
        first = max(0, n - m - w + 1)            # the first position that the window of some row reaches
        seen = lambda a, b: max(0, b - max(a, first)) + max(0, min(b, pre, max(first, a)) - a)  # noqa: E731
        total += hkv * (seen(0, s) + seen(s + N, n)) * 4 * d + hkv * seen(s, s + N) * _block_bytes(case) // case["group"]
        for p in (n - m, n - 1):                 # visible keys are linear in the row but for the corners: the mean of the ends
            pairs += m / 2 * (min(p + 1, w) + min(pre, max(0, p - w + 1)) + max(0, pre - p - 1))
    rows = sum(_n_q(case))
    return {"bytes": total + rows * case["hq"] * d * (SIZES[case["dtype"]] + 2), "flops": 4 * d * case["hq"] * pairs}


# ---------------------------------------------------------------- inputs
def _quantize(x, dim, bits):
    """Codes, scale and least value of x (fp32 values) along dim: scale and least value in fp16, codes to the nearest level."""
    top = 2 ** bits - 1
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s, z = ((hi - lo) / top).half(), lo.half()
    codes = torch.where(s == 0, torch.zeros_like(x), torch.round((x - z.float()) / s.float()).clamp(0, top)).to(torch.uint8)
    return codes, s.squeeze(dim), z.squeeze(dim)


def _spec(case, seqs, most):
    from asymmetric_kv_cache_b200 import kvq
    return kvq.CacheSpec(case.get("kb", 4), case.get("vb", 2), case.get("group", 32), case["d"], case.get("hq", case["hkv"]),
                         case["hkv"], seqs, most, window=case.get("recent", 0), sink=case.get("sink", 0))


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed * 7919 + 13)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return {"attend": _prepare_attend, "rotary": _prepare_rotary, "reorder": _prepare_reorder}[case["op"]](case, g, randn)


def _prepare_attend(case, g, randn):
    lens, n_q, hkv, hq, d, G = _lens(case), _n_q(case), case["hkv"], case["hq"], case["d"], case["group"]
    B, n, S = len(lens), max(lens), case["sink"]
    # keys: a spread of its own for each channel; values: a norm of its own for each token, as caches hold them
    k = torch.stack([(torch.exp(randn(1, hkv, d)) * randn(n, hkv, d)).half() for _ in lens])
    v = torch.stack([torch.nn.functional.normalize(randn(n, hkv, d), dim=-1) * torch.exp(0.5 * randn(n, hkv, 1)) for _ in lens]).half()
    split = [_split(case, x) for x in lens]
    ng = max(N for _, N in split) // G
    kq, vq = (x[:, S:S + ng * G].float() for x in (k, v))
    kc, ks, kz = _quantize(kq.view(B, ng, G, hkv, d), 2, case["kb"]) if ng else (None,) * 3
    vc, vs, vz = _quantize(vq.view(B, ng * G, hkv, d // G, G), 4, case["vb"]) if ng else (None,) * 3
    # the fp16 tokens: (sequence, position) of each and their rows
    at = torch.tensor([(b, p) for b, (s, N) in enumerate(split) for p in [*range(s), *range(s + N, lens[b])]] or [(0, 0)],
                      device="cuda")[: sum(x - N for x, (_, N) in zip(lens, split))]
    state = {"case": case, "lens": lens, "n_q": n_q, "kc": kc, "ks": ks, "kz": kz, "vc": vc, "vs": vs, "vz": vz, "b": at[:, 0],
             "p": at[:, 1], "kt": k[at[:, 0], at[:, 1]], "vt": v[at[:, 0], at[:, 1]],
             "q": randn(sum(n_q), hq, d).to(DTYPES[case["dtype"]]),
             "row_b": torch.tensor([b for b, m in enumerate(n_q) for _ in range(m)], device="cuda"),
             "row_i": torch.tensor([i for m in n_q for i in range(m)], device="cuda"),
             "dev_lens": torch.tensor(lens, device="cuda"), "dev_n_q": torch.tensor(n_q, device="cuda"),
             "slopes": 2.0 ** (-8.0 * (torch.arange(hq, device="cuda") + 1.0) / hq) if case["slopes"] else None,
             "prefix": torch.full((B,), case["prefix"], dtype=torch.int32, device="cuda") if case["prefix"] else None}
    if own:
        from asymmetric_kv_cache_b200 import kvq
        cache = kvq.KVQCache(_spec(case, B, n))
        cache.append(torch.cat([k[b, :x] for b, x in enumerate(lens)]), torch.cat([v[b, :x] for b, x in enumerate(lens)]), lens)
        state["cache"] = cache
    return state


def _prepare_rotary(case, g, randn):
    rows, d, hq, hkv = _ragged(case, case["batch"], case["lo"], case["hi"], "rows"), case["d"], case["hq"], case["hkv"]
    dt, n, pairs = DTYPES[case["dtype"]], sum(rows), case["pairs"]
    lens = torch.randint(0, case["pos_hi"], (len(rows),), generator=g, device="cuda", dtype=torch.int32)
    state = {"case": case, "rows": rows, "qkv": (randn(n, (hq + 2 * hkv) * d) * torch.exp(randn(1, (hq + 2 * hkv) * d) / 2)).to(dt),
             "inv_freq": (500000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)).float(),
             "lens": lens, "row_b": torch.tensor([b for b, m in enumerate(rows) for _ in range(m)], device="cuda"),
             "row_i": torch.tensor([i for m in rows for i in range(m)], device="cuda"),
             "qw": (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None, "kw": (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None,
             "positions": None, "sections": None}
    if case["axes"]:
        state["positions"] = torch.randint(0, case["pos_hi"], (case["axes"], n), generator=g, device="cuda", dtype=torch.int32)
        cut = pairs // case["axes"]
        state["sections"] = [cut] * (case["axes"] - 1) + [pairs - cut * (case["axes"] - 1)]
    if own:
        from asymmetric_kv_cache_b200 import kvq
        spec = kvq.CacheSpec(2, 2, 32, d, hq, hkv, len(rows), case["pos_hi"] + max(rows))
        cache = kvq.KVQCache(spec)
        cache.device_lengths().copy_(lens)
        cache.sync_lengths()
        state["cache"] = cache
    return state


def _beams(case):
    """Lengths and parents of every sequence, and how many first tokens the beams of a request share."""
    r = random.Random("%d beams" % case["salt"])
    lens, parents = [], []
    for i in range(case["requests"]):
        n = r.randint(case["lo"], case["hi"])
        lens += [n] * case["beams"]
        parents += [i * case["beams"] + r.randrange(case["beams"]) for _ in range(case["beams"])]
    if all(b == p for b, p in enumerate(parents)):
        parents[0] = 1
    G, R = case["group"], case["recent"]
    shared = max(0, min(case["lo"], min(lens) - R)) // G * G if case["shared"] else 0
    return lens, parents, min(shared, min(lens))


def _prepare_reorder(case, g, randn):
    lens, parents, shared = _beams(case)
    hkv, d, G, B = case["hkv"], case["d"], case["group"], len(lens)
    most, W, bb = max(lens), case["recent"] + case["group"], _block_bytes(case)
    ng = torch.tensor([_split(case, n)[1] // G for n in lens], device="cuda")
    blocks = torch.randint(0, 256, (B, hkv, most // G, bb), generator=g, device="cuda", dtype=torch.uint8)
    live = torch.arange(most // G, device="cuda") < ng[:, None]
    blocks *= live[:, None, :, None]
    # what the beams of a request share is the same in all of them
    first = torch.arange(B, device="cuda") // case["beams"] * case["beams"]
    blocks[:, :, : shared // G] = blocks[first][:, :, : shared // G]
    tail = torch.zeros(B, hkv, 2, W, d, dtype=torch.float16, device="cuda")
    for b, n in enumerate(lens):
        N = _split(case, n)[1]
        at = torch.tensor([p % W for p in range(N, n)], dtype=torch.long, device="cuda")
        tail[b, :, 0, at] = randn(hkv, n - N, d).half()
        pairs = tail[b, :, 1].view(hkv, W // 2, d, 2)
        pairs[:, at // 2, :, at % 2] = randn(n - N, hkv, d).half()
    state = {"case": case, "shared": shared, "parents": parents, "parent": torch.tensor(parents, device="cuda"),
             "first": torch.tensor(shared // G), "blocks": blocks, "tails": tail.view(B, hkv, -1).view(torch.uint8),
             "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if own:
        from asymmetric_kv_cache_b200 import kvq
        cache = kvq.KVQCache(_spec(case, B, most))
        L = cache.layout
        for name, at, like in (("blocks", "blocks_offset", blocks), ("tails", "tails_offset", state["tails"])):
            view = cache.buffer[L[at]: L[at] + like.numel()].view(like.shape)
            state[name] = view.copy_(like)
        cache.device_lengths().copy_(state["lens"])
        cache.sync_lengths()
        state["lens"], state["cache"] = cache.device_lengths(), cache
    return state


# ---------------------------------------------------------------- the operators
def run(state):
    return {"attend": _run_attend, "rotary": _run_rotary, "reorder": _run_reorder}[state["case"]["op"]](state)


def _run_attend(st):
    case = st["case"]
    if own:
        return st["cache"].attend(st["q"], st["n_q"], cap=case["cap"], window=case["window"], slopes=st["slopes"],
                                  prefix=st["prefix"])
    hq, hkv, d, G, S = case["hq"], case["hkv"], case["d"], case["group"], case["sink"]
    B, n, m = len(st["lens"]), max(st["lens"]), max(st["n_q"])
    k = torch.zeros(B, n, hkv, d, device="cuda")
    v = torch.zeros_like(k)
    if st["kc"] is not None:
        kd = st["kc"].float() * st["ks"].float()[:, :, None] + st["kz"].float()[:, :, None]
        vd = st["vc"].float() * st["vs"].float()[..., None] + st["vz"].float()[..., None]
        t = kd.shape[1] * G
        k[:, S:S + t] = kd.view(B, t, hkv, d)
        v[:, S:S + t] = vd.view(B, t, hkv, d)
    k[st["b"], st["p"]] = st["kt"].float()
    v[st["b"], st["p"]] = st["vt"].float()
    q = torch.zeros(B, m, hq, d, device="cuda")
    q[st["row_b"], st["row_i"]] = st["q"].float()
    q = q.view(B, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, hq, m, n) * (1 / math.sqrt(d))
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    at = (st["dev_lens"] - st["dev_n_q"])[:, None] + torch.arange(m, device="cuda")      # position of each row
    j = torch.arange(n, device="cuda")
    ahead = at[:, :, None] - j                                                          # [B, m, n]
    seen = ahead >= 0
    if case["window"]:
        seen &= ahead < case["window"]
    if st["prefix"] is not None:
        seen |= j < st["prefix"][:, None, None]
    seen &= j < st["dev_lens"][:, None, None]
    if st["slopes"] is not None:
        s = s - st["slopes"][None, :, None, None] * ahead.abs()[:, None].float()
    s = torch.where(seen[:, None], s, torch.full((), -math.inf, device="cuda"))
    top = s.amax(-1, keepdim=True)
    s = torch.exp(s - top)
    s = s / s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, hkv, -1, n), v.permute(0, 2, 1, 3)).view(B, hq, m, d)
    return o[st["row_b"], :, st["row_i"]].half()


def _run_rotary(st):
    case = st["case"]
    d, hq, hkv, pairs = case["d"], case["hq"], case["hkv"], case["pairs"]
    out = DTYPES[case["out"]]
    x = st["qkv"].view(len(st["qkv"]), hq + 2 * hkv, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if own:
        return st["cache"].norm_rotary(q, k, v, st["rows"], st["inv_freq"], q_weight=st["qw"], k_weight=st["kw"], eps=1e-6,
                                       positions=st["positions"], sections=st["sections"], interleaved=case["interleaved"],
                                       out_dtype=out)
    if st["positions"] is None:
        angle = (st["lens"][st["row_b"]] + st["row_i"]).double()[:, None] * st["inv_freq"].double()
    else:
        axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"), torch.tensor(st["sections"], device="cuda"))
        angle = st["positions"][axis].t().double() * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(y, w):
        y = y.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        r = y.clone()
        if case["interleaved"]:
            a, b = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
        else:
            a, b = slice(0, pairs), slice(pairs, 2 * pairs)
        r[..., a] = y[..., a] * cos - y[..., b] * sin
        r[..., b] = y[..., b] * cos + y[..., a] * sin
        return r.to(out)

    return turned(q, st["qw"]), turned(k, st["kw"]), v.float().to(out)


def _run_reorder(st):
    if own:
        st["cache"].reorder(st["parents"], shared=st["shared"])
    else:
        f = st["shared"] // st["case"]["group"]
        st["blocks"][:, :, f:] = st["blocks"][:, :, f:][st["parent"]]
        st["tails"][:] = st["tails"][st["parent"]]
        st["lens"][:] = st["lens"][st["parent"]]
    return {"blocks": st["blocks"], "tails": st["tails"], "lens": st["lens"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "reorder":
        return None
    st = prepare(case, seed)
    case = st["case"]
    return _exact_rotary(case, st) if case["op"] == "rotary" else _exact_attend(case, st)


def _exact_rotary(case, st):
    d, hq, hkv, P = case["d"], case["hq"], case["hkv"], case["pairs"]
    x = st["qkv"].double().view(-1, hq + 2 * hkv, d)
    rows = []
    if st["positions"] is None:
        for b, m in enumerate(st["rows"]):
            rows.append(st["lens"][b].double() + torch.arange(m, device="cuda", dtype=torch.float64))
        pos = torch.cat(rows)[:, None].expand(-1, P)
    else:
        for a, m in enumerate(st["sections"]):
            rows.append(st["positions"][a].double()[:, None].expand(-1, m))
        pos = torch.cat(rows, 1)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(pos.shape), pos * st["inv_freq"].double())[:, None]

    def head(y, w):
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        a = y[..., :2 * P]
        a = a.unflatten(-1, (P, 2)) if case["interleaved"] else a.unflatten(-1, (2, P)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(a.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), y[..., 2 * P:]], -1)

    return head(x[:, :hq], st["qw"]), head(x[:, hq:hq + hkv], st["kw"]), x[:, hq + hkv:]


def _exact_attend(case, st):
    hq, hkv, d, G, S = case["hq"], case["hkv"], case["d"], case["group"], case["sink"]
    out, row = torch.empty(len(st["q"]), hq, d, dtype=torch.float64, device="cuda"), 0
    for b, (n, m) in enumerate(zip(st["lens"], st["n_q"])):
        s0, N = _split(case, n)
        mine = st["b"] == b
        for h in range(hkv):
            k, v = torch.empty(2, n, d, dtype=torch.float64, device="cuda")
            for x, c, s, z in ((k, st["kc"], st["ks"], st["kz"]), (v, st["vc"], st["vs"], st["vz"])):
                if not N:
                    continue
                if x is k:
                    c, s, z = (y[b, : N // G, ..., h, :].double() for y in (c, s, z))
                    x[s0:s0 + N] = (c * s[:, None] + z[:, None]).reshape(N, d)
                else:
                    c, s, z = (y[b, :N, h].double() for y in (c, s, z))
                    x[s0:s0 + N] = (c * s[..., None] + z[..., None]).reshape(N, d)
            k[st["p"][mine]], v[st["p"][mine]] = st["kt"][mine, h].double(), st["vt"][mine, h].double()
            j = torch.arange(n, device="cuda")
            far = (n - m + torch.arange(m, device="cuda"))[:, None] - j[None]
            hide = far < 0
            if case["window"]:
                hide = hide | (far >= case["window"])
            if case["prefix"]:
                hide = hide & (j >= case["prefix"])
            for i in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = st["q"][row:row + m, i].double() @ k.t() / math.sqrt(d)
                if case["cap"]:
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                if st["slopes"] is not None:
                    x = x - st["slopes"][i].double() * far.abs()
                out[row:row + m, i] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v
        row += m
    return out
