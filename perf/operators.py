"""Cases, plain forms and calls of the prompt-side operators: rotary positions
fused with the cache append (rope_append), attention of ragged chunks of new
tokens over the paged cache (paged_chunk_attn), and the same with a sliding
window and first tokens that stay visible, each over bf16 and FP8 (E4M3) caches.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases
def _rope(name, **kw):
    case = dict(op="rope", name=name, tokens=8, ctx=32768, hq=32, hkv=8, d=128, rot=128, off=0,
                interleaved=False, latent=0, e4m3=False, fp32_q=False, block=16, theta=10000.0,
                stretch=1.0)
    case.update(kw)
    return case


def _chunk(name, **kw):
    case = dict(op="chunk", name=name, seqs=1, new=2048, ctx=0, ragged=False, lens_seed=1, hq=32,
                hkv=8, d=128, block=16, e4m3=False, window=0, sinks=0)
    case.update(kw)
    return case


def listed():
    return [
        # one decode step of 8 sequences at 32K: the new token of each, q kept in fp32 for
        # the decode attention that follows; latency
        _rope("rope-decode", tokens=8, fp32_q=True),
        # one prompt chunk of a whole batch, odd length
        _rope("rope-prompt", tokens=8191),
        # FP8 cache, interleaved layout, half of the head rotated, far positions with
        # interpolated frequencies
        _rope("rope-fp8-long", tokens=2500, ctx=200000, hq=64, rot=64, interleaved=True,
              e4m3=True, theta=500000.0, stretch=8.0),
        # latent (MLA-shaped) rows: 128 heads, the last 64 of 576 dims rotated, values
        # inside the keys
        _rope("rope-latent", tokens=1024, hq=128, hkv=1, d=576, rot=64, off=512,
              interleaved=True, latent=512, block=64),
        # prompts of the continuous-batching mix: 16 sequences of 8 to 32 tokens; latency
        _chunk("chunk-mix", seqs=16, new=32, ragged=True),
        # one 8K prompt from an empty cache
        _chunk("chunk-prompt", new=8192),
        # the last 2,048 tokens of a 32K context
        _chunk("chunk-32k", new=2048, ctx=30720),
        # a serving batch: 24 sequences, some bringing one token, some up to 512, ragged contexts
        _chunk("chunk-ragged", seqs=24, new=512, ctx=4096, ragged=True, hq=64, lens_seed=5),
        # a 1,000-token chunk over an FP8 cache, head groups of 8
        _chunk("chunk-fp8", new=1000, ctx=16384, hq=64, e4m3=True),
        # single tokens of 64 sequences, window of 4,096 and 4 first tokens
        _chunk("window-decode", seqs=64, new=1, ctx=32767, window=4096, sinks=4),
        # an 8K prompt under a short window, small heads, larger blocks
        _chunk("window-prompt", new=8192, ctx=1000, hq=64, d=64, block=32, window=1024, sinks=16),
        # single tokens and small chunks over an FP8 cache at 64K, window of 8,192
        _chunk("window-fp8", seqs=12, new=4, ctx=65000, ragged=True, hq=64, e4m3=True,
               window=8192, sinks=4, lens_seed=3),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    if rng.random() < 0.3:
        case = _rope("", tokens=_spread(rng, 1, 8192), ctx=_spread(rng, 128, 200000),
                     block=rng.choice([16, 32, 64]), theta=rng.choice([10000.0, 500000.0]),
                     stretch=rng.choice([1.0, 1.0, 4.0, 8.0]))
        case["interleaved"] = rng.random() < 0.5
        if rng.random() < 0.2:
            case.update(tokens=min(case["tokens"], 1024), hq=rng.choice([16, 128]), hkv=1, d=576,
                        rot=64, off=512, latent=512, block=64)
        else:
            case["hq"], case["hkv"] = rng.choice([(32, 8), (64, 8), (8, 8), (28, 4), (40, 8)])
            case["d"] = rng.choice([64, 128])
            case["rot"] = case["d"] if rng.random() < 0.5 else case["d"] // 2
            case["e4m3"] = rng.random() < 0.4
            case["fp32_q"] = rng.random() < 0.3
            if case["hq"] > 32:
                case["tokens"] = min(case["tokens"], 4096)
    else:
        most = max(work(c)["flops"] for c in listed())
        while True:
            case = _chunk("", seqs=_spread(rng, 1, 64), new=_spread(rng, 1, 8192),
                          ctx=_spread(rng, 1, 65536) - 1, ragged=rng.random() < 0.6,
                          lens_seed=rng.randrange(1 << 20), block=rng.choice([16, 32, 64, 128]))
            case["hq"], case["hkv"] = rng.choice([(32, 8), (64, 8), (8, 8), (28, 4), (40, 8),
                                                  (16, 1)])
            case["d"] = rng.choice([64, 128, 128])
            case["e4m3"] = case["d"] == 128 and rng.random() < 0.3
            if rng.random() < 0.4:
                case["window"] = _spread(rng, 16, 8192)
                case["sinks"] = rng.choice([0, 1, 4, 16, 100])
            # the plain form holds every score of the padded batch
            news, lens = lengths(case)
            scores = case["seqs"] * case["hq"] * max(news) * max(lens)
            keys = case["seqs"] * max(lens) * case["hkv"] * case["d"]
            if scores <= 2.5e9 and keys <= 1.2e9 and work(case)["flops"] <= most:
                break
    case.pop("name")
    return case


def lengths(case):
    """New and stored tokens (new ones among them) of each sequence."""
    rng = random.Random(case["lens_seed"])
    news, lens = [], []
    for _ in range(case["seqs"]):
        n = _spread(rng, 1, case["new"]) if case["ragged"] else case["new"]
        c = rng.randint(0, case["ctx"]) if case["ragged"] else case["ctx"]
        news.append(n)
        lens.append(c + n)
    return news, lens


def _visible_pairs(n, length, window, sinks):
    """(query, key) pairs that are attended, and the distinct keys among them."""
    first = length - n
    if window <= 0:
        return n * first + n * (n + 1) // 2, length
    pairs = 0
    for p in range(first, length):
        low = max(0, p - window + 1)
        pairs += p + 1 - low + min(sinks, low)
    low = max(0, first - window + 1)
    return pairs, length - low + min(sinks, low)


def work(case):
    if case["op"] == "rope":
        t, d, dv = case["tokens"], case["d"], case["d"]
        kept = 1 if case["e4m3"] else 2
        if case["latent"]:
            dv = 0
        rows = case["hkv"] * (d + dv)
        bytes_ = t * (case["hq"] * d * (2 + (4 if case["fp32_q"] else 2)) + rows * (2 + kept) + 16)
        pairs = case["rot"] // 2 * (case["hq"] + case["hkv"])
        return {"bytes": bytes_ + case["rot"] * 4, "flops": t * pairs * 6}
    news, lens = lengths(case)
    pairs = keys = pages = 0
    for n, length in zip(news, lens):
        a, b = _visible_pairs(n, length, case["window"], case["sinks"])
        pairs, keys, pages = pairs + a, keys + b, pages + -(-b // case["block"])
    rows = sum(news) * case["hq"]
    kept = 1 if case["e4m3"] else 2
    bytes_ = rows * (4 * case["d"] + 4) + keys * case["hkv"] * 2 * case["d"] * kept + 4 * pages
    return {"bytes": bytes_ + 8 * len(news), "flops": 4 * case["d"] * case["hq"] * pairs}


# ------------------------------------------------------------- their inputs
def _pools(case, blocks, gen):
    """K and V pools (bf16, or E4M3 codes with a scale per KV head) of N(0, 1) values."""
    shape = (blocks, case["hkv"], case["block"], case["d"])
    pools, scales = [], []
    for _ in range(1 if case.get("latent") else 2):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        if case["e4m3"]:
            # a head's largest magnitudes (about 4.5 to 5.5 deviations) at the top of the range
            s = (4.5 + torch.rand(case["hkv"], generator=gen, device="cuda")) / 448
            x = (x.float() / s.view(1, -1, 1, 1)).clamp_(-448, 448).to(E4M3).view(torch.uint8)
            scales.append(s)
        pools.append(x)
    return (pools + [None])[:2], scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    s = {"case": case}
    if case["op"] == "rope":
        t, bs = case["tokens"], case["block"]
        blocks = -(-t // bs) + 3
        (s["k_pool"], s["v_pool"]), s["scales"] = _pools(case, blocks, gen)
        s["q"] = normal(t, case["hq"], case["d"])
        s["k"] = normal(t, case["hkv"], case["d"])
        s["v"] = None if case["latent"] else normal(t, case["hkv"], case["d"])
        # a few sequences' runs of positions, anywhere in the context
        runs = max(1, min(8, t))
        start = torch.randint(0, case["ctx"], (runs,), generator=gen, device="cuda")
        at = torch.arange(t, device="cuda")
        per = -(-t // runs)
        s["positions"] = (start[at // per] + at % per).to(torch.int64)
        order = torch.randperm(blocks, generator=gen, device="cuda")
        s["slots"] = order[at // bs] * bs + at % bs
        i = torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = case["theta"] ** (-i / case["rot"]) / case["stretch"]
        return s
    news, lens = lengths(case)
    bs = case["block"]
    per = -(-max(lens) // bs)
    used = sum(-(-x // bs) for x in lens)
    blocks = used + 7
    (s["k_pool"], s["v_pool"]), s["scales"] = _pools(case, blocks, gen)
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    tables = torch.zeros(len(lens), per, device="cuda", dtype=torch.int32)
    at = 0
    for b, x in enumerate(lens):
        n = -(-x // bs)
        tables[b, :n] = order[at:at + n]
        at += n
    s["tables"] = tables
    s["q"] = normal(sum(news), case["hq"], case["d"])
    s["cu"] = torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], device="cuda",
                           dtype=torch.int32)
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    # the batch's largest lengths, which its scheduler knows
    s["most"] = (max(news), max(lens))
    return s


# ------------------------------------------------------------- the operators
def run(s):
    case = s["case"]
    if own:
        return _own_rope(s, case) if case["op"] == "rope" else _own_chunk(s, case)
    return _plain_rope(s, case) if case["op"] == "rope" else _plain_chunk(s, case)


def _shown(pool, case):
    """A pool as the values it holds."""
    return pool.view(E4M3) if case["e4m3"] else pool


def _rope_out(s, case, q):
    got = {"q": q, "k_pool": _shown(s["k_pool"], case)}
    if s["v_pool"] is not None:
        got["v_pool"] = _shown(s["v_pool"], case)
    return got


def _own_rope(s, case):
    import paged_kv_cache_93_gb300 as pkv
    v_pool = pkv.ValuesInKeys(case["latent"]) if case["latent"] else s["v_pool"]
    how = dict(interleaved=case["interleaved"], rotary_offset=case["off"],
               q_dtype=torch.float32 if case["fp32_q"] else torch.bfloat16)
    if case["e4m3"]:
        q = pkv.rope_append_e4m3(s["k_pool"], v_pool, s["q"], s["k"], s["v"], s["positions"],
                                 s["slots"], s["inv_freq"], *s["scales"], **how)
    else:
        q = pkv.rope_append(s["k_pool"], v_pool, s["q"], s["k"], s["v"], s["positions"],
                            s["slots"], s["inv_freq"], **how)
    return _rope_out(s, case, q)


def _own_chunk(s, case):
    import paged_kv_cache_93_gb300 as pkv
    scale = 1.0 / math.sqrt(case["d"])
    how = dict(window=case["window"], sink_tokens=case["sinks"])
    if case["e4m3"]:
        out, lse = pkv.paged_chunk_attn_e4m3(s["q"], s["cu"], s["k_pool"], s["v_pool"],
                                             *s["scales"], s["tables"], s["lens"], scale, **how)
    else:
        out, lse = pkv.paged_chunk_attn(s["q"], s["cu"], s["k_pool"], s["v_pool"], s["tables"],
                                        s["lens"], scale, **how)
    return {"out": out, "lse": lse}


def _rotate(x, cos, sin, case):
    """x [tokens, heads, d] in fp32 with its rotary part turned by the tokens' angles."""
    off, rot = case["off"], case["rot"]
    part = x[:, :, off:off + rot]
    if case["interleaved"]:
        a, b = part[:, :, 0::2], part[:, :, 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(2)
    else:
        a, b = part[:, :, :rot // 2], part[:, :, rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((x[:, :, :off], turned, x[:, :, off + rot:]), dim=-1)


def _store(pool, x, slots, scale, case):
    """Rows x [tokens, hkv, d] (fp32) into the pool at their slots."""
    block, at = slots // case["block"], slots % case["block"]
    if case["e4m3"]:
        x = (x / scale.view(1, -1, 1)).clamp(-448, 448).to(E4M3).view(torch.uint8)
    pool[block, :, at] = x.to(pool.dtype)


def _plain_rope(s, case):
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float(), cos, sin, case)
    ks, vs = s["scales"] if case["e4m3"] else (None, None)
    _store(s["k_pool"], _rotate(s["k"].float(), cos, sin, case), s["slots"], ks, case)
    if s["v"] is not None:
        _store(s["v_pool"], s["v"].float(), s["slots"], vs, case)
    return _rope_out(s, case, q if case["fp32_q"] else q.to(torch.bfloat16))


def _gathered(pool, rows, scale, case):
    """Stored rows of every sequence, [seqs, hkv, tokens, d] in fp32."""
    bs = case["block"]
    x = _shown(pool, case).transpose(1, 2).reshape(-1, case["hkv"], case["d"])
    x = x.view(torch.uint8)[rows].view(E4M3) if case["e4m3"] else x[rows]
    x = x.transpose(1, 2).float()
    return x if scale is None else x * scale.view(1, -1, 1, 1)


def _plain_chunk(s, case):
    tmax, lmax = s["most"]
    n, bs, hkv, d = case["seqs"], case["block"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    cu, lens = s["cu"].long(), s["lens"].long()
    news = cu[1:] - cu[:-1]
    j = torch.arange(lmax, device="cuda")
    rows = s["tables"].long()[:, j // bs] * bs + j % bs
    ks, vs = s["scales"] if case["e4m3"] else (None, None)
    stored = (j < lens[:, None])[:, None, :, None]
    k = _gathered(s["k_pool"], rows, ks, case)
    v = _gathered(s["v_pool"], rows, vs, case).masked_fill_(~stored, 0)
    # queries padded to [seqs, hkv, group * tmax, d]
    t = torch.arange(tmax, device="cuda")
    at = (cu[:-1, None] + t).clamp_(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(n, tmax, hkv, group, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(n, hkv, group * tmax, d), k.transpose(2, 3))
    del k
    x = x.view(n, hkv, group, tmax, lmax).mul_(1.0 / math.sqrt(d))
    p = (lens - news)[:, None] + t
    seen = (j <= p[:, :, None]) & (t < news[:, None])[:, :, None]
    if case["window"]:
        seen &= (j > p[:, :, None] - case["window"]) | (j < case["sinks"])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m.masked_fill_(m == -math.inf, 0)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(n, hkv, group * tmax, lmax), v).view(n, hkv, group, tmax, d)
    del x, v
    out = out / total
    lse = (m + total.log()).squeeze(-1)
    # back to the packed rows: row r is token r - cu[b] of sequence b
    r = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, tmax, hkv * group, d)[b, r - cu[b]]
    lse = lse.permute(0, 3, 1, 2).reshape(n, tmax, hkv * group)[b, r - cu[b]]
    return {"out": out.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------- their definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s, case) if case["op"] == "rope" else _exact_chunk(s, case)


def _exact_rope(s, case):
    off, rot, bs = case["off"], case["rot"], case["block"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * s["inv_freq"][None, :])[:, None, :]

    def turned(x):
        x = x.double()
        y = x.clone()
        first = slice(off, off + rot, 2) if case["interleaved"] else slice(off, off + rot // 2)
        second = (slice(off + 1, off + rot, 2) if case["interleaved"]
                  else slice(off + rot // 2, off + rot))
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def stored(pool, x, scale):
        y = _shown(pool, case).double()
        if case["e4m3"]:
            x = (x / scale.double()[:, None]).clamp(-448, 448)
        flat = y.transpose(1, 2).reshape(-1, case["hkv"], case["d"])
        flat[s["slots"]] = x
        return flat.view(y.shape[0], bs, case["hkv"], case["d"]).transpose(1, 2)

    ks, vs = s["scales"] if case["e4m3"] else (None, None)
    got = {"q": turned(s["q"]), "k_pool": stored(s["k_pool"], turned(s["k"]), ks)}
    if s["v"] is not None:
        got["v_pool"] = stored(s["v_pool"], s["v"].double(), vs)
    return got


def _exact_chunk(s, case):
    news, lens = lengths(case)
    if sum(n * x for n, x in zip(news, lens)) * case["hq"] * case["d"] * 4 > 6e12:
        return None
    group = case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(news, lens)):
        pages = s["tables"][b, :-(-length // case["block"])].long()
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None, :]
        hidden = key > pos
        if case["window"]:
            hidden |= (key <= pos - case["window"]) & (key >= case["sinks"])
        for g in range(case["hkv"]):
            k = _shown(s["k_pool"], case)[pages, g].double().flatten(0, 1)[:length]
            v = _shown(s["v_pool"], case)[pages, g].double().flatten(0, 1)[:length]
            if case["e4m3"]:
                k, v = k * s["scales"][0][g].double(), v * s["scales"][1][g].double()
            for h in range(g * group, (g + 1) * group):
                x = s["q"][at:at + n, h].double() @ k.t() / math.sqrt(case["d"])
                x[hidden] = -math.inf
                z = torch.logsumexp(x, 1)
                out[at:at + n, h] = torch.exp_(x.sub_(z[:, None])) @ v
                lse[at:at + n, h] = z
        at += n
    return {"out": out, "lse": lse}
