"""Cases, plain forms and calls of what a server needs around a 4-bit cache: decode
attention over a cache held in 4 bits and the quantising append into it, block tables
and slot maps kept on the GPU from request lengths, and rotary positions of several
axes (time, height, width) fused with the append.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases
def _int4(name, **kw):
    case = dict(op="int4", name=name, seqs=8, ctx=32768, ragged=False, lens_seed=1, toks=1, hq=32,
                hkv=8, d=128, block=16)
    case.update(kw)
    return case


def _append(name, **kw):
    case = dict(op="append", name=name, tokens=64, hkv=8, d=128, block=16)
    case.update(kw)
    return case


def _axes(name, **kw):
    case = dict(op="axes", name=name, tokens=64, ctx=32768, hq=28, hkv=4, d=128, first=16,
                second=24, interleaved=False, e4m3=False, fp32_q=False, block=16, theta=1000000.0)
    case.update(kw)
    return case


def _tables(name, **kw):
    case = dict(op="tables", name=name, seqs=256, ctx=32768, new=1, ragged=False, lens_seed=1,
                block=16, blocks_left=1.0)
    case.update(kw)
    return case


def listed():
    return [
        # the continuous-batching mix: 16 sequences of 24 to 128 tokens; latency
        _int4("int4-mix", seqs=16, ctx=128, ragged=True),
        # the 8 x 32K decode step of the benchmark's headline, over 4 bits
        _int4("int4-32k"),
        # a serving batch of unequal lengths, head groups of 8, larger blocks
        _int4("int4-ragged", seqs=48, ctx=16384, ragged=True, hq=64, block=64, lens_seed=5),
        # four tokens a sequence, drafted and to be verified
        _int4("int4-spec", ctx=32768, toks=4),
        # one sequence of 200,000 tokens
        _int4("int4-200k", seqs=1, ctx=200000, hq=64),
        # small heads, two tokens a sequence, an odd length
        _int4("int4-d64", seqs=32, ctx=4095, toks=2, d=64, block=32),
        # a decode step's append of 64 sequences; latency
        _append("append-decode"),
        # a prompt chunk's append, odd length
        _append("append-prompt", tokens=8191),
        # prompts with images: 4,999 tokens with time, height and width
        _axes("axes-image", tokens=4999),
        # a decode step of 48 sequences into an FP8 cache, q kept in fp32; latency
        _axes("axes-decode-fp8", tokens=48, hq=64, hkv=8, e4m3=True, fp32_q=True),
        # a decode step's bookkeeping of 256 sequences; latency
        _tables("tables-decode"),
        # 1,000 sequences that bring 1 to 512 tokens each
        _tables("tables-batch", seqs=1000, new=512, ragged=True, ctx=4096, lens_seed=7),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    kind = rng.random()
    if kind < 0.5:
        most = max(work(c)["bytes"] for c in listed())
        while True:
            case = _int4("", seqs=_spread(rng, 1, 64), ctx=_spread(rng, 1, 200000),
                         ragged=rng.random() < 0.5, lens_seed=rng.randrange(1 << 20),
                         toks=rng.choice([1, 1, 1, 2, 3, 5, 8]), d=rng.choice([64, 128, 128]),
                         block=rng.choice([8, 16, 32, 64, 128]))
            case["hq"], case["hkv"] = rng.choice([(32, 8), (64, 8), (8, 8), (28, 4), (40, 8),
                                                  (16, 1)])
            keys = case["seqs"] * case["ctx"] * case["hkv"] * case["d"]
            scores = case["seqs"] * case["ctx"] * case["hq"] * case["toks"]
            if work(case)["bytes"] <= most and keys <= 6e8 and scores <= 2e8:
                break
    elif kind < 0.65:
        case = _append("", tokens=_spread(rng, 1, 8192), hkv=rng.choice([1, 4, 8]),
                       d=rng.choice([64, 96, 128, 256]), block=rng.choice([16, 32, 64]))
    elif kind < 0.8:
        case = _axes("", tokens=_spread(rng, 1, 5000), ctx=_spread(rng, 128, 200000),
                     interleaved=rng.random() < 0.5, e4m3=rng.random() < 0.4,
                     fp32_q=rng.random() < 0.3, block=rng.choice([16, 32, 64]),
                     theta=rng.choice([10000.0, 1000000.0]))
        case["hq"], case["hkv"] = rng.choice([(32, 8), (28, 4), (40, 8), (8, 8)])
        case["d"] = rng.choice([64, 128])
        case["first"] = rng.choice([8, 11, 16])
        case["second"] = rng.choice([8, 10])
    else:
        case = _tables("", seqs=_spread(rng, 1, 1024), ctx=_spread(rng, 1, 32768),
                       new=_spread(rng, 1, 512), ragged=rng.random() < 0.7,
                       lens_seed=rng.randrange(1 << 20), block=rng.choice([16, 32, 64]),
                       blocks_left=rng.choice([1.0, 1.0, 0.6]))
    case.pop("name")
    return case


def lengths(case):
    """Stored tokens of each sequence (int4: the new ones among them)."""
    rng = random.Random(case["lens_seed"])
    low = case.get("toks", 0) if case["op"] == "int4" else 0
    least = max(low, 24 if case["op"] == "int4" and case["ctx"] <= 128 else 0)
    most = max(case["ctx"], low)
    return [rng.randint(min(least, most), most) if case["ragged"] else most
            for _ in range(case["seqs"])]


def brought(case):
    """Tokens that each sequence of a `tables` case brings: some bring none."""
    rng = random.Random(case["lens_seed"] + 1)
    if not case["ragged"]:
        return [case["new"]] * case["seqs"]
    return [0 if rng.random() < 0.1 else _spread(rng, 1, case["new"])
            for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "int4":
        lens, d, t = lengths(case), case["d"], case["toks"]
        rows = case["seqs"] * t * case["hq"]
        pages = sum(-(-x // case["block"]) for x in lens)
        bytes_ = (sum(lens) * case["hkv"] * 2 * (d // 2 + 4) + rows * (8 * d + 4) + 4 * pages +
                  4 * len(lens))
        pairs = sum(t * x - t * (t - 1) // 2 for x in lens)
        return {"bytes": bytes_, "flops": 4 * d * case["hq"] * pairs}
    if case["op"] == "append":
        rows = case["tokens"] * case["hkv"] * 2
        return {"bytes": rows * (2 * case["d"] + case["d"] // 2 + 4) + 8 * case["tokens"],
                "flops": rows * case["d"] * 4}
    if case["op"] == "axes":
        t, d = case["tokens"], case["d"]
        kept = 1 if case["e4m3"] else 2
        bytes_ = t * (case["hq"] * d * (2 + (4 if case["fp32_q"] else 2)) +
                      2 * case["hkv"] * d * (2 + kept) + 8 + 3 * 8)
        return {"bytes": bytes_ + d * 4 + d // 2 * 4,
                "flops": t * d // 2 * (case["hq"] + case["hkv"]) * 6}
    lens, new, bs = lengths(case), brought(case), case["block"]
    taken = sum(-(-(a + n) // bs) + -a // bs for a, n in zip(lens, new))
    # extend: lengths, new lengths, the blocks taken, a token's position and slot; trim:
    # lengths and the blocks given back
    return {"bytes": 16 * sum(new) + 28 * len(lens) + 16 * taken, "flops": 2 * sum(new)}


# ------------------------------------------------------------- their inputs
def _quantise(x):
    """Rows of x (its last dim) as 4-bit codes, two to a byte, and their (scale, offset):
    an element is scale * code + offset."""
    x = x.float()
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    offset = low.to(torch.bfloat16)
    scale = ((high - offset.float()) * (1.0 / 15)).to(torch.bfloat16)
    s = scale.float()
    inverse = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    codes = ((x - offset.float()) * inverse).round_().clamp_(0, 15).to(torch.uint8)
    return codes[..., 0::2] | codes[..., 1::2] << 4, torch.cat((scale, offset), -1)


def _cache(case, blocks, gen):
    """K and V pools in 4 bits of N(0, 1) values; a few of the keys' channels larger."""
    pools = []
    for which in range(2):
        gain = 1 + 3 * (torch.rand(case["d"], generator=gen, device="cuda") < 0.03).bfloat16()
        codes, params = [], []
        # in parts: the values in fp32 would be eight times the cache
        for at in range(0, blocks, 4096):
            shape = (min(4096, blocks - at), case["hkv"], case["block"], case["d"])
            x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
            c, p = _quantise(x * gain if which == 0 else x)
            codes.append(c)
            params.append(p)
        pools += [torch.cat(codes), torch.cat(params)]
    return pools


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"] == "int4":
        lens, bs = lengths(case), case["block"]
        used = [-(-x // bs) for x in lens]
        blocks = sum(used) + 3
        s["k"], s["k_params"], s["v"], s["v_params"] = _cache(case, blocks, gen)
        order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        s["tables"] = torch.zeros(len(lens), max(used), device="cuda", dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            s["tables"][b, :n] = order[at:at + n]
            at += n
        s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["most"] = max(lens)
        shape = (case["seqs"], case["toks"], case["hq"], case["d"])
        s["q"] = normal(*shape, dtype=torch.float32)
        return s
    if case["op"] == "append":
        t, d, bs = case["tokens"], case["d"], case["block"]
        blocks = -(-t // bs) + 3
        s["k"], s["k_params"], s["v"], s["v_params"] = _cache(case, blocks, gen)
        s["k_new"], s["v_new"] = normal(t, case["hkv"], d), normal(t, case["hkv"], d)
        at = torch.arange(t, device="cuda")
        order = torch.randperm(blocks, generator=gen, device="cuda")
        s["slots"] = order[at // bs] * bs + at % bs
        return s
    if case["op"] == "axes":
        t, d, bs = case["tokens"], case["d"], case["block"]
        blocks = -(-t // bs) + 3
        shape = (blocks, case["hkv"], bs, d)
        s["k"], s["v"], s["scales"] = normal(*shape), normal(*shape), []
        if case["e4m3"]:
            s["scales"] = [(4.5 + torch.rand(case["hkv"], generator=gen, device="cuda")) / 448
                           for _ in range(2)]
            s["k"], s["v"] = ((x.float() / c.view(1, -1, 1, 1)).clamp_(-448, 448).to(E4M3)
                              .view(torch.uint8) for x, c in zip((s["k"], s["v"]), s["scales"]))
        s["q"] = normal(t, case["hq"], d)
        s["k_new"], s["v_new"] = normal(t, case["hkv"], d), normal(t, case["hkv"], d)
        # runs of text (all axes alike) and of images, 24 patches wide
        at = torch.arange(t, device="cuda")
        start = torch.randint(0, case["ctx"], (1,), generator=gen, device="cuda")
        image = (at // 500) % 2 == 1
        begin = start + at // 500 * 500
        within = at % 500
        s["positions"] = torch.stack((torch.where(image, begin, start + at),
                                      torch.where(image, begin + within // 24, start + at),
                                      torch.where(image, begin + within % 24, start + at)))
        pair = torch.arange(d // 2, device="cuda")
        s["pair_axis"] = ((pair >= case["first"]).to(torch.int32) +
                          (pair >= case["first"] + case["second"]).to(torch.int32))
        order = torch.randperm(blocks, generator=gen, device="cuda")
        s["slots"] = order[at // bs] * bs + at % bs
        s["inv_freq"] = case["theta"] ** (-2.0 * pair.double() / d)
        return s
    lens, new, bs = lengths(case), brought(case), case["block"]
    width = max(-(-(a + n) // bs) for a, n in zip(lens, new)) + 1
    held = [-(-a // bs) for a in lens]
    taken = sum(-(-(a + n) // bs) - h for a, n, h in zip(lens, new, held))
    free = max(1, int((taken + 5) * case["blocks_left"]))
    s["num_blocks"] = sum(held) + free
    order = torch.randperm(s["num_blocks"], generator=gen, device="cuda").to(torch.int32)
    s["free"] = order.clone()
    s["state"] = torch.tensor([free, 0, 0, 0], device="cuda", dtype=torch.int32)
    s["tables"] = torch.zeros(len(lens), width, device="cuda", dtype=torch.int32)
    held = torch.tensor(held, device="cuda")
    column = torch.arange(width, device="cuda")
    first = free + held.cumsum(0) - held
    s["tables"] = torch.where(column < held[:, None],
                              order[(first[:, None] + column).clamp_(max=len(order) - 1)],
                              s["tables"])
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["kept"] = s["lens"].clone()
    s["new"] = torch.tensor(new, device="cuda", dtype=torch.int32)
    # the rows of a captured step: the batch's tokens, rounded up
    s["rows"] = -(-max(1, sum(new)) // 64) * 64
    return s


# ------------------------------------------------------------- the operators
def run(s):
    case = s["case"]
    if case["op"] == "int4":
        out, lse = (_own_int4 if own else _plain_int4)(s, case)
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        (_own_append if own else _plain_append)(s, case)
        # codes are whole numbers, two to a byte
        return {n: s[n] for n in ("k", "k_params", "v", "v_params")}
    if case["op"] == "axes":
        q = (_own_axes if own else _plain_axes)(s, case)
        k, v = (x.view(E4M3) if case["e4m3"] else x for x in (s["k"], s["v"]))
        return {"q": q, "k": k, "v": v}
    # a step's tokens are placed and, all of them refused, taken back: the state is what
    # it was
    cu, positions, slots = (_own_tables if own else _plain_tables)(s, case)
    return {"cu": cu, "positions": positions, "slots": slots, "tables": s["tables"],
            "lens": s["lens"], "free": s["free"], "count": s["state"][:1]}


def _own_int4(s, case):
    import paged_kv_cache_93_gb300 as pkv
    scale = 1.0 / math.sqrt(case["d"])
    pools = (s["k"], s["k_params"], s["v"], s["v_params"])
    if case["toks"] > 1:
        return pkv.paged_decode_attn_multi_int4(s["q"], *pools, s["tables"], s["lens"], scale)
    out, lse = pkv.paged_decode_attn_int4(s["q"][:, 0], *pools, s["tables"], s["lens"], scale)
    return out[:, None], lse[:, None]


def _own_append(s, case):
    import paged_kv_cache_93_gb300 as pkv
    pkv.kv_append_int4(s["k"], s["k_params"], s["v"], s["v_params"], s["k_new"], s["v_new"],
                       s["slots"])


def _own_axes(s, case):
    import paged_kv_cache_93_gb300 as pkv
    call = pkv.rope_append_e4m3 if case["e4m3"] else pkv.rope_append
    return call(s["k"], s["v"], s["q"], s["k_new"], s["v_new"], s["positions"], s["slots"],
                s["inv_freq"], *s["scales"], interleaved=case["interleaved"],
                pair_axis=s["pair_axis"],
                q_dtype=torch.float32 if case["fp32_q"] else torch.bfloat16)


def _own_tables(s, case):
    import paged_kv_cache_93_gb300 as pkv
    pool = (s["free"], s["state"], case["block"])
    got = pkv.extend_sequences(s["tables"], s["lens"], s["new"], *pool, s["rows"])
    pkv.trim_sequences(s["tables"], s["lens"], s["kept"], *pool)
    return got


def _plain_int4(s, case):
    n, t, hkv, d, bs = case["seqs"], case["toks"], case["hkv"], case["d"], case["block"]
    group = case["hq"] // hkv
    j = torch.arange(s["most"], device="cuda")
    rows = s["tables"].long()[:, j // bs] * bs + j % bs
    lens = s["lens"].long()
    stored = (j < lens[:, None])[:, None, :, None]

    def gathered(pool, params):
        """The sequences' rows [seqs, hkv, tokens, d] in fp32."""
        at = pool.transpose(1, 2).reshape(-1, hkv, d // 2)[rows].transpose(1, 2)
        p = params.transpose(1, 2).reshape(-1, hkv, 2)[rows].transpose(1, 2).float()
        x = torch.stack((at & 15, at >> 4), -1).flatten(-2).float()
        return x.mul_(p[..., :1]).add_(p[..., 1:])

    k = gathered(s["k"], s["k_params"])
    q = s["q"].view(n, t, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * t, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    del k
    last = lens[:, None] - t + torch.arange(t, device="cuda")
    x = x.view(n, hkv, group, t, s["most"])
    x.masked_fill_((j > last[:, :, None])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m.masked_fill_(m == -math.inf, 0)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    v = gathered(s["v"], s["v_params"]).masked_fill_(~stored, 0)
    out = torch.matmul(x.view(n, hkv, group * t, s["most"]), v).view(n, hkv, group, t, d) / total
    lse = (m + total.log()).squeeze(-1)
    return (out.permute(0, 3, 1, 2, 4).reshape(n, t, case["hq"], d),
            lse.permute(0, 3, 1, 2).reshape(n, t, case["hq"]))


def _plain_append(s, case):
    block, at = s["slots"] // case["block"], s["slots"] % case["block"]
    for x, pool, params in (("k_new", "k", "k_params"), ("v_new", "v", "v_params")):
        s[pool][block, :, at], s[params][block, :, at] = _quantise(s[x])


def _plain_axes(s, case):
    # each pair's position is its axis's
    at = s["positions"][s["pair_axis"].long()].t().double()
    angle = at * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(2)
        a, b = x.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)

    def store(pool, x, scale):
        if case["e4m3"]:
            x = (x / scale.view(1, -1, 1)).clamp(-448, 448).to(E4M3).view(torch.uint8)
        pool[s["slots"] // case["block"], :, s["slots"] % case["block"]] = x.to(pool.dtype)

    ks, vs = s["scales"] if case["e4m3"] else (None, None)
    store(s["k"], turned(s["k_new"]), ks)
    store(s["v"], s["v_new"].float(), vs)
    q = turned(s["q"])
    return q if case["fp32_q"] else q.to(torch.bfloat16)


def _plain_tables(s, case):
    bs, tables, free = case["block"], s["tables"], s["free"]
    count = s["state"][0].long()
    old, new = s["lens"].long(), s["new"].long()
    column = torch.arange(tables.shape[1], device="cuda")
    # extend: from the first sequence whose blocks are not there on, those that need a
    # block bring nothing
    held = (old + bs - 1) // bs
    need = (old + new + bs - 1) // bs - held
    upto = need.cumsum(0)
    new = torch.where((need == 0) | (upto <= count), new, torch.zeros_like(new))
    now = (old + new + bs - 1) // bs
    before = upto - need
    at = (count - 1 - (before[:, None] + column - held[:, None])).clamp_(0, len(free) - 1)
    fresh = (column >= held[:, None]) & (column < now[:, None])
    tables.copy_(torch.where(fresh, free[at], tables))
    taken = (now - held).sum()
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    row = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(cu[1:], row, right=True).clamp_(max=len(old) - 1)
    live = row < cu[-1]
    position = old[b] + row - cu[b]
    slot = tables[b, (position // bs).clamp_(max=tables.shape[1] - 1)].long() * bs + position % bs
    positions = torch.where(live, position, -torch.ones_like(position))
    slots = torch.where(live, slot, -torch.ones_like(slot))
    s["lens"].copy_(old + new)
    # trim: the blocks past each kept length, the last sequence's last block first
    keep = s["kept"].long()
    left = (keep + bs - 1) // bs
    gone = now - left
    after = gone.flip(0).cumsum(0).flip(0) - gone
    back = (column >= left[:, None]) & (column < now[:, None])
    to = count - taken + after[:, None] + now[:, None] - 1 - column
    to = torch.where(back, to, torch.full_like(to, len(free)))
    longer = torch.cat((free, free.new_zeros(1)))
    longer.scatter_(0, to.flatten(), tables.flatten())
    free.copy_(longer[:-1])
    s["state"][0] = (count - taken + gone.sum()).to(torch.int32)
    s["lens"].copy_(keep)
    return cu.to(torch.int32), positions, slots


# ------------------------------------------------- their definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "int4":
        return _exact_int4(s, case)
    if case["op"] == "append":
        got = {}
        for new, params in (("k_new", "k_params"), ("v_new", "v_params")):
            x, p = s[new].double(), s[params].double()
            low = x.min(-1).values
            rows = torch.stack(((x.max(-1).values - low) / 15, low), -1)
            flat = p.transpose(1, 2).reshape(-1, case["hkv"], 2)
            flat[s["slots"]] = rows
            shape = (p.shape[0], case["block"], case["hkv"], 2)
            got[params] = flat.view(shape).transpose(1, 2)
        return {"k": None, "k_params": got["k_params"], "v": None, "v_params": got["v_params"]}
    if case["op"] == "axes":
        return _exact_axes(s, case)
    return None


def _exact_int4(s, case):
    t, d, bs, group = case["toks"], case["d"], case["block"], case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, length in enumerate(lengths(case)):
        pages = s["tables"][b, :-(-length // bs)].long()
        hidden = (torch.arange(length, device="cuda")[None, :] >
                  length - t + torch.arange(t, device="cuda")[:, None])
        for g in range(case["hkv"]):

            def rows(pool, params):
                byte = pool[pages, g].flatten(0, 1)[:length].int()
                p = params[pages, g].flatten(0, 1)[:length].double()
                x = torch.empty(length, d, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = (byte % 16).double(), (byte // 16).double()
                return p[:, :1] * x + p[:, 1:]

            k, v = rows(s["k"], s["k_params"]), rows(s["v"], s["v_params"])
            for h in range(g * group, (g + 1) * group):
                x = s["q"][b, :, h].double() @ k.t() / math.sqrt(d)
                x[hidden] = -math.inf
                z = torch.logsumexp(x, 1)
                out[b, :, h] = torch.exp(x - z[:, None]) @ v
                lse[b, :, h] = z
    return {"out": out, "lse": lse}


def _exact_axes(s, case):
    d, bs = case["d"], case["block"]
    at = torch.stack([s["positions"][a] for a in s["pair_axis"].tolist()], 1)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       at.double() * s["inv_freq"][None, :])[:, None, :]
    first, second = ((slice(0, d, 2), slice(1, d, 2)) if case["interleaved"]
                     else (slice(0, d // 2), slice(d // 2, d)))

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def stored(pool, x, scale):
        y = (pool.view(E4M3) if case["e4m3"] else pool).double()
        if case["e4m3"]:
            x = (x / scale.double()[:, None]).clamp(-448, 448)
        flat = y.transpose(1, 2).reshape(-1, case["hkv"], d)
        flat[s["slots"]] = x
        return flat.view(y.shape[0], bs, case["hkv"], d).transpose(1, 2)

    ks, vs = s["scales"] if case["e4m3"] else (None, None)
    return {"q": turned(s["q"]), "k": stored(s["k"], turned(s["k_new"]), ks),
            "v": stored(s["v"], s["v_new"].double(), vs)}
