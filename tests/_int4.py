"""The 4-bit cache in plain torch on the CPU: its rows, its inputs, and decode attention
over it in 64 bits, shared by the tests."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

LEAST = 2.0 ** -126


def quantise(x):
    """Rows of x (fp32 or bf16) -> (codes uint8, two to a byte; params bf16), each
    operation rounded to binary32 as documented."""
    x = x.float()
    odd = ~torch.isfinite(x).all(-1, keepdim=True)
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    offset = low.to(torch.bfloat16)
    spread = (high - offset.float()).clamp_min(0)
    odd |= ~torch.isfinite(spread)
    scale = (spread * torch.tensor(1 / 15, dtype=torch.float32)).to(torch.bfloat16)
    scale = torch.where(scale.float() < LEAST, torch.zeros_like(scale), scale)
    s = scale.float()
    inverse = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    codes = ((x - offset.float()) * inverse).round().clamp(0, 15)
    codes = torch.where(odd, torch.zeros_like(codes), codes).to(torch.uint8)
    params = torch.cat((scale, offset), -1)
    params = torch.where(odd, torch.full_like(params, math.nan), params)
    return codes[..., 0::2] | codes[..., 1::2] << 4, params


def values(pool, params):
    """What the rows read back as, in 64 bits."""
    x = torch.stack((pool & 15, pool >> 4), -1).flatten(-2).double()
    return params[..., :1].double() * x + params[..., 1:].double()


def sizes(pool, params):
    """|scale| code + |offset| of every element: what its rounding errors scale with."""
    x = torch.stack((pool & 15, pool >> 4), -1).flatten(-2).double()
    return params[..., :1].double().abs() * x + params[..., 1:].double().abs()


@dataclass
class Case:
    q: torch.Tensor               # [B, T, Hq, Dk] fp32
    k: torch.Tensor
    k_params: torch.Tensor
    v: torch.Tensor
    v_params: torch.Tensor
    tables: torch.Tensor
    lens: torch.Tensor
    scale: float

    def pools(self, device="cuda"):
        return [t.to(device) for t in (self.k, self.k_params, self.v, self.v_params)]


def make(seed, lens, hq, hkv, dk, dv, bs, T=1, poison=True, wide=False, width=None, scale=None):
    """poison: every pool row that no sequence holds reads as NaN, its codes arbitrary;
    wide: the rows' scales spread over many powers of ten."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // bs) for n in lens]
    nb = sum(counts) + 2
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max(counts + [1]) if width is None else width), -1,
                        dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        tables[b, :c] = perm[at:at + c]
        at += c
    pools = []
    for d in (dk, dv):
        x = torch.randn(nb, hkv, bs, d, generator=g)
        if wide:
            x = x * 10 ** (6 * torch.rand(nb, hkv, bs, 1, generator=g) - 5) + \
                torch.randn(nb, hkv, bs, 1, generator=g)
        codes, params = quantise(x.to(torch.bfloat16))
        pools += [codes, params]
    if poison:
        held = torch.zeros(nb, bs, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(n):
                held[int(tables[b, j // bs]), j % bs] = True
        for params in (pools[1], pools[3]):
            params[~held[:, None].expand(nb, hkv, bs)] = math.nan
    q = torch.randn(len(lens), T, hq, dk, generator=g)
    return Case(q, *pools, tables, torch.tensor(lens, dtype=torch.int32),
                1.0 / math.sqrt(dk) if scale is None else scale)


def attend(c: Case):
    """-> out, lse, and how far each may be off (see `close`), in 64 bits."""
    B, T, Hq, Dk = c.q.shape
    hkv, bs = c.k.shape[1], c.k.shape[2]
    dv = 2 * c.v.shape[3]
    out = torch.zeros(B, T, Hq, dv, dtype=torch.float64)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        L = int(c.lens[b])
        pages = c.tables[b, :-(-L // bs)].long()
        for g in range(hkv):
            def rows(of, pool, params):
                return of(pool[pages, g].flatten(0, 1)[:L], params[pages, g].flatten(0, 1)[:L])
            k, v = rows(values, c.k, c.k_params), rows(values, c.v, c.v_params)
            ka, va = rows(sizes, c.k, c.k_params), rows(sizes, c.v, c.v_params)
            for t in range(T):
                n = L - T + 1 + t
                if n <= 0:
                    continue
                hs = slice(g * (Hq // hkv), (g + 1) * (Hq // hkv))
                q = c.q[b, t, hs].double()
                s = c.scale * q @ k[:n].T
                z = torch.logsumexp(s, 1)
                p = torch.exp(s - z[:, None])
                out[b, t, hs], lse[b, t, hs] = p @ v[:n], z
                # a score's error: 2^-18 of the sum of its terms' sizes (a product of 22
                # significant bits or more, at most 40 roundings of 2^-24 or 16 of 2^-23 in
                # its sum), and in base 2 half a step of its own size
                e = 2.0 ** -18 * abs(c.scale) * (q.abs() @ ka[:n].T).max(1).values
                e = e + 2.0 ** -22 * s.abs().max(1).values
                # both ends of the quotient, and 2^-18 for the exponential, the weights' 22
                # bits and the sums
                tol[b, t, hs] = (2 * e + 2.0 ** -18)[:, None] * (p @ va[:n])
                ltol[b, t, hs] = e + 2.0 ** -20 * (1 + z.abs())
    return out, lse, tol, ltol


def close(got, lse, ref):
    ro, rl, tol, ltol = ref
    got, lse = got.cpu().double().view(ro.shape), lse.cpu().double().view(rl.shape)
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert torch.all(got[empty] == 0)
    err = (got - ro).abs()
    assert torch.all(err <= tol), float((err / tol.clamp_min(1e-300)).max())
    err = (lse - rl).abs()[~empty]
    assert torch.all(err <= ltol[~empty]), float((err / ltol[~empty]).max())
