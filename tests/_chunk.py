"""Inputs and the plain 64-bit definition of chunk attention, shared by its tests."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch


@dataclass
class ChunkCase:
    q: torch.Tensor              # [T, Hq, Dk] bf16 (padding rows included)
    cu: torch.Tensor             # [B + 1] int32
    k_pool: torch.Tensor         # bf16, or uint8 E4M3 codes
    v_pool: torch.Tensor | None  # None: values inside the keys
    dv: int
    tables: torch.Tensor
    lens: torch.Tensor
    scale: float
    window: int
    sinks: int
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None


def make(seed, chunks, hq, hkv, dk, bs, dv=None, latent=False, window=0, sinks=0, pad=(0, 0),
         e4m3=False, poison=False, scale=None):
    """`chunks`: (stored before, new) of each sequence; pad: rows before the
    first and after the last sequence; poison: every pool row that no sequence
    holds, and every block that only masked positions lie in, is NaN."""
    g = torch.Generator().manual_seed(seed)
    dv = dk if dv is None else dv
    lens = [c + n for c, n in chunks]
    counts = [-(-n // bs) for n in lens]
    nb = sum(counts) + 2
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((len(chunks), max(counts + [1])), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        tables[b, :c] = perm[at:at + c]
        at += c
    cu = [pad[0]]
    for _, n in chunks:
        cu.append(cu[-1] + n)
    T = cu[-1] + pad[1]
    bf = torch.bfloat16
    q = torch.randn(T, hq, dk, generator=g).to(bf)
    k = torch.randn(nb, hkv, bs, dk, generator=g).to(bf)
    v = None if latent else torch.randn(nb, hkv, bs, dv, generator=g).to(bf)
    ks = vs = None
    if e4m3:
        ks = (4 + torch.rand(hkv, generator=g)) / 448
        vs = (4 + torch.rand(hkv, generator=g)) / 448
        k = (k.float() / ks.view(1, -1, 1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v.float() / vs.view(1, -1, 1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    case = ChunkCase(q, torch.tensor(cu, dtype=torch.int32), k, v, dv, tables,
                     torch.tensor(lens, dtype=torch.int32),
                     1.0 / math.sqrt(dk) if scale is None else scale, window, sinks, ks, vs)
    if poison:
        held = torch.zeros(nb, bs, dtype=torch.bool)
        for b, (c, n) in enumerate(chunks):
            j = torch.arange(c + n)
            seen = j >= 0
            if window:
                seen = (j > c - window) | (j < sinks)       # by the first new token
            held[tables[b, j // bs].long(), j % bs] = seen
        for pool in (k, v):
            if pool is None:
                continue
            p = pool.transpose(1, 2)
            p[~held] = 0x7f if e4m3 else float("nan")
        # blocks that hold nothing any new token sees may have stale entries
        for b, (c, n) in enumerate(chunks):
            for i in range(counts[b]):
                if window and not held[tables[b, i].long()].any():
                    tables[b, i] = -1
    return case


def values(pool, scale):
    if pool.dtype == torch.uint8:
        return pool.view(torch.float8_e4m3fn).double() * scale.double().view(1, -1, 1, 1)
    return pool.double()


def reference(case):
    """out, lse, and the bounds' ingredients: sum_j p_j |v_j| (absv), the largest
    scale * sum_d |q_d k_d| of a row (mag), sum_j |v_j| over the sum of the
    probabilities taken against the row's largest (low), and the largest
    scale * max_d |q_d| * sum_d |k_d| (qlow).  Rows of padding are NaN."""
    T, hq, dk = case.q.shape
    hkv, bs = case.k_pool.shape[1], case.k_pool.shape[2]
    kp = values(case.k_pool, case.k_scale)
    vp = kp[..., :case.dv] if case.v_pool is None else values(case.v_pool, case.v_scale)
    out = torch.full((T, hq, case.dv), math.nan, dtype=torch.float64)
    absv, lse = out.clone(), torch.full((T, hq), math.nan, dtype=torch.float64)
    mag, qlow, low = lse.clone(), lse.clone(), out.clone()
    for b in range(case.lens.numel()):
        lo, hi = int(case.cu[b]), int(case.cu[b + 1])
        n, L = hi - lo, int(case.lens[b])
        if n == 0:
            continue
        p = L - n + torch.arange(n)
        j = torch.arange(L)
        seen = j[None] <= p[:, None]
        if case.window:
            seen &= (j[None] > p[:, None] - case.window) | (j[None] < case.sinks)
        blocks = case.tables[b, j // bs].long().clamp(min=0)
        for h in range(hq):
            gk = h * hkv // hq
            k, v = kp[blocks, gk, j % bs], vp[blocks, gk, j % bs]
            any_seen = seen.any(0)
            k, v = k.clone(), v.clone()
            k[~any_seen], v[~any_seen] = 0, 0
            qh = case.q[lo:hi, h].double()
            s = (qh @ k.T * case.scale).masked_fill(~seen, -math.inf)
            m = s.amax(-1, keepdim=True) if L else torch.full((n, 1), -math.inf)
            m = m.masked_fill(m == -math.inf, 0)
            e = torch.exp(s - m)
            l = e.sum(-1, keepdim=True)
            pr = torch.where(l > 0, e / l.clamp(min=1e-300), 0)
            out[lo:hi, h] = pr @ v
            absv[lo:hi, h] = pr @ v.abs()
            lse[lo:hi, h] = (m + l.log())[:, 0]
            low[lo:hi, h] = seen.double() @ v.abs() / l.clamp(min=1)
            a = (qh.abs() @ k.abs().T * case.scale).masked_fill(~seen, 0)
            mag[lo:hi, h] = a.amax(-1) if L else 0
            a = (qh.abs().amax(-1)[:, None] * k.abs().sum(-1) * case.scale).masked_fill(~seen, 0)
            qlow[lo:hi, h] = a.amax(-1) if L else 0
    return out, lse, absv, mag, low, qlow


def run(pkv, case, dev="cuda", flags=0, out=None, lse=None, workspace=None, stream=None):
    to = lambda t: None if t is None else t.to(dev)
    v = pkv.ValuesInKeys(case.dv) if case.v_pool is None else to(case.v_pool)
    how = dict(window=case.window, sink_tokens=case.sinks, flags=flags, out=out, lse=lse,
               workspace=workspace, stream=stream)
    if case.k_scale is not None:
        return pkv.paged_chunk_attn_e4m3(to(case.q), to(case.cu), to(case.k_pool), v,
                                         to(case.k_scale), to(case.v_scale), to(case.tables),
                                         to(case.lens), case.scale, **how)
    return pkv.paged_chunk_attn(to(case.q), to(case.cu), to(case.k_pool), v, to(case.tables),
                                to(case.lens), case.scale, **how)


def check(case, out, lse):
    """out and lse against the definition.

    out: each probability is rounded by at most 2^-8 of itself for the value
    product (bf16; E4M3 caches fp16, 2^-11), which moves out by at most
    2^-8 sum p |v|; the result is rounded by at most 2^-8 of itself; fp32
    sums, and probabilities from scores that are off as below, are covered by
    the score term.  fp16 steps by 2^-24 where the row's largest probability is 1
    or more: however small a probability, it is off by at most 2^-24 of the
    largest, 2^-24 sum |v|.
    lse, and each score: dk products summed in fp32, (dk + 2) 2^-24 of the sum
    of their magnitudes; the sum of probabilities 2^-17 relative.  E4M3: the
    second term of a query element steps by 2^-9 where the row's largest is 2^7
    or more, an element is off by up to 2^-17 of that."""
    ref, ref_lse, absv, mag, low, qlow = reference(case)
    out, lse = out.cpu().double(), lse.cpu().double()
    real = ~torch.isnan(ref_lse)
    empty = ref_lse == -math.inf
    assert torch.equal(torch.isinf(lse[real]), empty[real])
    assert torch.all(out[real & empty] == 0)
    rows = real & ~empty
    dk = case.q.shape[2]
    score = (dk + 2) * 2.0 ** -24 * mag[rows] + 2.0 ** -17
    if case.k_scale is not None:
        score = score + 2.0 ** -17 * qlow[rows]
    d_lse = (lse[rows] - ref_lse[rows]).abs()
    assert torch.all(d_lse <= score), float((d_lse - score).max())
    e4m3 = case.k_scale is not None
    vanish = 2.0 ** -24 * low[rows] if e4m3 else 0.0
    tol = ((2.0 ** -11 if e4m3 else 2.0 ** -8) + 2 * score[:, None]) * absv[rows] + 2.0 ** -8 * ref[rows].abs() + vanish
    d = (out[rows] - ref[rows]).abs()
    assert torch.all(d <= tol), float((d - tol).max())
    # the whole result is nearer than the worst case of every element at once
    rel = float(d.norm() / ref[rows].norm())
    assert rel <= 5e-3, rel
