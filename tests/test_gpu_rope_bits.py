"""What rope_append copies without turning it keeps its bits."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_rope import call, make, pkv, rows  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

# NaNs of either sign, quiet and signalling, with bits below; infinities; subnormals
ODD = [0x7fa1, -0x3d, 0x7f81, -0x7f, 0x7fff, -1, 0x7f80, -0x80, 0x0001, -0x7fff, -0x8000, 0x7fc0]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [3, 6000])
# heads of a power of two by a warp, other heads in units of 16, and what neither
# takes: vectors of 8 and single elements
@pytest.mark.parametrize("shape,rot,off", [
    ((4, 2, 128, 128, 16), 64, 32), ((4, 2, 128, 128, 16), 128, 0), ((6, 1, 576, None, 64), 64, 512),
    ((4, 2, 96, 64, 16), 32, 16), ((4, 2, 128, 128, 16), 16, 8), ((4, 2, 128, 128, 16), 6, 3)])
def test_copied_elements_keep_their_bits(pkv, shape, rot, off, T, interleaved):  # noqa: F811
    hq, hkv, dk, dv, bs = shape
    t = make(5, T, hq, hkv, dk, dv, bs)
    odd = torch.tensor(ODD, dtype=torch.int16)
    out = [i for i in range(dk) if not off <= i < off + rot]
    for name in ("q", "k", "v"):
        if t[name] is None:
            continue
        b = t[name].view(torch.int16)
        n = 4 * T * len(ODD)
        at = torch.randint(0, b.shape[2], (n,), generator=torch.Generator().manual_seed(n))
        if name != "v":
            if not out:
                continue
            at = torch.tensor(out)[at % len(out)]
        j = torch.arange(n)
        b[j % T, (j // T) % b.shape[1], at] = odd[j % len(ODD)]
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    q, kp, vp = call(pkv, t, inv, latent_dv=512, rotary_offset=off, interleaved=interleaved)
    same = lambda x, y: torch.equal(x.cpu().contiguous().view(torch.int16),
                                    y.contiguous().view(torch.int16))
    assert same(q[..., out], t["q"][..., out])
    assert same(rows(kp, t["slots"], bs)[..., out], t["k"][..., out])
    if vp is not None:
        assert same(rows(vp, t["slots"], bs), t["v"])
    # the fp32 queries hold the same numbers
    q, _, _ = call(pkv, t, inv, latent_dv=512, rotary_offset=off, interleaved=interleaved,
                   q_dtype=torch.float32)
    want = t["q"][..., out].float()
    assert torch.equal(q.cpu()[..., out].nan_to_num(7.0), want.nan_to_num(7.0))
    assert pkv.device_status(reset=True) == 0
