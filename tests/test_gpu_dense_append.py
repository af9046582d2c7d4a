"""GPU: the append's rows next to the borders of their roundings, code for code."""
import numpy as np
import pytest
import torch

from oracle import csa2_oracle as O
from tests.test_gpu_dense import BF, DEV, FP, HF, blank_cache, csa2, freqs, gen, normed, turned  # noqa: F401

pytestmark = pytest.mark.gpu


def row_of_fp32(y):
    """Oracle codes and scales of float64 rows: rounded to fp32, that to bf16, then the FP4 rule."""
    bits = y.cpu().float().to(BF).view(torch.int16).numpy().view(np.uint16)
    return [torch.from_numpy(t).to(DEV) for t in O.quantize_rows(bits)]


def append(csa2, lat, pos=None, **kw):  # noqa: F811
    """One sequence of as many rows as the positions need; codes and scales of the tokens' rows."""
    n = lat.shape[0]
    pos = torch.arange(n, device=DEV) if pos is None else pos
    total = int(pos.max()) + 1
    codes, scales, _, _ = blank_cache(total)
    csa2.append_rope(csa2.append_args(latent=lat, pos=pos, seq=torch.zeros(n, dtype=torch.int32, device=DEV), codes=codes,
                                      scales=scales, kv_offsets=torch.tensor([0, total], device=DEV), **kw))
    return codes[pos], scales[pos]


# Halfway between two bf16 values of which the even one is a border of E2M1 at scale 1 (6 in the
# group): the border's side that a magnitude next to it takes depends on where it is rounded.
# From below 3.5 and 1.75 (ties to 4 and 2), from above 2.5, 1.25 and 5 (to 2, 1 and 4).
HALFWAY = [3.4921875, 1.74609375, 2.5078125, 1.25390625, 5.015625]


@pytest.mark.parametrize("by,src,below", [("norm", BF, True), ("norm", HF, True), ("norm", FP, True), ("norm", FP, False),
                                          ("rotation", FP, True), ("rotation", FP, False)])
def test_values_halfway_are_rounded_to_fp32_first(csa2, by, src, below):  # noqa: F811
    """Real numbers 2^-37 (or so) of themselves off such a halfway value: fp32 holds that value, and
    its rounding to bf16 is the even neighbour."""
    w = torch.full((32, 16), 6.0)
    for i, b in enumerate(HALFWAY):
        w[:, 2 * (i + 1)] = b
    w[1::2] *= -1
    w = w.flatten()
    if by == "norm":
        # mean(x^2) is 1 and eps 2^-36: 1 / rms = 1 - 2^-37; or 2^-32 less and no eps: 1 + 2^-33
        x, eps = torch.ones(3, 512), 2.0 ** -36
        if not below:
            x[:, 0], eps = 1 - 2.0 ** -24, 0.0
        lat, pos, kw = x.to(src).to(DEV), torch.arange(3, device=DEV), dict(weight=w.to(DEV), eps=eps)
        y = normed(lat.double(), kw["weight"], eps)
    else:
        # (u, 0) at a = p 2^-18 has u cos a = u (1 - p^2 2^-37); (u, -u 2^-17) has u (1 + (4 p - p^2) 2^-37)
        u = w.view(256, 2)[:, :1]
        lat = torch.cat([u, torch.zeros_like(u) if below else -u * 2.0 ** -17], 1).view(1, 512).repeat(3, 1).to(DEV)
        pos, kw = torch.arange(1, 4, device=DEV), dict(norm=False, inv_freq=torch.full((256,), 2.0 ** -18, device=DEV))
        y = turned(lat.double(), pos, kw["inv_freq"])
    assert ((y.abs() < w.abs().to(DEV)) == below)[:, 2:12:2].all()
    codes, scales = append(csa2, lat, pos, **kw)
    want = row_of_fp32(y)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("half", [False, True])
def test_a_chunk_of_normed_and_rotated_tokens_is_exact(csa2, seed, half):  # noqa: F811
    n = 8192
    g = gen(1000 + seed)
    lat = torch.randn(n, 512, generator=g, device=DEV)
    lat[:, ::64] *= 4
    lat = lat.to((BF, HF, FP)[seed % 3])
    w = torch.rand(512, generator=g, device=DEV) + 0.5
    pos = torch.randperm(1 << 17, generator=g, device=DEV)[:n]
    r = (64, 512)[seed // 3]
    codes, scales = append(csa2, lat, pos, weight=w, eps=1e-6, inv_freq=freqs(r), half=half)
    y = turned(normed(lat.double(), w, float(np.float32(1e-6))), pos, freqs(r), half)
    want = row_of_fp32(y)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
