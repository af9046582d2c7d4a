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


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("ri", [2, 32, 62])
@pytest.mark.parametrize("far", [False, True])
def test_indexer_channels_outside_the_rotation_are_copied(csa2, ri, half, far):  # noqa: F811
    """Infinities, NaN and zeros of both signs beside finite values, in the channels that are not
    turned: the codes and scales of append_kv.  The turned ones are finite and stand at position 0, or
    are zeros at far positions."""
    inf, nan, keep = float("inf"), float("nan"), 64 - ri
    special = [inf, -inf, nan, -nan, 0.0, -0.0, 448.0, -1e-30]
    n = len(special) ** 2
    proj = torch.randn(n, 64, generator=gen(ri), device=DEV)
    for i in range(n):                       # every pair of them, at an even and at an odd channel
        at = i % (keep - 1)
        proj[i, at], proj[i, at + 1] = special[i // len(special)], special[i % len(special)]
        if not i % 3:
            proj[i, :keep] = proj[i, :keep].nan_to_num(nan=-0.0, posinf=0.0, neginf=-0.0)
    pos = torch.zeros(n, dtype=torch.int64, device=DEV)
    if far:
        proj[:, keep:] = 0.0
        pos += torch.arange(n, device=DEV) * 1001 + 5
    lat, rows = torch.zeros(n, 512, dtype=BF, device=DEV), torch.arange(n, device=DEV)
    a, b = blank_cache(n), blank_cache(n)
    csa2.append_kv(lat, proj, rows, *a)
    # far: every page of sequence i is page i
    table = rows.to(torch.int32).view(n, 1).repeat(1, 1000)
    if far:
        b = blank_cache(128 * n)
        csa2.append_rope(csa2.append_args(latent=lat, pos=pos, codes=b[0], scales=b[1], page_table=table, page_rows=128, norm=False,
                                          half=half, idx_proj=proj, idx_inv_freq=freqs(ri), idx_k=b[2], idx_kscale=b[3]))
        b = [t[rows * 128 + pos % 128] for t in b]
    else:
        offs = torch.arange(n + 1, device=DEV)
        csa2.append_rope(csa2.append_args(latent=lat, pos=pos, codes=b[0], scales=b[1], kv_offsets=offs, norm=False, half=half,
                                          idx_proj=proj, idx_inv_freq=freqs(ri), idx_k=b[2], idx_kscale=b[3]))
    assert torch.equal(a[2][:, :keep], b[2][:, :keep])
    assert torch.equal(a[3].view(torch.int32), b[3].view(torch.int32))
    if not far:
        assert torch.equal(a[2], b[2])


@pytest.mark.parametrize("r", [0, 64])
def test_weights_that_bring_back_what_fp32_loses(csa2, r):  # noqa: F811
    """x / rms below fp32's normal range keeps 14 bits there, and a weight of 2^127 makes it count."""
    n = 4096
    g = gen(60)
    x = torch.randn(n, 512, generator=g, device=DEV)
    tiny = torch.zeros(512, dtype=torch.bool, device=DEV)
    tiny[32:96], tiny[200:216] = True, True
    x[:, tiny] = torch.randn(n, int(tiny.sum()), generator=g, device=DEV) * 2.0 ** -134
    w = torch.rand(512, generator=g, device=DEV) + 0.5
    w[tiny] *= 2.0 ** 127
    codes, scales = append(csa2, x, weight=w, eps=1e-6, inv_freq=freqs(r))
    y = turned(normed(x.double(), w, float(np.float32(1e-6))), torch.arange(n, device=DEV), freqs(r))
    want = row_of_fp32(y)
    assert (want[1][:, 2:6] > 0).any()
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
