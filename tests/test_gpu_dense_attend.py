"""GPU: attention over the cache against float64 of the query that the library documents (the bf16
query in a 16-bit fixed point of its head), so that the bound is a sum's rounding and nothing else."""
import math

import pytest
import torch

from tests.test_gpu_dense import BF, DEV, FP, csa2, gen, make_cache, row_of, rows64, seen_positions, table_for  # noqa: F401

pytestmark = pytest.mark.gpu


def fixed_point(q):
    """rint(q 2^k) / 2^k in float64, k = min(15 - e, 126), the head's largest element in [2^e, 2^(e+1))."""
    q = q.double()
    top = q.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1].double() - 1, torch.full_like(top, -127.0))
    k = torch.clamp(15 - e, max=126.0)
    return torch.round(q * 2.0 ** k) * 2.0 ** -k


def check_row(q, kv, sm_scale, out, lse=None, out_type=None):
    """One query row [16][512] over the rows kv (float64); returns the largest error over its bound."""
    q64 = fixed_point(q)
    s = q64 @ kv.T * sm_scale
    w = torch.softmax(s, -1)
    # a logit: six digits' sums of eight MMA steps and five additions, about 54 roundings of 2^-23
    # of partial sums that Cauchy-Schwarz bounds: 2^-17 in all.  It counts by the key's weight.
    ds = 2.0 ** -17 * abs(sm_scale) * q64.norm(dim=-1, keepdim=True) * kv.norm(dim=-1)
    mean = (w * ds).sum(-1, keepdim=True)
    n_add = 2.0 ** -23 * (kv.shape[0] / 16 + 32)                # P V adds 16 positions per step
    want, a = w @ kv, kv.abs()
    # P in f16: 2^-11, and 2^-36 of the largest weight where it is subnormal; exp2 2^-20
    tol = (w * ds) @ a + (mean + 2.0 ** -20 + 2.0 ** -11 + n_add) * (w @ a) + 2.0 ** -36 * a.sum(0)
    tol = tol + torch.finfo(out_type or out.dtype).eps / 2 * want.abs() * 1.01 + 1e-30
    worst = float(((out.double() - want).abs() / tol).max())
    if lse is not None:
        le = torch.logsumexp(s, -1)
        worst = max(worst, float(((lse.double() - le).abs() / (mean[:, 0] + n_add + 2.0 ** -20 + 2.0 ** -22 * le.abs())).max()))
    return worst


def attend(csa2, q, out, codes, scales, offs, max_n, ws=None, **kw):  # noqa: F811
    """One call over q.shape[0] rows; the workspace is its own unless one is given."""
    kw = dict(batch=offs.numel() - 1, max_n=max_n, kv_offsets=offs, codes=codes, scales=scales, q=q, out=out, **kw)
    if ws is None:
        ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
    csa2.attend_cache(csa2.cache_args(workspace=ws, **kw))
    assert csa2.check_device_status(ws) == 0


@pytest.mark.parametrize("max_n,batches", [(1024, [64, 62, 30, 5, 1, 63]), (512, [32, 31, 40, 16, 3])])
def test_one_workspace_serves_every_smaller_batch(csa2, max_n, batches):  # noqa: F811
    """Sized once for the largest batch; the sequences that remain are served as they end."""
    most = max(batches)
    codes, scales = make_cache(most * max_n, 1)
    every = rows64(codes, scales)
    q = torch.randn(most, 16, 512, generator=gen(2), device=DEV).to(BF)
    out = torch.empty(most, 16, 512, device=DEV)
    ws = None
    for batch in batches:
        lens = torch.tensor([max_n - 7 * (i % 50) for i in range(batch)])
        offs = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(DEV)
        if ws is None:
            a = csa2.cache_args(batch=most, max_n=max_n, kv_offsets=torch.zeros(most + 1, dtype=torch.int64, device=DEV), codes=codes,
                                scales=scales, q=q, out=out)
            ws = csa2.alloc_workspace(csa2.cache_workspace_size(a))
        out.fill_(7.0)
        attend(csa2, q[:batch], out[:batch], codes, scales, offs, max_n, ws=ws, sm_scale=512 ** -0.5)
        for b in range(0, batch, 5):
            assert check_row(q[b], every[offs[b]:offs[b + 1]], 512 ** -0.5, out[b]) <= 1
        assert (out[batch:] == 7.0).all()


@pytest.mark.parametrize("lens,window,q_per_seq", [([5000, 3, 0, 997], 0, 1), ([900, 130] * 40, 0, 1), ([9000, 700, 20], 1000, 3),
                                                   ([3, 1] * 700, 0, 1)])
def test_waits_that_give_up_anywhere_end_the_call(csa2, lens, window, q_per_seq):  # noqa: F811
    """Bounds from one poll to many: each call ends, with the timeout flagged or with the result, and
    leaves nothing behind for the next one."""
    B, rows = len(lens), len(lens) * q_per_seq
    codes, scales = make_cache(sum(lens), 8)
    offs = torch.tensor([0] + lens).cumsum(0).to(DEV)
    q = torch.randn(rows, 16, 512, generator=gen(9), device=DEV).to(BF)
    outs = [torch.empty(rows, 16, 512, device=DEV) for _ in range(2)]
    kw = dict(batch=B, q_per_seq=q_per_seq, max_n=max(lens), kv_offsets=offs, codes=codes, scales=scales, q=q, sm_scale=512 ** -0.5,
              window=window, sinks=4)
    if q_per_seq > 1:
        kw["q_pos"] = torch.tensor([max(0, n - q_per_seq) for n in lens], device=DEV)
    ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(out=outs[0], **kw)))
    csa2.attend_cache(csa2.cache_args(out=outs[0], workspace=ws, **kw))
    assert csa2.check_device_status(ws) == 0
    a = csa2.cache_args(out=outs[1], workspace=ws, **kw)
    for polls in (1, 2, 3, 5, 8, 13, 30, 60, 100, 200, 400, 1000, 3000, 10000):
        outs[1].fill_(5.0)
        csa2.set_wait_limit(ws, polls)
        csa2.attend_cache(a)
        status = csa2.check_device_status(ws)
        assert status in (0, 5) and (status == 5 or torch.equal(outs[0], outs[1]))
    csa2.set_wait_limit(ws, 0)
    csa2.attend_cache(a)
    assert csa2.check_device_status(ws) == 0 and torch.equal(outs[0], outs[1])
