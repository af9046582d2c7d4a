"""GPU: attention over the cache against float64 of the query that the library documents (the bf16
query in a 16-bit fixed point of its head), so that the bound is a sum's rounding and nothing else."""
import math

import pytest
import torch

from tests.test_gpu_dense import (BF, DEV, FP, blank_cache, csa2, freqs, gen, make_cache, row_of, rows64,  # noqa: F401
                                  seen_positions, table_for, turned)

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
    # a logit: six digits' sums of eight MMA steps and five additions of them, 54 roundings of up to
    # 2^-23 of partial sums; the digits' magnitudes add up to 3 |q| at most (4 = 8 - 4).  It counts
    # by the key's weight.
    ds = 54 * 3 * 2.0 ** -23 * abs(sm_scale) * (q64.abs() @ kv.abs().T)
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


def place(lens, page, seed):
    """Offsets, page table (or None) and rows of a cache of these lengths."""
    offs = torch.tensor([0] + lens).cumsum(0).to(DEV)
    if not page:
        return offs, None, max(1, sum(lens))
    pages = max(1, max(-(-n // page) for n in lens))
    return offs, table_for(len(lens), pages, len(lens) * pages + 3, seed), (len(lens) * pages + 3) * page


def run_and_check(csa2, lens, q_of, page=0, window=0, sinks=0, q_per_seq=1, q_pos=None, ratio=1, sm_scale=512 ** -0.5, spread=1.0,  # noqa: F811
                  out_type=FP, cache=None):
    offs, table, total = place(lens, page, 5)
    codes, scales = cache or make_cache(total, 6, spread)
    rows, max_n = len(lens) * q_per_seq, max(1, max(lens))
    q = q_of(rows).to(BF)
    out, lse = torch.empty(rows, 16, 512, dtype=out_type, device=DEV), torch.empty(rows, 16, device=DEV)
    attend(csa2, q, out, codes, scales, offs, max_n, q_per_seq=q_per_seq, window=window, sinks=sinks, ratio=ratio, sm_scale=sm_scale,
           lse=lse, page_table=table, page_rows=page, q_pos=None if q_pos is None else torch.tensor(q_pos, device=DEV))
    for r in range(rows):
        b, i = divmod(r, q_per_seq)
        p = seen_positions(lens[b], None if q_pos is None else q_pos[b] + i, ratio, window, sinks)
        if not p.numel():
            assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
            continue
        at = row_of(torch.full_like(p, b), p, offs, table, page)
        assert check_row(q[r], rows64(codes[at], scales[at]), sm_scale, out[r], lse[r]) <= 1, f"row {r}"


def test_the_bound_sees_one_position_of_500():
    """The check itself: float64 attention over one row more or less, or a row twice, is out of its bound."""
    kv = rows64(*make_cache(501, 1))
    q = torch.zeros(16, 512, dtype=BF, device=DEV)
    out, lse = kv[:500].mean(0).expand(16, 512), torch.full((16,), math.log(500.0), device=DEV, dtype=torch.float64)
    assert check_row(q, kv[:500], 0.1, out, lse, out_type=FP) <= 1
    for other in (kv, kv[:499], kv[1:500], torch.cat([kv[:499], kv[:1]])):
        assert check_row(q, other, 0.1, out, out_type=FP) > 2


def normal(gain, seed=3):
    return lambda rows: torch.randn(rows, 16, 512, generator=gen(seed), device=DEV) * gain


# gain 0: every key weighs the same, and one key more or less of 500 is several times the bound
@pytest.mark.parametrize("gain", [0.0, 0.3, 2.0])
@pytest.mark.parametrize("window,sinks,page", [(0, 0, 0), (0, 0, 128), (130, 5, 256), (128, 0, 0), (1, 1, 0), (700, 300, 128)])
def test_no_position_more_or_less(csa2, gain, window, sinks, page):  # noqa: F811
    run_and_check(csa2, [513, 128, 1, 0, 129, 1300, 255, 384], normal(gain), page=page, window=window, sinks=sinks)


@pytest.mark.parametrize("ratio", [1, 2])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 9)])
def test_no_position_more_or_less_for_drafts(csa2, ratio, window, sinks):  # noqa: F811
    run_and_check(csa2, [500, 260, 17, 0, 385], normal(0.0), window=window, sinks=sinks, q_per_seq=4, ratio=ratio,
                  q_pos=[1, 260 * ratio - 4, 1000, 3, 380 * ratio])


@pytest.mark.parametrize("n", [700, 5000])
@pytest.mark.parametrize("by", [1e2, 1e4, 1e6])
def test_a_channel_far_above_the_rest_of_its_query(csa2, n, by):  # noqa: F811
    """The rest is held to 2^-16 of the largest, as documented: the reference has the same fixed point."""
    def q_of(rows):
        q = normal(1.0)(rows)
        for h in range(16):
            q[:, h, 32 * h + h] = by
        return q
    run_and_check(csa2, [n, 50], q_of, sm_scale=512 ** -0.5 / by ** 0.5)


@pytest.mark.parametrize("gain,spread,sm_scale", [(2.0, 60.0, 512 ** -0.5), (20.0, 1.0, 512 ** -0.5), (2.0, 1.0, 1.0), (1e-30, 1.0, 1e30),
                                                  (2.0, 0.004, 1.0), (1e30, 1.0, 1e-31), (3e38, 1.0, 1e-38)])
def test_peaked_softmax_and_far_magnitudes(csa2, gain, spread, sm_scale):  # noqa: F811
    run_and_check(csa2, [900, 3, 2500], lambda rows: normal(1.0)(rows).clamp(-1, 1) * gain, spread=spread, sm_scale=sm_scale)


@pytest.mark.parametrize("falling", [False, True])
def test_running_reference(csa2, falling):  # noqa: F811
    """Tiles whose logits rise or fall throughout, for one head; the others see them in any order."""
    n = 4096
    codes, scales = make_cache(n, 12)
    q = normal(2.0)(1)
    order = torch.argsort(rows64(codes, scales) @ q[0, 3].to(BF).double(), descending=falling)
    run_and_check(csa2, [n], lambda rows: q, cache=(codes[order].contiguous(), scales[order].contiguous()), sm_scale=0.25)


@pytest.mark.parametrize("graph", [False, True])
def test_a_step_of_a_dense_layer_each_operator_from_what_the_last_one_left(csa2, graph):  # noqa: F811
    """Append, query, attention, rotation back and read-back of three steps, eager or as one captured
    graph that is replayed on new inputs; each result against float64 of the operands that it had."""
    g = gen(70)
    B, page, r = 3, 128, 64
    table = table_for(B, 5, 20, 3)
    codes, scales, _, _ = blank_cache(20 * page)
    lens = torch.tensor([126, 0, 511], device=DEV)
    old = torch.cat([torch.arange(int(n), device=DEV) for n in lens])
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), lens).to(torch.int32)
    csa2.append_rope(csa2.append_args(latent=torch.randn(old.numel(), 512, generator=g, device=DEV).to(BF), pos=old, seq=seq, codes=codes,
                                      scales=scales, page_table=table, page_rows=page))
    wq, wk, f = torch.rand(512, generator=g, device=DEV) + 0.5, torch.rand(512, generator=g, device=DEV) + 0.5, freqs(r)
    proj, pos = torch.empty(B, 17 * 512, dtype=BF, device=DEV), torch.empty(B, dtype=torch.int64, device=DEV)
    offs, rows = torch.zeros(B + 1, dtype=torch.int64, device=DEV), torch.empty(B, dtype=torch.int64, device=DEV)
    q, out = torch.empty(B, 16, 512, dtype=BF, device=DEV), torch.empty(B, 16, 512, device=DEV)
    back, got = torch.empty(B, 16, 512, dtype=BF, device=DEV), torch.empty(B, 512, dtype=BF, device=DEV)
    new = csa2.append_args(latent=proj[:, 8192:], pos=pos, codes=codes, scales=scales, page_table=table, page_rows=page, weight=wk,
                           inv_freq=f)
    query = csa2.rope_args(x=proj[:, :8192].unflatten(1, (16, 512)), out=q, pos=pos, inv_freq=f, weight=wq)
    kw = dict(batch=B, max_n=600, kv_offsets=offs, codes=codes, scales=scales, q=q, out=out, sm_scale=512 ** -0.5, page_table=table,
              page_rows=page)
    ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
    every = csa2.cache_args(workspace=ws, **kw)
    turn = csa2.rope_args(x=out, out=back, pos=pos, inv_freq=f, norm=False, inverse=True)

    def step():
        csa2.append_rope(new)
        csa2.norm_rope(query)
        csa2.attend_cache(every)
        csa2.norm_rope(turn)
        csa2.dequantize_kv(codes, scales, got, src_row=rows)

    def inputs(k):
        proj.copy_(torch.randn(B, 17 * 512, generator=gen(80 + k), device=DEV))
        pos.copy_(lens + k)
        offs[1:] = (pos + 1).cumsum(0)
        rows.copy_(row_of(torch.arange(B, device=DEV), pos, None, table, page))

    run = step
    if graph:
        inputs(0)
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        run = captured.replay
    for k in range(3):
        inputs(k)
        run()
        torch.cuda.synchronize()
        assert csa2.check_device_status(ws) == 0
        assert torch.equal(got.double(), rows64(codes[rows], scales[rows]))
        for b in range(B):
            p = torch.arange(int(pos[b]) + 1, device=DEV)
            at = row_of(torch.full_like(p, b), p, None, table, page)
            assert check_row(q[b], rows64(codes[at], scales[at]), 512 ** -0.5, out[b]) <= 1
        want = turned(out.double(), pos, f, sign=-1.0)
        # fp32 rotation 36 u32 of |u| + |v| <= 2 max, then one rounding to bf16
        tol = 72 * 2.0 ** -24 * out.abs().amax(-1, keepdim=True) + 2.0 ** -8 * want.abs()
        assert ((back.double() - want).abs() <= tol).all()


def test_selected_attention_right_behind_the_append(csa2):  # noqa: F811
    """csa2_attend launched behind the append of rows that it reads: as if the append had been waited for."""
    n, B = 400, 4
    offs = torch.arange(B + 1, device=DEV) * n
    lat = torch.randn(B * n, 512, generator=gen(90), device=DEV).to(BF)
    seq, pos = torch.arange(B, device=DEV).to(torch.int32).repeat_interleave(n), torch.arange(n, device=DEV).repeat(B)
    q, swa = torch.randn(B, 16, 512, generator=gen(91), device=DEV).to(BF), torch.randn(B, 128, 512, generator=gen(92), device=DEV).to(BF)
    topk = torch.full((B, 512), -1, dtype=torch.int32, device=DEV)
    topk[:, :n] = torch.arange(n, device=DEV)
    codes, scales, _, _ = blank_cache(B * n)
    outs = []
    new = csa2.append_args(latent=lat, pos=pos, seq=seq, codes=codes, scales=scales, kv_offsets=offs, inv_freq=freqs(64))
    for wait in (True, False, False):
        codes.fill_(0), scales.fill_(0)
        out = torch.empty(B, 16, 512, device=DEV)
        kw = dict(mode=csa2.MODE_REUSE, batch=B, q_per_seq=1, max_n=n, kv_offsets=offs, codes=codes, scales=scales, topk_idx=topk, q=q,
                  swa_kv=swa, out=out, sm_scale=512 ** -0.5)
        layer = csa2.layer_args(workspace=csa2.alloc_workspace(csa2.workspace_size(csa2.layer_args(**kw))), **kw)
        torch.cuda.synchronize()
        csa2.append_rope(new)
        if wait:
            torch.cuda.synchronize()
        csa2.attend(layer)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("window,ratio", [(0, 1), (130, 1), (0, 2), (1, 2)])
def test_many_queries_of_a_sequence(csa2, window, ratio):  # noqa: F811
    """A chunk's queries, each from its own position on: more than the row table holds, and a sequence
    that ends inside the chunk."""
    run_and_check(csa2, [300, 40, 0], normal(0.3), page=128, window=window, sinks=3 if window else 0, q_per_seq=101, ratio=ratio,
                  q_pos=[300 * ratio - 101, 0, 5])


@pytest.mark.parametrize("paged", [False, True])
def test_rows_past_32_bits_of_bytes(csa2, paged):  # noqa: F811
    """A cache of 17 M rows (4.35 GB of codes): append, read-back and attention at its end."""
    total, n, B = 17_000_064, 700, 2
    codes, scales = torch.empty(total, 256, dtype=torch.uint8, device=DEV), torch.empty(total, 32, dtype=torch.uint8, device=DEV)
    lat = torch.randn(B * n, 512, generator=gen(1), device=DEV).to(BF)
    seq, pos = torch.arange(B, device=DEV).to(torch.int32).repeat_interleave(n), torch.arange(n, device=DEV).repeat(B)
    table, offs = None, torch.tensor([total - 2 * n, total - n, total], device=DEV)
    if paged:
        last = total // 128 - 1
        table = torch.tensor([[last, 3, last - 2, last - 7, 0, last - 1], [5, last - 3, last - 5, last - 6, last - 4, 1]],
                             dtype=torch.int32, device=DEV)
    csa2.append_rope(csa2.append_args(latent=lat, pos=pos, seq=seq, codes=codes, scales=scales, page_table=table,
                                      kv_offsets=None if paged else offs, page_rows=128 if paged else 0, norm=False))
    rows = row_of(seq, pos, offs, table, 128)
    want = [torch.empty(B * n, k, dtype=torch.uint8, device=DEV) for k in (256, 32)]
    csa2.quantize_kv(lat, 1, *want)
    assert torch.equal(codes[rows], want[0]) and torch.equal(scales[rows], want[1])
    back = torch.empty(B * n, 512, dtype=BF, device=DEV)
    csa2.dequantize_kv(codes, scales, back, src_row=rows)
    kv = rows64(*want)
    assert torch.equal(back.double(), kv)
    q, out = normal(1.0)(B).to(BF), torch.empty(B, 16, 512, device=DEV)
    lens = torch.tensor([0, n, 2 * n], device=DEV) if paged else offs
    attend(csa2, q, out, codes, scales, lens, n, sm_scale=512 ** -0.5, page_table=table, page_rows=128 if paged else 0)
    for b in range(B):
        assert check_row(q[b], kv[b * n:(b + 1) * n], 512 ** -0.5, out[b]) <= 1


def test_queries_at_strides_past_32_bits(csa2):  # noqa: F811
    """Tokens 2^31 elements apart: what is read and written there, compared with the same tokens packed."""
    far = torch.empty((1 << 32) + 256, dtype=BF, device=DEV).as_strided((3, 2, 64), (1 << 31, 128, 1))
    x = torch.randn(3, 2, 64, generator=gen(5), device=DEV).to(BF)
    far.copy_(x)
    kw = dict(pos=torch.tensor([5, 1 << 40, 7], device=DEV), inv_freq=freqs(64))
    want, out = torch.empty_like(x), torch.empty_like(x)
    csa2.norm_rope(csa2.rope_args(x=x, out=want, **kw))
    csa2.norm_rope(csa2.rope_args(x=far, out=out, **kw))
    assert torch.equal(out, want)
    csa2.norm_rope(csa2.rope_args(x=far, out=far, **kw))
    assert torch.equal(far.contiguous(), want)


@pytest.mark.parametrize("rows,heads,dim,r", [(7, 16, 512, 64), (301, 3, 72, 30), (2, 1, 8, 8), (33, 2, 1024, 1024)])
def test_half_split_pairs_in_place(csa2, rows, heads, dim, r):  # noqa: F811
    x = torch.randn(rows, heads, dim, generator=gen(6), device=DEV).to(BF)
    out = torch.empty_like(x)
    kw = dict(pos=torch.arange(rows, device=DEV) * 77, inv_freq=freqs(r), half=True)
    csa2.norm_rope(csa2.rope_args(x=x, out=out, **kw))
    csa2.norm_rope(csa2.rope_args(x=x, out=x, **kw))
    assert torch.equal(x, out)


def test_two_graphs_that_share_a_workspace_in_turn(csa2):  # noqa: F811
    """Captured calls of different batches and plans over one workspace, replayed in turn on one stream."""
    lens = {"cut": [3000, 1, 777], "uncut": [128] * 70, "window": [5000] * 9}
    most = csa2.cache_workspace_size(csa2.cache_args(batch=70, max_n=5000, kv_offsets=torch.zeros(71, dtype=torch.int64, device=DEV),
                                                     codes=torch.empty(1, 256, dtype=torch.uint8, device=DEV),
                                                     scales=torch.empty(1, 32, dtype=torch.uint8, device=DEV),
                                                     q=normal(1.0)(70).to(BF), out=normal(1.0)(70)))
    ws, graphs = csa2.alloc_workspace(most), {}
    for name, n in lens.items():
        codes, scales = make_cache(sum(n), 4)
        q, out = normal(1.0)(len(n)).to(BF), torch.empty(len(n), 16, 512, device=DEV)
        a = csa2.cache_args(batch=len(n), max_n=max(n), kv_offsets=torch.tensor([0] + n).cumsum(0).to(DEV), codes=codes, scales=scales, q=q,
                            out=out, sm_scale=512 ** -0.5, window=300 if name == "window" else 0, sinks=4, workspace=ws)
        csa2.attend_cache(a)
        torch.cuda.synchronize()
        alone, g = out.clone(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            csa2.attend_cache(a)
        graphs[name] = (g, a, out, alone)
    for _ in range(3):
        for _, _, out, _ in graphs.values():
            out.fill_(9.0)
        for g, _, _, _ in graphs.values():
            g.replay()
        torch.cuda.synchronize()
        assert csa2.check_device_status(ws) == 0
        assert all(torch.equal(out, alone) for _, _, out, alone in graphs.values())
