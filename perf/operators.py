"""The dense-cache operators of libcsa2 as measurable cases: the query's head norm with its
position rotation, the cache append with norm and rotation on the way, the read-back of
cache rows, and the attention of new tokens over the whole FP4 cache (or over a sliding
window of it plus the first positions).

Each case is a dict of plain values.  ``run`` computes it in elementary torch operations,
or, with ``own`` set, through the library's entry points; ``exact`` computes it in float64
from the definitions.
"""
import math

import torch

own = False

D, HEADS, GROUP, IDX = 512, 16, 16, 64
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------------------ cases

def _norm(name, rows, heads, dim, rope, src="bf16", dst="bf16", strided=False, inverse=False, half=False):
    return {"name": name, "op": "norm_rope", "rows": rows, "heads": heads, "dim": dim, "rope": rope, "src": src,
            "dst": dst, "strided": strided, "inverse": inverse, "half": half}


def _append(name, batch, per_seq, n, page_rows, idx=True, strided=True, src="bf16", rope=64, idx_rope=64):
    return {"name": name, "op": "append", "batch": batch, "per_seq": per_seq, "n": n, "page_rows": page_rows,
            "idx": idx, "strided": strided, "src": src, "rope": rope, "idx_rope": idx_rope}


def _deq(name, rows, total, gather):
    return {"name": name, "op": "dequantize", "rows": rows, "total": total, "gather": gather}


def _attend(name, batch, n, ragged=False, page_rows=0, window=0, sinks=0, q=1, ratio=1):
    return {"name": name, "op": "attend", "batch": batch, "n": n, "ragged": ragged, "page_rows": page_rows,
            "window": window, "sinks": sinks, "q": q, "ratio": ratio}


def listed():
    return [
        # the queries of one decode step: 64 sequences, 16 heads of 512 with 64 rotated, cut out of a wider projection
        _norm("norm_rope_decode_64", 64, 16, 512, 64, strided=True),
        # the indexer queries of a small prefill chunk: 4 heads of 64, all of it rotated, half-split pairs
        _norm("norm_rope_index_1000", 1000, 4, 64, 64, half=True),
        # two 2,048-token prefill chunks: turns the fp32 attention output back by its query's angle
        _norm("norm_rope_back_4096", 4096, 16, 512, 64, src="f32", inverse=True),
        # one new position for each of 64 sequences in a paged cache, main row and indexer row
        _append("append_decode_64", 64, 1, 512, 256),
        # a prefill chunk's own tokens: two sequences, 4,096 positions each, packed cache
        _append("append_chunk_8192", 2, 4096, 8192, 0),
        # the rows of one Top-512 selection of 8 sequences read back
        _deq("dequantize_top512_8", 4096, 32768, True),
        # a cache of 131,072 rows read back whole
        _deq("dequantize_cache_128k", 131072, 131072, False),
        # one sequence with a short odd context
        _attend("attend_b1_1501", 1, 1501),
        # a ragged decode batch, pages of 128 rows, one sequence empty and one with a single position
        _attend("attend_b64_8k_paged", 64, 8192, ragged=True, page_rows=128),
        # long contexts, ragged, packed cache
        _attend("attend_b8_256k", 8, 262144, ragged=True),
        # a 128-position window and four first positions of long contexts
        _attend("window128_b64_32k_paged", 64, 32768, page_rows=512, window=128, sinks=4),
        # four drafted tokens per sequence over a 4,096-position window and four first positions
        _attend("window4k_b16_64k_draft4", 16, 65536, ragged=True, window=4096, sinks=4, q=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "dequantize", "attend", "attend", "window", "window"])
    if op == "norm_rope":
        dim = rng.choice([64, 128, 192, 256, 512])
        rope = rng.choice([r for r in (2, 32, 64, 128, dim) if r <= dim])
        heads = rng.choice([1, 2, 4, 7, 16, 32])
        rows = _log(rng, 1, max(1, 4096 * 16 * 512 // (heads * dim)) if heads * dim > 512 else 16384)
        inverse = rng.random() < 0.3
        return _norm("", rows, heads, dim, rope, rng.choice(["bf16", "bf16", "f16", "f32"]),
                     rng.choice(["bf16", "bf16", "f16", "f32"]), rng.random() < 0.5, inverse, rng.random() < 0.5)
    if op == "append":
        batch = _log(rng, 1, 128)
        per_seq = _log(rng, 1, max(1, 8192 // batch))
        page = rng.choice([0, 128, 256, 512])
        n = per_seq + rng.randrange(0, max(1, 16384 // batch - per_seq) + 1)
        return _append("", batch, per_seq, n, page, rng.random() < 0.7, rng.random() < 0.5,
                       rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([2, 32, 64, 128, 512]),
                       rng.choice([32, 64]))
    if op == "dequantize":
        total = _log(rng, 100, 131072)
        return _deq("", rng.randrange(1, total + 1), total, rng.random() < 0.5)
    ragged, page = rng.random() < 0.6, rng.choice([0, 128, 256, 512])
    batch = _log(rng, 1, 64)
    if op == "attend":
        n = _log(rng, 1, (1600000 if ragged else 1050000) // batch)
        return _attend("", batch, min(n, 262144), ragged, page, q=1, ratio=1)
    q, ratio = rng.choice([1, 1, 1, 2, 4, 7]), rng.choice([1, 1, 2])
    window = _log(rng, 1, 4096)
    n = _log(rng, 8, 1000000 // batch)
    return _attend("", batch, min(n, 131072), ragged, page, window, rng.choice([0, 1, 4, 16, 130]), q, ratio)


def _lens(case):
    """Positions of each sequence: all n, or spread over n/4 .. n with an empty one and a single one."""
    b, n = case["batch"], case["n"]
    if not case.get("ragged"):
        return [n] * b
    lens = [n if i == 0 else max(1, int(n * (0.25 + 0.75 * ((i * 0.6180339887) % 1.0)))) for i in range(b)]
    if b >= 4:
        lens[1], lens[2] = 0, 1
    return lens


def _tokens(case):
    """Token of each sequence's last query: the one that sees the whole cache."""
    return [n * case["ratio"] - 1 for n in _lens(case)]


def _seen(case):
    """(positions that each query row sees, positions that any query of each sequence sees)."""
    rows, union = [], []
    w, s, r = case["window"], case["sinks"], case["ratio"]
    for n, t in zip(_lens(case), _tokens(case)):
        vis = [min(n, max(0, (t - case["q"] + 1 + i + 1) // r)) for i in range(case["q"])]
        rows += [v if not w else min(v, s) + max(0, v - max(min(v, s), v - w)) for v in vis]
        lo, hi = vis[0], vis[-1]
        union.append(hi if not w else min(hi, s) + max(0, hi - max(min(hi, s), lo - w)))
    return rows, union


def work(case):
    op = case["op"]
    if op == "norm_rope":
        n = case["rows"] * case["heads"] * case["dim"]
        return {"bytes": n * (SIZE[case["src"]] + SIZE[case["dst"]]) + case["rows"] * 8 + case["dim"] * 4, "flops": 5.0 * n}
    if op == "append":
        n = case["batch"] * case["per_seq"]
        row = D * SIZE[case["src"]] + 288 + (IDX * 4 + 68 if case["idx"] else 0) + 12
        return {"bytes": n * row * 1.0 + n * (288 + 2 * D), "flops": 10.0 * n * D}
    if op == "dequantize":
        return {"bytes": case["rows"] * (288.0 + 2 * D + (8 if case["gather"] else 0)), "flops": 1.0 * case["rows"] * D}
    rows, union = _seen(case)
    n_rows = len(rows)
    return {"bytes": 288.0 * sum(union) + n_rows * HEADS * D * 4.0, "flops": 4.0 * HEADS * D * sum(rows)}


# ------------------------------------------------------------------------------ inputs

def _inv_freq(rope):
    return (10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)).float().to(DEV)


def _values(shape, dtype, gen, strided):
    """N(0,1) with a few channels four times as large, contiguous or cut out of a wider matrix."""
    dim = shape[-1]
    wide = 1
    for s in shape[1:]:
        wide *= s
    buf = torch.empty(shape[0], wide + (64 if strided else 0), dtype=dtype, device=DEV)
    step = max(1, (1 << 27) // wide)
    gain = torch.ones(wide, device=DEV)
    gain[:: 64 if dim >= 64 else 8] = 4.0
    for i in range(0, shape[0], step):
        part = buf[i:i + step]
        part[:, :wide] = torch.randn(part.shape[0], wide, generator=gen, device=DEV) * gain
        if strided:
            part[:, wide:] = 1e4
    return buf[:, :wide].unflatten(1, shape[1:])


def _places(case, lens, gen):
    """kv_offsets, page table and rows of the whole cache; pages lie in a shuffled order."""
    page = case["page_rows"]
    offs = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(DEV)
    if not page:
        return offs, None, max(1, sum(lens))
    per = max(1, max(-(-n // page) for n in lens))
    need = per * case["batch"]
    order = torch.randperm(need + 3, generator=gen, device=DEV)[:need]
    return offs, order.to(torch.int32).view(case["batch"], per).contiguous(), (need + 3) * page


def _fill_cache(total, gen, want_idx):
    """A cache with every row written: codes and scales of N(0,1) latents with larger channels."""
    codes = torch.empty(total, 256, dtype=torch.uint8, device=DEV)
    scales = torch.empty(total, 32, dtype=torch.uint8, device=DEV)
    for i in range(0, total, 131072):
        m = min(131072, total - i)
        x = _values((m, D), torch.bfloat16, gen, False)
        codes[i:i + m], scales[i:i + m] = _quantize(x)
    if not want_idx:
        return codes, scales, None, None
    idx_k = torch.randn(total, IDX, generator=gen, device=DEV).mul_(100).to(torch.float8_e4m3fn).view(torch.uint8)
    idx_s = torch.rand(total, generator=gen, device=DEV) * 0.01 + 0.001
    return codes, scales, idx_k, idx_s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "norm_rope":
        st["x"] = _values((case["rows"], case["heads"], case["dim"]), TYPES[case["src"]], gen, case["strided"])
        st["out"] = torch.empty(case["rows"], case["heads"], case["dim"], dtype=TYPES[case["dst"]], device=DEV)
        st["pos"] = torch.randint(0, 1 << 20, (case["rows"],), generator=gen, device=DEV)
        st["inv_freq"] = _inv_freq(case["rope"])
        st["weight"] = None if case["inverse"] else torch.rand(case["dim"], generator=gen, device=DEV) + 0.5
    elif op == "append":
        lens, per = [case["n"]] * case["batch"], case["per_seq"]
        st["offs"], st["table"], total = _places(case, lens, gen)
        st["codes"], st["scales"], st["idx_k"], st["idx_s"] = _fill_cache(total, gen, case["idx"])
        n = case["batch"] * per
        st["seq"] = torch.arange(case["batch"], device=DEV, dtype=torch.int32).repeat_interleave(per)
        st["pos"] = torch.arange(case["n"] - per, case["n"], device=DEV).repeat(case["batch"])
        st["latent"] = _values((n, D), TYPES[case["src"]], gen, case["strided"])
        st["proj"] = _values((n, IDX), torch.float32, gen, case["strided"]) if case["idx"] else None
        st["weight"] = torch.rand(D, generator=gen, device=DEV) + 0.5
        st["inv_freq"], st["idx_inv_freq"] = _inv_freq(case["rope"]), _inv_freq(case["idx_rope"]) if case["idx"] else None
        st["rows"] = _cache_rows(st, st["seq"].long(), st["pos"])
        st["back"] = torch.empty(n, D, dtype=torch.bfloat16, device=DEV)
    elif op == "dequantize":
        st["codes"], st["scales"], _, _ = _fill_cache(case["total"], gen, False)
        st["rows"] = torch.randint(0, case["total"], (case["rows"],), generator=gen, device=DEV) if case["gather"] else None
        st["out"] = torch.empty(case["rows"], D, dtype=torch.bfloat16, device=DEV)
    else:
        lens = _lens(case)
        st["offs"], st["table"], total = _places(case, lens, gen)
        st["codes"], st["scales"], _, _ = _fill_cache(total, gen, False)
        rows = case["batch"] * case["q"]
        st["q"] = (torch.randn(rows, HEADS, D, generator=gen, device=DEV) * 2).to(torch.bfloat16)
        st["out"] = torch.empty(rows, HEADS, D, dtype=torch.bfloat16, device=DEV)
        first = [t - case["q"] + 1 for t in _tokens(case)]
        st["q_pos"] = torch.tensor(first, dtype=torch.int64, device=DEV) if case["q"] > 1 or case["ratio"] > 1 else None
        st["max_n"] = max(1, max(lens))
        st["scale"] = 1.0 / math.sqrt(D)
    return st


# ------------------------------------------------------------------------------ plain forms

def _cache_rows(st, seq, pos):
    """Row in the cache of each (sequence, position)."""
    page = st["case"]["page_rows"]
    if not page:
        return st["offs"][seq] + pos
    return st["table"].long()[seq, torch.div(pos, page, rounding_mode="floor")] * page + pos % page


def _quantize(x):
    """bf16 rows -> codes [n][256], scales [n][32]: E4M3 of amax / 6, E2M1 of |x| / scale, to nearest even."""
    g = x.float().view(x.shape[0], 32, GROUP)
    scale = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    y = torch.where(s > 0, g.abs() / s, torch.zeros_like(g))
    mag = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = (mag + torch.signbit(g) * 8).view(x.shape[0], 256, 2)
    return (code[..., 0] + code[..., 1] * 16).to(torch.uint8), scale.view(torch.uint8)


def _rows_as_float(codes, scales):
    """The values of FP4 rows, fp32 [...][512]."""
    lut = torch.tensor(E2M1, device=DEV)
    pairs = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], -1)
    v = pairs[codes.int()].flatten(-2).unflatten(-1, (32, GROUP))
    return (v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _rotate(y, pos, inv_freq, half, inverse):
    """Rotates the last 2 len(inv_freq) channels of y [n][...][dim] by pos * inv_freq; the angles in 64 bits."""
    r = 2 * inv_freq.numel()
    a = pos.double().view([-1] + [1] * (y.dim() - 1)) * inv_freq.double()
    c, s = torch.cos(a).to(y.dtype), torch.sin(a).to(y.dtype)
    s = -s if inverse else s
    keep, tail = y[..., :-r], y[..., -r:]
    u, v = (tail[..., : r // 2], tail[..., r // 2:]) if half else (tail[..., 0::2], tail[..., 1::2])
    a, b = u * c - v * s, v * c + u * s
    return torch.cat([keep, torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)], -1)


def _normed(x, weight, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _plain_norm_rope(st):
    case, x = st["case"], st["x"].float()
    y = x if st["weight"] is None else _normed(x, st["weight"], 1e-6)
    st["out"].copy_(_rotate(y, st["pos"], st["inv_freq"], case["half"], case["inverse"]))
    return st["out"]


def _plain_append(st):
    # 64 bits up to the rounding to bf16: the FP4 codes that follow change at borders
    y = _rotate(_normed(st["latent"].double(), st["weight"].double(), 1e-6), st["pos"], st["inv_freq"], False, False)
    st["codes"][st["rows"]], st["scales"][st["rows"]] = _quantize(y.to(torch.bfloat16))
    if st["proj"] is not None:
        k = _rotate(st["proj"], st["pos"], st["idx_inv_freq"], False, False)
        ks = k.abs().amax(-1) / 448.0
        code = torch.where(ks.unsqueeze(-1) > 0, k / ks.unsqueeze(-1), torch.zeros_like(k)).clamp(-448.0, 448.0)
        st["idx_k"][st["rows"]] = code.to(torch.float8_e4m3fn).view(torch.uint8)
        st["idx_s"][st["rows"]] = ks
    st["back"].copy_(_rows_as_float(st["codes"][st["rows"]], st["scales"][st["rows"]]))


def _appended(st):
    out = [st["back"], st["scales"].view(torch.float8_e4m3fn)]
    return out + [st["idx_k"].view(torch.float8_e4m3fn), st["idx_s"]] if st["idx_k"] is not None else out


def _plain_dequantize(st):
    rows, n = st["rows"], st["case"]["rows"]
    c, s = (st["codes"][:n], st["scales"][:n]) if rows is None else (st["codes"][rows], st["scales"][rows])
    st["out"].copy_(_rows_as_float(c, s))
    return st["out"]


def _keys_of(st):
    """Positions [rows][L] that each query row sees, and which of them count."""
    case = st["case"]
    n = (st["offs"][1:] - st["offs"][:-1]).repeat_interleave(case["q"])
    if st["q_pos"] is not None:
        t = (st["q_pos"].unsqueeze(1) + torch.arange(case["q"], device=DEV)).flatten()
        n = torch.minimum(n, torch.div(t + 1, case["ratio"], rounding_mode="floor").clamp(min=0))
    n = n.unsqueeze(1)
    if not case["window"]:
        p = torch.arange(st["max_n"], device=DEV).expand(n.shape[0], -1)
        return p, p < n
    first = torch.arange(case["sinks"], device=DEV).expand(n.shape[0], -1)
    last = n - case["window"] + torch.arange(case["window"], device=DEV)
    return torch.cat([first, last], 1), torch.cat([first < n, last >= case["sinks"]], 1) & (n > 0)


def _plain_attend(st):
    case = st["case"]
    p, ok = _keys_of(st)
    seq = torch.arange(case["batch"], device=DEV).repeat_interleave(case["q"]).unsqueeze(1)
    rows = _cache_rows(st, seq, torch.where(ok, p, torch.zeros_like(p))).clamp(max=st["codes"].shape[0] - 1)
    kv = _rows_as_float(st["codes"][rows], st["scales"][rows])
    s = torch.matmul(st["q"].float(), kv.transpose(1, 2)) * st["scale"]
    s = s.masked_fill(~ok.unsqueeze(1), -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(s - m)
    st["out"].copy_(torch.matmul(w, kv) / w.sum(-1, keepdim=True).clamp(min=1e-30))
    return st["out"]


# ------------------------------------------------------------------------------ the library's calls

def _args(st):
    """The argument block and workspace that a serving loop keeps for its buffers."""
    from fp4_kv_cache_04_b200 import csa2
    if "args" in st:
        return csa2, st["args"]
    case = st["case"]
    if case["op"] == "norm_rope":
        st["args"] = csa2.rope_args(x=st["x"], out=st["out"], pos=st["pos"], inv_freq=st["inv_freq"], weight=st["weight"],
                                    norm=st["weight"] is not None, eps=1e-6, half=case["half"], inverse=case["inverse"])
    elif case["op"] == "append":
        st["args"] = csa2.append_args(
            latent=st["latent"], pos=st["pos"], seq=st["seq"], codes=st["codes"], scales=st["scales"],
            kv_offsets=None if st["table"] is not None else st["offs"], page_table=st["table"], page_rows=case["page_rows"],
            weight=st["weight"], eps=1e-6, inv_freq=st["inv_freq"], idx_proj=st["proj"], idx_inv_freq=st["idx_inv_freq"],
            idx_k=st["idx_k"], idx_kscale=st["idx_s"])
    else:
        kw = dict(batch=case["batch"], q_per_seq=case["q"], max_n=st["max_n"], kv_offsets=st["offs"], codes=st["codes"],
                  scales=st["scales"], q=st["q"], out=st["out"], window=case["window"], sinks=case["sinks"], q_pos=st["q_pos"],
                  ratio=case["ratio"], sm_scale=st["scale"], page_table=st["table"], page_rows=case["page_rows"])
        st["workspace"] = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
        st["args"] = csa2.cache_args(workspace=st["workspace"], **kw)
    return csa2, st["args"]


def run(st):
    op = st["case"]["op"]
    if op == "norm_rope":
        if own:
            csa2, a = _args(st)
            csa2.norm_rope(a)
            return st["out"]
        return _plain_norm_rope(st)
    if op == "append":
        if own:
            csa2, a = _args(st)
            csa2.append_rope(a)
            csa2.dequantize_kv(st["codes"], st["scales"], st["back"], src_row=st["rows"])
        else:
            _plain_append(st)
        return _appended(st)
    if op == "dequantize":
        if own:
            from fp4_kv_cache_04_b200 import csa2
            csa2.dequantize_kv(st["codes"], st["scales"], st["out"], src_row=st["rows"])
            return st["out"]
        return _plain_dequantize(st)
    if own:
        csa2, a = _args(st)
        csa2.attend_cache(a)
        return st["out"]
    return _plain_attend(st)


# ------------------------------------------------------------------------------ 64 bits

def _x_turn(y, pos, inv_freq, half, sign):
    """Rotation as a product of complex numbers."""
    r = 2 * inv_freq.numel()
    tail = y[..., -r:]
    z = torch.complex(tail[..., : r // 2].contiguous(), tail[..., r // 2:].contiguous()) if half else \
        torch.view_as_complex(tail.contiguous().unflatten(-1, (r // 2, 2)))
    w = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                    sign * torch.outer(pos.double(), inv_freq.double()))
    z = torch.view_as_real(z * w.view([w.shape[0]] + [1] * (y.dim() - 2) + [w.shape[1]]))
    out = y.clone()
    out[..., -r:] = torch.cat([z[..., 0], z[..., 1]], -1) if half else z.flatten(-2)
    return out


def _x_rms(x, weight):
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * weight.double()


def _x_e4m3(v):
    """Nearest E4M3 value of v >= 0 (ties to the even code), by search in the table of all of them."""
    table = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    hi = torch.searchsorted(table, v.clamp(max=448.0)).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    a, b = v.clamp(max=448.0) - table[lo], table[hi] - v.clamp(max=448.0)
    return table[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]


def _x_fp4_values(x):
    """The values that FP4 rows of x (bf16 values held in float64) stand for, and their scales."""
    g = x.unflatten(-1, (32, GROUP))
    s = _x_e4m3(g.abs().amax(-1) / 6.0)
    grid = torch.tensor(E2M1[:8], dtype=torch.float64, device=DEV)
    y = torch.where(s.unsqueeze(-1) > 0, g.abs() / s.unsqueeze(-1), torch.zeros_like(g))
    best = torch.zeros_like(y)
    for i in range(1, 8):                      # past the midpoint, or on it where the upper code is even
        mid = (grid[i - 1] + grid[i]) / 2
        best = torch.where((y > mid) | ((y == mid) & (i % 2 == 0)), grid[i], best)
    return (best * s.unsqueeze(-1) * torch.sign(g)).flatten(-2), s


def _x_rows(codes, scales):
    c = codes.long()
    both = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    mag, grid = both & 7, torch.tensor(E2M1[:8], dtype=torch.float64, device=DEV)
    v = torch.where(both > 7, -grid[mag], grid[mag])
    return v * scales.view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, -1)


def _x_place(st, b, p):
    """Row in the cache of positions p of sequence b."""
    page = st["case"]["page_rows"]
    if not page:
        return p + int(st["offs"][b])
    return st["table"][b].long().index_select(0, p // page) * page + p.remainder(page)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        x = st["x"].double()
        y = x if st["weight"] is None else _x_rms(x, st["weight"])
        return _x_turn(y, st["pos"], st["inv_freq"], case["half"], -1.0 if case["inverse"] else 1.0)
    if op == "append":
        y = _x_turn(_x_rms(st["latent"].double(), st["weight"]), st["pos"], st["inv_freq"], False, 1.0)
        back, s = _x_fp4_values(y.to(torch.bfloat16).double())
        scales = st["scales"].view(torch.float8_e4m3fn).double()
        scales[st["rows"]] = s
        if st["idx_k"] is None:
            return [back, scales]
        k = _x_turn(st["proj"].double(), st["pos"], st["idx_inv_freq"], False, 1.0)
        ks = k.abs().amax(-1) / 448.0
        idx_k, idx_s = st["idx_k"].view(torch.float8_e4m3fn).double(), st["idx_s"].double()
        idx_k[st["rows"]] = _x_e4m3(k.abs() / ks.unsqueeze(-1)) * torch.sign(k)
        idx_s[st["rows"]] = ks
        return [back, scales, idx_k, idx_s]
    if op == "dequantize":
        rows = torch.arange(case["rows"], device=DEV) if st["rows"] is None else st["rows"]
        return _x_rows(st["codes"][rows], st["scales"][rows])
    out = torch.zeros(case["batch"], case["q"], HEADS, D, dtype=torch.float64, device=DEV)
    lens, last = _lens(case), _tokens(case)
    for b in range(case["batch"]):
        every = torch.arange(lens[b], device=DEV)
        if not lens[b]:
            continue
        for i in range(case["q"]):
            seen = min(lens[b], (last[b] - case["q"] + 1 + i + 1) // case["ratio"])
            p = every[:max(0, seen)]
            p = p if not case["window"] else p[(p < case["sinks"]) | (p >= seen - case["window"])]
            if not p.numel():
                continue
            rows = _x_place(st, b, p)
            kv = _x_rows(st["codes"][rows], st["scales"][rows])
            w = torch.softmax(st["q"][b * case["q"] + i].double() @ kv.T * st["scale"], -1)
            out[b, i] = w @ kv
    return out.flatten(0, 1)
