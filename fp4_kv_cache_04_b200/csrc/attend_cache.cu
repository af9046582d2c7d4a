// Attention of new tokens over the FP4 cache without an index: every visible position, or
// the last `window` and the first `sinks` of them.  Per query row and head h
//     out_h = softmax_j(sm_scale * q_h . row_j) . rows   (row = the dequantised latent)
//
// Work split: the visible 128-position tiles of all rows form one list (first-position
// tiles, then window tiles, row after row), cut into equal ranges, one per CTA.  A row that
// lies inside one range is finished there; a row cut by range ends leaves one partial
// (running max m, sum l, unnormalised O) per range, joined by the second kernel in range
// order.  A range leaves at most two partials: of the row it starts in and of the row it
// ends in, so the workspace does not grow with the batch.
#include <algorithm>

#include "dense.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

// What a query row sees: positions j < n_vis with j < sinks or j >= w_beg, in `tiles`
// tiles: the first `ts` tiles of the sequence, then those from tile w0 on.
struct RowView {
    int n_vis, w_beg, ts, w0, tiles;
    __device__ __forceinline__ int pos(int tile) const { return (tile < ts ? tile : w0 + tile - ts) * CACHE_TILE; }
};

__device__ __forceinline__ RowView row_view(const CacheParams& p, int64_t row) {
    const int64_t b = row / p.q_per_seq;
    int64_t n = __ldg(p.kv_offsets + b + 1) - __ldg(p.kv_offsets + b);
    n = max(static_cast<int64_t>(0), min(n, p.max_n));
    if (p.q_pos) {
        const int64_t t = __ldg(p.q_pos + b) + row % p.q_per_seq + 1;
        n = min(n, max(static_cast<int64_t>(0), t / p.ratio));
    }
    RowView v;
    v.n_vis = static_cast<int>(n);
    const int64_t w = p.window > 0 ? max(static_cast<int64_t>(0), n - p.window) : 0;
    v.w_beg = static_cast<int>(w);
    const int64_t s = p.window > 0 ? min(p.sinks, n) : 0;
    v.w0 = static_cast<int>(w / CACHE_TILE);
    v.ts = static_cast<int>(min(ceil_div(s, CACHE_TILE), static_cast<int64_t>(v.w0)));
    v.tiles = n > 0 ? v.ts + static_cast<int>(ceil_div(n, CACHE_TILE)) - v.w0 : 0;
    return v;
}

__device__ __forceinline__ bool visible(const CacheParams& p, const RowView& v, int j) {
    return j < v.n_vis && (j >= v.w_beg || j < p.sinks);
}

constexpr int AC_THREADS = 256;
constexpr int AC_WARPS = AC_THREADS / 32;

// This CTA's range of the tile list: the row it starts in, the tile inside that row, and
// how many tiles follow.  Whole block; red: >= 33 words of shared memory.
struct Range {
    int64_t row;
    int tile;
    int64_t count;
};

template <int THREADS>
__device__ __forceinline__ Range my_range(const CacheParams& p, int64_t (&red)[34]) {
    constexpr int WARPS = THREADS / 32;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    int64_t sum = 0;
    for (int64_t r = tid; r < rows; r += THREADS) sum += row_view(p, r).tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) total += red[w];
    __syncthreads();
    // with fewer tiles than ranges the first `total` ranges take one each: a cut row's
    // ranges are always consecutive
    const int64_t c = blockIdx.x, g = min(static_cast<int64_t>(p.ranges), total);
    if (c >= g) return Range{0, 0, 0};
    const int64_t t0 = total * c / g, t1 = total * (c + 1) / g;
    Range out{0, 0, t1 - t0};
    if (tid == 0) red[32] = -1;
    int64_t base = 0;
    for (int64_t r0 = 0; r0 < rows; r0 += THREADS) {
        const int64_t r = r0 + tid;
        const int mine = r < rows ? row_view(p, r).tiles : 0;
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) red[warp] = inc;
        __syncthreads();
        int64_t before = base, all = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += red[w];
            all += red[w];
        }
        const int64_t first = before + inc - mine;
        if (mine > 0 && t0 >= first && t0 < first + mine) {
            red[32] = r;
            red[33] = t0 - first;
        }
        base += all;
        __syncthreads();
        if (red[32] >= 0) break;
        __syncthreads();
    }
    out.row = red[32];
    out.tile = static_cast<int>(red[33]);
    return out;
}

__device__ __forceinline__ void store_out(const CacheParams& p, int64_t row, int h, int c, float v) {
    const int64_t at = (row * HEADS + h) * D + c;
    if (p.out_f32) static_cast<float*>(p.out)[at] = v;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}

// Rows that see nothing: zeros, lse -inf (dealt over the CTAs, a warp each).
__device__ __forceinline__ void empty_rows(const CacheParams& p, int warp, int warps) {
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    const int lane = threadIdx.x & 31;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * warps + warp; r < rows; r += static_cast<int64_t>(gridDim.x) * warps) {
        if (row_view(p, r).tiles > 0) continue;
        for (int i = lane; i < HEADS * D; i += 32) store_out(p, r, i / D, i % D, 0.0f);
        if (p.lse && lane < HEADS) p.lse[r * HEADS + lane] = -INFINITY;
    }
}

// Warp w takes heads 4 (w % 4) .. + 3 of keys w / 4, w / 4 + 2, ...; lane l holds channels
// 16 l .. + 15 of the query and of O.
__global__ void __launch_bounds__(AC_THREADS)
attend_cache_kernel(CacheParams p) {
    __shared__ int64_t red[34];
    __shared__ float half_o[4][4][D];                 // O of the odd keys' warps
    __shared__ float half_m[4][4], half_l[4][4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int h0 = 4 * (warp % 4), odd = warp / 4;
    const Range range = my_range<AC_THREADS>(p, red);
    empty_rows(p, warp, AC_WARPS);
    if (tid < 2) p.meta[2 * blockIdx.x + tid] = -1;
    __syncthreads();

    int64_t row = range.row;
    int tile = range.tile;
    int64_t left = range.count;
    const float c = p.sm_scale * 1.4426950408889634f;
    while (left > 0) {
        const RowView v = row_view(p, row);
        if (v.tiles == 0) {
            ++row;
            continue;
        }
        const int end = static_cast<int>(min(static_cast<int64_t>(v.tiles), tile + left));
        const int64_t b = row / p.q_per_seq, off = __ldg(p.kv_offsets + b);
        float q[4][16], o[4][16] = {}, m[4], l[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                q[h][i] = bf16_bits_to_float(__ldg(p.q + (row * HEADS + h0 + h) * D + lane * GROUP + i));
        }
        for (int t = tile; t < end; ++t) {
            const int base = v.pos(t);
            const int64_t r0 = p.rows.row(b, off, base);
            const bool bad = r0 < 0 || r0 >= p.total_n;
            if (bad && tid == 0) atomicOr(p.err, ERR_DEVICE);
            for (int j = odd; j < CACHE_TILE && !bad; j += 2) {
                if (!visible(p, v, base + j) || r0 + j >= p.total_n) continue;
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.codes + (r0 + j) * ROW_CODES) + lane);
                const float s = e4m3_to_float(__ldg(p.scales + (r0 + j) * ROW_SCALES + lane));
                float k[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t code = ((i < 8 ? w.x : w.y) >> (4 * (i & 7))) & 15u;
                    const uint32_t e = (code >> 1) & 3u, f = code & 1u;
                    const float a = e ? static_cast<float>((2u + f) << (e - 1)) * 0.5f : 0.5f * static_cast<float>(f);
                    k[i] = (code & 8u ? -a : a) * s;
                }
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float d = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) d = fmaf(q[h][i], k[i], d);
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
                    d *= c;
                    const float mn = fmaxf(m[h], d), al = exp2f(m[h] - mn), pr = exp2f(d - mn);
                    m[h] = mn;
                    l[h] = l[h] * al + pr;
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[h][i] = fmaf(pr, k[i], o[h][i] * al);
                }
            }
        }
        // join the two key halves
        if (odd) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
#pragma unroll
                for (int i = 0; i < 16; ++i) half_o[warp % 4][h][lane * GROUP + i] = o[h][i];
                if (lane == 0) {
                    half_m[warp % 4][h] = m[h];
                    half_l[warp % 4][h] = l[h];
                }
            }
        }
        __syncthreads();
        const bool whole = tile == 0 && end == v.tiles;
        const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);     // 0: the row this range starts in
        if (!odd) {
            float* part = p.part + static_cast<int64_t>(slot) * CACHE_PART_FLOATS;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float m2 = half_m[warp][h], mn = fmaxf(m[h], m2);
                const float a = m[h] == -INFINITY ? 0.0f : exp2f(m[h] - mn), a2 = m2 == -INFINITY ? 0.0f : exp2f(m2 - mn);
                const float ls = l[h] * a + half_l[warp][h] * a2;
                const float inv = whole ? (ls > 0.0f ? 1.0f / ls : 0.0f) : 1.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int ch = lane * GROUP + i;
                    const float val = (o[h][i] * a + half_o[warp][h][ch] * a2) * inv;
                    if (whole) store_out(p, row, h0 + h, ch, val);
                    else part[2 * HEADS + (h0 + h) * D + ch] = val;
                }
                if (lane == 0) {
                    if (!whole) {
                        part[h0 + h] = mn;
                        part[HEADS + h0 + h] = ls;
                    } else if (p.lse) {
                        p.lse[row * HEADS + h0 + h] = (mn + log2f(ls)) * 0.6931471805599453f;
                    }
                }
            }
            if (!whole && tid == 0) p.meta[slot] = static_cast<int32_t>(row);
        }
        __syncthreads();
        left -= end - tile;
        tile = 0;
        ++row;
    }
}

// Joins the partials of one cut row.  Block (x, y): the x-th cut row (the x-th range whose
// first partial is its row's last one), 512 / AJ_SLICES channels.  A row's partials are
// partial 1 of the range it starts in and partials 0 of the following ones, in that order.
constexpr int AJ_SLICES = 16;
constexpr int AJ_THREADS = 128;

__global__ void __launch_bounds__(AJ_THREADS)
join_cache_kernel(CacheParams p) {
    __shared__ int sh[2];
    __shared__ int32_t meta[2 * CACHE_MAX_RANGES];
    const int tid = threadIdx.x;
    for (int i = tid; i < 2 * p.ranges; i += AJ_THREADS) meta[i] = p.meta[i];
    __syncthreads();
    if (tid == 0) {
        int seen = 0, last = -1;
        for (int g = 0; g < p.ranges; ++g) {
            const int32_t r = meta[2 * g];
            if (r < 0 || (g + 1 < p.ranges && meta[2 * (g + 1)] == r)) continue;
            if (seen++ == static_cast<int>(blockIdx.x)) {
                last = g;
                break;
            }
        }
        int first = last;
        if (last >= 0) {
            const int32_t r = meta[2 * last];
            while (first > 0 && meta[2 * first + 1] != r) --first;
        }
        sh[0] = first;
        sh[1] = last;
    }
    __syncthreads();
    const int first = sh[0], last = sh[1];
    if (last < 0) return;
    const int64_t row = meta[2 * last];
    const int h = tid / 8, c = blockIdx.y * (D / AJ_SLICES) + (tid % 8) * 4;
    float m = -INFINITY;
    for (int g = first; g <= last; ++g)
        m = fmaxf(m, p.part[static_cast<int64_t>(2 * g + (g == first ? 1 : 0)) * CACHE_PART_FLOATS + h]);
    float l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = first; g <= last; ++g) {
        const float* part = p.part + static_cast<int64_t>(2 * g + (g == first ? 1 : 0)) * CACHE_PART_FLOATS;
        const float a = part[h] == -INFINITY ? 0.0f : exp2f(part[h] - m);
        const float4 v = *reinterpret_cast<const float4*>(part + 2 * HEADS + h * D + c);
        l = fmaf(a, part[HEADS + h], l);
        o.x = fmaf(a, v.x, o.x);
        o.y = fmaf(a, v.y, o.y);
        o.z = fmaf(a, v.z, o.z);
        o.w = fmaf(a, v.w, o.w);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    store_out(p, row, h, c, o.x * inv);
    store_out(p, row, h, c + 1, o.y * inv);
    store_out(p, row, h, c + 2, o.z * inv);
    store_out(p, row, h, c + 3, o.w * inv);
    if (p.lse && blockIdx.y == 0 && tid % 8 == 0) p.lse[row * HEADS + h] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

int cache_ranges(int64_t rows, int64_t max_n, int64_t window, int64_t sinks) {
    // tiles of a row at most: the window may straddle one tile more than its length
    int64_t tiles = ceil_div(max_n, CACHE_TILE);
    if (window > 0) {
        const int64_t w = std::min(window, max_n), s = std::min(sinks, max_n);
        tiles = std::min(tiles, ceil_div(w, CACHE_TILE) + 1 + ceil_div(s, CACHE_TILE));
    }
    if (rows >= CACHE_MAX_RANGES || tiles >= CACHE_MAX_RANGES) return CACHE_MAX_RANGES;
    return static_cast<int>(std::min<int64_t>(CACHE_MAX_RANGES, std::max<int64_t>(1, rows * tiles)));
}

csa2_status launch_attend_cache(const CacheParams& p, cudaStream_t stream) {
    attend_cache_kernel<<<p.ranges, AC_THREADS, 0, stream>>>(p);
    csa2_status st = check_launch("attend_cache_kernel");
    if (st != CSA2_OK || p.ranges == 1) return st;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    const int cut = static_cast<int>(std::min<int64_t>(rows, p.ranges - 1));
    join_cache_kernel<<<dim3(cut, AJ_SLICES), AJ_THREADS, 0, stream>>>(p);
    return check_launch("join_cache_kernel");
}

}  // namespace csa2
