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

// Rows that see nothing: zeros, lse -inf.  One warp of each CTA; CTA c looks at rows 32 c ..
// + 31 of every 32 x grid rows at once.
__device__ __forceinline__ void empty_rows(const CacheParams& p) {
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    const int lane = threadIdx.x & 31;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * 32) {
        unsigned none = __ballot_sync(0xFFFFFFFFu, r0 + lane < rows && row_view(p, r0 + lane).tiles == 0);
        for (; none; none &= none - 1) {
            const int64_t r = r0 + __ffs(none) - 1;
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + r * HEADS * D * (p.out_f32 ? 4 : 2));
            for (int i = lane; i < HEADS * D * (p.out_f32 ? 4 : 2) / 16; i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse && lane < HEADS) p.lse[r * HEADS + lane] = -INFINITY;
        }
    }
}

// ---------------------------------------------------------------- the kernel
constexpr int AC_THREADS = 512;
constexpr int AC_WARPS = AC_THREADS / 32;
constexpr int AC_PV_WARPS = 8;                     // warps 0-7: P V
constexpr int AC_SM_WARP = 8;                      // warps 8-11: softmax (TMEM lane quarters 0-3)
constexpr int AC_TMA_WARP = 12;
constexpr int AC_MMA_WARP = 13;
constexpr int AC_SYNC = AC_THREADS - 32;           // every warp but the producer
constexpr int AC_STAGES = 5;
constexpr int AC_CODE_BYTES = CACHE_TILE * ROW_CODES;                    // two panels of 16 KB
constexpr int AC_STAGE_BYTES = AC_CODE_BYTES + CACHE_TILE * ROW_SCALES;  // 36 KB
constexpr int AC_DIGITS = 6;
constexpr int AC_N = AC_DIGITS * HEADS;            // columns of S: digit d of head h in 16 d + h
constexpr int AC_QPANEL = AC_N * 128;
constexpr int AC_P_BYTES = CACHE_TILE * HEADS * 2;
// tensor memory: two S accumulators, the tile's scales twice, the digits' scales
constexpr uint32_t AT_COLS = 512, AT_S = 0, AT_S_STEP = 128, AT_SFA = 256, AT_SFB = 320;
// named barriers
constexpr int BAR_ROW = 1, BAR_VOTE = 2, BAR_MAX = 3, BAR_PV = 4;
constexpr float AC_GAP = 4.0f;                     // the reference maximum moves by more than 2^4 ...
constexpr float AC_SHIFT = 11.0f;                  // ... and P is kept times 2^11, at most 2^15 in f16
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct alignas(1024) CacheSmem {
    uint8_t stage[AC_STAGES][AC_STAGE_BYTES];
    union {
        struct {
            uint8_t q[2 * AC_QPANEL];              // query digits, K-major SW128 panels
            uint8_t p[2][AC_P_BYTES];              // P [key][head] f16
        } a;
        float4 x[AC_PV_WARPS][8][32];              // O exchanged between the two key halves
    } u;
    uint8_t sf[2][8][512];                         // a tile's scales as 32 x 16 B blocks
    uint64_t full[AC_STAGES], empty[AC_STAGES], s_full[2], s_empty[2], p_full[2], p_empty[2], drain;
    float alpha[2][HEADS];
    float part_m[4][HEADS], l[4][HEADS], m[HEADS], f[HEADS];
    int moved[2];
    int issued[AC_STAGES];                         // copies issued into each stage
    uint32_t tmem;
    int64_t red[34];
};
static_assert(sizeof(CacheSmem) + 1024 <= 232448, "shared memory of one SM");
static_assert(sizeof(CacheSmem::u) == 32768, "O exchange over the query digits and P");

// kind::mxf4nvf4, A = B = E2M1, scales E4M3, M = 128 keys, N = 96
constexpr uint32_t AC_IDESC = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(AC_N >> 3) << 17) |
                              (static_cast<uint32_t>(CACHE_TILE >> 4) << 24);

// Descriptor of a 32-row x 16-byte block without swizzle (8-row groups 128 bytes apart).
__device__ __forceinline__ uint64_t desc_rows16(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// 32 rows of 16 bytes -> 4 columns of tensor memory, in every quarter of the lanes.
__device__ __forceinline__ void tmem_copy_rows16(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ bool vote_barrier(int id, int threads, bool v) {
    uint32_t r;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %3, 0; barrier.cta.red.or.pred q, %1, %2, p; selp.u32 %0, 1, 0, q; }"
                 : "=r"(r) : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v)) : "memory");
    return r != 0;
}

// exp2; the hardware approximation is good to 2^-22
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Four bytes, each two E2M1 codes (low nibble first) -> four f16x2.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
    asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; "
        "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Next row at or after `row` that sees anything (whole warp; there is one).
__device__ __forceinline__ int64_t next_row(const CacheParams& p, int64_t row) {
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    for (; row < rows; row += 32) {
        const int64_t r = row + (threadIdx.x & 31);
        const unsigned any = __ballot_sync(0xFFFFFFFFu, r < rows && row_view(p, r).tiles > 0);
        if (any) return row + __ffs(any) - 1;
    }
    return rows - 1;
}

// Head h of the row's query as six balanced base-8 digits: n = rint(q 2^k), 2^15 <= |n| <
// 2^16 for the head's largest element, n = sum_d e_d 8^d with e_d in -4 .. 3, every one of
// which E2M1 holds.  Adding 4 to every digit (0o444444) makes them plain octal digits.
// One warp, lane l holds channels 16 l .. + 15.
__device__ __forceinline__ void put_query(const CacheParams& p, CacheSmem& sm, int64_t row, int h) {
    const int lane = threadIdx.x & 31;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (row * HEADS + h) * D + lane * GROUP);
    const uint4 v0 = __ldg(src), v1 = __ldg(src + 1);
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t top = 0;                                       // largest magnitude, as bf16 bits
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const int e = static_cast<int>(top >> 7) - 127;         // largest in [2^e, 2^(e+1))
    const int k = min(15 - e, 126);
    const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    uint32_t n[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        n[2 * i] = static_cast<uint32_t>(__float2int_rn(__uint_as_float(w[i] << 16) * up) + 0x24924);
        n[2 * i + 1] = static_cast<uint32_t>(__float2int_rn(__uint_as_float(w[i] & 0xFFFF0000u) * up) + 0x24924);
    }
    uint8_t* base = sm.u.a.q + (lane >> 4) * AC_QPANEL + (lane & 1) * 8;
    const int chunk = (lane & 15) >> 1;
#pragma unroll
    for (int d = 0; d < AC_DIGITS; ++d) {
        uint32_t out[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {                       // channels 8 j .. + 7: 4 bytes
            uint32_t even = 0, odd = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                even |= ((n[8 * j + 2 * i] >> (3 * d)) & 7u) << (4 * i);
                odd |= ((n[8 * j + 2 * i + 1] >> (3 * d)) & 7u) << (4 * i);
            }
            // E2M1 codes of -4 .. 3 looked up four at a time
            out[j] = __byte_perm(0x0A0C0D0Eu, 0x05040200u, even) | (__byte_perm(0x0A0C0D0Eu, 0x05040200u, odd) << 4);
        }
        const int r = d * HEADS + h;
        *reinterpret_cast<uint2*>(base + r * 128 + ((chunk ^ (r & 7)) << 4)) = make_uint2(out[0], out[1]);
    }
    if (lane == 0) sm.f[h] = p.sm_scale * LOG2E * __uint_as_float(static_cast<uint32_t>(9 - k + 127) << 23);
}

__global__ void __launch_bounds__(AC_THREADS, 1)
attend_cache_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ CUtensorMap tm_codes,
                    const __grid_constant__ CUtensorMap tm_scales) {
    extern __shared__ uint8_t raw[];
    CacheSmem& sm = *reinterpret_cast<CacheSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;

    if (tid == 0) {
        for (int i = 0; i < AC_STAGES; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], AC_PV_WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], 4);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.p_empty[i], AC_PV_WARPS);
        }
        mbar_init(&sm.drain, 1);
        for (int i = 0; i < AC_STAGES; ++i) sm.issued[i] = 0;
        mbar_fence_init();
    }
    if (warp == AC_MMA_WARP) tmem_alloc(&sm.tmem, AT_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    if (warp >= AC_SM_WARP && warp < AC_SM_WARP + 4) {
        // scale of column n (row n of the query operand): 8^(n / 16) 2^-9, in lane n % 32 of
        // each quarter, column 4 s + n / 32 for the 64 channels of step s
        constexpr uint64_t codes = 0x0000685038200801ull;   // E4M3 of 2^-9, 2^-6, .. 2^6
        uint32_t y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int d = min(2 * (i & 3) + (lane >> 4), AC_DIGITS - 1);
            y[i] = static_cast<uint32_t>((codes >> (8 * d)) & 0xFFu) * 0x01010101u;
        }
        tmem_st32(tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + AT_SFB, y);
        tc_fence_before();
    }
    griddep_launch_dependents();
    griddep_wait();                                         // nothing global is touched before
    const Range range = my_range<AC_THREADS>(p, sm.red);
    if (tid < 2) p.meta[2 * blockIdx.x + tid] = -1;
    __syncthreads();
    tc_fence_after();

    unsigned* err = p.err;
    const uint32_t limit = wait_limit(err);
    bool dead = false;                                      // a wait ran out: no more waiting, no more issuing
    auto wait = [&](uint64_t* bar, int phase) {
        if (!dead && !mbar_wait(bar, static_cast<uint32_t>(phase & 1), err, limit)) dead = true;
    };

    if (warp == AC_TMA_WARP) {
        // ---- producer: runs ahead over the rows, AC_STAGES tiles at most
        int it = 0;
        int64_t row = range.row, left = range.count;
        int tile = range.tile;
        while (left > 0) {
            row = next_row(p, row);
            const RowView v = row_view(p, row);
            const int end = static_cast<int>(min(static_cast<int64_t>(v.tiles), tile + left));
            const int64_t b = row / p.q_per_seq, off = __ldg(p.kv_offsets + b);
            for (int t0 = tile; t0 < end; t0 += 32) {
                int y = 0;                                  // each lane looks one tile's row up
                if (t0 + lane < end) {
                    const int64_t r0 = p.rows.row(b, off, v.pos(t0 + lane));
                    const bool bad = r0 < 0 || r0 >= p.total_n;
                    if (bad) atomicOr(err, ERR_DEVICE);
                    y = static_cast<int>(bad ? p.total_n : r0);      // past the end: reads zeros
                }
                for (int i = 0; i < 32 && t0 + i < end; ++i, ++it) {
                    const int yi = __shfl_sync(0xFFFFFFFFu, y, i);
                    if (lane == 0) {
                        const int st = it % AC_STAGES;
                        if (it >= AC_STAGES) wait(&sm.empty[st], it / AC_STAGES - 1);
                        if (!dead) {
                            uint8_t* dst = sm.stage[st];
                            mbar_arrive_expect_tx(&sm.full[st], AC_STAGE_BYTES);
                            tma_load_2d(dst, &tm_codes, 0, yi, &sm.full[st]);
                            tma_load_2d(dst + AC_CODE_BYTES / 2, &tm_codes, 128, yi, &sm.full[st]);
                            tma_load_2d(dst + AC_CODE_BYTES, &tm_scales, 0, yi, &sm.full[st]);
                            sm.issued[st] = it / AC_STAGES + 1;
                        }
                    }
                    __syncwarp();
                }
            }
            left -= end - tile;
            tile = 0;
            ++row;
        }
        if (lane == 0) {                                    // no copy may land after the CTA is gone
            for (int st = 0; st < AC_STAGES; ++st)
                if (sm.issued[st]) mbar_wait(&sm.full[st], static_cast<uint32_t>((sm.issued[st] - 1) & 1), err);
        }
    } else {
        if (warp == AC_WARPS - 1) empty_rows(p);
        int it = 0;
        int64_t row = range.row, left = range.count;
        int tile = range.tile;
        while (left > 0) {
            row = next_row(p, row);
            const RowView v = row_view(p, row);
            const int end = static_cast<int>(min(static_cast<int64_t>(v.tiles), tile + left));
            for (int h = warp < AC_TMA_WARP ? warp : warp - 1; h < HEADS; h += AC_WARPS - 1) put_query(p, sm, row, h);
            fence_proxy_async_smem();
            named_barrier(BAR_ROW, AC_SYNC);

            if (warp == AC_MMA_WARP) {
                for (int t = tile; t < end; ++t, ++it) {
                    const int st = it % AC_STAGES, buf = it & 1;
                    wait(&sm.full[st], it / AC_STAGES);
                    if (it >= 2) wait(&sm.s_empty[buf], (it >> 1) - 1);
                    tc_fence_after();
                    // scales [key][32 B] -> per 64-channel step s a block of 32 rows x 16 B:
                    // row l holds the scale words of keys l, l + 32, l + 64, l + 96
                    uint32_t w[4][8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4* src = reinterpret_cast<const uint4*>(sm.stage[st] + AC_CODE_BYTES + (32 * q + lane) * ROW_SCALES);
                        const uint4 a = src[0], c = src[1];
                        w[q][0] = a.x, w[q][1] = a.y, w[q][2] = a.z, w[q][3] = a.w;
                        w[q][4] = c.x, w[q][5] = c.y, w[q][6] = c.z, w[q][7] = c.w;
                    }
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        *reinterpret_cast<uint4*>(sm.sf[buf][s] + 16 * lane) = make_uint4(w[0][s], w[1][s], w[2][s], w[3][s]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && !dead) {
                        const uint32_t sfa = tm + AT_SFA + 32 * buf;
#pragma unroll
                        for (int s = 0; s < 8; ++s) tmem_copy_rows16(sfa + 4 * s, desc_rows16(smem_u32(sm.sf[buf][s])));
                        const uint32_t ca = smem_u32(sm.stage[st]), qa = smem_u32(sm.u.a.q);
#pragma unroll
                        for (int s = 0; s < 8; ++s) {
                            const uint64_t da = umma_desc_sw128(ca + (s >> 2) * (AC_CODE_BYTES / 2) + (s & 3) * 32, 16, 1024);
                            const uint64_t db = umma_desc_sw128(qa + (s >> 2) * AC_QPANEL + (s & 3) * 32, 16, 1024);
                            mma_nvf4(tm + AT_S + AT_S_STEP * buf, da, db, AC_IDESC, sfa + 4 * s, tm + AT_SFB + 4 * s, s > 0);
                        }
                        mma_commit(&sm.s_full[buf]);
                    }
                    __syncwarp();
                }
            } else if (warp >= AC_SM_WARP && warp < AC_SM_WARP + 4) {
                // ---- softmax: thread = key
                const int quarter = warp & 3, key = 32 * quarter + lane;
                float m[HEADS], l[HEADS];
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    m[h] = -INFINITY;
                    l[h] = 0.0f;
                }
                for (int t = tile; t < end; ++t, ++it) {
                    const int st = it % AC_STAGES, buf = it & 1;
                    const bool vis = visible(p, v, v.pos(t) + key);
                    wait(&sm.s_full[buf], it >> 1);
                    tc_fence_after();
                    float s[HEADS];
                    const uint32_t src = tm + (static_cast<uint32_t>(32 * quarter) << 16) + AT_S + AT_S_STEP * buf;
#pragma unroll
                    for (int i = 0; i < AC_N / 32; ++i) {
                        uint32_t r[32];
                        tmem_ld32(src + 32 * i, r);
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) {
                            const float two = __uint_as_float(r[h]) + __uint_as_float(r[16 + h]);
                            s[h] = i ? s[h] + two : two;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.s_empty[buf]);
                    float d = -INFINITY;
#pragma unroll
                    for (int h = 0; h < HEADS; ++h) {
                        s[h] = vis ? s[h] * sm.f[h] : -INFINITY;
                        d = fmaxf(d, s[h] - m[h]);           // (-inf) - (-inf): NaN, which fmaxf drops
                    }
                    if (it >= 2) wait(&sm.p_empty[buf], (it >> 1) - 1);
                    const bool moved = vote_barrier(BAR_VOTE, 128, d > AC_GAP);
                    if (moved) {
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) {
                            float x = s[h];
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                            if (lane == 0) sm.part_m[quarter][h] = x;
                        }
                        named_barrier(BAR_MAX, 128);
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) {
                            const float mn = fmaxf(fmaxf(fmaxf(sm.part_m[0][h], sm.part_m[1][h]),
                                                         fmaxf(sm.part_m[2][h], sm.part_m[3][h])), m[h]);
                            const float a = mn == -INFINITY ? 1.0f : fast_exp2(m[h] - mn);
                            m[h] = mn;
                            l[h] *= a;
                            if (tid == 32 * AC_SM_WARP) sm.alpha[buf][h] = a;
                        }
                    }
                    if (tid == 32 * AC_SM_WARP) sm.moved[buf] = moved;
                    uint32_t pk[HEADS / 2];
#pragma unroll
                    for (int h = 0; h < HEADS; h += 2) {
                        const float a = vis ? fast_exp2(s[h] - m[h] + AC_SHIFT) : 0.0f;
                        const float b = vis ? fast_exp2(s[h + 1] - m[h + 1] + AC_SHIFT) : 0.0f;
                        l[h] += a;
                        l[h + 1] += b;
                        const __half2 two = __floats2half2_rn(a, b);
                        pk[h / 2] = *reinterpret_cast<const uint32_t*>(&two);
                    }
                    uint8_t* dst = sm.u.a.p[buf] + key * 32;
                    const int x = ((key >> 2) & 1) << 4;
                    *reinterpret_cast<uint4*>(dst + x) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    *reinterpret_cast<uint4*>(dst + (x ^ 16)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    if (!vis) {
                        // rows behind the sequence or its mask may hold any bytes, NaN scales among
                        // them: 0 x NaN must not reach O
                        uint4* z = reinterpret_cast<uint4*>(sm.stage[st] + AC_CODE_BYTES + key * ROW_SCALES);
                        z[0] = z[1] = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();            // before the next copy into this stage
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[buf]);
                }
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    float x = l[h];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                    if (lane == 0) {
                        sm.l[quarter][h] = x;
                        if (quarter == 0) sm.m[h] = m[h];
                    }
                }
                named_barrier(BAR_ROW, AC_SYNC);
            } else if (warp < AC_PV_WARPS) {
                // ---- P V: warp owns channels 128 (w % 4) .. + 127 of keys 64 (w / 4) .. + 63; lane
                // (g, t) converts channels 16 g .. + 15 of those (one scale group) of the keys of its
                // B fragments, n-tile i being channel i of every group
                const int wq = warp & 3, kh = warp >> 2, g = lane >> 2, t4 = lane & 3;
                float o[16][4] = {};
                const uint32_t code_off = (wq >> 1) * (AC_CODE_BYTES / 2) + (g & 1) * 8;
                const uint32_t chunk = (wq & 1) * 4 + (g >> 1);
                for (int t = tile; t < end; ++t, ++it) {
                    const int st = it % AC_STAGES, buf = it & 1;
                    wait(&sm.full[st], it / AC_STAGES);
                    wait(&sm.p_full[buf], it >> 1);
                    if (sm.moved[buf]) {
                        const float a0 = sm.alpha[buf][g], a1 = sm.alpha[buf][g + 8];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            o[i][0] *= a0;
                            o[i][1] *= a0;
                            o[i][2] *= a1;
                            o[i][3] *= a1;
                        }
                    }
                    const uint8_t* codes = sm.stage[st] + code_off;
                    const uint8_t* scales = sm.stage[st] + AC_CODE_BYTES + wq * 8 + g;
                    const uint32_t pa = smem_u32(sm.u.a.p[buf]);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const int kb = 64 * kh + 16 * ks;
                        uint32_t a[4];
                        {
                            const int key = kb + ((lane >> 4) << 3) + (lane & 7);
                            ldmatrix_x4_trans(a, pa + key * 32 + ((((lane >> 3) ^ (key >> 2)) & 1) << 4));
                        }
                        uint2 c[4];
                        uint32_t sc[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int key = kb + 2 * t4 + (j & 1) + 8 * (j >> 1);
                            c[j] = *reinterpret_cast<const uint2*>(codes + key * 128 + ((chunk ^ (key & 7)) << 4));
                            sc[j] = scales[key * ROW_SCALES];
                        }
                        const uint32_t s0 = e4m3x2_to_f16x2(static_cast<uint16_t>(sc[0] | (sc[1] << 8)));
                        const uint32_t s1 = e4m3x2_to_f16x2(static_cast<uint16_t>(sc[2] | (sc[3] << 8)));
#pragma unroll
                        for (int hw = 0; hw < 2; ++hw) {     // channels 8 hw .. + 7
                            const uint32_t a0 = hw ? c[0].y : c[0].x, a1 = hw ? c[1].y : c[1].x;
                            const uint32_t b0 = hw ? c[2].y : c[2].x, b1 = hw ? c[3].y : c[3].x;
                            // two keys' codes interleaved: byte i of ev / od = channel 2 i / 2 i + 1 of both
                            uint32_t e0[4], e1[4], d0[4], d1[4];
                            e2m1x8_to_f16((a0 & 0x0F0F0F0Fu) | ((a1 << 4) & 0xF0F0F0F0u), e0);
                            e2m1x8_to_f16(((a0 >> 4) & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u), d0);
                            e2m1x8_to_f16((b0 & 0x0F0F0F0Fu) | ((b1 << 4) & 0xF0F0F0F0u), e1);
                            e2m1x8_to_f16(((b0 >> 4) & 0x0F0F0F0Fu) | (b1 & 0xF0F0F0F0u), d1);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                mma_16816(o[8 * hw + 2 * i], a, mul_f16x2(e0[i], s0), mul_f16x2(e1[i], s1));
                                mma_16816(o[8 * hw + 2 * i + 1], a, mul_f16x2(d0[i], s0), mul_f16x2(d1[i], s1));
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.p_empty[buf]);
                        mbar_arrive(&sm.empty[st]);
                    }
                }
                named_barrier(BAR_ROW, AC_SYNC);            // every MMA of the row has read its operands
                // ---- the two key halves swap half of their channels: warp finishes n-tiles 8 kh .. + 7
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float (&mine)[4] = kh ? o[i] : o[8 + i];
                    sm.u.x[warp][i][lane] = make_float4(mine[0], mine[1], mine[2], mine[3]);
                }
                named_barrier(BAR_PV, 32 * AC_PV_WARPS);
                const bool whole = tile == 0 && end == v.tiles;
                const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);     // 0: the row this range starts in
                float* part = p.part + static_cast<int64_t>(slot) * CACHE_PART_FLOATS;
                float r[8][4];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 other = sm.u.x[warp ^ 4][i][lane];
                    const float (&mine)[4] = kh ? o[8 + i] : o[i];
                    r[i][0] = mine[0] + other.x;
                    r[i][1] = mine[1] + other.y;
                    r[i][2] = mine[2] + other.z;
                    r[i][3] = mine[3] + other.w;
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int h = g + 8 * hh;
                    const float ls = sm.l[0][h] + sm.l[1][h] + sm.l[2][h] + sm.l[3][h];
                    const float inv = whole ? 1.0f / ls : 1.0f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int ch = 128 * wq + 16 * (2 * t4 + e) + 8 * kh;
                        float val[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) val[i] = r[i][2 * hh + e] * inv;
                        const int64_t at = (row * HEADS + h) * D + ch;
                        if (whole && !p.out_f32) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const __nv_bfloat162 two = __floats2bfloat162_rn(val[2 * i], val[2 * i + 1]);
                                w[i] = *reinterpret_cast<const uint32_t*>(&two);
                            }
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
                            float4* dst = reinterpret_cast<float4*>(whole ? static_cast<float*>(p.out) + at
                                                                          : part + 2 * HEADS + h * D + ch);
                            dst[0] = make_float4(val[0], val[1], val[2], val[3]);
                            dst[1] = make_float4(val[4], val[5], val[6], val[7]);
                        }
                    }
                    if (wq == 0 && kh == 0 && t4 == 0) {
                        if (!whole) {
                            part[h] = sm.m[h] - AC_SHIFT;
                            part[HEADS + h] = ls;
                        } else if (p.lse) {
                            p.lse[row * HEADS + h] = (sm.m[h] - AC_SHIFT + log2f(ls)) * LN2;
                        }
                    }
                }
                if (!whole && tid == 0) p.meta[slot] = static_cast<int32_t>(row);
            }
            if (warp >= AC_MMA_WARP) {
                it += warp == AC_MMA_WARP ? 0 : end - tile;
                named_barrier(BAR_ROW, AC_SYNC);
            }
            named_barrier(BAR_ROW, AC_SYNC);                // the exchange is read: the next query may be written
            left -= end - tile;
            tile = 0;
            ++row;
        }
        if (warp == AC_MMA_WARP && lane == 0) {
            mma_commit(&sm.drain);
            mbar_wait(&sm.drain, 0, err);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == AC_MMA_WARP) tmem_dealloc(tm, AT_COLS);
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
    griddep_wait();
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

csa2_status launch_attend_cache(const CacheParams& p, const CUtensorMap& codes, const CUtensorMap& scales,
                                cudaStream_t stream) {
    const int smem = static_cast<int>(sizeof(CacheSmem) + 1024);
    if (!opt_in_smem(reinterpret_cast<const void*>(attend_cache_kernel), smem))
        return check_launch("attend_cache_kernel smem attribute");
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ranges));
    cfg.blockDim = dim3(AC_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, attend_cache_kernel, p, codes, scales);
    csa2_status st = check_launch("attend_cache_kernel");
    if (st != CSA2_OK || p.ranges == 1) return st;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(rows, p.ranges - 1)), AJ_SLICES);
    cfg.blockDim = dim3(AJ_THREADS);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchKernelEx(&cfg, join_cache_kernel, p);
    return check_launch("join_cache_kernel");
}

}  // namespace csa2
