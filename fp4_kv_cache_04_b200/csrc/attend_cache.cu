// Attention of new tokens over the FP4 cache without an index: every visible position, or
// the last `window` and the first `sinks` of them.  Per query row and head h
//     out_h = softmax_j(sm_scale * q_h . row_j) . rows   (row = the dequantised latent)
// in one pass with a running reference m and sum l (rescaled when m moves).
//
// Work split: the visible 128-position tiles of all rows form one list (first-position
// tiles, then window tiles, row after row), cut into equal ranges, one per CTA (one CTA per
// SM).  A row that lies inside one range is finished there; a row cut by range ends leaves
// one partial (m, l, unnormalised O) per range, joined by the second kernel in range order,
// so results do not depend on timing.  A range leaves at most two partials: of the row it
// starts in and of the row it ends in, so the workspace does not grow with the batch.
//
// Logits on the block-scaled FP4 tensor core, straight from the stored codes: the bf16 query
// is written as six base-8 digits that E2M1 holds exactly (put_query), 16 heads x 6 digits =
// 96 columns, digit d under the scale 8^d; a tile is 8 tcgen05.mma M128 N96 K64 (57 cycles
// each, the instruction's least time, so the digits cost nothing over one), and its scales go
// to tensor memory by 8 tcgen05.cp.  P V on mma.sync, rows expanded in registers (the codes
// of two keys interleaved by nibble, cvt e2m1x2 -> f16x2, times the two keys' scales): 16
// heads fill its M = 16, while a tcgen05 MMA takes 45 to 57 cycles whatever its N up to 64 -
// 32 of them a tile, fed from tensor memory by the same conversions and beside the logits'
// MMAs, measured 2,500 cycles against 1,850 for this form alone.
//
// Roles (16 warps of 128 registers, all of the register file): 0-7 P V (warp = 128 channels
// of half the keys: 64-bit code loads without bank conflicts, 64 accumulators), 8-11
// softmax (thread = key, packed fp32), 12 TMA (4 stages of 36 KB), 13 and 14 scale words
// and MMAs of even and odd tiles, 15 the next row's query (with 13, 14) and the empty rows.
//
// Measured (1.83 GHz): 1.7 us a tile and SM, 3,140 cycles, against 1,580 for its 37 KB of
// HBM: P V alone takes 1,850, the logits' MMAs hold the tensor pipe for 490 more, and the
// softmax shares the issue slots (1,600 warp instructions a scheduler and tile).  1.07 M
// positions of 8 sequences: 118 us (47 at HBM's rate); 64 ragged sequences of up to 8,192 in
// pages: 55 us (15).  The first P is ready ~8 us into the launch (range 2.3, query 5, logits
// 7), a row's end costs 1.9 us, the join 3 to 7: these bound the short calls.
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

__device__ __forceinline__ int visible_positions(const CacheParams& p, int row) {
    const int b = p.q_per_seq == 1 ? row : row / p.q_per_seq;
    int n = static_cast<int>(max(static_cast<int64_t>(0), min(p.kv_offsets[b + 1] - p.kv_offsets[b], static_cast<int64_t>(p.max_n))));
    if (p.q_pos) {
        const int64_t t = min(p.q_pos[b], int64_t(1) << 40) + (row - b * p.q_per_seq) + 1;
        n = static_cast<int>(min(static_cast<int64_t>(n), max(static_cast<int64_t>(0), t) >> (p.ratio - 1)));
    }
    return n;
}

__device__ __forceinline__ RowView view_of(const CacheParams& p, int n) {
    RowView v;
    v.n_vis = n;
    v.w_beg = p.window > 0 ? max(0, n - p.window) : 0;
    v.w0 = v.w_beg / CACHE_TILE;
    v.ts = p.window > 0 ? min((min(p.sinks, n) + CACHE_TILE - 1) / CACHE_TILE, v.w0) : 0;
    v.tiles = n > 0 ? v.ts + (n + CACHE_TILE - 1) / CACHE_TILE - v.w0 : 0;
    return v;
}

__device__ __forceinline__ RowView row_view(const CacheParams& p, int row) { return view_of(p, visible_positions(p, row)); }

__device__ __forceinline__ bool visible(const CacheParams& p, const RowView& v, int j) {
    return j < v.n_vis && (j >= v.w_beg || j < p.sinks);
}

// This CTA's range of the tile list: the row it starts in, the tile inside that row, and
// how many tiles follow.  Whole block.
struct Range {
    int row, tile, count;
};

// Each warp sums an equal share of the rows; the share, then the row, in which the range
// starts is found from those sums.  red: 34 words.
template <int THREADS>
__device__ __forceinline__ Range my_range(const CacheParams& p, int (&red)[34]) {
    constexpr int WARPS = THREADS / 32;
    static_assert(WARPS <= 32, "one lane per warp");
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x;
    int lo = 0, hi = p.batch * p.q_per_seq;
    if (p.whole_rows) {                                     // rows dealt out uncut
        const int each = hi / p.ranges, more = hi % p.ranges;
        lo = c * each + min(c, more);
        hi = lo + each + (c < more ? 1 : 0);
    }
    const int share = (hi - lo + WARPS - 1) / WARPS, r0 = lo + warp * share, r1 = min(hi, r0 + share);
    int sum = 0;
    for (int r = r0 + lane; r < r1; r += 32) sum += row_view(p, r).tiles;
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    const int mine = lane < WARPS ? red[lane] : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += u;
    }
    const int total = __shfl_sync(0xFFFFFFFFu, upto, 31);
    int t0 = 0, count = total;
    if (!p.whole_rows) {
        // with fewer tiles than ranges the first `total` ranges take one each: a cut row's
        // ranges are always consecutive
        const int g = max(1, min(p.ranges, total)), each = total / g, more = total % g;
        t0 = c * each + min(c, more);
        count = c < g ? each + (c < more ? 1 : 0) : 0;
    }
    if (count == 0 || total == 0) return Range{0, 0, 0};
    const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, upto > t0)) - 1;
    if (warp == owner) {
        int before = __shfl_sync(0xFFFFFFFFu, upto - mine, owner);
        for (int r = r0; r < r1; r += 32) {
            const int n = r + lane < r1 ? row_view(p, r + lane).tiles : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += u;
            }
            const int first = before + inc - n;
            if (n > 0 && t0 >= first && t0 < first + n) {
                red[32] = r + lane;
                red[33] = t0 - first;
            }
            before += __shfl_sync(0xFFFFFFFFu, inc, 31);
            if (before > t0) break;
        }
    }
    __syncthreads();
    return Range{red[32], red[33], count};
}

// Rows that see nothing: zeros, lse -inf.  One warp of each CTA; CTA c looks at rows 32 c ..
// + 31 of every 32 x grid rows at once.
__device__ __forceinline__ void empty_rows(const CacheParams& p) {
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    const int lane = threadIdx.x & 31;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * 32) {
        unsigned none = __ballot_sync(0xFFFFFFFFu, r0 + lane < rows && row_view(p, static_cast<int>(r0) + lane).tiles == 0);
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
constexpr int AC_PV_WARPS = 8;                     // warps 0-3, 4-7: P V of a tile's first / last 64 keys
constexpr int AC_SM_WARP = 8;                      // warps 8-11: softmax (TMEM lane quarters 0-3)
constexpr int AC_TMA_WARP = 12;
constexpr int AC_MMA_WARP = 13;                    // warps 13, 14: scales and MMAs of even / odd tiles
constexpr int AC_Q_WARP = 15;                      // the next row's query, shared with warps 13 and 14
constexpr int AC_STAGES = 4;
constexpr int AC_ROWS = 32;                        // rows of a range that the table holds
constexpr int AC_CODE_BYTES = CACHE_TILE * ROW_CODES;                    // two panels of 16 KB
constexpr int AC_STAGE_BYTES = AC_CODE_BYTES + CACHE_TILE * ROW_SCALES;  // 36 KB
constexpr int AC_DIGITS = 6;
constexpr int AC_N = AC_DIGITS * HEADS;            // columns of S: digit d of head h in 16 d + h
constexpr int AC_QPANEL = AC_N * 128;
constexpr int AC_P_BYTES = CACHE_TILE * HEADS * 2;
// tensor memory: two S accumulators, the tile's scales twice, the digits' scales
constexpr uint32_t AT_COLS = 512, AT_S = 0, AT_S_STEP = 128, AT_SFA = 256, AT_SFB = 320;
// named barriers
constexpr int BAR_VOTE = 1, BAR_MAX = 2, BAR_PV = 3;   // BAR_PV + w: warps w and w + 4
constexpr float AC_GAP = 4.0f;                     // the reference maximum moves by more than 2^4 ...
constexpr float AC_SHIFT = 11.0f;                  // ... and P is kept times 2^11, at most 2^15 in f16
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct alignas(1024) CacheSmem {
    uint8_t stage[AC_STAGES][AC_STAGE_BYTES];
    uint8_t q[2][2 * AC_QPANEL];                   // query digits of two rows, K-major SW128 panels
    uint8_t p[2][AC_P_BYTES];                      // P [key][head] f16
    uint8_t sf[2][8][512];                         // a tile's scales as 32 x 16 B blocks
    float4 x[AC_PV_WARPS / 2][8][32];              // O passed between the two key halves
    // tiles: loaded / read, S written / read, P written / read; rows: query written / read,
    // statistics written / read
    uint64_t full[AC_STAGES], empty[AC_STAGES], s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t q_full[2], q_empty[2], r_full[2], r_empty[2], drain;
    // per row: logit factors, sums, minus the reference maxima (less AC_SHIFT: P = exp2(logit - m));
    // per tile: the reference its P stands at
    alignas(16) float f[2][HEADS], l[2][4][HEADS], minus_m[2][HEADS];
    alignas(16) float ref[2][HEADS], part_m[4][HEADS];
    int moved[2];
    int2 rows[AC_ROWS];                            // the range's first rows that see anything: row, positions
    int issued[AC_STAGES];                         // copies issued into each stage
    uint32_t tmem;
    int red[34];
};
static_assert(sizeof(CacheSmem) + 1024 <= 232448, "shared memory of one SM");

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

// Two E4M3 bytes -> f16x2.
__device__ __forceinline__ uint32_t scales_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(two));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// TMA box load of a stream that is read once: its lines leave L2 first, so that code, queries
// and partials stay.
__device__ __forceinline__ void tma_load_stream(void* smem_dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                                uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], "
        "[%4], %5;"
        :: "r"(smem_u32(smem_dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy) : "memory");
}

// Two floats in one register pair, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// x[h] = s[h] f[h] + c[h] for the 16 heads, packed; f and c in shared memory.
__device__ __forceinline__ void scale_heads(const uint64_t (&s)[HEADS / 2], const float* f, const float* c, float (&x)[HEADS]) {
#pragma unroll
    for (int i = 0; i < HEADS / 4; ++i) {
        const ulonglong2 fv = *reinterpret_cast<const ulonglong2*>(f + 4 * i), cv = *reinterpret_cast<const ulonglong2*>(c + 4 * i);
        const float2 a = unpack2(fma2(s[2 * i], fv.x, cv.x)), b = unpack2(fma2(s[2 * i + 1], fv.y, cv.y));
        x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
    }
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Next row at or after `row` that sees anything (whole warp; there is one).
__device__ __noinline__ int next_row(const CacheParams& p, int row) {
    const int rows = p.batch * p.q_per_seq;
    for (; row < rows; row += 32) {
        const int r = row + (threadIdx.x & 31);
        const unsigned any = __ballot_sync(0xFFFFFFFFu, r < rows && r >= row && row_view(p, r).tiles > 0);
        if (any) return row + __ffs(any) - 1;
        if (row > rows - 32) break;
    }
    return rows - 1;
}

// The k-th row of the range (k counts those that see anything): from the table, or behind the
// table's end from global memory, `row` being the (k - 1)-th.  Whole warp.
__device__ __forceinline__ RowView range_row(const CacheParams& p, const CacheSmem& sm, int k, int& row) {
    if (k < AC_ROWS) {
        const int2 r = sm.rows[k];
        row = r.x;
        return view_of(p, r.y);
    }
    row = next_row(p, row + 1);
    return row_view(p, row);
}

// Fills the table from row `row` on, as far as `tiles` tiles reach.  One warp.
__device__ __forceinline__ void list_rows(const CacheParams& p, CacheSmem& sm, int row, int64_t tiles) {
    const int rows = p.batch * p.q_per_seq, lane = threadIdx.x & 31;
    int have = 0;
    for (; row < rows && have < AC_ROWS && tiles > 0; row += 32) {
        const int n = row + lane < rows && row + lane >= row ? visible_positions(p, row + lane) : 0;
        const unsigned some = __ballot_sync(0xFFFFFFFFu, n > 0);
        const int k = have + __popc(some & ((1u << lane) - 1u));
        if (n > 0 && k < AC_ROWS) sm.rows[k] = make_int2(row + lane, n);
        have += __popc(some);
        tiles -= __reduce_add_sync(0xFFFFFFFFu, view_of(p, n).tiles);
        if (row > rows - 32) break;
    }
}

// The six octal digits (each plus 4) of rint(v), |v| < 2^16, in the low six nibbles.
__device__ __forceinline__ uint32_t spread_digits(float v) {
    uint32_t x = __float_as_uint(v + 12582912.0f) - 0x4B400000u + 0x24924u;      // 1.5 2^23: rounds to an integer
    x += 7 * (x & 0x3FE00u);                                // digits 3 .. 5 up by 3 bits
    x += x & 0x1F81F8u;                                     // 1, 2, 4 and 5 by 1
    x += x & 0x380380u;                                     // 2 and 5 by 1
    return x;
}

// E2M1 codes of four digits, a byte each: -4 .. 3 looked up.
__device__ __forceinline__ uint32_t digit_codes(uint32_t nibbles) { return __byte_perm(0x0A0C0D0Eu, 0x05040200u, nibbles); }

// Head h of a row's query as six balanced base-8 digits: n = rint(q 2^k), 2^15 <= |n| <
// 2^16 for the head's largest element, n = sum_d e_d 8^d with e_d in -4 .. 3, every one of
// which E2M1 holds.  Adding 4 to every digit (0o444444) makes them plain octal digits.
// One warp, lane l holds channels 16 l .. + 15.  Not inlined: one copy for all the warps that
// come here, as what a launch runs once is bound by fetching its code (3 copies: 52 us for 64
// rows of 4,096 positions, one 46.6).
struct QueryHead {
    uint4 a, b;
};

__device__ __forceinline__ QueryHead load_query(const CacheParams& p, int row, int h) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(row) * HEADS + h) * D + (threadIdx.x & 31) * GROUP);
    return QueryHead{src[0], src[1]};
}

__device__ __noinline__ void put_query(float sm_scale, CacheSmem& sm, int qb, int h, const QueryHead v) {
    const int lane = threadIdx.x & 31;
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
    uint32_t top = 0;                                       // largest magnitude, as bf16 bits
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const int e = static_cast<int>(top >> 7) - 127;         // largest in [2^e, 2^(e+1))
    const int k = min(15 - e, 126);
    const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    uint8_t* base = sm.q[qb] + (lane >> 4) * AC_QPANEL + h * 128 + ((((lane & 15) >> 1) ^ (h & 7)) << 4) + (lane & 1) * 8;
    uint32_t out[2][AC_DIGITS];                             // [half][digit]: channels 8 half .. + 7, 4 bits each
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t lo[4], hi[4];                              // channels 2 i, 2 i + 1: bytes of digits 0 .. 3, 4 and 5
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = w[4 * j + i];
            const uint32_t x = spread_digits(__uint_as_float(two << 16) * up), y = spread_digits(__uint_as_float(two & 0xFFFF0000u) * up);
            lo[i] = digit_codes(x) + 16 * digit_codes(y);
            hi[i] = digit_codes(x >> 16) + 16 * digit_codes(y >> 16);
        }
        // bytes [channel pair][digit] -> [digit][channel pair]
        const uint32_t a0 = __byte_perm(lo[0], lo[1], 0x5140), a1 = __byte_perm(lo[2], lo[3], 0x5140);
        const uint32_t b0 = __byte_perm(lo[0], lo[1], 0x7362), b1 = __byte_perm(lo[2], lo[3], 0x7362);
        const uint32_t c0 = __byte_perm(hi[0], hi[1], 0x5140), c1 = __byte_perm(hi[2], hi[3], 0x5140);
        out[j][0] = __byte_perm(a0, a1, 0x5410), out[j][1] = __byte_perm(a0, a1, 0x7632);
        out[j][2] = __byte_perm(b0, b1, 0x5410), out[j][3] = __byte_perm(b0, b1, 0x7632);
        out[j][4] = __byte_perm(c0, c1, 0x5410), out[j][5] = __byte_perm(c0, c1, 0x7632);
    }
#pragma unroll
    for (int d = 0; d < AC_DIGITS; ++d)                     // row 16 d + h
        *reinterpret_cast<uint2*>(base + d * HEADS * 128) = make_uint2(out[0][d], out[1][d]);
    if (lane == 0)                                          // a head with an infinity or NaN answers NaN
        sm.f[qb][h] = top >= 0x7F80u ? NAN : sm_scale * LOG2E * __uint_as_float(static_cast<uint32_t>(9 - k + 127) << 23);
}

// Cache row of position pos of sequence b (RowMap::row with a plain load: the page table may
// have been written by the kernel this one was launched behind).
__device__ __forceinline__ int64_t cache_row(const CacheParams& p, int64_t b, int64_t off, int64_t pos) {
    if (p.rows.page_table == nullptr) return off + pos;
    return static_cast<int64_t>(p.rows.page_table[b * p.rows.pages_per_seq + pos / p.rows.page_rows]) * p.rows.page_rows +
           pos % p.rows.page_rows;
}

// Per-head results of 32 lanes x 16 heads: each step halves the heads a lane still holds,
// so 16 shuffles do the work of 80.  Lane 2 i (and 2 i + 1) ends with head head_of(lane).
__device__ __forceinline__ int head_of(int lane) {
    return ((lane >> 4) & 1) * 8 + ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1);
}

template <bool MAX>
__device__ __forceinline__ float reduce_heads(const float (&v)[HEADS]) {
    const int lane = threadIdx.x & 31;
    float a[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) a[i] = v[i];
#pragma unroll
    for (int n = 8; n >= 1; n /= 2) {
        const bool up = lane & (2 * n);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? a[i] : a[n + i], 2 * n);
            const float mine = up ? a[n + i] : a[i];
            a[i] = MAX ? fmaxf(mine, got) : mine + got;
        }
    }
    const float got = __shfl_xor_sync(0xFFFFFFFFu, a[0], 1);
    return MAX ? fmaxf(a[0], got) : a[0] + got;
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
            sm.issued[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], 4);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.p_empty[i], AC_PV_WARPS);
            mbar_init(&sm.q_full[i], 3);
            mbar_init(&sm.q_empty[i], 4);                   // the softmax warps: they saw the row's last S
            mbar_init(&sm.r_full[i], 4);
            mbar_init(&sm.r_empty[i], AC_PV_WARPS);
        }
        mbar_init(&sm.drain, 2);
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
    // The join is not let in early: with a few SMs free its blocks would crowd there, ahead of the
    // ranges' end (1 row of 131,072: 37.6 us, against 29.0).
    griddep_wait();                                         // nothing global is touched before
    unsigned* err = p.err;
    const uint32_t bound = *reinterpret_cast<const volatile unsigned*>(err + 1);      // csa2_set_wait_limit's, or 0
    const Range range = my_range<AC_THREADS>(p, sm.red);
    if (tid < 2) p.meta[2 * blockIdx.x + tid] = -1;

    // Every wait is bounded: by `limit` polls (after a first one that never blocks, the default
    // bound's may suspend the thread for a while).  One that runs out flags ERR_TIMEOUT and sets
    // limit to 0: from then on this thread polls once per wait, issues no copy and no MMA, and
    // takes part in every barrier and arrival as before, so that all warps reach the end.
    uint32_t limit = bound ? bound : SPIN_LIMIT;
    const bool block = limit == SPIN_LIMIT;
    auto done = [&](uint64_t* bar, int phase) {             // one look
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(smem_u32(bar)), "r"(static_cast<uint32_t>(phase & 1)) : "memory");
        return ok;
    };
    auto wait = [&](uint64_t* bar, int phase) {
        const uint32_t addr = smem_u32(bar), parity = static_cast<uint32_t>(phase & 1);
        uint32_t n = 0, ok = done(bar, phase);
        while (!ok && ++n < limit) {
            if (block)
                asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                             : "=r"(ok) : "r"(addr), "r"(parity) : "memory");
            else
                ok = done(bar, phase);
        }
        if (!ok) {
            limit = 0;
            atomicOr(err, ERR_TIMEOUT);
        }
    };
    // Lanes leave a wait one by one: a __syncwarp() stands between it and an instruction that wants
    // the whole warp at once (tensor memory, ldmatrix, barriers).

    // every role walks the range's rows by itself: it counts tiles, rw rows
    int it = 0, rw = 0;
    int row = range.row, left = range.count, tile = range.tile;

    // the producer's copies: tile `it` from cache row y on, into its stage
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    auto copy_tile = [&](int y) {
        const int st = it % AC_STAGES;
        if (it >= AC_STAGES) {
            wait(&sm.empty[st], it / AC_STAGES - 1);
            wait(&sm.full[st], it / AC_STAGES - 1);         // landed, whoever gave up waiting for it
        }
        if (limit) {
            uint8_t* dst = sm.stage[st];
            mbar_arrive_expect_tx(&sm.full[st], AC_STAGE_BYTES);
            tma_load_stream(dst, &tm_codes, 0, y, &sm.full[st], policy);
            tma_load_stream(dst + AC_CODE_BYTES / 2, &tm_codes, 128, y, &sm.full[st], policy);
            tma_load_stream(dst + AC_CODE_BYTES, &tm_scales, 0, y, &sm.full[st], policy);
            sm.issued[st] = it / AC_STAGES + 1;
        }
    };
    // tiles [t0, end) of a row; each lane looks one tile's row up
    auto copy_tiles = [&](const RowView& v, int t0, int end) {
        const int b = row / p.q_per_seq;
        const int64_t off = p.kv_offsets[b];
        for (; t0 < end; t0 += 32) {
            int y = 0;
            if (t0 + lane < end) {
                const int at = v.pos(t0 + lane);
                const int64_t r0 = cache_row(p, b, off, at);
                const bool bad = r0 < 0 || r0 + min(CACHE_TILE, v.n_vis - at) > p.total_n;
                if (bad) atomicOr(err, ERR_DEVICE);
                y = static_cast<int>(bad ? p.total_n : r0);      // past the end: reads zeros
            }
            for (int i = 0; i < 32 && t0 + i < end; ++i, ++it) {
                const int yi = __shfl_sync(0xFFFFFFFFu, y, i);
                if (lane == 0) copy_tile(yi);
                __syncwarp();
            }
        }
    };

    // the first row's query, a head per warp; the first tiles are on their way before
    if (range.count > 0) {
        const QueryHead v = load_query(p, range.row, warp);
        if (warp == AC_TMA_WARP) {
            const RowView r = row_view(p, row);
            copy_tiles(r, tile, min(min(r.tiles, tile + left), tile + AC_STAGES));
        }
        if (warp == AC_Q_WARP) list_rows(p, sm, range.row, static_cast<int64_t>(range.tile) + range.count);
        put_query(p.sm_scale, sm, 0, warp, v);
        fence_proxy_async_smem();
    }
    __syncthreads();
    tc_fence_after();
    // the following rows' ones: heads [h0, h1) by this warp, the next one's values on their way
    int h0 = 0, h1 = 0, next = range.row;
    bool asked = false;
    auto next_query = [&](int qb) {                         // of row rw + 1, into buffer qb
        if (asked) return;
        asked = true;
        range_row(p, sm, rw + 1, next);
        QueryHead ahead = load_query(p, next, h0);
        if (rw >= 1) wait(&sm.q_empty[qb], ((rw + 1) >> 1) - 1);
#pragma unroll 1
        for (int h = h0; h < h1; ++h) {
            const QueryHead v = ahead;
            if (h + 1 < h1) ahead = load_query(p, next, h + 1);
            put_query(p.sm_scale, sm, qb, h, v);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[qb]);
    };

    if (warp == AC_TMA_WARP) {
        // ---- producer: runs ahead over the rows, AC_STAGES tiles at most
        while (left > 0) {
            const RowView v = range_row(p, sm, rw, row);
            const int end = min(v.tiles, tile + left);
            copy_tiles(v, rw ? tile : tile + it, end);      // the first row's first ones are on their way
            left -= end - tile;
            tile = 0;
            ++rw;
        }
        if (lane == 0) {                                    // no copy may land after the CTA is gone
            for (int st = 0; st < AC_STAGES; ++st)
                if (sm.issued[st]) mbar_wait(&sm.full[st], static_cast<uint32_t>((sm.issued[st] - 1) & 1), err);
        }
    } else {
        if (warp >= AC_MMA_WARP) {
            h0 = (warp - AC_MMA_WARP) * 5;
            h1 = warp == AC_Q_WARP ? HEADS : h0 + 5;
            if (left > 0 && lane == 0) mbar_arrive(&sm.q_full[0]);       // the first row's is there
        }
        if (warp == AC_Q_WARP) {
            while (left > 0) {
                const int end = min(range_row(p, sm, rw, row).tiles, tile + left);
                if (left > end - tile) next_query((rw & 1) ^ 1);
                asked = false;
                left -= end - tile;
                tile = 0;
                ++rw;
            }
            empty_rows(p);
        } else if (warp >= AC_MMA_WARP) {
            const int buf = warp - AC_MMA_WARP;             // tiles of this parity
            const uint64_t dq = umma_desc_sw128(smem_u32(sm.q[0]), 16, 1024);
            const uint64_t dc = umma_desc_sw128(smem_u32(sm.stage[0]), 16, 1024);
            const uint64_t ds = desc_rows16(smem_u32(sm.sf[0][0]));
            while (left > 0) {
                const int qb = rw & 1;
                wait(&sm.q_full[qb], rw >> 1);
                const int end = min(range_row(p, sm, rw, row).tiles, tile + left);
                // its share of the next row's query is prepared once its first tile of this row is
                // on its way, two tiles ahead of P V
                const bool more = left > end - tile;
                const uint64_t dqr = dq + qb * (2 * AC_QPANEL / 16);
                for (int t = tile; t < end; ++t, ++it) {
                    if ((it & 1) != buf) continue;
                    const int st = it % AC_STAGES;
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
                    if (lane == 0 && limit) {
                        const uint32_t sfa = tm + AT_SFA + 32 * buf, dst = tm + AT_S + AT_S_STEP * buf;
                        const uint64_t da = dc + st * (AC_STAGE_BYTES / 16), dsb = ds + buf * (8 * 512 / 16);
#pragma unroll
                        for (int s = 0; s < 8; ++s) tmem_copy_rows16(sfa + 4 * s, dsb + s * (512 / 16));
#pragma unroll
                        for (int s = 0; s < 8; ++s)
                            mma_nvf4(dst, da + (s >> 2) * (AC_CODE_BYTES / 2 / 16) + (s & 3) * 2,
                                     dqr + (s >> 2) * (AC_QPANEL / 16) + (s & 3) * 2, AC_IDESC, sfa + 4 * s,
                                     tm + AT_SFB + 4 * s, s > 0);
                        mma_commit(&sm.s_full[buf]);
                    }
                    __syncwarp();
                    if (more) next_query(qb ^ 1);
                }
                if (more) next_query(qb ^ 1);
                asked = false;
                left -= end - tile;
                tile = 0;
                ++rw;
            }
            if (lane == 0) {
                mma_commit(&sm.drain);
                mbar_wait(&sm.drain, 0, err);
            }
        } else if (warp >= AC_SM_WARP) {
            // ---- softmax: thread = key
            const int quarter = warp & 3, key = 32 * quarter + lane;
            while (left > 0) {
                const int rb = rw & 1;
                wait(&sm.q_full[rb], rw >> 1);
                const RowView v = range_row(p, sm, rw, row);
                const int end = min(v.tiles, tile + left);
                uint64_t l2[HEADS / 2];
#pragma unroll
                for (int i = 0; i < HEADS / 2; ++i) l2[i] = 0;
                if (rw >= 2) wait(&sm.r_empty[rb], (rw >> 1) - 1);
                if (warp == AC_SM_WARP && lane < HEADS) sm.minus_m[rb][lane] = 0.0f;     // the first tile sets it
                __syncwarp();
                named_barrier(BAR_MAX, 128);
                for (int t = tile; t < end; ++t, ++it) {
                    const int st = it % AC_STAGES, buf = it & 1, base = v.pos(t);
                    const bool vis = visible(p, v, base + key);
                    const bool all = base + CACHE_TILE <= v.n_vis && (base >= v.w_beg || base + CACHE_TILE <= p.sinks);
                    wait(&sm.s_full[buf], it >> 1);
                    __syncwarp();
                    tc_fence_after();
                    uint64_t s[HEADS / 2];                  // the digits' columns summed, two heads a pair
                    const uint32_t src = tm + (static_cast<uint32_t>(32 * quarter) << 16) + AT_S + AT_S_STEP * buf;
#pragma unroll
                    for (int i = 0; i < AC_DIGITS; i += 2) {
                        uint32_t r[2 * HEADS];
                        tmem_ld32(src + HEADS * i, r);
#pragma unroll
                        for (int h = 0; h < HEADS / 2; ++h) {
                            const uint64_t two = add2(pack2(__uint_as_float(r[2 * h]), __uint_as_float(r[2 * h + 1])),
                                                      pack2(__uint_as_float(r[16 + 2 * h]), __uint_as_float(r[17 + 2 * h])));
                            s[h] = i ? add2(s[h], two) : two;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.s_empty[buf]);
                    float x[HEADS];                         // logits less the reference, in powers of two
                    scale_heads(s, sm.f[rb], sm.minus_m[rb], x);
                    if (!all) {
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) x[h] = vis ? x[h] : -INFINITY;
                    }
                    float d = fmaxf(x[0], x[1]);
#pragma unroll
                    for (int h = 2; h < HEADS; h += 2) d = max3(d, x[h], x[h + 1]);
                    if (it >= 2) wait(&sm.p_empty[buf], (it >> 1) - 1);
                    __syncwarp();
                    const bool first = t == tile;
                    const bool moved = vote_barrier(BAR_VOTE, 128, d > AC_GAP + AC_SHIFT || first);
                    if (moved) {
                        // back to plain logits, their maximum over the tile's keys, and a new reference
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) x[h] = vis ? x[h] - sm.minus_m[rb][h] : -INFINITY;
                        const float top = reduce_heads<true>(x);
                        if (!(lane & 1)) sm.part_m[quarter][head_of(lane)] = top;
                        named_barrier(BAR_MAX, 128);
                        float mine = 0.0f;
#pragma unroll
                        for (int h = 0; h < HEADS; h += 2) {
                            float2 l = unpack2(l2[h / 2]);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float old = first ? -INFINITY : -sm.minus_m[rb][h + e];
                                const float mn = fmaxf(fmaxf(fmaxf(sm.part_m[0][h + e], sm.part_m[1][h + e]),
                                                             fmaxf(sm.part_m[2][h + e], sm.part_m[3][h + e])) - AC_SHIFT, old);
                                const float a = first ? 0.0f : fast_exp2(old - mn);
                                if (e) l.y *= a;
                                else l.x *= a;
                                if (lane == h + e) mine = mn;
                                x[h + e] -= mn;
                            }
                            l2[h / 2] = pack2(l.x, l.y);
                        }
                        named_barrier(BAR_MAX, 128);          // everyone has read the old ones
                        if (warp == AC_SM_WARP && lane < HEADS) sm.minus_m[rb][lane] = -mine;
                        named_barrier(BAR_MAX, 128);
                    }
                    if (warp == AC_SM_WARP) {                // the warps of P V rescale O where it moved
                        if (moved && lane < HEADS) sm.ref[buf][lane] = -sm.minus_m[rb][lane];
                        if (lane == 0) sm.moved[buf] = moved;
                    }
                    // P in f16, as the A operand of P V: 2^-11 of each weight, an eighth of a bf16 output's
                    // own rounding; an fp32 output is off by 6e-5 over 1,501 positions, 2.4e-5 over 65,536.
                    // The sums l are of the unrounded weights, in fp32.
                    uint32_t pk[HEADS / 2];
#pragma unroll
                    for (int h = 0; h < HEADS; h += 2) {
                        const float a = fast_exp2(x[h]), b = fast_exp2(x[h + 1]);
                        l2[h / 2] = add2(l2[h / 2], pack2(a, b));
                        const __half2 two = __floats2half2_rn(a, b);
                        pk[h / 2] = *reinterpret_cast<const uint32_t*>(&two);
                    }
                    uint8_t* dst = sm.p[buf] + key * 32;
                    const int swap = ((key >> 2) & 1) << 4;
                    *reinterpret_cast<uint4*>(dst + swap) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    *reinterpret_cast<uint4*>(dst + (swap ^ 16)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    if (!vis) {
                        // rows behind the sequence or its mask may hold any bytes, NaN scales among
                        // them: 0 x NaN must not reach O
                        uint4* z = reinterpret_cast<uint4*>(sm.stage[st] + AC_CODE_BYTES + key * ROW_SCALES);
                        z[0] = z[1] = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();            // before the next copy into this stage
                    }
                    wait(&sm.full[st], it / AC_STAGES);      // P V reads the tile on this word
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[buf]);
                }
                float l[HEADS];
#pragma unroll
                for (int h = 0; h < HEADS; h += 2) {
                    const float2 u = unpack2(l2[h / 2]);
                    l[h] = u.x, l[h + 1] = u.y;
                }
                const float sum = reduce_heads<false>(l);
                if (!(lane & 1)) sm.l[rb][quarter][head_of(lane)] = sum;
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.r_full[rb]);
                    mbar_arrive(&sm.q_empty[rb]);
                }
                left -= end - tile;
                tile = 0;
                ++rw;
            }
        } else {
            // ---- P V: warp owns channels 128 (w % 4) .. + 127 of keys 64 (w / 4) .. + 63; lane (g, t)
            // converts channels 16 g .. + 15 of those (one scale group) of the keys of its B
            // fragments, n-tile i being channel i of every group
            const int wq = warp & 3, kh = warp >> 2, g = lane >> 2, t4 = lane & 3;
            // byte offsets in a stage of the lane's codes of keys 2 t and 2 t + 1 (their swizzles),
            // and of their scales; in P of the row that the lane hands to ldmatrix
            const uint32_t panel = (wq >> 1) * (AC_CODE_BYTES / 2) + (64 * kh + 2 * t4) * 128 + (g & 1) * 8;
            const uint32_t chunk = (wq & 1) * 4 + (g >> 1);
            const uint32_t code0 = panel + ((chunk ^ (2 * t4)) << 4), code1 = panel + 128 + ((chunk ^ (2 * t4 + 1)) << 4);
            const uint32_t scale0 = AC_CODE_BYTES + (64 * kh + 2 * t4) * ROW_SCALES + wq * 8 + g;
            const uint32_t stage0 = smem_u32(sm.stage[0]);
            const uint32_t p0 = smem_u32(sm.p[0]) + (64 * kh + ((lane >> 4) << 3) + (lane & 7)) * 32 +
                                ((((lane >> 3) ^ (lane >> 2)) & 1) << 4);
            while (left > 0) {
                const int tiles = range_row(p, sm, rw, row).tiles;
                const int end = min(tiles, tile + left);
                float o[16][4] = {};
                float m0 = -INFINITY, m1 = -INFINITY;        // references of heads g, g + 8 that o stands at
                uint32_t ready = 0;                          // P of the next tile seen already
                for (int t = tile; t < end; ++t, ++it) {
                    const int st = it % AC_STAGES, buf = it & 1;
                    const uint32_t sa = stage0 + st * AC_STAGE_BYTES, pa = p0 + buf * AC_P_BYTES;
                    if (!ready) wait(&sm.p_full[buf], it >> 1);
                    __syncwarp();
                    // step ks + 1's operands are loaded while step ks is multiplied
                    uint32_t a[2][4], sc[2][4];
                    uint2 c[2][4];
                    auto load_step = [&](int ks) {           // keys 16 ks + 2 t + {0, 1, 8, 9}
                        const int n = ks & 1;
                        ldmatrix_x4_trans(a[n], pa + ks * 512);
                        c[n][0] = lds64(sa + code0 + ks * 2048);
                        c[n][1] = lds64(sa + code1 + ks * 2048);
                        c[n][2] = lds64(sa + code0 + ks * 2048 + 1024);
                        c[n][3] = lds64(sa + code1 + ks * 2048 + 1024);
                        sc[n][0] = lds8(sa + scale0 + ks * 512);
                        sc[n][1] = lds8(sa + scale0 + ks * 512 + 32);
                        sc[n][2] = lds8(sa + scale0 + ks * 512 + 256);
                        sc[n][3] = lds8(sa + scale0 + ks * 512 + 288);
                    };
                    load_step(0);
                    if (sm.moved[buf]) {
                        const float n0 = sm.ref[buf][g], n1 = sm.ref[buf][g + 8];
                        const float a0 = fast_exp2(m0 - n0), a1 = fast_exp2(m1 - n1);
                        m0 = n0;
                        m1 = n1;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            o[i][0] *= a0;
                            o[i][1] *= a0;
                            o[i][2] *= a1;
                            o[i][3] *= a1;
                        }
                    }
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const int n = ks & 1;
                        if (ks < 3) load_step(ks + 1);
                        else ready = t + 1 < end ? done(&sm.p_full[buf ^ 1], (it + 1) >> 1) : 0u;
                        const uint32_t s0 = scales_to_f16x2(__byte_perm(sc[n][0], sc[n][1], 0x40));
                        const uint32_t s1 = scales_to_f16x2(__byte_perm(sc[n][2], sc[n][3], 0x40));
#pragma unroll
                        for (int hw = 0; hw < 2; ++hw) {     // channels 8 hw .. + 7
                            const uint32_t a0 = hw ? c[n][0].y : c[n][0].x, a1 = hw ? c[n][1].y : c[n][1].x;
                            const uint32_t b0 = hw ? c[n][2].y : c[n][2].x, b1 = hw ? c[n][3].y : c[n][3].x;
                            // two keys' codes interleaved: byte i of e / d = channel 2 i / 2 i + 1 of both
                            uint32_t e0[4], e1[4], d0[4], d1[4];
                            e2m1x8_to_f16((a0 & 0x0F0F0F0Fu) | ((a1 << 4) & 0xF0F0F0F0u), e0);
                            e2m1x8_to_f16((b0 & 0x0F0F0F0Fu) | ((b1 << 4) & 0xF0F0F0F0u), e1);
                            e2m1x8_to_f16(((a0 >> 4) & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u), d0);
                            e2m1x8_to_f16(((b0 >> 4) & 0x0F0F0F0Fu) | (b1 & 0xF0F0F0F0u), d1);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                mma_16816(o[8 * hw + 2 * i], a[n], mul_f16x2(e0[i], s0), mul_f16x2(e1[i], s1));
                                mma_16816(o[8 * hw + 2 * i + 1], a[n], mul_f16x2(d0[i], s0), mul_f16x2(d1[i], s1));
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.p_empty[buf]);
                        mbar_arrive(&sm.empty[st]);
                    }
                }
                // ---- the key halves: warps 4-7 hand n-tiles 0 .. 7 over and take 8 .. 15
                const bool whole = tile == 0 && end == tiles;
                const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);     // 0: the row this range starts in
                float* part = p.part + static_cast<int64_t>(slot) * CACHE_PART_FLOATS;
                const int rb = rw & 1;
                wait(&sm.r_full[rb], rw >> 1);
                __syncwarp();
                if (kh) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sm.x[wq][i][lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                }
                named_barrier(BAR_PV + wq, 64);
                if (!kh) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 u = sm.x[wq][i][lane];
                        o[i][0] += u.x, o[i][1] += u.y, o[i][2] += u.z, o[i][3] += u.w;
                        sm.x[wq][i][lane] = make_float4(o[8 + i][0], o[8 + i][1], o[8 + i][2], o[8 + i][3]);
                    }
                }
                named_barrier(BAR_PV + wq, 64);
                if (kh) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 u = sm.x[wq][i][lane];
                        o[i][0] = o[8 + i][0] + u.x, o[i][1] = o[8 + i][1] + u.y;
                        o[i][2] = o[8 + i][2] + u.z, o[i][3] = o[8 + i][3] + u.w;
                    }
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int h = g + 8 * hh;
                    const float ls = sm.l[rb][0][h] + sm.l[rb][1][h] + sm.l[rb][2][h] + sm.l[rb][3][h];
                    const float inv = whole ? 1.0f / ls : 1.0f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {            // channels 16 (2 t + e) + 8 kh .. + 7 of the warp's
                        const int ch = 128 * wq + 16 * (2 * t4 + e) + 8 * kh;
                        float val[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) val[i] = o[i][2 * hh + e] * inv;
                        const int64_t at = (static_cast<int64_t>(row) * HEADS + h) * D + ch;
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
                    if (warp == 0 && t4 == 0) {
                        if (!whole) {
                            part[h] = -sm.minus_m[rb][h];
                            part[HEADS + h] = ls;
                        } else if (p.lse) {
                            p.lse[static_cast<int64_t>(row) * HEADS + h] = (log2f(ls) - sm.minus_m[rb][h]) * LN2;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.r_empty[rb]);
                if (!whole && tid == 0) p.meta[slot] = row;
                left -= end - tile;
                tile = 0;
                ++rw;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == AC_MMA_WARP) tmem_dealloc(tm, AT_COLS);
}

// Joins the partials of one cut row.  Block (x, y): the x-th cut row (the x-th range whose
// first partial is its row's last one), 512 / SLICES channels.  A row's partials are
// partial 1 of the range it starts in and
// partials 0 of the following ones, in that order: GROUPS groups of threads take every GROUPS-th
// and are added up in group order.  Bound by latency (4.8 MB of partials from L2 at most):
// 3 to 7 us behind the ranges' end.
constexpr int AJ_AHEAD = 2;
constexpr int AJ_THREADS = 512;
static_assert(AJ_THREADS >= CACHE_MAX_RANGES, "a thread per range");

template <int SLICES>
__global__ void __launch_bounds__(AJ_THREADS)
join_cache_kernel(CacheParams p) {
    constexpr int GROUP_THREADS = HEADS * (D / SLICES / 4), GROUPS = AJ_THREADS / GROUP_THREADS;
    __shared__ float w[CACHE_MAX_RANGES][HEADS], lw[CACHE_MAX_RANGES][HEADS];
    __shared__ int ends[AJ_THREADS / 32], sh_first, sh_last, sh_row;
    __shared__ float4 acc[GROUPS - 1][GROUP_THREADS];
    __shared__ float acc_l[GROUPS - 1][GROUP_THREADS], tops[AJ_THREADS / 32][HEADS];
    const int tid = threadIdx.x, lane = tid & 31;
    griddep_wait();
    // thread g: range g's partials' rows, and whether its first one ends a row
    int r0 = -1, r1 = -1;
    bool end = false;
    if (tid < p.ranges) {
        const int2 m = __ldcg(reinterpret_cast<const int2*>(p.meta) + tid);
        const int after = tid + 1 < p.ranges ? __ldcg(p.meta + 2 * tid + 2) : -1;
        r0 = m.x, r1 = m.y;
        end = r0 >= 0 && after != r0;
    }
    const unsigned mine = __ballot_sync(0xFFFFFFFFu, end);
    if (lane == 0) ends[tid / 32] = __popc(mine);
    if (tid == 0) sh_row = -1;
    __syncthreads();
    int before = __popc(mine & ((1u << lane) - 1u));
    for (int i = 0; i < tid / 32; ++i) before += ends[i];
    if (end && before == static_cast<int>(blockIdx.x)) {
        sh_last = tid;
        sh_row = r0;
    }
    __syncthreads();
    const int row = sh_row;
    if (row < 0) return;
    if (r1 == row) sh_first = tid;
    __syncthreads();
    const int first = sh_first, n = sh_last - first + 1;
    auto part = [&](int i) { return p.part + static_cast<int64_t>(2 * (first + i) + (i == 0 ? 1 : 0)) * CACHE_PART_FLOATS; };
    const int grp = tid / GROUP_THREADS, at = tid % GROUP_THREADS, h = at / (GROUP_THREADS / HEADS),
              c = blockIdx.y * (D / SLICES) + at % (GROUP_THREADS / HEADS) * 4;
    float4 v[AJ_AHEAD];                                     // the group's first ones, on their way with the statistics
#pragma unroll
    for (int k = 0; k < AJ_AHEAD; ++k) {
        const int i = grp + k * GROUPS;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) v[k] = __ldcg(reinterpret_cast<const float4*>(part(i) + 2 * HEADS + h * D + c));
    }
    float top = -INFINITY;                                  // of head tid % 16 over this thread's partials
    for (int i = tid; i < n * HEADS; i += AJ_THREADS) {
        const float mi = __ldcg(part(i / HEADS) + i % HEADS);
        w[i / HEADS][i % HEADS] = mi;
        lw[i / HEADS][i % HEADS] = __ldcg(part(i / HEADS) + HEADS + i % HEADS);
        top = fmaxf(top, mi);
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, HEADS));
    if (lane < HEADS) tops[tid / 32][lane] = top;
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < AJ_THREADS / 32; ++i) m = fmaxf(m, tops[i][h]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto take = [&](int i, const float4& u) {
        const float a = fast_exp2(w[i][h] - m);
        l = fmaf(a, lw[i][h], l);
        o.x = fmaf(a, u.x, o.x);
        o.y = fmaf(a, u.y, o.y);
        o.z = fmaf(a, u.z, o.z);
        o.w = fmaf(a, u.w, o.w);
    };
#pragma unroll
    for (int k = 0; k < AJ_AHEAD; ++k)
        if (grp + k * GROUPS < n) take(grp + k * GROUPS, v[k]);
#pragma unroll 4
    for (int i = grp + AJ_AHEAD * GROUPS; i < n; i += GROUPS)
        take(i, __ldcg(reinterpret_cast<const float4*>(part(i) + 2 * HEADS + h * D + c)));
    if (grp) {
        acc[grp - 1][at] = o;
        acc_l[grp - 1][at] = l;
    }
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int i = 0; i < GROUPS - 1; ++i) {
        const float4 u = acc[i][at];
        o.x += u.x, o.y += u.y, o.z += u.z, o.w += u.w;
        l += acc_l[i][at];
    }
    const float inv = 1.0f / l;
    const int64_t dst = (static_cast<int64_t>(row) * HEADS + h) * D + c;
    if (p.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + dst) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
    if (p.lse && blockIdx.y == 0 && at % (GROUP_THREADS / HEADS) == 0) p.lse[static_cast<int64_t>(row) * HEADS + h] = (m + log2f(l)) * LN2;
}

}  // namespace

CachePlan cache_plan(int64_t rows, int64_t max_n, int64_t window, int64_t sinks) {
    // tiles of a row at most: the window may straddle one tile more than its length
    int64_t tiles = ceil_div(max_n, CACHE_TILE);
    if (window > 0) {
        const int64_t w = std::min(window, max_n), s = std::min(sinks, max_n);
        tiles = std::min(tiles, ceil_div(w, CACHE_TILE) + 1 + ceil_div(s, CACHE_TILE));
    }
    // In tiles: uncut, the busiest CTA has whole rows to do, one for each time the rows go around
    // the SMs; cut, all have the same number and, where that is one, the join behind them (2 tiles,
    // one more for 20 rows); where it is more, most CTAs also change rows inside (5 with the join).
    // Measured over 1 .. 400 equal rows of 1 .. 8 tiles, uncut / cut (us): 1 row of 2 tiles 11.5 /
    // 12.5, of 4 14.8 / 12.9; 16 of 4 14.9 / 14.0, of 8 21.8 / 15.0; 28 of 4 15.2 / 15.9, of 7 20.3 /
    // 22.6; 36 of 6 18.6 / 19.0, of 8 22.3 / 19.3; 40 of 8 22.1 / 23.3; 64 of 4 15.5 / 19.0, of 8 22.4 /
    // 25.4, of 16 35.9 / 34.3; 149 of 6 32.6 / 30.9 (the rule's worst, 6 %), of 8 40.1 / 35.0; 200 of 8
    // 41.2 / 47.9; 300 of 4 36.5 / 38.4, of 8 56.6 / 53.0, of 16 98 / 81.
    CachePlan plan;
    const int64_t uncut = ceil_div(rows, CACHE_MAX_RANGES) * tiles, cut = ceil_div(rows * tiles, CACHE_MAX_RANGES);
    // long rows are always cut: their true lengths may lie far below max_n
    plan.whole_rows = tiles <= 8 && uncut <= cut + (cut == 1 ? 2 + rows / 20 : 5);
    plan.room = static_cast<int>(std::min<int64_t>(CACHE_MAX_RANGES, tiles >= CACHE_MAX_RANGES ? tiles : rows * tiles));
    plan.ranges = plan.whole_rows ? static_cast<int>(std::min<int64_t>(CACHE_MAX_RANGES, rows)) : plan.room;
    return plan;
}

csa2_status launch_attend_cache(const CacheParams& p, const CUtensorMap& codes, const CUtensorMap& scales,
                                cudaStream_t stream) {
    const int smem = static_cast<int>(sizeof(CacheSmem) + 1024);
    if (!opt_in_smem(reinterpret_cast<const void*>(attend_cache_kernel), smem))
        return check_launch("attend_cache_kernel smem attribute");
    launch_dependent(attend_cache_kernel, dim3(static_cast<unsigned>(p.ranges)), AC_THREADS, smem, stream, p, codes, scales);
    csa2_status st = check_launch("attend_cache_kernel");
    if (st != CSA2_OK || p.ranges == 1 || p.whole_rows) return st;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_per_seq;
    // A row in 32 or 16 slices as long as there are at most two blocks an SM, else in 8.  With 32 / 16 / 8
    // (us): 1 row of 131,072 29.0 / 31.5 / 34.5, 4 of 32,768 31.2 / 31.8 / 32.5, 9 of 8,192 21.6 / 21.7 /
    // 21.7, 16 of 8,192 33.2 / 31.8 / 32.0, 37 of 4,096 33.6 / 30.5 / 28.4, 64 of 8,192 76.8 / 71.4 / 69.2.
    const unsigned cut = static_cast<unsigned>(std::min<int64_t>(rows, p.ranges - 1));
    if (cut * 32 <= 2 * CACHE_MAX_RANGES) launch_dependent(join_cache_kernel<32>, dim3(cut, 32), AJ_THREADS, 0, stream, p);
    else if (cut * 16 <= 2 * CACHE_MAX_RANGES) launch_dependent(join_cache_kernel<16>, dim3(cut, 16), AJ_THREADS, 0, stream, p);
    else launch_dependent(join_cache_kernel<8>, dim3(cut, 8), AJ_THREADS, 0, stream, p);
    return check_launch("join_cache_kernel");
}

}  // namespace csa2
