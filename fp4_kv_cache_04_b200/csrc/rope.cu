// Head norm and rotary positions: queries (norm_rope_kernel) and the cache append with
// both on the way (append_rope_kernel).  Neither is described by the pages; the append
// writes the pages' FP4 main-KV row and FP8 indexer row (quantize.cu has the plain append).
//
//   y = x * w / sqrt(mean(x^2) + eps);  (u, v) -> (u cos a - v sin a, v cos a + u sin a),
//   a = position * inv_freq.
//
// The angle is formed in 64 bits and reduced there to a fraction of a turn, so a position
// of 2^30 still has its angle to 2^-22 of a turn; only then does sincospi see it.
#include "dense.cuh"
#include "tc.cuh"
#include "row_formats.cuh"

namespace csa2 {

namespace {

constexpr double INV_TWO_PI = 0.15915494309189533577;

// Fraction of a turn, in [-1/2, 1/2], of the angle pos * inv_freq (radians).
__device__ __forceinline__ double turn_fraction(int64_t pos, float inv_freq) {
    const double t = static_cast<double>(pos) * static_cast<double>(inv_freq) * INV_TWO_PI;
    return t - rint(t);
}

template <int T> struct Elem;
template <> struct Elem<CSA2_T_BF16> { using type = __nv_bfloat16; };
template <> struct Elem<CSA2_T_F16> { using type = __half; };
template <> struct Elem<CSA2_T_F32> { using type = float; };

// 8 elements -> fp32 (16-byte loads).
template <int T>
__device__ __forceinline__ void load8(const typename Elem<T>::type* p, float (&v)[8]) {
    if constexpr (T == CSA2_T_F32) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == CSA2_T_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

template <int T>
__device__ __forceinline__ void store8(typename Elem<T>::type* p, const float (&v)[8]) {
    if constexpr (T == CSA2_T_F32) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == CSA2_T_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Queries; bound by HBM (in + out once: 36 us for 4,096 x 16 fp32 vectors of 512 in and bf16
// out, 5.6 TB/s) or, for a step's few tokens, by the launch.  A block takes rows_per_block tokens: first their cos / sin tables (one per
// token, shared by its heads), then their vectors, `lanes` lanes (a power of two) per
// vector and 8 channels per lane and item.  The half-split pairing reaches across lanes,
// so there the vector goes through shared memory once.
constexpr int NR_THREADS = 256;
constexpr int NR_MAX_PAIRS = 2048;             // cos / sin pairs of a block (16 KB)

// Pairs of a block's table, rounded up so that the vectors behind it start 16-byte aligned.
__host__ __device__ __forceinline__ int table_pairs(int rows_per_block, int pairs) {
    return (rows_per_block * pairs + 1) & ~1;
}

template <int TI, int TO, int ITEMS, bool HALF>
__global__ void __launch_bounds__(NR_THREADS)
norm_rope_kernel(RopeParams p, int rows_per_block, int lanes) {
    extern __shared__ float2 nr_smem[];        // [rows_per_block][rope_dim / 2], then vectors
    griddep_launch_dependents();
    griddep_wait();
    const int pairs = p.rope_dim / 2;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_per_block;
    const int n_rows = static_cast<int>(min(static_cast<int64_t>(rows_per_block), p.rows - row0));
    for (int i = threadIdx.x; i < n_rows * pairs; i += NR_THREADS) {
        const int r = i / pairs, k = i - r * pairs;
        const float t = 2.0f * static_cast<float>(turn_fraction(p.pos[row0 + r], p.inv_freq[k]));
        float s, c;
        sincospif(t, &s, &c);
        nr_smem[i] = make_float2(c, p.inverse ? -s : s);
    }
    if (pairs) __syncthreads();

    const int sub = threadIdx.x / lanes, sl = threadIdx.x % lanes, subs = NR_THREADS / lanes;
    float* stage = reinterpret_cast<float*>(nr_smem + table_pairs(rows_per_block, pairs)) + sub * p.dim;
    const int start = p.dim - p.rope_dim;
    const int total = n_rows * p.heads;
    // every thread makes the same number of turns: the shuffles and barriers below are
    // whole-warp, and a vector past the end is worked on as the last one and not stored
    for (int v0 = 0; v0 < total; v0 += subs) {
        const int vi = min(v0 + sub, total - 1);
        const bool live = v0 + sub < total;
        const int r = vi / p.heads, h = vi - r * p.heads;
        const auto* x = static_cast<const typename Elem<TI>::type*>(p.x) + (row0 + r) * p.x_row_stride +
                        h * p.x_head_stride;
        float y[ITEMS][8];
        float ss = 0.0f;
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const int c = (it * lanes + sl) * 8;
            if (c < p.dim) {
                load8<TI>(x + c, y[it]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[it][j] = 0.0f;
            }
        }
        if (p.norm) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(y[it][j], y[it][j], ss);
            for (int o = lanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            const float rs = 1.0f / sqrtf(ss / static_cast<float>(p.dim) + p.eps);
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) {
                const int c = (it * lanes + sl) * 8;
                if (p.weight != nullptr && c < p.dim) {
                    float w[8];
                    load8<CSA2_T_F32>(p.weight + c, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[it][j] *= rs * w[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[it][j] *= rs;
                }
            }
        }
        const float2* cs = nr_smem + r * pairs;
        if constexpr (HALF) {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) {
                const int c = (it * lanes + sl) * 8;
                if (c < p.dim) store8<CSA2_T_F32>(stage + c, y[it]);
            }
            __syncwarp();
        }
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const int c = (it * lanes + sl) * 8;
            if (c >= p.dim) continue;
            if (c + 8 > start) {
                if constexpr (HALF) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int k = c + j - start;
                        if (k >= 0) {
                            const bool second = k >= pairs;
                            const float2 a = cs[second ? k - pairs : k];
                            const float other = stage[second ? c + j - pairs : c + j + pairs];
                            y[it][j] = second ? y[it][j] * a.x + other * a.y : y[it][j] * a.x - other * a.y;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        if (c + j >= start) {
                            const float2 a = cs[(c + j - start) >> 1];
                            const float u = y[it][j], v = y[it][j + 1];
                            y[it][j] = u * a.x - v * a.y;
                            y[it][j + 1] = v * a.x + u * a.y;
                        }
                    }
                }
            }
            if (live) {
                auto* o = static_cast<typename Elem<TO>::type*>(p.out) + (row0 + r) * p.out_row_stride +
                          h * p.out_head_stride;
                store8<TO>(o + c, y[it]);
            }
        }
        if constexpr (HALF) __syncwarp();
    }
}

// ------------------------------------------------------------------ append

// sin and cos of 2 pi t, |t| <= 1/2, in 64 bits: the nearest quarter turn taken off leaves
// |x| <= pi/4, where the Taylor series to x^13 and x^14 are off by less than 2^-45.
__device__ __forceinline__ double2 turn_cos_sin(double t) {
    const double q = rint(4.0 * t);
    const double x = (t - 0.25 * q) * 6.283185307179586477, z = x * x;
    double s = 1.0 / 6227020800.0, c = -1.0 / 87178291200.0;
    s = fma(s, z, -1.0 / 39916800.0);
    c = fma(c, z, 1.0 / 479001600.0);
    s = fma(s, z, 1.0 / 362880.0);
    c = fma(c, z, -1.0 / 3628800.0);
    s = fma(s, z, -1.0 / 5040.0);
    c = fma(c, z, 1.0 / 40320.0);
    s = fma(s, z, 1.0 / 120.0);
    c = fma(c, z, -1.0 / 720.0);
    s = fma(s, z, -1.0 / 6.0);
    c = fma(c, z, 1.0 / 24.0);
    s = fma(s * z, x, x);
    c = fma(c, z, -0.5);
    c = fma(c, z, 1.0);
    const int n = static_cast<int>(q) & 3;                  // quarter turns
    const double cc = (n & 1) ? s : c, ss = (n & 1) ? c : s;
    return make_double2(n == 1 || n == 2 ? -cc : cc, n >= 2 ? -ss : ss);
}

// A 64-bit result's bf16 value: rounded to fp32, then to bf16, to nearest even both.
__device__ __forceinline__ uint16_t bf16_by_f32(double m) {
    const __nv_bfloat16 h = __float2bfloat16_rn(__double2float_rn(m));
    return *reinterpret_cast<const uint16_t*>(&h);
}

// 72 registers a thread: an SM holds 7 blocks of 4 warps, or 3 of 8.  8,192 tokens (and their
// read-back) take 14.8 us with 4, 14.9 with 2, 15.8 with 8.
constexpr int AR_WARPS = 4;

template <int T>
__device__ __forceinline__ float load1(const typename Elem<T>::type* p) {
    if constexpr (T == CSA2_T_BF16) return __bfloat162float(*p);
    else if constexpr (T == CSA2_T_F16) return __half2float(*p);
    else return *p;
}

// One warp per token, one lane per 16-channel group (as in quantize.cu).  The FP4 codes
// change by a whole step at a border, so the value they are made of is defined to the bit: the
// real number rounded to fp32, as the indexer row's values are, and that to bf16 (what a
// program has that casts its fp32 or fp64 result; off by half a bf16 step and half an fp32
// step at most).  The sum of squares in 64 bits, 1/sqrt by one 64-bit step of Newton-Raphson
// from the fp32 one (2^-43); x * w * r in fp32 (off by 3 units at most), and again in 64 bits
// by the whole warp where one of its 512 results lies within 4 units of a bf16 rounding border
// (1 token in 14; elsewhere both fp32 values round to the same bf16); the rotated channels in
// 64 bits throughout, a pair per lane and turn, handed to their group's lane through shared
// memory.
//
// Bound by latency: a token is one chain (position, row, sum over 32 lanes, root, sine and
// cosine, rotation, shared memory, quantisation) of 900 instructions, 8,192 tokens are two
// waves of blocks, the issue slots are half busy and the 64-bit pipe 7 %.  What a token loads
// is asked for before its norm, which is worth 0.6 us; 64-bit products throughout took 21 us
// with the read-back, 14.6 now.  By itself 8,192 tokens 10.9 us, 64 tokens 3.1 (in a graph).
template <int TI>
__global__ void __launch_bounds__(32 * AR_WARPS)
append_rope_kernel(AppendParams p) {
    extern __shared__ uint16_t ar_smem[];                   // [warps][rope_dim rounded up to 8]: turned channels, bf16
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * AR_WARPS + warp;
    if (i >= p.n) return;
    const int64_t pos = p.pos[i], b = p.seq ? p.seq[i] : i;
    const auto* src = static_cast<const typename Elem<TI>::type*>(p.latent) + i * p.latent_stride + lane * GROUP;
    float x[16];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float a[8];
        load8<TI>(src + 8 * q, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[8 * q + j] = a[j];
    }
    float w[16];
    bool close = false;
    if (p.norm && p.weight) {
        float top = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float a[8];
            load8<CSA2_T_F32>(p.weight + lane * GROUP + 8 * q, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                w[8 * q + j] = a[j];
                top = fmaxf(top, fabsf(a[j]));
            }
        }
        // x r below 2^-126 has lost bits in fp32: under such a weight they count, under smaller ones
        // the result is below 2^-26, far from FP4's lowest border (2^-11)
        close = top > 0x1p100f;
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = 1.0f;
    }
    // asked for now, used behind the norm
    float freq = lane < p.rope_dim / 2 ? p.inv_freq[lane] : 0.0f;
    const int ip = p.idx_proj ? p.idx_rope_dim / 2 : 0, k0 = 2 * lane - 2 * (IDX_DIM / 2 - ip);
    const int pair = p.half ? lane : k0 >> 1;               // the indexer row's one that this lane turns by
    float2 k = make_float2(0.0f, 0.0f);
    float idx_freq = 0.0f;
    if (p.idx_proj) k = *reinterpret_cast<const float2*>(p.idx_proj + i * p.idx_stride + 2 * lane);
    if (pair >= 0 && pair < ip) idx_freq = p.idx_inv_freq[pair];
    if (pos < 0) return;
    // the row's place: looked up here, on its way until the row is stored
    int64_t base = -1, end = 0, in_page = 0;               // packed: first row and length; paged: page
    if (b >= 0 && b < p.batch) {
        if (p.rows.page_table) {
            if (pos < static_cast<int64_t>(p.rows.pages_per_seq) * p.rows.page_rows) {
                // 32-bit division wherever the position fits
                const int64_t in_seq = pos >> 32 ? pos / p.rows.page_rows
                                                 : static_cast<int64_t>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.rows.page_rows));
                base = p.rows.page_table[b * p.rows.pages_per_seq + in_seq];
                in_page = pos - in_seq * p.rows.page_rows;
            }
        } else {
            base = p.kv_offsets[b];
            end = p.kv_offsets[b + 1];
        }
    }

    double r = 1.0;
    if (p.norm) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss = fma(static_cast<double>(x[j]), static_cast<double>(x[j]), ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const double a = fma(ss, 1.0 / D, static_cast<double>(p.eps));
        // the fp32 root is good to 2^-22 where fp32 holds `a`; outside, the 64-bit one
        const float af = static_cast<float>(a);
        if (af > 1e-30f && af < 1e30f) {
            const double r0 = static_cast<double>(rsqrtf(af));
            r = r0 * fma(-0.5 * a * r0, r0, 1.5);
        } else {
            r = 1.0 / sqrt(a);
            close = true;                                   // and no fp32 products
        }
    }

    uint16_t h[16];
    {
        const float rf = static_cast<float>(r);
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            y[j] = (x[j] * rf) * w[j];                      // (x r stays below sqrt(512), whatever w is)
            close |= ((__float_as_uint(y[j]) - 0x7FFCu) & 0xFFFFu) <= 8u;
        }
        if (p.norm && __any_sync(0xFFFFFFFFu, close)) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                h[j] = bf16_by_f32(static_cast<double>(x[j]) * (static_cast<double>(w[j]) * r));
        } else {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(y[j], y[j + 1]);
                const uint32_t u = *reinterpret_cast<const uint32_t*>(&two);
                h[j] = static_cast<uint16_t>(u);
                h[j + 1] = static_cast<uint16_t>(u >> 16);
            }
        }
    }
    if (p.rope_dim) {
        const int pairs = p.rope_dim / 2, start = D - p.rope_dim;
        uint16_t* turned = ar_smem + warp * ((p.rope_dim + 7) & ~7);
        const auto* xr = static_cast<const typename Elem<TI>::type*>(p.latent) + i * p.latent_stride + start;
        for (int k = lane; k < pairs; k += 32) {
            const int iu = p.half ? k : 2 * k, iv = p.half ? k + pairs : 2 * k + 1;
            if (k >= 32) freq = p.inv_freq[k];
            const double2 a = turn_cos_sin(turn_fraction(pos, freq));
            double u = static_cast<double>(load1<TI>(xr + iu)), v = static_cast<double>(load1<TI>(xr + iv));
            if (p.norm) {
                u *= p.weight ? static_cast<double>(p.weight[start + iu]) * r : r;
                v *= p.weight ? static_cast<double>(p.weight[start + iv]) * r : r;
            }
            turned[iu] = bf16_by_f32(fma(u, a.x, -(v * a.y)));
            turned[iv] = bf16_by_f32(fma(v, a.x, u * a.y));
        }
        __syncwarp();
        const int c0 = lane * GROUP - start;                // first channel of the lane among the rotated
        if (c0 + GROUP > 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c0 + j >= 0) h[j] = turned[c0 + j];
        }
    }
    int64_t row = -1;
    if (base >= 0) {
        if (p.rows.page_table) row = base * p.rows.page_rows + in_page;
        else if (pos < end - base) row = base + pos;
    }
    if (row < 0 || row >= p.total_rows) {
        if (lane == 0 && p.err) atomicOr(p.err, ERR_DEVICE);
        return;
    }
    uint2 v;
    const uint8_t sc = nvfp4_group_hw(h, v);
    *reinterpret_cast<uint2*>(p.codes + row * ROW_CODES + lane * 8) = v;
    p.scales[row * ROW_SCALES + lane] = sc;

    if (!p.idx_proj) return;
    // indexer row: lane l holds values 2l, 2l+1 (a pair of the interleaved rotation); turned in 64
    // bits and rounded once to fp32, since its E4M3 codes change by whole steps too
    if (ip) {
        const double2 a = turn_cos_sin(turn_fraction(pos, idx_freq));
        const double u = static_cast<double>(k.x), v = static_cast<double>(k.y);
        if (!p.half) {
            // the others stay as they are: times cos 0 and sin 0 an infinity would reach its neighbour
            if (pair >= 0) k = make_float2(static_cast<float>(fma(u, a.x, -(v * a.y))), static_cast<float>(fma(v, a.x, u * a.y)));
        } else {
            float out[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const int kk = k0 + d;
                const bool second = kk >= ip;
                const int at = kk < 0 ? 0 : second ? kk - ip : kk, partner = (IDX_DIM - p.idx_rope_dim) + (second ? at : at + ip);
                const double c = __shfl_sync(0xFFFFFFFFu, a.x, at), s = __shfl_sync(0xFFFFFFFFu, a.y, at);
                const float o0 = __shfl_sync(0xFFFFFFFFu, k.x, partner >> 1), o1 = __shfl_sync(0xFFFFFFFFu, k.y, partner >> 1);
                const double other = static_cast<double>((partner & 1) ? o1 : o0), me = d ? v : u;
                out[d] = kk < 0 ? (d ? k.y : k.x) : static_cast<float>(second ? fma(me, c, other * s) : fma(me, c, -(other * s)));
            }
            k = make_float2(out[0], out[1]);
        }
    }
    store_idx_row(k, lane, p.idx_k + row * IDX_DIM, p.idx_kscale + row);
}

template <int TI, int TO, int ITEMS>
csa2_status launch_norm(const RopeParams& p, int rows_per_block, int lanes, int smem, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(ceil_div(p.rows, rows_per_block));
    if (p.half) launch_dependent(norm_rope_kernel<TI, TO, ITEMS, true>, grid, NR_THREADS, smem, stream, p, rows_per_block, lanes);
    else launch_dependent(norm_rope_kernel<TI, TO, ITEMS, false>, grid, NR_THREADS, smem, stream, p, rows_per_block, lanes);
    return check_launch("norm_rope_kernel");
}

template <int TI, int TO>
csa2_status launch_norm_items(const RopeParams& p, int rpb, int lanes, int smem, cudaStream_t stream) {
    const int items = (p.dim / 8 + lanes - 1) / lanes;
    if (items <= 1) return launch_norm<TI, TO, 1>(p, rpb, lanes, smem, stream);
    if (items <= 2) return launch_norm<TI, TO, 2>(p, rpb, lanes, smem, stream);
    return launch_norm<TI, TO, 4>(p, rpb, lanes, smem, stream);
}

template <int TI>
csa2_status launch_norm_out(const RopeParams& p, int out_type, int rpb, int lanes, int smem, cudaStream_t stream) {
    if (out_type == CSA2_T_BF16) return launch_norm_items<TI, CSA2_T_BF16>(p, rpb, lanes, smem, stream);
    if (out_type == CSA2_T_F16) return launch_norm_items<TI, CSA2_T_F16>(p, rpb, lanes, smem, stream);
    return launch_norm_items<TI, CSA2_T_F32>(p, rpb, lanes, smem, stream);
}

}  // namespace

csa2_status launch_norm_rope(const RopeParams& p, int in_type, int out_type, cudaStream_t stream) {
    if (p.rows == 0) return CSA2_OK;
    int lanes = 1;
    while (lanes < 32 && lanes * 8 < p.dim) lanes *= 2;
    const int subs = NR_THREADS / lanes, pairs = p.rope_dim / 2;
    // enough vectors for every sub-warp of a block, within the table's share of shared memory
    int rpb = static_cast<int>(ceil_div(subs, p.heads));
    if (pairs && rpb * pairs > NR_MAX_PAIRS) rpb = NR_MAX_PAIRS / pairs;
    const int smem = table_pairs(rpb, pairs) * static_cast<int>(sizeof(float2)) + (p.half ? subs * p.dim * 4 : 0);
    if (ceil_div(p.rows, rpb) > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
    if (in_type == CSA2_T_BF16) return launch_norm_out<CSA2_T_BF16>(p, out_type, rpb, lanes, smem, stream);
    if (in_type == CSA2_T_F16) return launch_norm_out<CSA2_T_F16>(p, out_type, rpb, lanes, smem, stream);
    return launch_norm_out<CSA2_T_F32>(p, out_type, rpb, lanes, smem, stream);
}

csa2_status launch_append_rope(const AppendParams& p, int in_type, cudaStream_t stream) {
    if (p.n == 0) return CSA2_OK;
    const int smem = AR_WARPS * ((p.rope_dim + 7) & ~7) * 2;
    const int64_t grid = ceil_div(p.n, AR_WARPS);
    if (grid > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
    const unsigned g = static_cast<unsigned>(grid);
    if (in_type == CSA2_T_BF16) launch_dependent(append_rope_kernel<CSA2_T_BF16>, g, 32 * AR_WARPS, smem, stream, p);
    else if (in_type == CSA2_T_F16) launch_dependent(append_rope_kernel<CSA2_T_F16>, g, 32 * AR_WARPS, smem, stream, p);
    else launch_dependent(append_rope_kernel<CSA2_T_F32>, g, 32 * AR_WARPS, smem, stream, p);
    return check_launch("append_rope_kernel");
}

}  // namespace csa2
