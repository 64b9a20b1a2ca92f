// The row-wise kernels of the prompt path (include/tf_prompt.h): rotary positions, the append of a
// projection's rows (RMS norm, rotation, the write into the pages) and the rows back from the pages.
// All three read every value once and write it once, and are bounded by HBM; small calls by their launch.
//
// Angles.  Pair i turns by t_i full turns a position.  t_i is held as the integer T = round(t_i 2^64), and
// the product T * position wraps modulo 2^64, which is modulo one turn: its upper 32 bits, signed, are the
// angle in units of 2^-32 turns, whatever the position.  (An fp32 angle at position 10^6 is off by up to
// 0.03 radians.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "ptx.cuh"
#include "tf_internal.h"

namespace tf {

namespace rows {

// Row j of a packed call belongs to the last stream with off <= j, at position base + j.
struct Packed {
    int32_t S, n;                      // streams, rows
    int32_t off[TF_MAX_STREAMS];       // the stream's first row
    int32_t base[TF_MAX_STREAMS];      // its position minus that row
};

__device__ __forceinline__ int stream_of(const Packed &k, int row) {
    int s = 0;
    for (int a = k.S - 1; s < a;) {
        const int mid = (s + a + 1) >> 1;
        if (k.off[mid] <= row) s = mid; else a = mid - 1;
    }
    return s;
}

// (cos, sin) of a pair's angle at a position, times the amplitude.  The angle lies within half a turn, where the
// hardware's sine and cosine are off by 2^-21 at most, a 4,000th of the rounding to bf16 that follows (sincospif
// instead: turning 297,264 rows of one head takes 22.7 us against 20.1, appending them to FP8 pages 109 against 106).
__device__ __forceinline__ float2 turn_of(uint64_t turn, int pos, float amplitude) {
    const int32_t frac = (int32_t)(uint32_t)((turn * (uint64_t)(uint32_t)pos) >> 32);
    const float angle = (float)frac * (3.14159265358979f * 0x1p-31f);
    return make_float2(__cosf(angle) * amplitude, __sinf(angle) * amplitude);
}

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// x[i] of an array in registers.
__device__ __forceinline__ float pick(const float (&x)[16], int i) {
    float v = x[0];
#pragma unroll
    for (int k = 1; k < 16; ++k)
        if (i == k) v = x[k];
    return v;
}

__device__ __forceinline__ void turn_pair(float &a, float &b, float2 cs) {
    const float x = a;
    a = x * cs.x - b * cs.y;
    b = b * cs.x + x * cs.y;
}

// ---- rotary positions ----
constexpr int RT = 256;      // threads
constexpr int RTAB = 4096;   // (row, pair) entries of the block's table of cosines and sines, at most: 32 KB

struct RopeParams {
    const uint16_t *x;
    uint16_t *y;
    int64_t x_row, x_head, y_row, y_head;   // in values
    int32_t H, dim, cols, threads_per_row;  // cols: units of one row over all heads
    float amplitude;
    uint64_t turn[TF_ROPE_MAX_DIM / 2];
    Packed rows;
};

// A unit is what a thread turns at once: 8 neighbouring values (interleaved: 4 pairs), or 8 values and the 8
// that lie half the part further (8 pairs).  A thread keeps its unit's place in the row (head and pairs) and
// takes the rows r, r + lanes, ... of its block, IT of them with all loads in flight; the block's angles are made
// once for all heads and wait in shared memory (64 heads share 32 sines a row).  19,480 rows of 64 heads, 64 of
// 192 values each (319 MB moved): 50.8 us, 0.93 of the measured copy rate.
template <bool HALF, int IT>
__global__ void __launch_bounds__(RT) rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float2 tab[];   // as large as the block needs: 32 KB each left 7 blocks an SM (71 us against 52)
    ptx::griddep_launch_dependents();
    const int tpr = p.threads_per_row, lanes = RT / tpr, pairs = p.dim / 2;
    const int row0 = (int)blockIdx.x * lanes * IT;
    const int nrows = min(p.rows.n - row0, lanes * IT);
    {   // a thread makes one pair's angles, of every (RT / pairs)-th row (one search for their streams: 297,264 rows
        // of one head 26.7 -> 20 us)
        const int r0 = (int)threadIdx.x / pairs, pair = (int)threadIdx.x - r0 * pairs, step = RT / pairs;
        const uint64_t turn = p.turn[pair];
        if (r0 < step && r0 < nrows) {
            int s = stream_of(p.rows, row0 + r0);
            int base = p.rows.base[s], next = s + 1 < p.rows.S ? p.rows.off[s + 1] : p.rows.n;
            for (int r = r0; r < nrows; r += step) {
                while (row0 + r >= next) {
                    ++s;
                    base = p.rows.base[s];
                    next = s + 1 < p.rows.S ? p.rows.off[s + 1] : p.rows.n;
                }
                tab[r * pairs + pair] = turn_of(turn, base + row0 + r, p.amplitude);
            }
        }
    }
    __syncthreads();
    ptx::griddep_wait();
    const int lane = (int)threadIdx.x / tpr, col = (int)blockIdx.y * tpr + (int)threadIdx.x - lane * tpr;
    if (lane >= lanes || col >= p.cols) return;
    const int per_head = HALF ? p.dim / 16 : p.dim / 8;
    const int h = col / per_head, c = col - h * per_head;
    const uint16_t *x = p.x + h * p.x_head + c * 8;
    uint16_t *y = p.y + h * p.y_head + c * 8;
    const int half = p.dim / 2;
    uint4 a[IT], b[IT];
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int r = lane + k * lanes;
        if (r >= nrows) break;
        const uint16_t *src = x + (row0 + r) * p.x_row;
        a[k] = *reinterpret_cast<const uint4 *>(src);
        if (HALF) b[k] = *reinterpret_cast<const uint4 *>(src + half);
    }
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int r = lane + k * lanes;
        if (r >= nrows) break;
        const float2 *cs = tab + r * pairs + (HALF ? c * 8 : c * 4);
        uint32_t w[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
        uint16_t *dst = y + (row0 + r) * p.y_row;
        if (HALF) {
            uint32_t v[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 t = *reinterpret_cast<const float4 *>(cs + 2 * i);
                float u0 = lo(w[i]), u1 = hi(w[i]), v0 = lo(v[i]), v1 = hi(v[i]);
                turn_pair(u0, v0, make_float2(t.x, t.y));
                turn_pair(u1, v1, make_float2(t.z, t.w));
                w[i] = ptx::pack_bf16x2(u0, u1);
                v[i] = ptx::pack_bf16x2(v0, v1);
            }
            *reinterpret_cast<uint4 *>(dst + half) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float4 t = *reinterpret_cast<const float4 *>(cs + i);
                float u0 = lo(w[i]), u1 = hi(w[i]), v0 = lo(w[i + 1]), v1 = hi(w[i + 1]);
                turn_pair(u0, u1, make_float2(t.x, t.y));
                turn_pair(v0, v1, make_float2(t.z, t.w));
                w[i] = ptx::pack_bf16x2(u0, u1);
                w[i + 1] = ptx::pack_bf16x2(v0, v1);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The larger value; NaN if one of them is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest of a warp's absolute values: as their bits, of which those of a NaN are above all others.
__device__ __forceinline__ float warp_amax(float a) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a))); }

// ---- append of a projection's rows ----
struct AppendParams {
    const int32_t *pt;       // [S][max_pages] or null (windows)
    const uint16_t *x;
    const uint4 *gain;       // null: no norm
    char *cache_base;        // page 0 of this cache
    DevErr *err;
    int64_t x_row;           // in values
    int32_t max_pages, num_pages;
    float eps, amplitude;
    int32_t rotate;
    uint64_t turn[kRope / 2];
    Packed rows;
};

// The page of a stream's row, or -1 (recorded).
__device__ __forceinline__ int page_of(const int32_t *pt, int max_pages, int num_pages, int s, int pos, DevErr *err,
                                       bool tell) {
    const int page = pt ? __ldg(pt + (int64_t)s * max_pages + (pos >> 9)) : s * max_pages + (pos >> 9);
    if (page >= 0 && page < num_pages) return page;
    if (tell) ptx::record_error(err, TF_E_DEVICE, page);
    return -1;
}

// One warp a row: lane l has latent values 8l .. 8l + 7 and 256 more of them further on, so that loads and stores are
// whole lines, and rope pair l.  The row's square sum is added in fp32, 16 values a lane and then across the warp.
// BF16, 297,264 rows (685 MB): 102 to 103 us, 0.99 of the measured copy rate (bare, without norm and rotation, 97);
// FP8 (534 MB): 105 us, 0.75: what the codes add to each row's chain (amax, scale, quotients) shows.  Six blocks an
// SM: 108 and 111 us with five, 113 and 104 to 113 with seven, which spill some 48 bytes (of the four forms one spills 8 at
// six).  Two rows a warp: 104 and 124.
template <bool FP8, bool HALF>
__global__ void __launch_bounds__(256, 6) append_rope_kernel(const __grid_constant__ AppendParams p) {
    __shared__ uint64_t turns[kRope / 2];
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w8 = threadIdx.x >> 5;
    const int row = (int)blockIdx.x * 8 + w8;
    // a parameter is read for one index at a time: 32 of them once a block, not once a row (112 us)
    if (lane < 4) turns[4 * w8 + lane] = p.turn[4 * w8 + lane];
    __syncthreads();
    if (row >= p.rows.n) return;
    const int s = stream_of(p.rows, row);
    const int pos = p.rows.base[s] + row;
    const uint16_t *src = p.x + row * p.x_row;
    const int ca = lane, cb = lane + 32;   // 16-byte chunks (8 bytes as codes)
    ptx::griddep_wait();
    // the row is on its way while the page is looked up and the angle made
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(src) + ca), b = __ldg(reinterpret_cast<const uint4 *>(src) + cb);
    uint32_t kw;   // the rope pair
    if (HALF)
        kw = __ldg(src + kLat + lane) | (uint32_t)__ldg(src + kLat + kRope / 2 + lane) << 16;
    else
        kw = __ldg(reinterpret_cast<const uint32_t *>(src + kLat) + lane);
    const int page = page_of(p.pt, p.max_pages, p.num_pages, s, pos, p.err, lane == 0);
    const float2 cs = p.rotate ? turn_of(turns[lane], pos, p.amplitude) : make_float2(1.f, 0.f);
    if (page < 0) return;
    const int r = pos & (kPageRows - 1);
    float k0 = lo(kw), k1 = hi(kw);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = lo(w[i]);
        x[2 * i + 1] = hi(w[i]);
    }
    if (p.gain) {
        const uint4 ga = __ldg(p.gain + ca), gb = __ldg(p.gain + cb);
        const uint32_t g[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) q = ptx::fma2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(x[2 * i], x[2 * i + 1]), q);
        float sum = q.x + q.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float f = rsqrtf(sum * (1.0f / kLat) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = ptx::mul2(ptx::mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(f, f)), make_float2(lo(g[i]), hi(g[i])));
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
    }
    if (p.rotate) turn_pair(k0, k1, cs);
    char *pg = p.cache_base + (size_t)page * (FP8 ? kF8PageBytes : kPageBytes);
    if (FP8) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = max_or_nan(amax, fabsf(x[i]));
        amax = warp_amax(amax);
        const bool nan = amax != amax;
        if (nan) {   // the scale is that of the other values, which keep theirs; 0 where there are none (or only zeros)
            amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
            amax = warp_amax(amax);
        }
        const float scale = __fdiv_rn(amax, 448.0f);
        uint32_t code[4] = {0u, 0u, 0u, 0u};
        if (amax > 0.0f || nan) {
            // x / scale, correctly rounded: with y = 1 / scale rounded to nearest, q = x y and the remainder q scale - x
            // (exact by fma, and with this sign a zero keeps its own), q - remainder y is the nearest quotient (Markstein, 1990), as long as nothing underflows:
            // a product's last bit is 2^-10 2^-23 2^-23 scale at least where the code is not 0.  297,264 rows take 106 us
            // so and 135 with sixteen divisions a lane.
            // An infinite scale has no such remainder: finite values over it are 0, the infinite ones NaN.
            if (scale >= 0x1p-90f && scale < INFINITY) {
                const float y = __frcp_rn(scale);
                const float2 y2 = make_float2(y, y), ny2 = make_float2(-y, -y), s2 = make_float2(scale, scale);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 v = make_float2(x[i], x[i + 1]), q = ptx::mul2(v, y2);
                    const uint32_t two = __nv_cvt_float2_to_fp8x2(
                        ptx::fma2(ptx::fma2(q, s2, make_float2(-v.x, -v.y)), ny2, q), __NV_SATFINITE, __NV_E4M3);
                    code[i >> 2] |= two << (8 * (i & 2));
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {   // (a dynamic index: few instructions for what never happens)
                    float v = pick(x, i);
                    if (scale > 0.0f) v = __fdiv_rn(v, scale);   // else zeros and NaN, as they are
                    const uint32_t c = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (i >> 2 == k) code[k] |= c << (8 * (i & 3));
                }
            }
        }
        uint2 *dst = reinterpret_cast<uint2 *>(pg + (size_t)r * kLat);
        dst[ca] = make_uint2(code[0], code[1]);
        dst[cb] = make_uint2(code[2], code[3]);
        if (lane == 0) reinterpret_cast<float *>(pg + kF8ScaleOff)[r] = scale;
    } else {
        // without a norm the packed values are the bits that came
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p.gain) w[i] = ptx::pack_bf16x2(x[2 * i], x[2 * i + 1]);
        uint4 *dst = reinterpret_cast<uint4 *>(pg + (size_t)r * (kLat * 2));
        dst[ca] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[cb] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    uint16_t *key = reinterpret_cast<uint16_t *>(pg + (FP8 ? kF8RopeOff : kLatBlockBytes)) + (size_t)r * kRope;
    const uint32_t pair = ptx::pack_bf16x2(k0, k1);
    if (HALF) {
        key[lane] = (uint16_t)pair;
        key[kRope / 2 + lane] = (uint16_t)(pair >> 16);
    } else {
        reinterpret_cast<uint32_t *>(key)[lane] = pair;
    }
}

// ---- rows back from the pages ----
struct ReadParams {
    const int32_t *pt;
    const char *cache_base;
    uint16_t *lat, *rope;    // null: not wanted
    DevErr *err;
    int64_t lat_row, rope_row;   // in values
    int32_t max_pages, num_pages;
    Packed rows;
};

// One warp a row: 16 bytes a lane and load, whole lines in and out.  BF16, 100,000 rows (230 MB): 34.9 us,
// 0.97 of the measured copy rate; FP8, 297,270 rows (534 MB): 81 us, 0.97.
template <bool FP8>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int row = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= p.rows.n) return;
    const int s = stream_of(p.rows, row);
    const int pos = p.rows.base[s] + row;
    ptx::griddep_wait();
    const int page = page_of(p.pt, p.max_pages, p.num_pages, s, pos, p.err, lane == 0);
    if (page < 0) return;
    const int r = pos & (kPageRows - 1);
    const char *pg = p.cache_base + (size_t)page * (FP8 ? kF8PageBytes : kPageBytes);
    const uint4 *key = reinterpret_cast<const uint4 *>(pg + (FP8 ? kF8RopeOff : kLatBlockBytes) + (size_t)r * (kRope * 2));
    uint4 k;
    if (p.rope && lane < 8) k = __ldg(key + lane);
    if (p.lat) {
        uint4 *dst = reinterpret_cast<uint4 *>(p.lat + row * p.lat_row);
        if (FP8) {
            const uint2 *codes = reinterpret_cast<const uint2 *>(pg + (size_t)r * kLat);
            const uint2 c[2] = {__ldg(codes + lane), __ldg(codes + lane + 32)};
            const float scale = __ldg(reinterpret_cast<const float *>(pg + kF8ScaleOff) + r);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = ((i & 2) ? c[q].y : c[q].x) >> (16 * (i & 1));
                    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
                    const float2 f = __half22float2(__half2(hr));
                    o[i] = ptx::pack_bf16x2(f.x * scale, f.y * scale);
                }
                dst[lane + 32 * q] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        } else {
            const uint4 *src = reinterpret_cast<const uint4 *>(pg + (size_t)r * (kLat * 2));
            const uint4 a = __ldg(src + lane), b = __ldg(src + lane + 32);
            dst[lane] = a;
            dst[lane + 32] = b;
        }
    }
    if (p.rope && lane < 8) reinterpret_cast<uint4 *>(p.rope + row * p.rope_row)[lane] = k;
}

static void pack(Packed &k, const int64_t *h_pos, const int64_t *h_n, int S) {
    int64_t n = 0;
    for (int s = 0; s < S; ++s) {
        k.off[s] = (int32_t)n;
        k.base[s] = (int32_t)(h_pos[s] - n);
        n += h_n[s];
    }
    k.S = S;
    k.n = (int32_t)n;
}

}  // namespace rows

int launch_rope(const tf_rope *rope, const int64_t *h_pos, const int64_t *h_n, int S, int H, const void *d_x, int64_t x_row,
                int64_t x_head, void *d_y, int64_t y_row, int64_t y_head, cudaStream_t st) {
    using namespace rows;
    RopeParams p;
    pack(p.rows, h_pos, h_n, S);
    p.x = static_cast<const uint16_t *>(d_x);
    p.y = static_cast<uint16_t *>(d_y);
    p.x_row = x_row;
    p.x_head = x_head;
    p.y_row = y_row;
    p.y_head = y_head;
    p.H = H;
    p.dim = rope->dim;
    p.amplitude = rope->amplitude;
    for (int i = 0; i < rope->dim / 2; ++i) p.turn[i] = rope->turn[i];
    const bool half = rope->layout == TF_ROPE_HALF;
    p.cols = H * rope->dim / (half ? 16 : 8);
    p.threads_per_row = std::min(p.cols, RT);
    // Rows in flight a thread: as many as the table has room for, where the blocks still go round the SMs twice;
    // 19,480 rows of 64 heads take 50.6 us with four (half layout), 51.9 with two.
    const int lanes = RT / p.threads_per_row, gy = (p.cols + p.threads_per_row - 1) / p.threads_per_row;
    int it = half ? 4 : 8;
    if (lanes * it * (rope->dim / 2) > RTAB) it /= 2;
    if ((int64_t)p.rows.n * gy / (lanes * it) < 304) it = 1;
    const dim3 grid((unsigned)((p.rows.n + (int64_t)lanes * it - 1) / (lanes * it)), (unsigned)gy);
    auto *kern = half ? (it == 1 ? rope_kernel<true, 1> : it == 2 ? rope_kernel<true, 2> : rope_kernel<true, 4>)
                      : (it == 1 ? rope_kernel<false, 1> : it == 4 ? rope_kernel<false, 4> : rope_kernel<false, 8>);
    const cudaError_t e = launch_pdl(kern, grid, dim3(RT), sizeof(float2) * lanes * it * (rope->dim / 2), st, p);
    launch_counter()++;
    return e == cudaSuccess ? TF_OK : TF_E_CUDA;
}

int launch_append_rope(tf_kvpool *pool, int cache, const int32_t *d_pt, int max_pages, const int64_t *h_pos,
                       const int64_t *h_n, int S, const void *d_rows, int64_t row_stride, const void *d_gain, float eps,
                       const tf_rope *rope, cudaStream_t st) {
    using namespace rows;
    const bool f8 = is_fp8(pool->desc);
    rows::AppendParams p;
    pack(p.rows, h_pos, h_n, S);
    p.pt = d_pt;
    p.x = static_cast<const uint16_t *>(d_rows);
    p.gain = static_cast<const uint4 *>(d_gain);
    p.cache_base = pool->base + (size_t)cache * pool->desc.num_pages * page_bytes(pool->desc);
    p.err = pool->err;
    p.x_row = row_stride;
    p.max_pages = max_pages;
    p.num_pages = pool->desc.num_pages;
    p.eps = eps;
    p.rotate = rope != nullptr;
    p.amplitude = rope ? rope->amplitude : 1.f;
    for (int i = 0; i < kRope / 2; ++i) p.turn[i] = rope ? rope->turn[i] : 0;
    const bool half = rope && rope->layout == TF_ROPE_HALF;
    if (prepare_launch(pool, st) != TF_OK) return TF_E_CUDA;
    ProfScope prof(pool, kProfAppend, st);
    auto *kern = f8 ? (half ? append_rope_kernel<true, true> : append_rope_kernel<true, false>)
                    : (half ? append_rope_kernel<false, true> : append_rope_kernel<false, false>);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)((p.rows.n + (int64_t)7) / 8)), dim3(256), 0, st, p);
    launch_counter()++;
    return e == cudaSuccess ? TF_OK : TF_E_CUDA;
}

int launch_paged_read(tf_kvpool *pool, int cache, const int32_t *d_pt, int max_pages, const int64_t *h_from,
                      const int64_t *h_n, int S, void *d_latent, int64_t lat_stride, void *d_rope, int64_t rope_stride,
                      cudaStream_t st) {
    using namespace rows;
    const bool f8 = is_fp8(pool->desc);
    ReadParams p;
    pack(p.rows, h_from, h_n, S);
    p.pt = d_pt;
    p.cache_base = pool->base + (size_t)cache * pool->desc.num_pages * page_bytes(pool->desc);
    p.lat = static_cast<uint16_t *>(d_latent);
    p.rope = static_cast<uint16_t *>(d_rope);
    p.err = pool->err;
    p.lat_row = lat_stride;
    p.rope_row = rope_stride;
    p.max_pages = max_pages;
    p.num_pages = pool->desc.num_pages;
    if (prepare_launch(pool, st) != TF_OK) return TF_E_CUDA;
    ProfScope prof(pool, kProfCopy, st);
    const cudaError_t e = launch_pdl(f8 ? read_kernel<true> : read_kernel<false>,
                                     dim3((unsigned)((p.rows.n + (int64_t)7) / 8)), dim3(256), 0, st, p);
    launch_counter()++;
    return e == cudaSuccess ? TF_OK : TF_E_CUDA;
}

}  // namespace tf
