// Choosing blocks of rows for sparse attention: the mean row ("key") of every 64-row block of a
// paged latent cache, and the score of each visible block for every query row.  The scores go to
// the blocked top-k, whose lists tf_paged_mla_attend_blocks takes.
//
//   k_b        = mean of the rows of block b that the stream holds         (576 wide, bf16)
//   score[r,b] = sum_h w[r,h] max(0, scale q[r,h] . k_b)                    (fp32)
//
// Pooled index keys and the weighted sum of rectified products over heads are the TensorFold pages'
// (issue #1142, "What happens now": one pooled index key every few tokens; issue #1142, piece 2: the kernels that pool keys and score
// them take the page table).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <memory>

#include "per_device.h"
#include "ptx.cuh"
#include "tf_internal.h"

namespace tf {

namespace blk {

constexpr int ROWS = TF_BLOCK_ROWS;
constexpr int PER_PAGE = kPageRows / ROWS;   // 8 blocks a page

// ---- block keys ----
struct KeysParams {
    const int32_t *pt;       // [S][max_pages] or null (windows)
    const char *cache_base;  // page 0 of this cache
    uint16_t *bkeys;         // [pages][8][576] bf16
    DevErr *err;
    int32_t max_pages, num_pages, S;
    int64_t off[TF_MAX_STREAMS + 1];   // first numbered block of each stream
    int64_t len[TF_MAX_STREAMS];
    int32_t first[TF_MAX_STREAMS];     // first block to average
};

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Numbered block n of the call: its stream and its number there.
__device__ __forceinline__ int64_t block_of(const KeysParams &p, int64_t n, int &s) {
    s = 0;
    for (int a = p.S - 1; s < a;) {   // the last stream whose blocks begin at or before n
        const int mid = (s + a + 1) >> 1;
        if (p.off[mid] <= n) s = mid; else a = mid - 1;
    }
    return p.first[s] + (n - p.off[s]);
}

// The block's page and rows; false, recorded, for a page out of the pool.
__device__ __forceinline__ bool block_rows(const KeysParams &p, int s, int64_t b, int &page, int &rows) {
    const int lp = (int)(b / PER_PAGE);
    page = p.pt ? __ldg(p.pt + (int64_t)s * p.max_pages + lp) : s * p.max_pages + lp;
    if (page < 0 || page >= p.num_pages) {
        ptx::record_error(p.err, TF_E_DEVICE, page);
        return false;
    }
    const int64_t left = p.len[s] - b * ROWS;
    rows = left < ROWS ? (int)left : ROWS;
    return true;
}

// Values 2 i, 2 i + 1 of a block's key: the G sums of each, added in order, over the rows, rounded once.
template <int G>
__device__ __forceinline__ uint32_t mean_pair(const float (&part)[G][kDk], int i, int rows) {
    float a = 0.f, d = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) {
        a += part[k][2 * i];
        d += part[k][2 * i + 1];
    }
    return ptx::pack_bf16x2(__fdiv_rn(a, (float)rows), __fdiv_rn(d, (float)rows));
}

// BF16 pages, one CTA a block: thread (g, c) adds 16-byte chunk c (72 a row) of rows g, g + 4, ... in
// fp32, eight loads in flight.  Bound by HBM: 297,264 rows take 54.8 us, 0.94 of the measured copy rate.
constexpr int KC = kDk / 8, KG = 4;
__global__ void __launch_bounds__(KC *KG) block_keys_kernel(const __grid_constant__ KeysParams p) {
    __shared__ float part[KG][kDk];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    int s, page, rows;
    const int64_t b = block_of(p, blockIdx.x, s);
    if (!block_rows(p, s, b, page, rows)) return;
    const int c = (int)threadIdx.x % KC, g = (int)threadIdx.x / KC;
    const int ib = (int)(b % PER_PAGE), row0 = ib * ROWS;
    const char *pg = p.cache_base + (size_t)page * kPageBytes;
    constexpr int LC = kLat / 8;   // latent chunks
    const bool rope = c >= LC;
    const size_t stride = rope ? (size_t)kRope * 2 : (size_t)kLat * 2;
    const char *src = (rope ? pg + kLatBlockBytes + (c - LC) * 16 : pg + c * 16) + (size_t)row0 * stride;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    constexpr int U = 8;             // loads in flight
#pragma unroll
    for (int i0 = 0; i0 < ROWS / KG; i0 += U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = (i0 + u) * KG + g;
            v[u] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(src + (size_t)r * stride)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[2 * k] += lo(w[k]);
                acc[2 * k + 1] += hi(w[k]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[g][8 * c + i] = acc[i];
    __syncthreads();
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.bkeys + ((size_t)page * PER_PAGE + ib) * kDk);
    for (int i = threadIdx.x; i < kDk / 2; i += KC * KG) dst[i] = mean_pair(part, i, rows);
}

// FP8 pages: a row's latent value is bf16(code * scale), as the attention takes it, so a value costs
// about five instructions and the loads of a CTA that also computes leave HBM idle (35 us for
// 208,000 rows in the form above).  Here a CTA a SM walks the blocks: one warp copies a block's codes
// (32 KB), rope rows and scales into a ring, and teams of ten warps take the blocks in turn, thread
// (g, c) of a team chunk c of rows g, g + 8, ... (32 chunks of 16 codes and 8 of 8 rope values a row).
// One team is latency-bound (43 us).
constexpr int FC = kLat / 16 + kRope / 8, FG = 8, FT = FC * FG;   // 40 chunks, 8 row groups, 320 threads
constexpr int FTEAMS = 3;
constexpr int FSTAGES = 4;
constexpr int F_ROPE = ROWS * kLat, F_SCALE = F_ROPE + ROWS * kRope * 2, F_STAGE = F_SCALE + ROWS * 4;
struct KeysFp8Shared {
    alignas(128) uint8_t ring[FSTAGES][F_STAGE];
    float part[FTEAMS][FG][kDk];
    uint64_t full[FSTAGES], empty[FSTAGES];
    int rows[FSTAGES], dst[FSTAGES];   // rows of the stage's block (0: left out), its key's number
    int abort;
};
__global__ void __launch_bounds__(FTEAMS * FT + 32, 1) block_keys_fp8_kernel(const __grid_constant__ KeysParams p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    KeysFp8Shared &sh = *reinterpret_cast<KeysFp8Shared *>(smem_raw);
    ptx::griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < FSTAGES; ++i) {
            ptx::mbar_init(&sh.full[i], 1);
            ptx::mbar_init(&sh.empty[i], FT / 32);
        }
        sh.abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    ptx::griddep_wait();
    volatile int *abort = &sh.abort;
    const int64_t total = p.off[p.S];
    if (threadIdx.x >= FTEAMS * FT) {
        if (threadIdx.x != FTEAMS * FT) return;
        int64_t k = 0;
        for (int64_t n = blockIdx.x; n < total; n += gridDim.x, ++k) {
            const int st = (int)(k % FSTAGES);
            int s, page = 0, rows = 0;
            const int64_t b = block_of(p, n, s);
            const bool good = block_rows(p, s, b, page, rows);
            if (k >= FSTAGES && !ptx::mbar_wait(&sh.empty[st], (uint32_t)(k / FSTAGES - 1) & 1, abort, p.err, 40)) break;
            sh.rows[st] = good ? rows : 0;
            sh.dst[st] = page * PER_PAGE + (int)(b % PER_PAGE);
            if (!good) {
                ptx::mbar_arrive(&sh.full[st]);
                continue;
            }
            const char *pg = p.cache_base + (size_t)page * kF8PageBytes;
            const int row0 = (int)(b % PER_PAGE) * ROWS;
            const uint32_t sb = (rows * 4 + 15) / 16 * 16;   // whole 16 bytes of the page's scales
            ptx::mbar_arrive_expect_tx(&sh.full[st], rows * (kLat + kRope * 2) + sb);
            ptx::bulk_g2s(sh.ring[st], pg + (size_t)row0 * kLat, rows * kLat, &sh.full[st]);
            ptx::bulk_g2s(sh.ring[st] + F_ROPE, pg + kF8RopeOff + (size_t)row0 * kRope * 2, rows * kRope * 2, &sh.full[st]);
            ptx::bulk_g2s(sh.ring[st] + F_SCALE, pg + kF8ScaleOff + (size_t)row0 * 4, sb, &sh.full[st]);
        }
        // no copy may still be writing shared memory when the CTA exits
        for (int64_t j = k > FSTAGES ? k - FSTAGES : 0; j < k; ++j)
            ptx::mbar_wait(&sh.full[j % FSTAGES], (uint32_t)(j / FSTAGES) & 1, abort, p.err, 41, 1ll << 28);
        return;
    }
    const int team = (int)threadIdx.x / FT, tid = (int)threadIdx.x % FT;
    const int c = tid % FC, g = tid / FC;
    const bool rope = c >= kLat / 16;
    float(&part)[FG][kDk] = sh.part[team];
    int64_t k = team;
    bool ok = true;
    for (int64_t n = blockIdx.x + (int64_t)team * gridDim.x; n < total; n += FTEAMS * (int64_t)gridDim.x, k += FTEAMS) {
        const int st = (int)(k % FSTAGES);
        if (!ptx::mbar_wait_warp(&sh.full[st], (uint32_t)(k / FSTAGES) & 1, abort, p.err, 42)) ok = false;
        // the team's previous sums are read; its warps leave together when a wait ran out
        if (ptx::named_bar_or(1 + team, FT, !ok || *abort)) return;
        const int rows = sh.rows[st], dn = sh.dst[st];
        float2 acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = make_float2(0.f, 0.f);
        if (rope) {
            for (int r = g; r < rows; r += FG) {
                const uint4 v = *reinterpret_cast<const uint4 *>(sh.ring[st] + F_ROPE + r * kRope * 2 + (c - kLat / 16) * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = ptx::add2(acc[i], make_float2(lo(w[i]), hi(w[i])));
            }
        } else {
#pragma unroll 4
            for (int r = g; r < rows; r += FG) {
                const uint4 v = *reinterpret_cast<const uint4 *>(sh.ring[st] + r * kLat + c * 16);
                const float sc = reinterpret_cast<const float *>(sh.ring[st] + F_SCALE)[r];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                        (__nv_fp8x2_storage_t)((w[i / 2] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3);
                    const float2 f = ptx::mul2(__half22float2(__half2(hr)), make_float2(sc, sc));
                    const uint32_t x = ptx::pack_bf16x2(f.x, f.y);
                    acc[i] = ptx::add2(acc[i], make_float2(lo(x), hi(x)));
                }
            }
        }
        const int v0 = rope ? kLat + (c - kLat / 16) * 8 : c * 16;
        float2 *dst = reinterpret_cast<float2 *>(&part[g][v0]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!rope || i < 4) dst[i] = acc[i];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&sh.empty[st]);
        ptx::named_bar(1 + team, FT);
        if (rows > 0 && tid < kDk / 2)
            reinterpret_cast<uint32_t *>(p.bkeys + (size_t)dn * kDk)[tid] = mean_pair(part, tid, rows);
    }
}

// ---- block scores ----
// A GEMM of the block keys with the queries, blocks on the accumulator's lanes:
//   D[256 blocks][N columns] = K[256][576] . Q[N][576]^T      tcgen05.mma cta_group::2, M = 256,
//                                                             K in 9 boxes of 64
// so a thread of the epilogue holds one block and adds the rectified products of a query row's
// heads, which lie along its columns, in registers; a warp's stores are 128 bytes of a score row.
// A tile's columns are as many whole query rows as fit 256 columns.  A pair of CTAs walks a run of
// tiles, block tile by block tile, so the block keys (128 a CTA, 144 KB) stay in shared memory while
// query tiles stream through a ring of 64-wide boxes; two accumulators let a tile's products run
// under the last one's epilogue.  Why a pair: each CTA holds and loads half of a query box, so a box
// of 16 KB feeds 512 cycles of products instead of 256.  One CTA alone (M = 128, N = 128) needs 64
// bytes a cycle of its queries from L2 and 128 + 64 of shared memory's 128, and took 323 us for 2,048
// rows of 64 heads against 1,595 blocks, where the products alone take 126 us.
constexpr int M = 128;                        // blocks a CTA: 16 pages of 8
constexpr int MP = 2 * M;                     // blocks a pair
constexpr int TILE_PAGES = M / PER_PAGE;
constexpr int NMAX = 256;                     // columns a tile
constexpr int KBOX = kDk / 64;                // 9
constexpr int PAGE_KEYS = PER_PAGE * kDk * 2; // 9,216 bytes: [9 boxes][8 blocks][64 values], swizzled
constexpr int STAGES = 5;
constexpr int STAGE_BYTES = NMAX / 2 * 128;
constexpr int SMEM_A = 0;
constexpr int SMEM_B = SMEM_A + TILE_PAGES * PAGE_KEYS;
constexpr int SMEM_CTRL = SMEM_B + STAGES * STAGE_BYTES;
constexpr int EPI = 256;                      // 8 epilogue warps: two a TMEM quadrant
constexpr int THREADS = EPI + 64;             // and the TMA warp, the MMA warp
constexpr int TCOLS = 2 * NMAX;

// Barriers marked L are waited on in the leader (rank 0) only and reached from both CTAs; the
// others are each CTA's own, and the MMA warp's commits arrive on both.
struct Ctrl {
    uint64_t a_full, a_free;                    // L: both CTAs' block keys are there; the tile's products are done
    uint64_t b_full[STAGES], b_free[STAGES];    // L: both halves of a query box landed; its products are done
    uint64_t d_full[2], d_free[2];              // accumulator computed; L: read by both CTAs' epilogue warps
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    alignas(16) float w[NMAX];
};
constexpr int SMEM_TOTAL = SMEM_CTRL + (int)sizeof(Ctrl) + 1024;
static_assert(ROWS == 64, "positions are shifted by 6");
static_assert(SMEM_TOTAL <= 232448, "shared memory budget");

struct ScoreParams {
    CUtensorMap tm_q;   // 2D {576, S*R*H}, box {64, npad / 2}
    const char *bkeys;
    const int32_t *pt;
    const float *w;
    float *scores;
    int32_t *nblk;
    DevErr *err;
    float scale;
    int32_t max_pages, num_pages, S, R, H;
    int32_t rpt;        // query rows a tile
    int32_t nrt;        // row tiles a stream
    int32_t npad;       // columns a tile, rounded up to 32
    int32_t sink, local;
    int64_t cols, ld;   // columns written, row stride
    int64_t items;      // (stream, block tile, row tile)
    int64_t item0[TF_MAX_STREAMS];
    int64_t len[TF_MAX_STREAMS];
};

// The pair's items: a run of the numbering (stream, block tile, place in the block tile's order), in
// which a block tile stands for as many runs as share it.  The places of a block tile are its row
// tiles in the order of (time, pair): the j-th items of all its pairs come before the (j+1)-th ones.
// So all pairs, whatever their block tile, go through the query rows side by side and each query
// tile comes from DRAM once: read run by run instead, 2,048 rows against 7 block tiles took 1.04 GB
// of DRAM reads for 151 MB of queries.
struct Items {
    int64_t len, more;     // items a pair, and how many of the first pairs have one more
    int64_t i, i1;         // next item, end
    int64_t first;         // the pair's first item
    int64_t i0 = 0;        // the block tile's first item
    // the pairs that hold the block tile: f0 .. f0 + nfull - 1 with all their items, the pair before
    // them with its times [fa, fe) and the one behind them with its times [0, le)
    int f0 = 0, nfull = 0;
    int64_t fa = 0, fe = 0, le = 0;
    int pair, s = -1;
    int64_t bt = -1;
    bool fresh = false;    // another block tile than the last item's
    __device__ __forceinline__ int64_t start(int64_t q) const { return q * len + (q < more ? q : more); }
    __device__ __forceinline__ explicit Items(const ScoreParams &p) {
        const int pairs = gridDim.x / 2;
        pair = blockIdx.x / 2;
        len = p.items / pairs;
        more = p.items - len * pairs;
        first = i = start(pair);
        i1 = start(pair + 1);
    }
    __device__ __forceinline__ bool next(const ScoreParams &p) {
        if (i >= i1) return false;
        fresh = s < 0 || i == i0 + p.nrt;
        if (fresh) {
            int a = s < 0 ? 0 : s, z = p.S - 1;
            while (a < z) {
                const int mid = (a + z + 1) >> 1;
                if (p.item0[mid] <= i) a = mid; else z = mid - 1;
            }
            s = a;
            bt = (i - p.item0[s]) / p.nrt;
            i0 = p.item0[s] + bt * p.nrt;
            const int64_t end = i0 + p.nrt;
            int p0 = pair, p1 = pair;   // they hold its first and its last item
            while (start(p0) > i0) --p0;
            while (start(p1 + 1) < end) ++p1;
            f0 = p0;
            fa = fe = le = 0;
            const bool cut0 = start(p0) < i0, cut1 = start(p1 + 1) > end;
            if (cut0) {
                ++f0;
                fa = i0 - start(p0);
                fe = (p1 > p0 ? start(p0 + 1) : end) - start(p0);
            }
            if (cut1 && !(cut0 && p1 == p0)) le = end - start(p1);
            nfull = max(0, (cut1 ? p1 - 1 : p1) - f0 + 1);
        }
        ++i;
        return true;
    }
    // after next(): the item's row tile
    __device__ __forceinline__ int64_t row_tile(const ScoreParams &p) const {
        if (p.nrt == 1) return 0;
        const int64_t t = i - 1 - first;   // <= len, so every full pair has t items before time t
        const int before = (t < len ? pair : (int)min((int64_t)pair, more)) - f0;   // full pairs ahead of this one at time t
        return t * nfull + max(0, min(before, nfull)) + min(t, le) +
               (t < fa ? 0 : t >= fe ? fe - fa : t - fa + (f0 - 1 < pair));
    }
    // after next(): the last item of its block tile here
    __device__ __forceinline__ bool last_of_tile(const ScoreParams &p) const { return i >= i1 || i == i0 + p.nrt; }
};

// ---- a pair of CTAs ----
// the address, in the pair's shared memory, of this CTA's `p` in the leader
__device__ __forceinline__ uint32_t leader_addr(const void *p) { return ptx::cluster_addr(ptx::smem_u32(p), 0); }
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// TMA into this CTA's shared memory, completing on a barrier of the pair.
__device__ __forceinline__ void tma_queries(void *dst, const CUtensorMap *tm, uint32_t bar, int x, int row,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(row), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t *dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Four MMAs along K on one 64-value box (32 bytes of each operand's rows a step); one elected lane
// issues for the pair; `first` = 1 starts the accumulator.
__device__ __forceinline__ void pair_mma4_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t first) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "setp.eq.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(first)
        : "memory");
}
// Arrive once on this CTA's `bar` when the pair's MMAs issued so far complete.
__device__ __forceinline__ void pair_commit_own_warp(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(ptx::smem_u32(bar))
        : "memory");
}
// The same on `bar` of both CTAs.
__device__ __forceinline__ void pair_commit_warp(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 both;\n\tmov.b16 both, 3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n\t}" ::"r"(
            ptx::smem_u32(bar))
        : "memory");
}

// C: a divisor of H that the epilogue adds up without asking whether the query row ends (32, 8, 4 or 1):
// at C = 1 a warp's 128 questions a tile cost more than its products (2,048 rows of 20 heads against
// 1,563 blocks take 179 us with C = 1 and 77 with C = 4; 32 heads take 90 us with C = 32).
template <int C>
__global__ void __launch_bounds__(THREADS, 1) block_scores_kernel(const __grid_constant__ ScoreParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl &c = *reinterpret_cast<Ctrl *>(smem + SMEM_CTRL);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    const uint32_t rank = ptx::cluster_rank();
    if (threadIdx.x == 0) {
        ptx::mbar_init(&c.a_full, 2 * EPI / 32);
        ptx::mbar_init(&c.a_free, 1);
        for (int i = 0; i < STAGES; ++i) {
            ptx::mbar_init(&c.b_full[i], 1);
            ptx::mbar_init(&c.b_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&c.d_full[i], 1);
            ptx::mbar_init(&c.d_free[i], 2 * EPI / 32);
        }
        ptx::mbar_init(&c.drain, 1);
        c.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == EPI / 32 + 1) pair_tmem_alloc(&c.tmem_base, TCOLS);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // the peer's barriers are ready
    ptx::tc_fence_after();
    const uint32_t tmem = c.tmem_base;
    volatile int *abort = &c.abort;
    ptx::griddep_wait();

    if (warp == EPI / 32) {
        // ================= TMA =================
        // Lane 0 waits and loads this CTA's half of each query box; both land on the leader's barrier,
        // which the leader arms with the bytes of both.
        if (lane == 0) ptx::prefetch_tmap(&p.tm_q);
        const uint64_t pol_q = ptx::policy_evict_last();
        int64_t nb = 0;    // query boxes loaded
        bool ok = true;
        Items it(p);
        auto row_of = [&]() {
            return (int)(((int64_t)it.s * p.R + it.row_tile(p) * p.rpt) * p.H) + (int)rank * (p.npad / 2);
        };
        bool more = it.next(p);
        int qrow = more ? row_of() : 0;
        while (ok && more) {
            if (lane == 0) {
                for (int kb = 0; ok && kb < KBOX; ++kb) {
                    const int64_t n = nb + kb;
                    const int st = (int)(n % STAGES);
                    if (n >= STAGES && !ptx::mbar_wait(&c.b_free[st], (uint32_t)(n / STAGES - 1) & 1, abort, p.err, 31)) {
                        ok = false;
                        nb -= KBOX - kb;   // the boxes that were not loaded
                        break;
                    }
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&c.b_full[st], p.npad * 128);
                    tma_queries(smem + SMEM_B + st * STAGE_BYTES, &p.tm_q, leader_addr(&c.b_full[st]), kb * 64, qrow, pol_q);
                }
            }
            nb += KBOX;
            more = it.next(p);   // worked out while the boxes are on their way
            if (more) qrow = row_of();
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
        // No copy may still be writing shared memory when a CTA exits, nor a commit of the leader's be
        // on its way to a barrier of the peer's: what was loaded last has to be released.
        if (lane == 0) {
            for (int k = 0; k < STAGES; ++k)
                if (nb > k) {
                    const int64_t last = nb - 1 - k;
                    ptx::mbar_wait(&c.b_free[last % STAGES], (uint32_t)(last / STAGES) & 1, abort, p.err, 32, 1ll << 28);
                }
            // after a wait that ran out: the copies themselves (all land on the leader's barriers)
            if (*abort && rank == 0) {
                for (int k = 0; k < STAGES; ++k)
                    if (nb > k) {
                        const int64_t last = nb - 1 - k;
                        ptx::mbar_wait(&c.b_full[last % STAGES], (uint32_t)(last / STAGES) & 1, abort, p.err, 32, 1ll << 28);
                    }
            }
        }
        __syncwarp();
    } else if (warp == EPI / 32 + 1) {
        // ================= MMA (the leader, for the pair) =================
        const uint64_t a0 = ptx::sdesc_sw128(ptx::smem_u32(smem + SMEM_A), 16, PAGE_KEYS);
        const uint64_t b0 = ptx::sdesc_sw128(ptx::smem_u32(smem + SMEM_B), 16, 1024);
        const uint32_t idesc = ptx::idesc_bf16_f32(MP, p.npad, false, false);
        int na = 0;
        int64_t nb = 0, nd = 0;
        bool ok = rank == 0;
        for (Items it(p); ok && it.next(p); ++nd) {
            if (it.fresh) {
                if (!ptx::mbar_wait_warp(&c.a_full, na & 1, abort, p.err, 33)) break;
                ++na;
            }
            const int buf = (int)(nd & 1);
            if (nd >= 2 && !ptx::mbar_wait_warp(&c.d_free[buf], (uint32_t)(nd / 2 - 1) & 1, abort, p.err, 34)) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int kb = 0; kb < KBOX; ++kb, ++nb) {
                const int st = (int)(nb % STAGES);
                if (!ptx::mbar_wait_warp(&c.b_full[st], (uint32_t)(nb / STAGES) & 1, abort, p.err, 35)) {
                    ok = false;
                    break;
                }
                pair_mma4_warp(tmem + buf * NMAX, a0 + (uint64_t)((kb * 1024) >> 4),
                               b0 + (uint64_t)((st * STAGE_BYTES) >> 4), idesc, kb == 0);
                pair_commit_warp(&c.b_free[st]);
            }
            if (!ok) break;
            pair_commit_warp(&c.d_full[buf]);
            if (it.last_of_tile(p)) pair_commit_warp(&c.a_free);
        }
        // no MMA may still run when TMEM is freed
        if (rank == 0) {
            pair_commit_own_warp(&c.drain);
            if (lane == 0) ptx::mbar_wait(&c.drain, 0, abort, p.err, 36, 1ll << 29);
        }
        __syncwarp();
    } else {
        // ================= epilogue: a block a thread, half of the item's query rows a warp =================
        const int tid = (int)threadIdx.x;
        const int half = warp >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint64_t pol_k = ptx::policy_evict_last();
        int64_t nd = 0;
        bool ok = true;
        // The weights of an item's columns go to shared memory for all to read; those of the next are
        // fetched while this one's products run (a column a thread).
        Items it(p);
        bool more = it.next(p);
        bool fresh = false, freshn = more;
        int na = 0;   // block tiles loaded
        int64_t r0 = 0, r0n = more ? it.row_tile(p) * p.rpt : 0;   // first query row: this item's, the next one's
        int s = 0, sn = it.s;
        int64_t bt = 0, btn = it.bt;
        float wn = 0.f;
        auto fetch = [&]() {
            const int n = (int)(p.R - r0n < p.rpt ? p.R - r0n : p.rpt) * p.H;
            if (p.w && tid < n) wn = __ldg(p.w + ((int64_t)sn * p.R + r0n) * p.H + tid);
        };
        if (more) fetch();
        for (; more; ++nd) {
            const int buf = (int)(nd & 1);
            r0 = r0n;
            s = sn;
            bt = btn;
            fresh = freshn;
            if (fresh) {
                // The block tile's keys, once its predecessor's products are done: two pages a warp, 18
                // copies of 16 bytes a lane and page into the 128-byte-swizzled tile (as TMA boxes, 144 of
                // one 1 KB atom, they took 8,300 cycles to issue).  A page past the stream's is left
                // out (no score is made of it), and so is one out of the pool (its scores are undefined):
                // the other lanes of the product do not see it.
                if (na > 0 && !ptx::mbar_wait_warp(&c.a_free, (na - 1) & 1, abort, p.err, 30)) ok = false;
                const int64_t pages = (p.len[s] + kPageRows - 1) / kPageRows;
#pragma unroll 1
                for (int k = 2 * warp; ok && k < 2 * warp + 2; ++k) {
                    const int64_t lp = bt * (2 * TILE_PAGES) + rank * TILE_PAGES + k;
                    if (lp >= pages) break;
                    const int id = p.pt ? __ldg(p.pt + (int64_t)s * p.max_pages + lp) : s * p.max_pages + (int)lp;
                    if (id < 0 || id >= p.num_pages) {
                        if (lane == 0) ptx::record_error(p.err, TF_E_DEVICE, id);
                        continue;
                    }
                    const char *src = p.bkeys + (size_t)id * PAGE_KEYS;
                    uint8_t *dst = smem + SMEM_A + k * PAGE_KEYS;
#pragma unroll 6
                    for (int i = 0; i < PAGE_KEYS / 16 / 32; ++i) {
                        const int x = i * 32 + lane, row = x / (kDk / 8), ch = x % (kDk / 8);   // chunk ch of block `row`
                        ptx::cp_async16(dst + (ch >> 3) * 1024 + row * 128 + (((ch & 7) ^ row) << 4), src + x * 16, pol_k);
                    }
                }
                ptx::cp_async_wait_all();
                ptx::fence_proxy_async_smem();   // the tensor cores read them
                __syncwarp();
                if (lane == 0) arrive_at(leader_addr(&c.a_full));
                ++na;
            }
            // the previous item's weights are read; the warps leave together when a wait ran out
            if (ptx::named_bar_or(1, EPI, !ok || *abort)) break;
            if (p.w) {
                c.w[tid] = wn;
                ptx::named_bar(1, EPI);
            }
            more = it.next(p);
            if (more) {
                r0n = it.row_tile(p) * p.rpt;
                sn = it.s;
                btn = it.bt;
                freshn = it.fresh;
                fetch();
            }
            if (!ptx::mbar_wait_warp(&c.d_full[buf], (uint32_t)(nd / 2) & 1, abort, p.err, 37)) {
                ok = false;
                continue;
            }
            ptx::tc_fence_after();
            const int nr = (int)(p.R - r0 < p.rpt ? p.R - r0 : p.rpt);
            const int ra = half ? (nr + 1) / 2 : 0;                    // this warp's rows
            const int ncols = ((half ? nr : (nr + 1) / 2) - ra) * p.H;  // and its columns
            const float *w = c.w + ra * p.H;
            const uint32_t col = lane_base + buf * NMAX + ra * p.H;
            const int64_t b = bt * MP + rank * M + (tid & (M - 1));
            float *dst = p.scores + ((int64_t)s * p.R + r0 + ra) * p.ld + b;
            int64_t pos = p.len[s] - p.R + r0 + ra;   // the row's position
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            int left = p.H;
            // 32 columns at n0
            auto add = [&](int n0, const uint32_t (&v)[32]) {
#pragma unroll
                for (int j = 0; j < 32; j += C) {
                    if (n0 + j >= ncols) break;
                    if (C == 1) {
                        acc[0].x = fmaf(p.w ? w[n0 + j] : 1.f, ptx::relu_nan(__uint_as_float(v[j])), acc[0].x);
                    } else {
#pragma unroll
                        for (int k = j; k < j + C; k += 4) {
                            const float4 wk = p.w ? *reinterpret_cast<const float4 *>(w + n0 + k)
                                                  : make_float4(1.f, 1.f, 1.f, 1.f);
                            acc[0] = ptx::fma2(make_float2(wk.x, wk.y),
                                               make_float2(ptx::relu_nan(__uint_as_float(v[k])),
                                                           ptx::relu_nan(__uint_as_float(v[k + 1]))), acc[0]);
                            acc[1] = ptx::fma2(make_float2(wk.z, wk.w),
                                               make_float2(ptx::relu_nan(__uint_as_float(v[k + 2])),
                                                           ptx::relu_nan(__uint_as_float(v[k + 3]))), acc[1]);
                        }
                    }
                    left -= C;
                    if (left == 0) {
                        const int mine = (int)(pos >> 6);
                        float y = ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) * p.scale;
                        if (b < p.sink || b > mine - p.local) y = INFINITY;
                        if (b > mine) y = -INFINITY;
                        if (b < p.cols) *dst = y;
                        dst += p.ld;
                        ++pos;
                        acc[0] = acc[1] = make_float2(0.f, 0.f);
                        left = p.H;
                    }
                }
            };
            // the next 32 columns are on their way from TMEM while these are added
            uint32_t va[32], vb[32];
            if (ncols > 0) ptx::tmem_ld32(col, va);
            for (int n0 = 0; n0 < ncols; n0 += 64) {
                ptx::tmem_ld_wait();
                if (n0 + 32 < ncols) ptx::tmem_ld32(col + n0 + 32, vb);
                add(n0, va);
                if (n0 + 32 >= ncols) break;
                ptx::tmem_ld_wait();
                if (n0 + 64 < ncols) ptx::tmem_ld32(col + n0 + 64, va);
                add(n0 + 32, vb);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(leader_addr(&c.d_free[buf]));
        }
        // the leader's last commit has to have reached this CTA's barrier before it exits
        if (na > 0) ptx::mbar_wait_warp(&c.a_free, (na - 1) & 1, abort, p.err, 32, 1ll << 28);
        // rows of streams with fewer block tiles than the longest: no block there; and every row's
        // visible blocks
        for (int64_t r = blockIdx.x; r < (int64_t)p.S * p.R; r += gridDim.x) {
            const int s = (int)(r / p.R);
            const int64_t len = p.len[s];
            const int64_t nb = (len + ROWS - 1) / ROWS;
            for (int64_t b = (nb + MP - 1) / MP * MP + tid; b < p.cols; b += EPI) p.scores[r * p.ld + b] = -INFINITY;
            if (p.nblk && tid == 0) p.nblk[r] = (int32_t)((len - p.R + (r - (int64_t)s * p.R)) / ROWS + 1);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // both CTAs are done with each other's barriers and TMEM
    ptx::tc_fence_after();
    if (warp == EPI / 32 + 1) pair_tmem_dealloc(tmem, TCOLS);
}

}  // namespace blk

// The current device's SMs, with every kernel opted in to its shared memory there; 0 when that failed.
static int device_ready() {
    using namespace blk;
    static PerDevice<int> sms;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int *n = sms.get(dev, [&](int &v) {
        bool ok = cudaFuncSetAttribute(block_keys_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(KeysFp8Shared)) == cudaSuccess;
        for (auto *kern : {block_scores_kernel<32>, block_scores_kernel<8>, block_scores_kernel<4>, block_scores_kernel<1>})
            ok = ok && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL) == cudaSuccess;
        ok = ok && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
        if (!ok) cudaGetLastError();
        return ok;
    });
    return n ? *n : 0;
}

int launch_block_keys(tf_kvpool *pool, int cache, const int32_t *d_pt, int max_pages, const int64_t *h_from,
                      const int64_t *h_len, int S, void *d_bkeys, cudaStream_t st) {
    using namespace blk;
    KeysParams p;
    const bool f8 = is_fp8(pool->desc);
    p.pt = d_pt;
    p.cache_base = pool->base + (size_t)cache * pool->desc.num_pages * page_bytes(pool->desc);
    p.bkeys = static_cast<uint16_t *>(d_bkeys);
    p.err = pool->err;
    p.max_pages = max_pages;
    p.num_pages = pool->desc.num_pages;
    p.S = S;
    int64_t n = 0;
    for (int s = 0; s < S; ++s) {
        p.off[s] = n;
        p.len[s] = h_len[s];
        p.first[s] = (int32_t)(h_from[s] / ROWS);
        if (h_from[s] < h_len[s]) n += (h_len[s] + ROWS - 1) / ROWS - p.first[s];
    }
    p.off[S] = n;
    if (n == 0) return TF_OK;
    if (n > 0x7FFFFFFF) return TF_E_UNSUPPORTED;
    const int sms = f8 ? device_ready() : 0;
    if (f8 && sms <= 0) return TF_E_CUDA;
    if (prepare_launch(pool, st) != TF_OK) return TF_E_CUDA;
    ProfScope prof(pool, kProfBlockKeys, st);
    const cudaError_t e = f8 ? launch_pdl(block_keys_fp8_kernel, dim3((unsigned)std::min<int64_t>(n, sms)),
                                          dim3(FTEAMS * FT + 32), sizeof(KeysFp8Shared), st, p)
                             : launch_pdl(block_keys_kernel, dim3((unsigned)n), dim3(KC * KG), 0, st, p);
    launch_counter()++;
    return e == cudaSuccess ? TF_OK : TF_E_CUDA;
}

int launch_block_scores(tf_kvpool *pool, const void *d_bkeys, const int32_t *d_pt, int max_pages, const int64_t *h_len,
                        int S, int R, int H, const void *d_q, const float *d_w, float scale, int sink, int local,
                        float *d_scores, int64_t ld, int32_t *d_nblk, cudaStream_t st) {
    using namespace blk;
    const int ready_sms = device_ready();
    if (ready_sms <= 0) return TF_E_CUDA;
    thread_local std::unique_ptr<ScoreParams> pp;
    if (!pp) pp.reset(new ScoreParams());
    ScoreParams &p = *pp;
    p.bkeys = static_cast<const char *>(d_bkeys);
    p.rpt = std::min(R, std::max(1, NMAX / H));
    // a warp of the epilogue reads 32 columns at a time from its first row on, up to the buffer's end
    auto reach = [&](int nr) { return (nr + 1) / 2 * H + (nr / 2 * H + 31) / 32 * 32; };
    for (int nr = 1; nr <= p.rpt; ++nr)
        if (reach(nr) > NMAX) p.rpt = nr - 1;
    p.nrt = (R + p.rpt - 1) / p.rpt;
    p.npad = (p.rpt * H + 31) / 32 * 32;
    {
        const uint64_t dims[2] = {(uint64_t)kDk, (uint64_t)S * R * H};
        const uint64_t strides[1] = {(uint64_t)kDk * 2};
        const uint32_t box[2] = {64, (uint32_t)p.npad / 2};
        if (!encode_tmap_bf16(&p.tm_q, const_cast<void *>(d_q), 2, dims, strides, box)) return TF_E_CUDA;
    }
    p.pt = d_pt;
    p.w = d_w;
    p.scores = d_scores;
    p.nblk = d_nblk;
    p.err = pool->err;
    p.scale = scale;
    p.max_pages = max_pages;
    p.num_pages = pool->desc.num_pages;
    p.S = S;
    p.R = R;
    p.H = H;
    p.sink = sink;
    p.local = local;
    p.ld = ld;
    p.cols = 0;
    p.items = 0;
    for (int s = 0; s < S; ++s) {
        const int64_t nb = (h_len[s] + ROWS - 1) / ROWS;
        p.cols = std::max(p.cols, nb);
        p.len[s] = h_len[s];
        p.item0[s] = p.items;
        p.items += (nb + MP - 1) / MP * p.nrt;
    }
    const int ctas = 2 * (int)std::min<int64_t>(p.items, std::max(1, ready_sms / 2));
    if (prepare_launch(pool, st) != TF_OK) return TF_E_CUDA;
    auto *kern = H % 32 == 0  ? block_scores_kernel<32>
                 : H % 8 == 0 ? block_scores_kernel<8>
                 : H % 4 == 0 ? block_scores_kernel<4>
                              : block_scores_kernel<1>;
    ProfScope prof(pool, kProfBlockScores, st);
    const cudaError_t e = launch_pdl_pairs(kern, dim3((unsigned)ctas), dim3(THREADS), SMEM_TOTAL, st, p);
    launch_counter()++;
    return e == cudaSuccess ? TF_OK : TF_E_CUDA;
}

}  // namespace tf
