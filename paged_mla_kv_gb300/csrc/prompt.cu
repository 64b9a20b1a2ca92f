// Attention of packed prompts whose heads have keys and values of their own (include/tf_prompt.h): the form
// of the attention that a layer uses where the projected keys cost less than the absorbed ones (2 (192 + 128)
// operations a query, key and head against 2 (576 + 512)).
//
//   S = Q K^T            [128 query rows x 128 keys], tcgen05, accumulated in TMEM
//   P = 2^(c S - m)      c = scale log2(e); the running maximum m moves only when a row passes it by 2^8
//   O = O + P V          P in TMEM (over S), V as it lies (MN-major)
//   out = O / l, lse = (m + log2 l) ln 2
//
// A query tile is 128 rows: tokens times the H / Hkv heads that share a key head, so that the keys of a
// single token's heads are read once.  A work item is a key head and a block of one or two such tiles over a
// range of 128-key tiles; two softmax warpgroups keep a tile each.  With two query tiles each takes one of
// them, over the same keys; with one, they take every other key tile of it and join what they have at the end.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <memory>
#include <type_traits>

#include "per_device.h"
#include "ptx.cuh"
#include "tf_internal.h"

namespace tf {

namespace prm {

constexpr int BM = 128;              // rows of a query tile
constexpr int BN = 128;              // keys of a tile
constexpr int BOX = 64;              // values of a box's row: 128 bytes, one swizzle atom
constexpr int VH = 64;               // keys of a half of a value tile
// Warps: two softmax warpgroups, one for the outputs, the MMA warp (for both warpgroups), the TMA warp, and the item warp, which
// asks for the next item and works out what it is; the last one does nothing.
constexpr int THREADS = 512;
constexpr int OUT_WARP = 8, MMA_WARP = 12, TMA_WARP = 13, ITEM_WARP = 14;
// Registers a thread: 128 at launch, of which the softmax takes more and the others less.
constexpr int REGS_SOFTMAX = 192, REGS_OUT = 64, REGS_OTHER = 64;
static_assert(2 * REGS_SOFTMAX + REGS_OUT + REGS_OTHER <= 4 * 128, "a split above the launch's total would wait forever");
constexpr int MAX_UNITS = 24;
constexpr int MAX_SMS = TF_PLAN_MAX_RANGES;

// Shared memory (bytes): the two query tiles, then a ring of units the size of half a value tile (64 keys), in
// which key tiles (KU units) and halves of value tiles follow one another in the order of their use; 224 KB in each
// form.  One ring for both holds a step more than two: at 192 wide, 8 units of 16 KB against 5 a step.
template <int DQK, int DV>
struct Lay {
    static constexpr int QB = DQK / BOX, VB = DV / BOX;
    static constexpr int Q_TILE = BM * DQK * 2, K_TILE = BN * DQK * 2, UNIT = VH * DV * 2;
    static constexpr int KU = K_TILE / UNIT, BU = BN * 128 / UNIT;   // units of a key tile, of one of its boxes
    // Groups of a key tile: boxes with a barrier of their own where the ring holds less than two steps, so that the
    // next keys' first boxes come while the last values are still in use (2,048 rows behind 100,000: 4.80 ms with one group,
    // 4.60 so; the halves of the values on their own as well: 4.77; at 128 wide, two steps and a half, 1.07 ms with one, 1.16 with two).
    static constexpr int KG = DQK == 192 ? QB : 1;
    static constexpr int OFF_R = 2 * Q_TILE, BYTES = 229376, U = (BYTES - OFF_R) / UNIT;
    // a box does not wrap: it starts on a multiple of its own size, as keys and pairs of value halves do
    static_assert(U * UNIT + OFF_R == BYTES && U <= MAX_UNITS && K_TILE % UNIT == 0 && U % BU == 0 && 2 % BU == 0, "the ring's form");
};

// A place in the ring: group (of a key tile, or a value tile) number `g` modulo U, its phase, its first unit.
template <int U>
struct Ring {
    int g = 0, u = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int units) {
        if (++g == U) {
            g = 0;
            phase ^= 1;
        }
        u += units;
        if (u >= U) u -= U;
    }
    template <typename L>
    __device__ __forceinline__ void keys() {
#pragma unroll
        for (int i = 0; i < L::KG; ++i) step(L::KU / L::KG);
    }
};

// Key tiles of an item, at most.  The tensor cores cut an accumulated sum where fp32 would round it: a sum of values of
// one sign loses 2^-23 of itself with every 16 keys.  Unsplit, 524,288 keys came out 0.4% low, as much as a rounding to
// bf16, 2^20 keys 0.75%, 2^24 10%; in parts of 131,072, which are joined in fp32, any number loses 0.1%.  It also keeps an
// item (3 to 4 million cycles then) far below the limit of the waits that last as long as one.
constexpr int LONGEST = 1024;

// Streams in the order of their work, the longest first.
struct Params {
    CUtensorMap q, k, kr, v;
    uint16_t *out;
    float *lse;
    float *part;                     // [slots][BM][DV], then (m, l) [slots][BM]
    struct {                         // a tensor as plain memory, for outputs that are made again
        const uint16_t *p;
        int64_t row, head;
    } mq, mk, mkr, mv;
    DevErr *err;
    int64_t out_row, out_head, slots;
    float scale_log2, thr;           // c; 8 / c
    int32_t S, H, Hkv, G, tpt, causal, has_kr;   // tpt: tokens of a query tile
    int32_t more;                    // more items than SMs
    int32_t out32;                   // output rows lie on 32 bytes
    int32_t item0[TF_MAX_STREAMS];   // first item
    int32_t qoff[TF_MAX_STREAMS], nq[TF_MAX_STREAMS], koff[TF_MAX_STREAMS], nk[TF_MAX_STREAMS];
    int32_t chunk[TF_MAX_STREAMS];   // key tiles of a split
    int32_t slot0[TF_MAX_STREAMS];   // first slot of a stream whose keys are split, or -1
    int16_t nsp[TF_MAX_STREAMS];     // splits
    int16_t hg[TF_MAX_STREAMS];      // key heads side by side
};

__host__ __device__ inline int ceil_div(int a, int b) { return (int)(((unsigned)a + b - 1) / b); }   // 0 <= a <= INT_MAX

// What an item is.  Items of a stream: groups of hg key heads; in a group blocks from the last (the longest of a
// causal prompt) to the first, in a block its splits, in a split the group's heads.  The heads of a group read
// keys that fit L2 together, and blocks of one head share them there.
struct alignas(16) Item {
    int h;                   // key head
    int tok0, ntok;          // first token in the stream, tokens
    int qrow, krow;          // rows of that token and of the stream's first key
    int nk, lag;             // the stream's keys; those before its first query row's own
    int c0;                  // first key tile
    int n0, n1;              // key tiles of each warpgroup; n0 < 0: no item
    int slot;                // slot of query tile 0, or -1
    int pair;                // two query tiles

    // Item i (-1: none).  Divisions and a search: the item warp does it ahead of time and the others read the result.
    __device__ __forceinline__ void decode(const Params &p, int i) {
        if (i < 0) {
            n0 = n1 = -1;
            return;
        }
        int st = 0;
        for (int a = p.S - 1; st < a;) {
            const int mid = (st + a + 1) >> 1;
            if (p.item0[mid] <= i) st = mid; else a = mid - 1;
        }
        const int nq = p.nq[st], nsp = p.nsp[st], hg = p.hg[st];
        const int blocks = ceil_div(nq, 2 * p.tpt);
        int x = i - p.item0[st];
        const int per = blocks * nsp * hg, g = x / per;
        x -= g * per;
        const int heads = min(hg, p.Hkv - g * hg);
        const int b = x / (nsp * heads);
        x -= b * nsp * heads;
        const int sp = x / heads, blk = blocks - 1 - b;
        h = g * hg + x - sp * heads;
        tok0 = blk * 2 * p.tpt;
        ntok = min(nq - tok0, 2 * p.tpt);
        qrow = p.qoff[st] + tok0;
        krow = p.koff[st];
        nk = p.nk[st];
        lag = nk - nq;
        pair = ntok > p.tpt;
        c0 = sp * p.chunk[st];
        const int end = c0 + p.chunk[st];
        n0 = max(0, min(end, ceil_div(seen(p, min(ntok, p.tpt)), BN)) - c0);
        if (pair) {
            n1 = max(0, min(end, ceil_div(seen(p, ntok), BN)) - c0);
        } else {
            n1 = n0 / 2;
            n0 -= n1;
        }
        slot = p.slot0[st] < 0 ? -1 : p.slot0[st] + ((h * blocks + blk) * nsp + sp) * 2;
    }
    __device__ __forceinline__ int n(int w) const { return w ? n1 : n0; }
    // Keys that the first `t` tokens of the block see at most.
    __device__ __forceinline__ int seen(const Params &p, int t) const {
        return p.causal ? max(0, min(nk, lag + tok0 + t)) : nk;
    }
    // One past the last key of its tiles.
    __device__ __forceinline__ int stop() const { return (int)min((int64_t)nk, (int64_t)(c0 + (pair ? n1 : n0 + n1)) * BN); }
    // Key tile of warpgroup w's step j.
    __device__ __forceinline__ int key_tile(int w, int j) const { return pair ? c0 + j : c0 + 2 * j + w; }
    // Keys of that tile that any row of warpgroup w's query tile sees, rounded up to the 16 of a product step.
    __device__ __forceinline__ int steps(const Params &p, int w, int kt) const {
        const int t = pair && w == 0 ? p.tpt : ntok;
        return min(BN / 16, ceil_div(seen(p, t) - kt * BN, 16));
    }
};

struct Ctl {
    uint64_t q_full[2], q_free[2];
    uint64_t full[MAX_UNITS], free[MAX_UNITS];     // of the ring's groups
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t ml_full[2], ml_free[2]; // the rows' maxima and sums
    uint64_t o_free[2];              // the sums have been read
    uint64_t ask, answer;            // time to ask for another item (from the TMA warp); the answer has come
    uint64_t item_full[2], item_free[2];
    uint64_t drain;
    alignas(16) uint4 next;          // the answer
    Item item[4];                    // two on their way, and those that outputs are written of
    float2 ml[2][BM];                // (m, l) of each row
    uint32_t tmem;
    int abort, busy;                 // roles gave up; warps that make outputs again
};
constexpr int SMEM = 229376 + (int)((sizeof(Ctl) + 127) / 128 * 128);
static_assert(SMEM <= 232448, "227 KB");

// ---- the next item: a CTA that has not been launched yet is taken over (cluster launch control) ----
__device__ __forceinline__ void ask_next(uint4 *dst, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     ptx::smem_u32(dst)),
                 "r"(ptx::smem_u32(bar))
                 : "memory");
}
// Its index, or -1 when there is none left.
__device__ __forceinline__ int read_next(const uint4 *src) {
    uint64_t a, b;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(ptx::smem_u32(src)) : "memory");
    int r;
    asm volatile(
        "{\n\t.reg .b128 x;\n\t.reg .pred c;\n\t"
        "mov.b128 x, {%1, %2};\n\t"
        "mov.u32 %0, -1;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 c, x;\n\t"
        "@c clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, x;\n\t}"
        : "=r"(r)
        : "l"(a), "l"(b));
    return r;
}

// One lane of a warp that stays together: addresses and coordinates then lie in uniform registers (40 prompts of 300
// rows, 64 heads: 250 us with a branch for lane 0, 240 so).
__device__ __forceinline__ void tma_load_3d_warp(uint32_t dst, const CUtensorMap *tm, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// Half of a value tile: all of its boxes one behind another (the fourth coordinate).
__device__ __forceinline__ void tma_load_4d_warp(uint32_t dst, const CUtensorMap *tm, uint64_t *bar, int c1, int c2) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %3}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(ptx::smem_u32(bar)), "r"(0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void expect_warp(uint64_t *bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(
            ptx::smem_u32(bar)),
        "r"(bytes)
        : "memory");
}

// `n` products of 16 keys: P from TMEM (8 columns a step), V MN-major (two 1 KB groups of 8 keys a step; its halves'
// descriptors are `b` and `b4`).
__device__ __forceinline__ void pv_warp(uint32_t d, uint32_t a, uint64_t b, uint64_t b4, uint32_t idesc, uint32_t acc, int n) {
#pragma unroll 1
    for (int i = 0; i < n; ++i, a += 8, b += 2048 >> 4, acc = 1) {
        if (i == 4) b = b4;
        ptx::mma_bf16_ts_warp(d, a, b, idesc, acc);
    }
}

// All eight of a tile, in one block: the loop issues them at half the pace of the tensor cores.
__device__ __forceinline__ void pv8_warp(uint32_t d, uint32_t a, uint64_t b, uint64_t b4, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b32 a1, a2, a3, a4, a5, a6, a7;\n\t.reg .b64 b1, b2, b3, b5, b6, b7;\n\t"
        "add.u32 a1, %1, 8;\n\t"
        "add.u32 a2, %1, 16;\n\t"
        "add.u32 a3, %1, 24;\n\t"
        "add.u32 a4, %1, 32;\n\t"
        "add.u32 a5, %1, 40;\n\t"
        "add.u32 a6, %1, 48;\n\t"
        "add.u32 a7, %1, 56;\n\t"
        "add.u64 b1, %2, 128;\n\tadd.u64 b5, %3, 128;\n\t"
        "add.u64 b2, %2, 256;\n\tadd.u64 b6, %3, 256;\n\t"
        "add.u64 b3, %2, 384;\n\tadd.u64 b7, %3, 384;\n\t"
        "setp.ne.b32 p, %5, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %4, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %4, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], %3, %4, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %4, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %4, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %4, 1;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "l"(b4), "r"(idesc), "r"(acc)
        : "memory");
}

// One look at a barrier.  Without a time to sleep it costs 38 cycles where the phase is complete, with one 70.
__device__ __forceinline__ bool look(uint64_t *bar, uint32_t parity) {
    uint32_t seen;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(seen)
        : "r"(ptx::smem_u32(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, seen);
}

// Whether a wait that began at t0 is to be given up: past its limit (recorded), or as another role gave up.  Outputs
// that are made again (abort[1] warps at it, which wait for nobody) do not count.
__device__ __forceinline__ bool expired(long long &t0, long long limit, volatile int *abort, DevErr *err, int site) {
    bool stop = *abort != 0;
    if (abort[1] != 0) t0 = clock64();
    if (!stop && clock64() - t0 > limit) {
        ptx::record_error(err, TF_E_TIMEOUT, site);
        *abort = 1;
        stop = true;
    }
    return __any_sync(0xffffffffu, stop);
}

// ptx::mbar_wait_warp without the call to its polling loop: a call would hold the registers around it to
// what the whole kernel was launched with.  Bounded in the same way.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort, DevErr *err, int site,
                                     long long limit = 1ll << 31) {
    if (look(bar, parity)) return true;
    long long t0 = clock64();
    for (uint32_t spins = 1;; ++spins) {
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
        if ((spins & 255u) == 0 && expired(t0, limit, abort, err, site)) return false;
    }
}

// 16 columns of a warp's 32 lanes of TMEM, a lane a thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 32 columns of a warp's 32 lanes of TMEM, a lane a thread, and their largest value (NaN aside).
// The load finds the maximum on its way: 128 comparisons a row less (8,192 rows of 64 heads 64 wide 582 -> 548 us).
__device__ __forceinline__ void tmem_ld32_max(uint32_t taddr, uint32_t (&r)[32], float &top) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=f"(top)
        : "r"(taddr));
}

// 32 bytes at once, 32-byte aligned.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The same without sleeping, for the warp that the tensor cores wait for.
__device__ __forceinline__ bool spin(uint64_t *bar, uint32_t parity, volatile int *abort, DevErr *err, int site) {
    long long t0 = clock64();
    for (uint32_t spins = 1; !look(bar, parity); ++spins)
        if ((spins & 4095u) == 0 && expired(t0, 1ll << 31, abort, err, site)) return false;
    return true;
}

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(const uint32_t &w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }

// The items of this CTA, as the roles that do not find them read them.
struct Walk {
    uint32_t count = 0;
    // The next item; false at the end or after a timeout.
    __device__ __forceinline__ bool next(Ctl &c, const Params &p, Item &x, int lane) {
        const int b = count & 1;
        if (!wait(&c.item_full[b], (count >> 1) & 1, &c.abort, p.err, 50)) return false;
        // through a shuffle, so that the compiler knows the values to be the same in all lanes: loops and descriptors
        // that hang on them then stay in uniform registers (8,192 rows of 64 heads
        // over 8 key heads: 768 us without it, 652 with)
        const int *src = reinterpret_cast<const int *>(&c.item[count & 3]);
        int *dst = reinterpret_cast<int *>(&x);
        const int mine = src[min(lane, (int)(sizeof(Item) / 4) - 1)];
#pragma unroll
        for (int k = 0; k < (int)(sizeof(Item) / 4); ++k) dst[k] = __shfl_sync(0xffffffffu, mine, k);
        if (lane == 0) ptx::mbar_arrive(&c.item_free[b]);
        ++count;
        return x.n0 >= 0;
    }
};

// Two neighbouring bf16 values.
__device__ __forceinline__ uint32_t load2(const uint16_t *at) {
    uint32_t v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(at));
    return v;
}

// ---- outputs made again ----
// P is 0 where the mask hides a key, but 0 times a NaN or an infinity is NaN: a value that is not finite reaches every row of a
// query tile that its key tile is multiplied with.  Rows that do not see it get the columns that it spoilt from here, in
// fp32 from the tensors themselves: a warp a row, eight keys at once, the row's maximum and sum as they are.  `rows`: the
// warp's rows whose outputs hold a NaN; m and l: a row's, a lane each.
// It runs only then, at some 600 cycles a key and row: a NaN in the last value row of 4,096 rows of 64 heads costs 41 ms,
// NaN everywhere 0.9 (a row that sees a NaN among its last keys stays).  Looking for such rows costs outputs 0 to 4%, of some split
// calls up to 8 (40 prompts of 300 rows 220 -> 227 us, 4,096 rows 216 -> 218).  Instead of it, a look by a warp of its own through
// the tiles that the mask cuts, before their use: 254 us; the whole item again after such a look: 264, for the longer code that all
// roles go through.
template <int DQK, int DV>
__device__ __forceinline__ void make_again(const Params &p, const Item &x, int w, int row0, uint32_t rows, float m, float l) {
    constexpr int V = DV / 32;   // a lane's columns
    const int lane = (int)threadIdx.x & 31, from = x.c0 * BN, stop = x.stop();
    const uint16_t *vals = p.mv.p + (int64_t)x.krow * p.mv.row + x.h * p.mv.head + lane * V;
    auto value = [&](int j, uint32_t (&v)[V]) {   // fp32 bits of key j's
        uint32_t u[V / 2];
        if (V == 4) {
            const uint2 two = __ldg(reinterpret_cast<const uint2 *>(vals + j * p.mv.row));
            u[0] = two.x, u[V / 2 - 1] = two.y;
        } else {
            u[0] = __ldg(reinterpret_cast<const uint32_t *>(vals + j * p.mv.row));
        }
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = k & 1 ? u[k / 2] & 0xFFFF0000u : u[k / 2] << 16;
    };
    auto sees = [&](int r, int &tok) {   // keys of these tiles that row r sees, behind the last one
        tok = (row0 + r) / p.G + (x.pair ? w * p.tpt : 0);
        return max(from, min(stop, x.seen(p, tok + 1)));
    };
    __syncwarp();   // the rows' own threads have written them
    // Of each column: the last value that is not finite and the first NaN, from two tiles before the first row's last key on.
    int bad[V], nan[V], tok;
#pragma unroll
    for (int k = 0; k < V; ++k) bad[k] = -1, nan[k] = INT_MAX;
#pragma unroll 4
    for (int j = max(from, sees(__ffs(rows) - 1, tok) - 2 * BN); j < stop; ++j) {
        uint32_t v[V];
        value(j, v);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t size = v[k] & 0x7FFFFFFFu;
            if (size >= 0x7F800000u) bad[k] = j;
            if (size > 0x7F800000u) nan[k] = min(nan[k], j);
        }
    }
#pragma unroll 1
    for (; rows; rows &= rows - 1) {
        const int r = __ffs(rows) - 1, upto = sees(r, tok);
        uint32_t again = 0;   // a bit a column: spoilt by a value that the row does not see, and no NaN before that it sees
#pragma unroll
        for (int k = 0; k < V; ++k) again |= (uint32_t)(bad[k] >= upto && nan[k] >= upto) << k;
        if (!__any_sync(0xffffffffu, again != 0)) continue;
        const float mr = __shfl_sync(0xffffffffu, m, r), lr = __shfl_sync(0xffffffffu, l, r), cl = p.scale_log2;
        const float mc = mr == -INFINITY ? 0.f : mr * cl;
        const int head = x.h * p.G + (row0 + r) % p.G;
        const int64_t token = (int64_t)x.qrow + tok;
        constexpr int B = DQK / BOX;   // a lane has two neighbouring values of each box
        const uint16_t *keys = p.mk.p + (int64_t)x.krow * p.mk.row + x.h * p.mk.head + 2 * lane;
        const uint16_t *last = p.has_kr ? p.mkr.p + (int64_t)x.krow * p.mkr.row + 2 * lane : keys + (B - 1) * BOX;
        const int64_t last_row = p.has_kr ? p.mkr.row : p.mk.row;
        uint32_t q[B];
#pragma unroll
        for (int i = 0; i < B; ++i) q[i] = load2(p.mq.p + token * p.mq.row + head * p.mq.head + i * BOX + 2 * lane);
        float acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        // the keys' loads in flight together, then the values' (asm volatile: they are not moved to their uses)
        constexpr int N = 8;
#pragma unroll 1
        for (int j0 = from; j0 < upto; j0 += N) {
            uint32_t u[N][B];
            float e[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int j = min(j0 + i, upto - 1);
#pragma unroll
                for (int d = 0; d < B; ++d) u[i][d] = load2(d + 1 < B ? keys + j * p.mk.row + d * BOX : last + j * last_row);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                e[i] = 0.f;
#pragma unroll
                for (int d = 0; d < B; ++d) {
                    e[i] = fmaf(__uint_as_float(u[i][d] << 16), __uint_as_float(q[d] << 16), e[i]);
                    e[i] = fmaf(__uint_as_float(u[i][d] & 0xFFFF0000u), __uint_as_float(q[d] & 0xFFFF0000u), e[i]);
                }
            }
            uint32_t v[N][V / 2];
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int k = 0; k < V / 2; ++k) v[i][k] = load2(vals + min(j0 + i, upto - 1) * p.mv.row + 2 * k);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < N; ++i) e[i] += __shfl_xor_sync(0xffffffffu, e[i], o);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = ptx::ex2(fmaf(e[i], cl, -mc));
                if (j0 + i < upto) {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        acc[k] = fmaf(f, __uint_as_float(k & 1 ? v[i][k / 2] & 0xFFFF0000u : v[i][k / 2] << 16), acc[k]);
                }
            }
        }
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (!(again >> k & 1)) continue;
            const int col = lane * V + k;
            if (x.slot >= 0) p.part[(((int64_t)x.slot + w) * BM + row0 + r) * DV + col] = acc[k];
            else p.out[token * p.out_row + head * p.out_head + col] = (uint16_t)ptx::pack_bf16x2(acc[k] * inv, 0.f);
        }
        __syncwarp();
    }
}

template <int DQK, int DV>
__global__ void __launch_bounds__(THREADS, 1) prompt_kernel(const __grid_constant__ Params p) {
    using L = Lay<DQK, DV>;
    extern __shared__ __align__(1024) uint8_t smem[];   // swizzle atoms lie on 1 KB
    Ctl &c = *reinterpret_cast<Ctl *>(smem + L::BYTES);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = (int)threadIdx.x & 31;

    ptx::griddep_launch_dependents();
    if (threadIdx.x == 0) {
        c.abort = c.busy = 0;
        for (int i = 0; i < L::U; ++i) ptx::mbar_init(&c.full[i], 1), ptx::mbar_init(&c.free[i], 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&c.q_full[i], 1);
            ptx::mbar_init(&c.q_free[i], 1);
            ptx::mbar_init(&c.s_full[i], 1);
            ptx::mbar_init(&c.p_full[i], 4);
            ptx::mbar_init(&c.o_full[i], 1);
            ptx::mbar_init(&c.ml_full[i], 4);
            ptx::mbar_init(&c.ml_free[i], 4);
            ptx::mbar_init(&c.o_free[i], 4);
            ptx::mbar_init(&c.item_full[i], 1);
            ptx::mbar_init(&c.item_free[i], 14);
        }
        ptx::mbar_init(&c.ask, 1);
        ptx::mbar_init(&c.answer, 1);
        ptx::mbar_init(&c.drain, 1);
        ptx::fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        ptx::tmem_alloc(&c.tmem, 512);
        ptx::tmem_relinquish();
    }
    if (warp == TMA_WARP && lane == 0) {
        ptx::prefetch_tmap(&p.q);
        ptx::prefetch_tmap(&p.k);
        ptx::prefetch_tmap(&p.v);
        if (p.has_kr) ptx::prefetch_tmap(&p.kr);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
    ptx::griddep_wait();

    if (warp == TMA_WARP) {
        // ================= TMA; it also says when the next item is to be asked for =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        Ring<L::U> head, tail;     // the next group, the oldest that is not known to be free
        int room = L::U;           // free units
        uint32_t keys = 0;         // which groups are key tiles
        uint32_t groups = 0;       // so far, up to U
        int nq[2] = {0, 0};        // uses of each query tile
        const uint32_t ring = ptx::smem_u32(smem + L::OFF_R);
        bool ok = true;
        Walk it;
        Item x;
        while (it.next(c, p, x, lane)) {
            // The next item is asked for shortly before this one's last tiles are copied.  Asked for at an item's start it
            // is taken from an SM that has none yet, or waits behind an item while others end.
            auto ask = [&]() {
                if (p.more && lane == 0) ptx::mbar_arrive(&c.ask);
            };
            // The next group's barrier, once there is room for it.
            auto group = [&](int units, bool is_keys) -> uint64_t * {
                for (; room < units; tail.step(0)) {
                    if (!wait(&c.free[tail.g], tail.phase, &c.abort, p.err, 53)) return nullptr;
                    room += (keys >> tail.g & 1) ? L::KU / L::KG : 2;
                }
                room -= units;
                keys = (keys & ~(1u << head.g)) | (uint32_t)is_keys << head.g;
                if (groups < L::U) ++groups;
                return &c.full[head.g];
            };
            auto load_k = [&](int kt) {
#pragma unroll 1
                for (int i = 0; i < L::KG; ++i) {
                    uint64_t *bar = group(L::KU / L::KG, true);
                    if (!bar) return false;
                    expect_warp(bar, L::K_TILE / L::KG);
                    int u = head.u;
#pragma unroll
                    for (int k = 0; k < L::QB / L::KG; ++k) {
                        const int b = i * (L::QB / L::KG) + k;
                        const bool shared = p.has_kr && b == L::QB - 1;
                        tma_load_3d_warp(ring + u * L::UNIT, shared ? &p.kr : &p.k, bar, shared ? 0 : b * BOX, shared ? 0 : x.h,
                                         x.krow + kt * BN);
                        u = u + L::BU == L::U ? 0 : u + L::BU;
                    }
                    head.step(L::KU / L::KG);
                }
                return true;
            };
            auto load_v = [&](int kt) {
                uint64_t *bar = group(2, false);
                if (!bar) return false;
                expect_warp(bar, 2 * L::UNIT);
                const int u1 = head.u + 1 == L::U ? 0 : head.u + 1;
                tma_load_4d_warp(ring + head.u * L::UNIT, &p.v, bar, x.h, x.krow + kt * BN);
                tma_load_4d_warp(ring + u1 * L::UNIT, &p.v, bar, x.h, x.krow + kt * BN + VH);
                head.step(2);
                return true;
            };
            auto load_q = [&](int w) {
                if (nq[w] > 0 && !wait(&c.q_free[w], (uint32_t)(nq[w] - 1) & 1, &c.abort, p.err, 52)) return false;
                ++nq[w];
                expect_warp(&c.q_full[w], (uint32_t)(L::QB * p.tpt * p.G * 128));
#pragma unroll
                for (int b = 0; b < L::QB; ++b)
                    tma_load_3d_warp(ring - L::OFF_R + w * L::Q_TILE + b * (BM * 128), &p.q, &c.q_full[w], b * BOX, x.h * p.G, x.qrow + w * p.tpt);
                return true;
            };
            if (x.n0 + x.n1 == 0) ask();
            // in the order in which the MMA warp takes them
            if (x.pair) {
                if (x.n1 > 0) ok = load_q(0) && load_k(x.key_tile(1, 0)) && load_q(1);
                for (int j = 0; ok && j < x.n1; ++j) {
                    if (j == max(0, x.n1 - 2)) ask();
                    ok = load_v(x.key_tile(1, j));
                    if (ok && j + 1 < x.n1) ok = load_k(x.key_tile(1, j + 1));
                }
            } else {
                if (x.n0 > 0) ok = load_q(0) && load_k(x.key_tile(0, 0));
                if (ok && x.n1 > 0) ok = load_k(x.key_tile(1, 0));
                for (int j = 0; ok && j < x.n0; ++j) {
                    if (j == max(0, x.n0 - 2)) ask();
                    for (int w = 0; ok && w < 2; ++w) {
                        if (j < x.n(w)) ok = load_v(x.key_tile(w, j));
                        if (ok && j + 1 < x.n(w)) ok = load_k(x.key_tile(w, j + 1));
                    }
                }
            }
            if (!ok) break;
        }
        // no copy may still be on its way into this CTA's shared memory when it ends
        constexpr long long LIMIT = 1ll << 28;
        for (int w = 0; w < 2; ++w)
            if (nq[w] > 0) wait(&c.q_full[w], (uint32_t)(nq[w] - 1) & 1, &c.abort, p.err, 55, LIMIT);
        for (; groups > 0; --groups) {   // from the last one back
            if (head.g == 0) head.phase ^= 1;
            head.g = head.g == 0 ? L::U - 1 : head.g - 1;
            wait(&c.full[head.g], head.phase, &c.abort, p.err, 55, LIMIT);
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        // ================= MMA =================
        // One warp for both warpgroups, first one's values and next keys, then the other's: in that order the tensor cores work
        // for one while the other's softmax runs.  (Two warps, each at its own pace, came to run side by side: both products
        // interleaved, both ended late, both softmaxes together, the tensor cores idle meanwhile.)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        const uint64_t dq = ptx::sdesc_sw128(ptx::smem_u32(smem), 16, 1024);
        const uint64_t dk = ptx::sdesc_sw128(ptx::smem_u32(smem + L::OFF_R), 16, 1024);
        const uint64_t dv = ptx::sdesc_sw128(ptx::smem_u32(smem + L::OFF_R), VH * 128, 1024);
        constexpr uint32_t IQK = ptx::idesc_bf16_f32(BM, BN, false, false);
        constexpr uint32_t IPV = ptx::idesc_bf16_f32(BM, DV, false, true);
        Ring<L::U> r;
        uint32_t np0 = 0, np1 = 0;   // softmax tiles of each warpgroup
        uint32_t no0 = 0, no1 = 0;   // outputs
        uint32_t nq0 = 0, nq1 = 0;   // uses of the query tiles
        bool ok = true;
        Walk it;
        Item x, y;
        Ring<L::U> keys, vals;
        bool early = false, known = false;   // the next item (y) is known, its first scores are made
        // Scores of warpgroup w from the keys at `k`; `last`: the query tile's last product; `look_first`: the keys may
        // still be on their way.  (Loops are not unrolled here: every instruction of this warp is fetched again between items.
        // Unrolled, 4,096 rows in eight prompts took 92 us for 72.)
        auto scores = [&](int w, Ring<L::U> k, bool pair, bool last, bool look_first) {
            ptx::tc_fence_after();
            const uint64_t a = dq + (uint64_t)(((pair ? w : 0) * L::Q_TILE) >> 4);
#pragma unroll 1
            for (int g = 0; g < L::KG; ++g) {
                if (look_first && !spin(&c.full[k.g], k.phase, &c.abort, p.err, 61)) return false;
                int u = k.u;
#pragma unroll
                for (int b = 0; b < L::QB / L::KG; ++b) {
                    const int i = g * (L::QB / L::KG) + b;
                    ptx::mma4_bf16_ss_warp(tmem + w * BN, a + (uint64_t)((i * BM * 128) >> 4), dk + (uint64_t)((u * L::UNIT) >> 4), IQK, i == 0);
                    u = u + L::BU == L::U ? 0 : u + L::BU;
                }
                if (g + 1 == L::KG) ptx::mma_commit_warp(&c.s_full[w]);
                if (w == 1 || !pair) ptx::mma_commit_warp(&c.free[k.g]);
                k.step(L::KU / L::KG);
            }
            if (last) ptx::mma_commit_warp(&c.q_free[pair ? w : 0]);
            return true;
        };
        for (;;) {
            if (!known && !it.next(c, p, y, lane)) break;
            x = y;
            known = false;
            const int n0 = x.n0, n1 = x.n1;
            if (n0 < 0) break;
            if (n0 + n1 == 0) continue;
            const bool pair = x.pair;
            // With two query tiles both warpgroups use a tile's keys, and the first to come takes them from the ring; so with
            // the values.
            auto qk = [&](int w, int j) {
                const bool first = w == 0 || !pair || j >= n0;
                if (first) {
                    keys = r;
                    r.template keys<L>();
                }
                return scores(w, keys, pair, pair ? j + 1 == (w ? n1 : n0) : w == (n1 == n0) && j + 1 == n0, first);
            };
            // Once warpgroup 0 has had its last product, while warpgroup 1 still works: the first scores of the next item,
            // if all that they need is there.  Without them the tensor cores wait through the last softmax.
            auto start_next = [&](int left_j) {
                if (early) return;
                if (!known) {
                    if (!look(&c.item_full[it.count & 1], (it.count >> 1) & 1)) return;
                    it.next(c, p, y, lane);
                    known = true;
                }
                if (y.n0 <= 0 || !look(&c.q_full[0], nq0 & 1)) return;
                Ring<L::U> at = r;     // behind what this item still takes
                if (pair) {
                    for (int j = left_j + 1; j < n1; ++j) {
                        at.template keys<L>();
                        at.step(2);
                    }
                }
                const Ring<L::U> begin = at;
#pragma unroll
                for (int g = 0; g < L::KG; ++g) {
                    if (!look(&c.full[at.g], at.phase)) return;
                    at.step(L::KU / L::KG);
                }
                scores(0, begin, y.pair, y.pair ? y.n0 == 1 : y.n0 == 1 && y.n1 == 0, false);
                early = true;
            };
            // The product of step j's P and values.  `whole`: not the warpgroup's last step, all keys count; `alone`:
            // warpgroup 0 has ended.  (P as a whole: handed over in halves it was taken 400 to 600 cycles late all the same, and
            // this warp's longer code cost 40 prompts of 300 rows 240 us for 218; at length the two are alike.)
            auto pv = [&](int w, int j, auto is_whole, auto is_alone) {
                constexpr bool whole = decltype(is_whole)::value, alone = decltype(is_alone)::value;
                if (w == 0 || !pair || j >= n0) {
                    if (!spin(&c.full[r.g], r.phase, &c.abort, p.err, 63)) return false;
                    vals = r;
                    r.step(2);
                }
                int steps = BN / 16;
                if (!whole) {
                    const int kt = x.key_tile(w, j), tail = x.nk - kt * BN;
                    steps = x.steps(p, w, kt);
                    if (tail < BN && (tail & 15)) {
                        // Rows behind the stream's last key, up to the 16 of a product's step: whatever they hold, 0
                        // times it has to be 0.  (16-byte chunks, whatever their order in a row.)
                        int u = vals.u + (tail >= VH);
                        if (u >= L::U) u -= L::U;
                        const int chunks = (16 - (tail & 15)) * 8;
                        uint8_t *dst = smem + L::OFF_R + u * L::UNIT + (tail & (VH - 1)) * 128;
                        for (int i = lane; i < chunks * L::VB; i += 32)
                            *reinterpret_cast<uint4 *>(dst + i / chunks * (VH * 128) + i % chunks * 16) = make_uint4(0, 0, 0, 0);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                const uint32_t np = w ? np1 : np0, no = w ? no1 : no0;
                if (alone) {
                    long long t0 = clock64();
                    for (uint32_t spins = 1; !look(&c.p_full[w], np & 1); ++spins) {
                        start_next(j);
                        if ((spins & 1023u) == 0 && expired(t0, 1ll << 31, &c.abort, p.err, 62)) return false;
                    }
                } else if (!spin(&c.p_full[w], np & 1, &c.abort, p.err, 62)) {
                    return false;
                }
                // the sums of the item before are read out
                if (j == 0 && no > 0 && !wait(&c.o_free[w], (no - 1) & 1, &c.abort, p.err, 66)) return false;
                ptx::tc_fence_after();
                const uint32_t ts = tmem + w * BN, to = tmem + 2 * BN + w * DV;
                const int u = vals.u + 1 == L::U ? 0 : vals.u + 1;
                const uint64_t b0 = dv + (uint64_t)((vals.u * L::UNIT) >> 4), b1 = dv + (uint64_t)((u * L::UNIT) >> 4);
                if (whole) {
                    pv8_warp(to, ts, b0, b1, IPV, j > 0);
                } else {
                    pv_warp(to, ts, b0, b1, IPV, j > 0, steps);
                }
                if (w == 1 || !pair) ptx::mma_commit_warp(&c.free[vals.g]);
                if (!whole && j + 1 == (w ? n1 : n0)) ptx::mma_commit_warp(&c.o_full[w]);
                if (w) ++np1; else ++np0;
                return true;
            };
            constexpr std::true_type yes{};
            constexpr std::false_type none{};
            if (early) {
                keys = r;
                r.template keys<L>();
                early = false;
            } else {
                ok = wait(&c.q_full[0], nq0 & 1, &c.abort, p.err, 60);
                if (ok && n0 > 0) ok = qk(0, 0);
                if (pair && n0 == 0) ptx::mma_commit_warp(&c.q_free[0]);
            }
            ++nq0;
            if (ok && pair) ok = wait(&c.q_full[1], nq1++ & 1, &c.abort, p.err, 60);
            if (ok && n1 > 0) ok = qk(1, 0);
            // steps that neither warpgroup ends with
            int j = 0;
#pragma unroll 1
            for (; ok && j + 1 < min(n0, n1); ++j)
#pragma unroll 1
                for (int w = 0; ok && w < 2; ++w) ok = pv(w, j, yes, none) && qk(w, j + 1);
            // the rest: warpgroup 0's last steps, then warpgroup 1's
#pragma unroll 1
            for (; ok && j < n0; ++j) {
                ok = pv(0, j, none, none) && (j + 1 == n0 || qk(0, j + 1));
                if (j + 1 == n0) break;
                if (ok && j < n1) ok = pv(1, j, none, none);
            }
#pragma unroll 1
            for (; ok && j < n1; ++j) ok = pv(1, j, none, yes) && (j + 1 == n1 || qk(1, j + 1));
            if (!ok) break;
            no0 += n0 > 0;
            no1 += n1 > 0;
        }
        // no product may still run when TMEM is freed
        ptx::mma_commit_warp(&c.drain);
        wait(&c.drain, 0, &c.abort, p.err, 64, 1ll << 29);
    } else if (warp < OUT_WARP) {
        // ================= softmax: a query row a thread =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        const int w = warp >> 2;
        const int row = (int)threadIdx.x & (BM - 1);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + w * BN + lanes, to = tmem + 2 * BN + w * DV + lanes;
        const float cl = p.scale_log2;
        const int rt = row / p.G;   // the row's token in the tile
        uint32_t ns = 0;
        uint32_t nml = 0;   // items with keys
        bool ok = true;
        Walk it;
        Item x;
        while (it.next(c, p, x, lane)) {
            const int n = x.n(w);
            const int tok = x.tok0 + (x.pair ? w * p.tpt : 0) + rt;
            const bool live = rt < p.tpt && tok < x.tok0 + x.ntok;
            // keys that the row sees; rows of no token take whatever comes, and a warp of them nothing at all
            const int vis = live ? x.seen(p, tok - x.tok0 + 1) : INT_MAX;
            const bool idle = __all_sync(0xffffffffu, !live);
            float m = -INFINITY, l = 0.f;
            for (int j = 0; ok && j < n; ++j, ++ns) {
                const int kt = x.key_tile(w, j);
                const int limit = vis - kt * BN;   // columns of this tile that the row sees
                if (!wait(&c.s_full[w], (uint32_t)ns & 1, &c.abort, p.err, 70)) {
                    ok = false;
                    break;
                }
                if (idle) {
                    if (lane == 0) ptx::mbar_arrive(&c.p_full[w]);
                    continue;
                }
                ptx::tc_fence_after();
                if (__any_sync(0xffffffffu, limit < BN)) {
                    // Hidden columns become -inf where they lie, 16 at a time: a small loop, as it runs once or twice an item
                    // and has to be fetched each time (128 selects in a row on the loaded scores: 2,000 cycles).
#pragma unroll 1
                    for (int k = 0; k < BN; k += 16) {
                        if (__all_sync(0xffffffffu, limit >= k + 16)) continue;
                        uint32_t v[16];
                        tmem_ld16(ts + k, v);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (k + i >= limit) v[i] = 0xFF800000u;
                        __syncwarp();
                        tmem_st16(ts + k, v);
                    }
                    ptx::tmem_st_wait();
                }
                uint32_t s[4][32];
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32_max(ts + 32 * q, s[q], mx[q]);
                ptx::tmem_ld_wait();
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                // the maximum moves only by more than 2^8: P stays far below bf16's largest value
                const bool move = top > m + p.thr || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, move)) {
                    float f = 1.f;
                    if (move) {
                        f = m == -INFINITY ? 0.f : ptx::ex2((m - top) * cl);
                        m = top;
                        l *= f;
                    }
                    __syncwarp();   // loads from TMEM are a whole warp's
                    if (j > 0) {   // O up to the tile before: its products are done, S of this one came after them
#pragma unroll 1
                        for (int q = 0; q < DV; q += 32) {
                            uint32_t o[32];
                            ptx::tmem_ld32(to + q, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            ptx::tmem_st32(to + q, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.f : m * cl;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const uint32_t (&v)[32] = s[q + i / 16];
                        const float2 t = ptx::fma2(make_float2(__uint_as_float(v[2 * i % 32]), __uint_as_float(v[2 * i % 32 + 1])),
                                                   make_float2(cl, cl), make_float2(-mc, -mc));
                        const float2 e = make_float2(ptx::ex2(t.x), ptx::ex2(t.y));
                        sum[i & 1] = ptx::add2(sum[i & 1], e);
                        pk[i] = ptx::pack_bf16x2(e.x, e.y);
                    }
                    ptx::tmem_st32(ts + 16 * q, pk);
                }
                ptx::tmem_st_wait();   // with it what the maximum's move changed in O
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&c.p_full[w]);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (ok && n > 0) {
                if (nml > 0) ok = wait(&c.ml_free[w], (nml - 1) & 1, &c.abort, p.err, 71);
                ++nml;
                c.ml[w][row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&c.ml_full[w]);
            }
            if (!ok) break;
        }
    } else if (warp < MMA_WARP) {
        // ================= outputs: a query row a thread, beside the next item's softmax =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OUT));
        const int row = (int)threadIdx.x & (BM - 1);
        const uint32_t to = tmem + 2 * BN + ((uint32_t)((warp & 3) * 32) << 16);
        const float cl = p.scale_log2;
        const int rt = row / p.G, rh = row - rt * p.G;   // the row's token in the tile, and its head
        uint32_t no0 = 0, no1 = 0;                       // outputs of each warpgroup
        bool ok = true;
        Walk it;
        Item x;
        while (it.next(c, p, x, lane)) {
            const bool join = !x.pair && x.n1 > 0;   // one query tile: the two warpgroups' sums are joined
            // A warpgroup's maxima and sums, and its O after its last product.
            auto ready = [&](int w, float &m, float &l) {
                m = -INFINITY;
                l = 0.f;
                if (x.n(w) == 0) return true;
                const uint32_t k = w ? no1++ : no0++;
                if (!wait(&c.ml_full[w], k & 1, &c.abort, p.err, 72)) return false;
                const float2 t = c.ml[w][row];
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&c.ml_free[w]);
                m = t.x;
                l = t.y;
                if (!wait(&c.o_full[w], k & 1, &c.abort, p.err, 73)) return false;
                ptx::tc_fence_after();
                return true;
            };
#pragma unroll 1
            for (int w = 0; w < (x.pair ? 2 : 1); ++w) {
                float m, l, f0 = 1.f, f1 = 0.f;
                ok = ready(w, m, l);
                if (ok && join) {
                    float m1, l1;
                    ok = ready(1, m1, l1);
                    const float top = fmaxf(m, m1);
                    f0 = m == -INFINITY ? 0.f : ptx::ex2((m - top) * cl);
                    f1 = m1 == -INFINITY ? 0.f : ptx::ex2((m1 - top) * cl);
                    l = l * f0 + l1 * f1;
                    m = top;
                }
                if (!ok) break;
                const int t = rt + (x.pair ? w * p.tpt : 0);   // the row's token in the block
                const bool live = rt < p.tpt && t < x.ntok;
                const int head = x.h * p.G + rh;
                const int64_t orow = (int64_t)x.qrow + t;
                if (x.slot < 0) f0 *= l == 0.f ? 0.f : 1.f / l, f1 *= l == 0.f ? 0.f : 1.f / l;
                uint16_t *out = p.out + orow * p.out_row + head * p.out_head;
                const int64_t slot = (int64_t)x.slot + w;
                float *part = p.part + (slot * BM + row) * DV;
                __nv_bfloat162 nil = __float2bfloat162_rn(0.f);   // sums of products of outputs: NaN where one of them is
#pragma unroll 1
                for (int q = 0; q < DV; q += 16) {
                    uint32_t o[16];
                    __syncwarp();   // after rows that are not live
                    if (x.n(w) > 0) {
                        tmem_ld16(to + w * DV + q, o);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = 0u;
                    }
                    if (join) {
                        uint32_t u[16];
                        tmem_ld16(to + DV + q, u);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(fmaf(__uint_as_float(u[i]), f1, __uint_as_float(o[i])));
                    }
                    if (!live) continue;
                    if (x.slot < 0) {
                        uint32_t v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = ptx::pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
#pragma unroll
                        for (int i = 0; i < 8; i += 2) nil = __hfma2(as_bf16x2(v[i]), as_bf16x2(v[i + 1]), nil);
                        if (p.out32) {
                            store32(out + q, v);
                        } else {
                            *reinterpret_cast<uint4 *>(out + q) = make_uint4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<uint4 *>(out + q + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i += 8) {
                            uint32_t v[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) v[k] = o[i + k];
#pragma unroll
                            for (int k = 0; k < 8; k += 4)   // the upper halves are NaN where the whole is
                                nil = __hfma2(as_bf16x2(__byte_perm(v[k], v[k + 1], 0x7632)), as_bf16x2(__byte_perm(v[k + 2], v[k + 3], 0x7632)), nil);
                            store32(part + q + i, v);
                        }
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane < 2 && (lane == w || join) && x.n(lane) > 0) ptx::mbar_arrive(&c.o_free[lane]);
                if (live) {
                    if (x.slot >= 0)
                        reinterpret_cast<float2 *>(p.part + p.slots * BM * DV)[slot * BM + row] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[orow * p.H + head] = l == 0.f ? -INFINITY : (m * cl + log2f(l)) * 0.69314718055994531f;
                }
                const uint32_t spoilt = __ballot_sync(0xffffffffu, __hisnan(__low2bfloat16(nil)) || __hisnan(__high2bfloat16(nil)));
                if (spoilt && p.causal) {
                    Item y;   // again, so that what only this needs takes no registers of the others
                    const int *src = reinterpret_cast<const int *>(&c.item[(it.count - 1) & 3]);
                    int *dst = reinterpret_cast<int *>(&y);
#pragma unroll
                    for (int k = 0; k < (int)(sizeof(Item) / 4); ++k) dst[k] = *const_cast<const volatile int *>(src + k);
                    if (lane == 0) atomicAdd(&c.busy, 1);
                    make_again<DQK, DV>(p, y, w, (warp & 3) * 32, spoilt, m, l);
                    if (lane == 0) atomicAdd(&c.busy, -1);
                }
            }
            if (!ok) break;
        }
    } else if (warp == ITEM_WARP) {
        // ================= the next item =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        int asked = 0;
        int i = (int)blockIdx.x;
        for (uint32_t count = 0;; ++count) {
            Item x;
            x.decode(p, i);
            if (count >= 2 && !wait(&c.item_free[count & 1], (count / 2 - 1) & 1, &c.abort, p.err, 51)) break;
            if (lane == 0) {
                c.item[count & 3] = x;
                ptx::mbar_arrive(&c.item_full[count & 1]);
            }
            if (i < 0) break;
            i = -1;
            if (!p.more) continue;
            if (!wait(&c.ask, count & 1, &c.abort, p.err, 56)) break;
            if (lane == 0) {
                ptx::fence_proxy_async_smem();   // the answer before has been read
                ptx::mbar_arrive_expect_tx(&c.answer, 16);
                ask_next(&c.next, &c.answer);
            }
            ++asked;
            __syncwarp();
            if (!wait(&c.answer, count & 1, &c.abort, p.err, 57)) break;
            i = __shfl_sync(0xffffffffu, read_next(&c.next), 0);
        }
        // no answer may still be on its way into this CTA's shared memory when it ends
        if (asked > 0) wait(&c.answer, (uint32_t)(asked - 1) & 1, &c.abort, p.err, 55, 1ll << 28);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == MMA_WARP) ptx::tmem_dealloc(tmem, 512);
}

// The splits of one row joined in order: a warp a row, DV / 32 values a lane.
template <int DV>
__global__ void __launch_bounds__(128) prompt_combine_kernel(const __grid_constant__ Params p) {
    ptx::griddep_launch_dependents();
    const int lane = (int)threadIdx.x & 31;
    const int st = (int)blockIdx.y;
    if (p.slot0[st] < 0) return;
    const int64_t i = (int64_t)blockIdx.x * 4 + ((int)threadIdx.x >> 5);   // (token, head), heads inner
    const int nq = p.nq[st], nsp = p.nsp[st];
    if (i >= (int64_t)nq * p.H) return;
    const int tok = (int)(i / p.H), head = (int)(i - (int64_t)tok * p.H);
    const int h = head / p.G, rh = head - h * p.G;
    const int blocks = ceil_div(nq, 2 * p.tpt), blk = tok / (2 * p.tpt), in = tok - blk * 2 * p.tpt;
    const int tile = in / p.tpt, row = (in - tile * p.tpt) * p.G + rh;
    const int64_t slot = (int64_t)p.slot0[st] + (int64_t)(h * blocks + blk) * nsp * 2 + tile;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part + p.slots * BM * DV);
    ptx::griddep_wait();
    float m = -INFINITY;
    for (int s = lane; s < nsp; s += 32) m = fmaxf(m, ml[(slot + 2 * s) * BM + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float cl = p.scale_log2;
    constexpr int V = DV / 32;
    float acc[V], l = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int s = 0; s < nsp; ++s) {
        const float2 t = ml[(slot + 2 * s) * BM + row];
        const float f = t.x == -INFINITY ? 0.f : ptx::ex2((t.x - m) * cl);
        l = fmaf(t.y, f, l);
        const float *src = p.part + ((slot + 2 * s) * BM + row) * DV + lane * V;
        float v[V];
        if (V == 4) {
            const float4 u = *reinterpret_cast<const float4 *>(src);
            v[0] = u.x, v[1] = u.y, v[2 % V] = u.z, v[3 % V] = u.w;
        } else {
            const float2 u = *reinterpret_cast<const float2 *>(src);
            v[0] = u.x, v[1] = u.y;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(v[k], f, acc[k]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t orow = (int64_t)p.qoff[st] + tok;
    uint16_t *out = p.out + orow * p.out_row + head * p.out_head + lane * V;
    if (V == 4) {
        *reinterpret_cast<uint2 *>(out) = make_uint2(ptx::pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                     ptx::pack_bf16x2(acc[2 % V] * inv, acc[3 % V] * inv));
    } else {
        *reinterpret_cast<uint32_t *>(out) = ptx::pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
    if (lane == 0 && p.lse) p.lse[orow * p.H + head] = l == 0.f ? -INFINITY : (m * cl + log2f(l)) * 0.69314718055994531f;
}

// ---- the plan ----
// Fills in what depends on the lengths.  Streams' keys are split where there are fewer items than SMs to
// take them; with `invariant` only where a stream is longer than an item may be, at places that hang on nothing else.
struct Plan {
    int64_t items = 0, slots = 0;
    int splits = 1;
};

static int plan(Params &p, const int64_t *h_nq, const int64_t *h_nk, int S, int H, int Hkv, int dqk, int dv, int causal,
                int sms, bool invariant, Plan *out) {
    const int G = H / Hkv, tpt = BM / G;
    p.H = H;
    p.Hkv = Hkv;
    p.G = G;
    p.tpt = tpt;
    p.causal = causal;
    // streams with rows, the most key tiles first
    struct Str {
        int64_t tiles, blocks;
        int32_t qoff, koff, nq, nk;
    };
    Str e[TF_MAX_STREAMS];
    int n = 0;
    int64_t q = 0, k = 0, most = 1;
    for (int s = 0; s < S; ++s) {
        if (h_nq[s] > 0) {
            const int64_t blocks = (h_nq[s] + 2 * tpt - 1) / (2 * tpt), tiles = (h_nk[s] + BN - 1) / BN;
            e[n++] = {tiles, blocks, (int32_t)q, (int32_t)k, (int32_t)h_nq[s], (int32_t)h_nk[s]};
            most = std::max(most, tiles);
        }
        q += h_nq[s];
        k += h_nk[s];
    }
    std::stable_sort(e, e + n, [](const Str &a, const Str &b) { return a.tiles > b.tiles; });
    // Splits of `chunk` key tiles.  The chunk with the smallest estimate of the time, in key tiles: one wave takes
    // the longest item; more of them the mean load and half of the longest item among the last ones, for what they
    // leave uneven.  An item's start and end count as START tiles, a split's partial sums as PART more, and the
    // launch that joins them as JOIN.
    constexpr int64_t START = 2, PART = 2, JOIN = 3;
    most = std::min<int64_t>(most, LONGEST);
    int64_t chunk = most;
    double best = 1e300, whole = 0;
    for (int64_t c = most; c >= 1 && !invariant; c = c > 16 ? c - c / 8 : c - 1) {
        int64_t cnt = 0, load = 0, longest = 0, tail = 0;
        bool split = false;
        for (int i = n - 1; i >= 0; --i) {
            const int64_t sp = std::max<int64_t>(1, (e[i].tiles + c - 1) / c), each = std::min(e[i].tiles, c) + START + (sp > 1 ? PART : 0);
            if (cnt < sms) tail = std::max(tail, each);
            longest = std::max(longest, each);
            cnt += e[i].blocks * Hkv * sp;
            // a causal prompt's blocks see half of its own keys on average
            const int64_t own = causal ? std::min<int64_t>(e[i].tiles, (e[i].nq + BN - 1) / BN) : 0;
            load += e[i].blocks * Hkv * (2 * e[i].tiles - own) / 2 + e[i].blocks * Hkv * sp * (START + (sp > 1 ? PART : 0));
            split = split || sp > 1;
        }
        const double t = (cnt <= sms ? (double)longest : std::max((double)longest, (double)load / sms + 0.5 * tail)) + (split ? JOIN : 0);
        if (t < best) {
            best = t;
            chunk = c;
        }
        // shorter splits only add work: near the unsplit load there is nothing to gain
        if (c == most) whole = (double)load / sms;
        if (best <= 1.03 * whole || cnt > 32 * (int64_t)sms) break;
    }
    out->items = 0;
    out->slots = 0;
    out->splits = 1;
    for (int i = 0; i < n; ++i) {
        const int64_t sp = std::max<int64_t>(1, (e[i].tiles + chunk - 1) / chunk);
        if (sp > INT16_MAX) return TF_E_UNSUPPORTED;
        const int64_t bytes = std::max<int64_t>(1, (int64_t)e[i].nk * (dqk + dv) * 2);
        p.item0[i] = (int32_t)out->items;
        p.qoff[i] = e[i].qoff;
        p.nq[i] = e[i].nq;
        p.koff[i] = e[i].koff;
        p.nk[i] = e[i].nk;
        p.nsp[i] = (int16_t)sp;
        p.chunk[i] = (int32_t)(sp > 1 ? chunk : std::max<int64_t>(1, e[i].tiles));
        // All heads side by side where their keys and values fit L2 together: the longest blocks of all come first then,
        // and the last items are short.  Else in groups of a like size that take up to 48 MB: a last group of few heads leaves
        // SMs idle behind its longest blocks (16,384 rows of 16 heads: 815 us with groups of 32 MB and a rest,
        // 714 so; 4,096 rows of 64 heads 235 and 209; like groups of 32, 64 and 90 MB: 220, 211 and 215).
        const int64_t fit = std::max<int64_t>(1, (48 << 20) / bytes), groups = bytes * Hkv <= (96 << 20) ? 1 : (Hkv + fit - 1) / fit;
        p.hg[i] = (int16_t)((Hkv + groups - 1) / groups);
        p.slot0[i] = sp > 1 ? (int32_t)out->slots : -1;
        const int64_t cnt = e[i].blocks * Hkv * sp;
        if (sp > 1) out->slots += cnt * 2;
        out->items += cnt;
        out->splits = std::max(out->splits, (int)sp);
        if (out->items > INT32_MAX / 2 || out->slots > INT32_MAX / 2) return TF_E_UNSUPPORTED;
    }
    p.S = n;
    p.slots = out->slots;
    p.more = out->items > sms;
    return TF_OK;
}

static size_t ws_bytes_of(const Plan &pl, int dv) {
    return ((size_t)pl.slots * BM * (dv * 4 + 8) + 255) / 256 * 256;
}

}  // namespace prm

// The current device's SMs, or an upper bound when no device answers.
static int prompt_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return prm::MAX_SMS;
    }
    return std::min(n, prm::MAX_SMS);
}

// The parameter block of this host thread's next launch (a launch copies it).
static prm::Params &prompt_params() {
    thread_local std::unique_ptr<prm::Params> pp;
    if (!pp) pp.reset(new prm::Params());
    return *pp;
}

int prompt_plan(const int64_t *h_nq, const int64_t *h_nk, int S, int H, int Hkv, int dqk, int dv, int causal, int sms,
                tf_prompt_plan *info, size_t *bytes) {
    prm::Plan pl;
    if (sms <= 0) sms = prompt_sms();
    const int rc = prm::plan(prompt_params(), h_nq, h_nk, S, H, Hkv, dqk, dv, causal, std::min(sms, prm::MAX_SMS), false, &pl);
    if (rc != TF_OK) return rc;
    if (info) {
        info->items = pl.items;
        info->slots = pl.slots;
        info->rows = 2 * (prm::BM / (H / Hkv)) * (H / Hkv);
        info->splits = pl.splits;
    }
    if (bytes) *bytes = prm::ws_bytes_of(pl, dv);
    return TF_OK;
}

int launch_prompt_attend(tf_kvpool *pool, const int64_t *h_nq, const int64_t *h_nk, int S, int H, int Hkv, int dqk, int dv,
                         const tf_heads *q, const tf_heads *k, const void *d_kr, int64_t kr_row, const tf_heads *v,
                         float scale, int causal, const tf_heads *out, float *d_lse, void *d_ws, size_t ws_bytes,
                         cudaStream_t st) {
    using namespace prm;
    Params &p = prompt_params();
    Plan pl;
    using Kern = void (*)(const Params);
    const Kern kern = dqk == 192 ? prompt_kernel<192, 128> : dqk == 128 ? prompt_kernel<128, 128> : prompt_kernel<64, 64>;
    static PerDevice<int> ready;   // SMs, once the kernels are opted in to their shared memory
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError(), dev = -1;
    const int *sms = ready.get(dev, [&](int &n) {
        n = prompt_sms();
        bool ok = true;
        for (const Kern f : {prompt_kernel<192, 128>, prompt_kernel<128, 128>, prompt_kernel<64, 64>})
            ok = ok && cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) == cudaSuccess;
        if (!ok) cudaGetLastError();
        return ok;
    });
    const bool invariant = (pool->desc.flags & TF_POOL_BATCH_INVARIANT) != 0;   // never more slots than by default
    const int rc = plan(p, h_nq, h_nk, S, H, Hkv, dqk, dv, causal, sms ? *sms : prompt_sms(), invariant, &pl);
    if (rc != TF_OK) return rc;
    const size_t need = ws_bytes_of(pl, dv);
    if (need > 0 && (!d_ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0))
        return d_ws && ws_bytes < need ? TF_E_NOMEM : TF_E_ARG;
    if (pl.items == 0) return TF_OK;
    if (!sms) return TF_E_CUDA;

    int64_t rows = 0, keys = 0;
    for (int s = 0; s < S; ++s) rows += h_nq[s], keys += h_nk[s];
    auto map = [&](CUtensorMap *tm, const void *d_p, int64_t row, int64_t head, int values, int heads, int64_t n, uint32_t box_h,
                   uint32_t box_n) {
        const uint64_t dims[3] = {(uint64_t)values, (uint64_t)heads, (uint64_t)n};
        // the stride of a single head is never used
        const uint64_t strides[2] = {(uint64_t)(heads > 1 ? head : values) * 2, (uint64_t)row * 2};
        const uint32_t box[3] = {BOX, box_h, box_n};
        return encode_tmap_bf16(tm, const_cast<void *>(d_p), 3, dims, strides, box);
    };
    if (!map(&p.q, q->d_p, q->row, q->head, dqk, H, rows, (uint32_t)p.G, (uint32_t)p.tpt)) return TF_E_CUDA;
    p.has_kr = d_kr != nullptr;
    if (keys > 0) {
        if (!map(&p.k, k->d_p, k->row, k->head, dqk - (d_kr ? 64 : 0), Hkv, keys, 1, BN)) return TF_E_CUDA;
        // the values' boxes of 64 as a dimension of their own
        const uint64_t vdims[4] = {BOX, (uint64_t)Hkv, (uint64_t)keys, (uint64_t)(dv / BOX)};
        const uint64_t vstrides[3] = {(uint64_t)(Hkv > 1 ? v->head : dv) * 2, (uint64_t)v->row * 2, BOX * 2};
        const uint32_t vbox[4] = {BOX, 1, VH, (uint32_t)(dv / BOX)};
        if (!encode_tmap_bf16(&p.v, v->d_p, 4, vdims, vstrides, vbox)) return TF_E_CUDA;
        if (!d_kr) p.kr = p.k;
        else if (!map(&p.kr, d_kr, kr_row, 64, 64, 1, keys, 1, BN)) return TF_E_CUDA;
    } else {
        p.k = p.kr = p.v = p.q;   // nothing is loaded through them
    }
    p.mq = {static_cast<const uint16_t *>(q->d_p), q->row, q->head};
    if (keys > 0) {
        p.mk = {static_cast<const uint16_t *>(k->d_p), k->row, k->head};
        p.mkr = {static_cast<const uint16_t *>(d_kr), kr_row, 0};
        p.mv = {static_cast<const uint16_t *>(v->d_p), v->row, v->head};
    }
    p.out = static_cast<uint16_t *>(out->d_p);
    p.out_row = out->row;
    p.out_head = out->head;
    p.out32 = ((reinterpret_cast<uintptr_t>(out->d_p) | (uintptr_t)out->row * 2 | (H > 1 ? (uintptr_t)out->head * 2 : 0)) & 31) == 0;
    p.lse = d_lse;
    p.part = static_cast<float *>(d_ws);
    p.err = pool->err;
    p.scale_log2 = scale * 1.44269504088896341f;
    p.thr = 8.0f / p.scale_log2;
    if (prepare_launch(pool, st) != TF_OK) return TF_E_CUDA;
    {
        ProfScope prof(pool, kProfAttend, st);
        const cudaError_t e = launch_pdl(kern, dim3((unsigned)pl.items), dim3(THREADS), SMEM, st, p);
        launch_counter()++;
        if (e != cudaSuccess) return TF_E_CUDA;
    }
    if (pl.slots == 0) return TF_OK;
    int64_t most = 0;
    for (int i = 0; i < p.S; ++i)
        if (p.slot0[i] >= 0) most = std::max<int64_t>(most, p.nq[i]);
    ProfScope prof(pool, kProfCombine, st);
    auto *join = dv == 128 ? prompt_combine_kernel<128> : prompt_combine_kernel<64>;
    const cudaError_t e = launch_pdl(join, dim3((unsigned)((most * H + 3) / 4), (unsigned)p.S), dim3(128), 0, st, p);
    launch_counter()++;
    return e == cudaSuccess ? TF_OK : TF_E_CUDA;
}

}  // namespace tf
