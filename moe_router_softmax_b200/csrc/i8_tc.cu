// i8_tc.cu -- int8 x int8 products on the 5th-generation tensor cores
// (tcgen05.mma kind::i8: int8 codes from shared memory, int32 sums in TMEM).
//
// The same two products as i8_gemv.cu for more than a few tokens: the dense
// product (moe_linear_int8) and the two grouped products of the FFN with int8
// activations.  Both operands are codes, so TMA puts them into shared memory in
// the 128-byte-swizzled K-major layout that the MMA reads and nothing touches
// them on the way; scales are applied to the sums.
//
// The weight rows are the M = 128 operand, the tokens (an expert's routes) N, up
// to 256 per block:
//   linear   D[128 x N] = Wq[m0..m0+127] . Xq^T        y[t][m] = D sx[t] sw[m]
//   phase 1  D rows: 16 gate rows of W13, their 16 up rows, the next 16 gate rows,
//            ...: a gate row and its up row are 16 lanes apart in one TMEM
//            quadrant, so an epilogue warp pairs them with one shuffle per two columns
//            (one half of the lanes finishes the even column, the other the odd one)
//            h[s][i] = gelu_tanh(g) * u  (fp32)
//   phase 2  as linear, per expert, over the codes of h; rows[s][m] = D sh[s] s2[m]
//
// The dense product runs on CTA pairs (tcgen05 cta_group::2) where its tiles fill the
// GPU: M = 256, each CTA holding 128 of the weight rows and half of the tokens, so that
// a stage brings 32 KB into an SM instead of 48 and six fit instead of four.  The loads of both
// CTAs report to the leader's barriers, its MMA warp issues for both, and its
// commits free the slots of both.
//
// Measured on B200 (device time): linear 4096 x 8192 x 2816 in 65 us, 2.92 POP/s (one
// CTA per tile: 79; bound by the tensor pipe and power); FFN of 64 tokens (128 experts,
// hidden 2816, intermediate 704, top-8; 107 experts with routes), combine included, 115 us, 5.5 TB/s of those
// experts' weights; of 2047 tokens 283 us.  Pairs gained the phases nothing (287 to 304 us).
//
// Persistent CTAs, one per SM; warp 0 TMA producer of the weights, warp 1 TMEM
// allocation and the MMA issuer, warps 2..9 epilogue (TMEM -> registers ->
// global; warp w reads lanes 32 (w % 4) ..), warp 10 TMA producer of the tokens.
// Two rings of stages of K, one of weight tiles and one of token blocks, whose slots
// share the CTA's memory by the launch's largest block: the weights come from HBM and
// want many bytes in flight, the tokens from L2.  Two accumulators of
// 256 columns, so that an item's epilogue overlaps the next item's products.  Every
// wait is bounded: on a timeout the kernel records it and every role drains out.
#include <cuda_bf16.h>

#include <algorithm>

#include "i8_math.cuh"
#include "ops.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kM = 128;                        // weight rows per tile
constexpr int kKB = 128;                       // codes of K per swizzle row (an atom of a stage)
constexpr int kNMax = 256;                     // tokens per block
constexpr uint32_t kABytes = kM * kKB;         // 16 KB: an atom of a weight stage
constexpr int kRing = 198 * 1024;
constexpr int kMaxStages = 12;                 // of either ring
constexpr int kEpiWarps = 8;                   // two per TMEM quadrant
constexpr int kWarpB = 2 + kEpiWarps;
constexpr int kThreads = 32 * (kWarpB + 1);
constexpr int kTmemCols = 512;

enum { kLinear = 0, kLinearF32 = 1, kPhase1 = 2, kPhase2 = 3 };

// First problem a kernel of this file recorded (0 = none), read and cleared by
// moe_take_device_errors(): 0x1000 | warp for a wait that gave up, 0x2006 a slot
// past the pool, 0x2008 a route block out of range, 0x2009 a route out of range.
__device__ unsigned int g_i8tc_error;
__device__ unsigned int g_i8tc_error_info;
__device__ __forceinline__ void record_error(unsigned code, unsigned info) {
    if (atomicCAS(&g_i8tc_error, 0u, code) == 0u) g_i8tc_error_info = info;
}
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    return mbar_wait_bounded(bar, parity, abort_flag, [=] {
        record_error(0x1000u | (threadIdx.x >> 5), (unsigned)((smem_u32(bar) << 1) | (parity & 1)));
    });
}

struct TcI8Params {
    LayerView L;                     // phases
    const int32_t *counts, *offsets; // phases
    int E;                           // 1 for linear
    int R;                           // token rows
    int K, M;                        // length of the products; output rows: N, I (phase 1) or H
    const float *brow;               // scale per token row
    const float *wscale;             // linear: scale per output row
    void *out;                       // y, h or rows
};

// Called by a whole warp; one lane issues.  CG = 2: for the CTA pair (its leader's
// warp), M = 256, each CTA holding its half of both operands and of the sums.
template <int CG>
__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// One arrival on `bar` when the products issued so far are done; CG = 2: on that
// barrier of both CTAs.
template <int CG>
__device__ __forceinline__ void tc_commit_warp(uint64_t *bar) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
            ::"r"(smem_u32(bar)), "h"((uint16_t)3)
            : "memory");
}
// Address of the pair leader's copy of a shared variable.
__device__ __forceinline__ uint32_t leader_u32(const void *p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
// Arrival of an epilogue warp on the leader's barrier.  What it orders are TMEM reads
// (tcgen05.fence); a release at cluster scope would wait for the warp's global
// stores as well, a microsecond an item.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// TMA boxes into this CTA's shared memory; the barrier `bar` (an address) is its
// own or, CG = 2, the pair leader's.
template <int CG>
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y, uint64_t pol) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "l"(pol)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "l"(pol)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void load_3d(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z,
                                        uint64_t pol) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5}], [%2], %6;"
            ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(pol)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%3, %4, %5}], [%2], %6;"
            ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(pol)
            : "memory");
}
// {x, row, 16-row block, gate or up, blob} box of W13.
__device__ __forceinline__ void load_5d(void *dst, const CUtensorMap *map, uint32_t bar, int x, int b, int z,
                                        uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %4, %6}], [%2], %7;"
        ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(0), "r"(b), "r"(z), "l"(pol)
        : "memory");
}

struct Items {
    int n_act, total, b_rows, a_slots, b_slots;  // b_rows: of a CTA's token slot
};

// Slots of the two rings for token blocks of `rows` rows and stages of ATOMS atoms
// of K.  Every role waits and signals once a stage, while an
// SM's share of HBM brings a weight atom in ~700 cycles.  So the phases take two atoms
// at a time where experts hold few routes (FFN of 64 tokens 120 -> 116 us); with many,
// two atoms were slower (2047 tokens: 315 us, one 296), as they leave fewer stages in
// flight, and three token slots leave the weights the rest of the memory.  The dense
// product's operands both come from L2 and get the same number of slots.
template <int MODE, int ATOMS, int CG>
__device__ __forceinline__ void split_ring(int rows, Items *it) {
    rows /= CG;  // a CTA of a pair holds half of the token rows
    const int a = ATOMS * (int)kABytes, b = ATOMS * rows * kKB, even = min(kMaxStages, kRing / (a + b));
    it->b_rows = rows;
    it->b_slots = MODE < kPhase1 || rows <= 64 ? even : 4 - ATOMS;
    it->a_slots = MODE < kPhase1 ? even : min(kMaxStages, (kRing - it->b_slots * b) / a);
}
constexpr int kFewRoutes = 32;  // two atoms a stage up to so many routes per expert on average

// Blocks of an expert's n routes: as few as kNMax allows, of even size, a
// multiple of 16 (the MMA's N; of 32 for a CTA pair).
__host__ __device__ __forceinline__ int blocks_of(int n) { return (n + kNMax - 1) / kNMax; }
template <int CG>
__host__ __device__ __forceinline__ int block_rows(int n) {
    const int nb = blocks_of(n), step = 16 * CG;
    return ((n + nb - 1) / nb + step - 1) / step * step;
}

// Up to 32 columns of one output row, `stride` values apart (whole chunks without
// a check per column).
__device__ __forceinline__ void put(float *o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *o, float v) { *o = __float2bfloat16_rn(v); }
template <class T>
__device__ __forceinline__ void store_cols(T *o, int stride, const float v[32], int n) {
    if (n >= 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) put(o + (size_t)j * stride, v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < n) put(o + (size_t)j * stride, v[j]);
    }
}

struct ItemInfo {
    int e, row0, n, n_mma, mt, z;
    bool pool;
};

// Boxes of the token rows: dense, the block of the launch; phases, 16 << i rows.
struct TokenMaps {
    CUtensorMap m[4];
};

template <int MODE, int ATOMS, int CG>
__global__ void __launch_bounds__(kThreads, 1)
k_i8_tc(const __grid_constant__ CUtensorMap map_home, const __grid_constant__ CUtensorMap map_pool,
        const __grid_constant__ TokenMaps map_b, const TcI8Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ int s_base[kMaxE + 1];     // first item of each active expert
    __shared__ int s_row0[kMaxE];
    __shared__ int s_cnt[kMaxE];          // routes of each expert, then of each active expert
    __shared__ uint16_t s_blk[kMaxE];     // rows of its blocks
    __shared__ uint16_t s_act[kMaxE];
    __shared__ Items s_items;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ uint64_t a_full[kMaxStages], a_empty[kMaxStages], b_full[kMaxStages], b_empty[kMaxStages];
    __shared__ uint64_t tfull[2], tempty[2];
    __shared__ __align__(16) float s_scale[kEpiWarps][kNMax];  // scales of the item's token rows, a copy per epilogue warp

    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A CTA's tile: 128 rows of the weights (64 columns of h in phase 1).  A pair takes
    // two neighbouring ones; rank: which of them (the leader's is 0).  (The item loops
    // read blockIdx and gridDim themselves: from variables they ran 4% slower.)
    constexpr int kRows = MODE == kPhase1 ? 64 : kM;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;
    const int m_tiles = (p.M + CG * kRows - 1) / (CG * kRows);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&a_full[i], MODE < kPhase1 ? 2 : 1);  // dense: both producers
            mbar_init(&a_empty[i], 1);
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], CG * kEpiWarps);
        }
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        if (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    // dense: one expert that holds every token.  phases: the experts with routes
    if (MODE >= kPhase1) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) s_cnt[e] = __ldg(p.counts + e);
        __syncthreads();
    }
    if (warp == 0) {
        int n_act = 0, run = 0, rows = 16 * CG;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.E ? (MODE < kPhase1 ? p.R : s_cnt[e]) : 0;
            const int off = MODE < kPhase1 || e >= p.E ? 0 : __ldg(p.offsets + e);
            __syncwarp();  // every lane has read its count before any is written in place
            const bool act = n > 0;
            const unsigned m = __ballot_sync(kAll, act);
            const int items = act ? m_tiles * blocks_of(n) : 0;
            if (act) rows = max(rows, block_rows<CG>(n));
            int inc = items;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kAll, inc, o);
                if (lane >= o) inc += v;
            }
            if (act) {
                const int pos = n_act + __popc(m & ((1u << lane) - 1u));
                s_act[pos] = (uint16_t)e;
                s_cnt[pos] = n;
                s_blk[pos] = (uint16_t)block_rows<CG>(n);
                s_row0[pos] = off;
                s_base[pos] = run + inc - items;
            }
            run += __shfl_sync(kAll, inc, 31);
            n_act += __popc(m);
        }
        rows = (int)__reduce_max_sync(kAll, (unsigned)rows);
        if (lane == 0) {
            s_base[n_act] = run;
            s_items.n_act = n_act;
            s_items.total = run;
            split_ring<MODE, ATOMS, CG>(rows, &s_items);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();  // the other CTA's barriers are set up
    tc_fence_after();
    // The next launch may take over SMs as this grid's CTAs finish.  The dense product
    // waits for the launch before it first: a later one that reads its own weights ahead
    // of its wait (the FFN's second phases do) may rely on all that came before this.
    if (MODE < kPhase1) pdl_wait();
    pdl_launch_dependents();
    const uint32_t tmem = s_tmem;
    const int total = s_items.total, n_act = s_items.n_act;
    const int SA = s_items.a_slots, SB = s_items.b_slots;
    const int n_atoms = (p.K + kKB - 1) / kKB, nk = (n_atoms + ATOMS - 1) / ATOMS;
    auto atoms_at = [&](int kk) { return min(ATOMS, n_atoms - kk * ATOMS); };
    const uint32_t b_atom = (uint32_t)s_items.b_rows * kKB, b_bytes = ATOMS * b_atom, a_bytes = ATOMS * kABytes;
    uint8_t *ringb = ring + SA * a_bytes;
    // The dense product's rings go round together (both operands come from L2): one
    // pair of barriers, so one wait and one commit a stage (5% at 4096x8192x2816)
    uint64_t *bf = MODE < kPhase1 ? a_full : b_full, *be = MODE < kPhase1 ? a_empty : b_empty;

    // Item -> (active expert, block of its routes, M tile), M tiles fastest.  A role
    // takes its items in order, so the search goes on from the last one's expert.
    int cur = 0;
    auto decode = [&](int item) {
        while (cur + 1 < n_act && s_base[cur + 1] <= item) ++cur;
        ItemInfo r;
        r.mt = item - s_base[cur];
        const int blk = s_blk[cur];
        int first = 0;
        for (; r.mt >= m_tiles; r.mt -= m_tiles) first += blk;
        r.e = s_act[cur];
        r.row0 = s_row0[cur] + first;
        r.n = min(blk, s_cnt[cur] - first);
        r.n_mma = (max(r.n, 1) + 16 * CG - 1) & ~(16 * CG - 1);
        r.z = 0;
        r.pool = false;
        if (MODE >= kPhase1) {
            bool bad;
            const int slot = expert_slot(p.L, r.e, &bad);
            r.pool = slot >= 0;
            r.z = slot >= 0 ? slot : r.e;
            if (bad) record_error(0x2006u, (unsigned)__ldg(p.L.slot_table + r.e));
            if (r.row0 < 0 || r.n < 0 || r.row0 > p.R - r.n) {
                record_error(0x2008u, (unsigned)item);
                bad = true;
            }
            if (bad) {  // nothing is written for it; its weights are read from home
                r.n = 0;
                r.n_mma = 16 * CG;
                r.row0 = 0;
            }
        }
        return r;
    };

    if (warp == 0) {
        // -------------------------------------------------- weights
        if (lane == 0) {
            // (the phases' launches follow this library's own, gather and codes of h,
            // which have waited for all before them and write no weights)
            const uint64_t pol = MODE < kPhase1 ? l2_policy_normal() : l2_policy_first();
            int st = 0;
            uint32_t ph = 0;
            for (int item = blockIdx.x / CG; item < total && !s_abort; item += gridDim.x / CG) {
                const ItemInfo it = decode(item);
                const CUtensorMap *ma = it.pool ? &map_pool : &map_home;
                bool ok = true;
                for (int kk = 0; kk < nk; ++kk) {
                    if (!mbar_wait(&a_empty[st], ph ^ 1, &s_abort)) { ok = false; break; }
                    const int na = atoms_at(kk);
                    const uint32_t bar = CG == 2 ? leader_u32(&a_full[st]) : smem_u32(&a_full[st]);
                    // a pair's leader expects the bytes of both CTAs
                    if (rank == 0) mbar_arrive_expect_tx(&a_full[st], CG * na * kABytes);
                    for (int a = 0; a < na; ++a) {
                        uint8_t *dst = ring + st * a_bytes + a * kABytes;
                        const int x = (kk * ATOMS + a) * kKB;
                        if (MODE == kPhase1) {
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                load_5d(dst + b * (kABytes / 4), ma, bar, x, it.mt * 4 + b, it.z, pol);
                        } else {
                            load_3d<CG>(dst, ma, bar, x, (it.mt * CG + rank) * kM, it.z, pol);
                        }
                    }
                    if (++st == SA) { st = 0; ph ^= 1; }
                }
                if (!ok) break;
            }
        }
    } else if (warp == kWarpB) {
        // -------------------------------------------------- tokens
        if (lane == 0) {
            pdl_wait();
            const uint64_t pol = MODE < kPhase1 ? l2_policy_normal() : l2_policy_last();
            int st = 0;
            uint32_t ph = 0;
            for (int item = blockIdx.x / CG; item < total && !s_abort; item += gridDim.x / CG) {
                const ItemInfo it = decode(item);
                // dense: the CTA's part of the block in one box (rows past the last token read
                // as zeros); phases: boxes of 128, 64, 32 and 16 rows
                const int rows = MODE < kPhase1 ? s_items.b_rows : it.n_mma / CG;
                const int y = it.row0 + rank * (it.n_mma / CG);
                bool ok = true;
                for (int kk = 0; kk < nk; ++kk) {
                    if (!mbar_wait(&be[st], ph ^ 1, &s_abort)) { ok = false; break; }
                    const int na = atoms_at(kk);
                    const uint32_t bar = CG == 2 ? leader_u32(&bf[st]) : smem_u32(&bf[st]);
                    if (rank == 0) mbar_arrive_expect_tx(&bf[st], (uint32_t)(CG * na * rows * kKB));
                    for (int a = 0; a < na; ++a) {
                        uint8_t *dst = ringb + st * b_bytes + a * b_atom;
                        const int x = (kk * ATOMS + a) * kKB;
                        if (MODE < kPhase1) {
                            load_2d<CG>(dst, &map_b.m[0], bar, x, y, pol);
                        } else {
                            int j = 0;
                            for (; j + 128 <= rows; j += 128)
                                load_2d<CG>(dst + j * kKB, &map_b.m[3], bar, x, y + j, pol);
#pragma unroll
                            for (int i = 2; i >= 0; --i)
                                if (rows & (16 << i)) {
                                    load_2d<CG>(dst + j * kKB, &map_b.m[i], bar, x, y + j, pol);
                                    j += 16 << i;
                                }
                        }
                    }
                    if (++st == SB) { st = 0; ph ^= 1; }
                }
                if (!ok) break;
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------- MMA issuer (the pair's leader)
        // The whole warp walks the stages and an elected lane issues, so that the
        // descriptors stay in uniform registers.  A wait on a completed phase costs
        // ~130 cycles: the next stage's is tested before this one's products are issued.
        // (After an abort the waits fail and end the role, for all lanes alike; a look at the
        // flag of each lane's own might part them.  The epilogue's likewise.)
        int sa = 0, sb = 0, acc = 0;
        uint32_t pa = 0, pb = 0, aph = 0;
        bool ra = false, rb = false;
        const uint64_t desc_a = sw128_desc(smem_u32(ring)), desc_b = sw128_desc(smem_u32(ringb));
        for (int item = blockIdx.x / CG; rank == 0 && item < total; item += gridDim.x / CG) {
            const ItemInfo it = decode(item);
            if (!__all_sync(kAll, mbar_wait(&tempty[acc], aph ^ 1, &s_abort))) break;
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(acc * kNMax);
            // int32 sums, both operands signed 8-bit, N and M of the tile
            const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(it.n_mma >> 3) << 17) |
                                   ((uint32_t)((CG * kM) >> 4) << 24);
            bool ok = true;
            for (int kk = 0; kk < nk; ++kk) {
                if (!__all_sync(kAll, ra) && !__all_sync(kAll, mbar_wait(&a_full[sa], pa, &s_abort))) { ok = false; break; }
                if (MODE >= kPhase1 && !__all_sync(kAll, rb) &&
                    !__all_sync(kAll, mbar_wait(&b_full[sb], pb, &s_abort))) { ok = false; break; }
                tc_fence_after();
                const uint64_t ad = desc_a + (uint64_t)(sa * (a_bytes >> 4));
                const uint64_t bd = desc_b + (uint64_t)(sb * (b_bytes >> 4));
                uint64_t *done_a = &a_empty[sa], *done_b = &b_empty[sb];
                if (++sa == SA) { sa = 0; pa ^= 1; }
                if (++sb == SB) { sb = 0; pb ^= 1; }
                ra = mbar_test_wait(&a_full[sa], pa);
                if (MODE >= kPhase1) rb = mbar_test_wait(&b_full[sb], pb);
                // 32 codes of K per MMA: 32 bytes, 2 in the descriptor's address field.
                // The four of a whole atom are unrolled: 128 cycles each at N = 256 (the
                // tensor pipe's), where a counted loop took 144 to issue one
                const int na = atoms_at(kk);
                for (int a = 0; a < na; ++a) {
                    const uint64_t ada = ad + (uint64_t)(a * (kABytes >> 4)), bda = bd + (uint64_t)(a * (b_atom >> 4));
                    const int left = p.K - (kk * ATOMS + a) * kKB;
                    if (left >= kKB) {
#pragma unroll
                        for (int j = 0; j < kKB / 32; ++j)
                            tc_mma_i8<CG>(d, ada + (uint64_t)(2 * j), bda + (uint64_t)(2 * j), idesc, (kk | a | j) != 0);
                    } else {
                        const int steps = (left + 31) / 32;  // past K both operands hold zeros
                        for (int j = 0; j < steps; ++j)
                            tc_mma_i8<CG>(d, ada + (uint64_t)(2 * j), bda + (uint64_t)(2 * j), idesc, (kk | a | j) != 0);
                    }
                }
                tc_commit_warp<CG>(done_a);
                if (MODE >= kPhase1) tc_commit_warp<CG>(done_b);
            }
            if (!ok) break;
            tc_commit_warp<CG>(&tfull[acc]);
            acc ^= 1;
            aph ^= acc == 0;
        }
    } else {
        // -------------------------------------------------- epilogue
        const int q = warp & 3;         // TMEM lane quadrant
        const int eh = (warp - 2) >> 2;  // which of its two warps: they take every other 32 columns
        const int half = lane >> 4;
        int acc = 0;
        uint32_t aph = 0;
        const uint64_t h_pol = l2_policy_last();  // the next launch reads h
        pdl_wait();  // the token rows' scales come from the launch before
        for (int item = blockIdx.x / CG; item < total; item += gridDim.x / CG) {
            const ItemInfo it = decode(item);
            // output row of this thread, and its scale(s)
            const int m = (it.mt * CG + rank) * kRows + (MODE == kPhase1 ? q * 16 + (lane & 15) : q * 32 + lane);
            float sw = 0.0f, su = 0.0f;
            if (MODE < kPhase1) {
                if (m < p.M) sw = __ldg(p.wscale + m);
            } else {
                const uint8_t *blob = expert_blob(p.L, it.e);
                if (blob != nullptr) {
                    const float *sc =
                        reinterpret_cast<const float *>(blob + (MODE == kPhase1 ? p.L.off.s13 : p.L.off.s2));
                    if (m < p.M) sw = __ldg(sc + m);
                    if (MODE == kPhase1) su = __ldg(sc + p.M + m);
                }
            }
            float *sb = s_scale[warp - 2];
            for (int c = lane; c < kNMax; c += 32)
                if (c < it.n_mma) sb[c] = c < it.n ? __ldg(p.brow + it.row0 + c) : 0.0f;
            __syncwarp();
            if (!__all_sync(kAll, mbar_wait(&tfull[acc], aph, &s_abort))) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kNMax);
            for (int c0 = 32 * eh; c0 < it.n; c0 += 64) {
                int raw[32];
                tmem_ld32(taddr + (uint32_t)c0, raw);
                if (MODE == kPhase1) {
                    // even columns to the gates' lanes, odd columns to the ups'
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int own = half ? raw[2 * j + 1] : raw[2 * j];
                        const int oth = __shfl_xor_sync(kAll, half ? raw[2 * j] : raw[2 * j + 1], 16);
                        const float2 s2 = *reinterpret_cast<const float2 *>(sb + c0 + 2 * j);
                        v[j] = gate_up(half ? oth : own, half ? own : oth, half ? s2.y : s2.x, sw, su);
                    }
                    float *o = static_cast<float *>(p.out) + (size_t)(it.row0 + c0 + half) * p.M + m;
                    if (c0 + 32 <= it.n) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) st_f32_hint(o + (size_t)(2 * j) * p.M, v[j], h_pol);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c0 + half + 2 * j < it.n) st_f32_hint(o + (size_t)(2 * j) * p.M, v[j], h_pol);
                    }
                } else {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 s4 = *reinterpret_cast<const float4 *>(sb + c0 + j);
                        v[j] = scaled(raw[j], s4.x, sw);
                        v[j + 1] = scaled(raw[j + 1], s4.y, sw);
                        v[j + 2] = scaled(raw[j + 2], s4.z, sw);
                        v[j + 3] = scaled(raw[j + 3], s4.w, sw);
                    }
                    const size_t at = (size_t)(it.row0 + c0) * p.M + m;
                    if (m < p.M) {  // not a row past the matrix
                        if (MODE == kLinear) store_cols(static_cast<__nv_bfloat16 *>(p.out) + at, p.M, v, it.n - c0);
                        else store_cols(static_cast<float *>(p.out) + at, p.M, v, it.n - c0);
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) mbar_arrive_cluster(leader_u32(&tempty[acc]));
                else mbar_arrive(&tempty[acc]);
            }
            acc ^= 1;
            aph ^= acc == 0;
        }
    }

    if (s_abort) {
        // copies and products still in flight end long before this (2 ms)
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000ll) {}
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();  // neither CTA leaves while the other may still signal it
    if (warp == 1) {
        tc_fence_after();
        if (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ------------------------------------------------- dense product, split over K
// A small batch has too few tiles to fill the GPU (2816 output rows: 22), and one SM
// brings in a 360 KB weight tile in about 8 us.  Here a cluster of S CTAs takes a tile,
// each a share of K: after its products a CTA puts its int32 sums into its own shared
// memory (the ring is free by then), and CTA r adds up columns r, r + S, ... over the
// cluster through distributed shared memory, scales and stores them.  The sums are
// integers, so the split changes no bit.  One tile per cluster; warp 0 TMA producer,
// warp 1 TMEM and MMA issuer, warps 4..7 TMEM -> shared memory, all eight the sums.
constexpr int kSplitThreads = 256;
constexpr int kSplitStages = 8;
constexpr int kSplitTokens = 128;
struct SplitParams {
    const float *sx, *sw;
    int T, N, K, blk, m_tiles, stages;
    void *y;
};

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <int S, bool FP32>
__global__ void __launch_bounds__(kSplitThreads, 1)
k_i8_split(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const SplitParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t full[kSplitStages], empty[kSplitStages], tfull;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % S), tile = (int)(blockIdx.x / S);
    const int mt = tile % p.m_tiles, row0 = tile / p.m_tiles * p.blk;
    const int n = min(p.blk, p.T - row0), n_mma = (n + 15) & ~15;
    const int atoms = (p.K + kKB - 1) / kKB, a0 = atoms * rank / S, a1 = atoms * (rank + 1) / S;
    const uint32_t stage_bytes = kABytes + (uint32_t)(p.blk * kKB);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSplitStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&tfull, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(kNMax)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();  // operands and scales may come from the launch before
    pdl_launch_dependents();
    const uint32_t tmem = s_tmem;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = l2_policy_normal();
            int st = 0;
            uint32_t ph = 0;
            for (int a = a0; a < a1; ++a) {
                if (!mbar_wait(&empty[st], ph ^ 1, &s_abort)) break;
                mbar_arrive_expect_tx(&full[st], stage_bytes);
                uint8_t *dst = ring + st * stage_bytes;
                load_3d<1>(dst, &map_a, smem_u32(&full[st]), a * kKB, mt * kM, 0, pol);
                load_2d<1>(dst + kABytes, &map_b, smem_u32(&full[st]), a * kKB, row0, pol);
                if (++st == p.stages) { st = 0; ph ^= 1; }
            }
        }
    } else if (warp == 1) {
        int st = 0;
        uint32_t ph = 0;
        const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n_mma >> 3) << 17) |
                               ((uint32_t)(kM >> 4) << 24);
        const uint64_t desc0 = sw128_desc(smem_u32(ring));
        bool ok = true;
        for (int a = a0; a < a1 && ok; ++a) {
            ok = __all_sync(kAll, mbar_wait(&full[st], ph, &s_abort));
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = desc0 + (uint64_t)((st * stage_bytes) >> 4), bd = ad + (kABytes >> 4);
            if ((a + 1) * kKB <= p.K) {
#pragma unroll
                for (int j = 0; j < kKB / 32; ++j)
                    tc_mma_i8<1>(tmem, ad + (uint64_t)(2 * j), bd + (uint64_t)(2 * j), idesc, a != a0 || j != 0);
            } else {
                const int steps = (p.K - a * kKB + 31) / 32;  // past K both operands hold zeros
                for (int j = 0; j < steps; ++j)
                    tc_mma_i8<1>(tmem, ad + (uint64_t)(2 * j), bd + (uint64_t)(2 * j), idesc, a != a0 || j != 0);
            }
            tc_commit_warp<1>(&empty[st]);
            if (++st == p.stages) { st = 0; ph ^= 1; }
        }
        if (ok) tc_commit_warp<1>(&tfull);
    } else if (warp >= 4) {
        const int q = warp & 3;
        int *part = reinterpret_cast<int *>(ring) + q * 32 + lane;  // [column][128 rows]
        if (__all_sync(kAll, mbar_wait(&tfull, 0, &s_abort))) {
            tc_fence_after();
            for (int c0 = 0; c0 < n; c0 += 32) {
                int v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c0 + j < n) part[(c0 + j) * kM] = v[j];
            }
        }
    }
    if (s_abort) {
        // copies and products still in flight end long before this (2 ms)
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000ll) {}
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // every CTA's sums are in its shared memory
    {
        const int row = threadIdx.x & (kM - 1), m = mt * kM + row;
        uint32_t base[S];
#pragma unroll
        for (int i = 0; i < S; ++i)
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base[i]) : "r"(smem_u32(ring) + 4 * row), "r"(i));
        const float sw = m < p.N ? __ldg(p.sw + m) : 0.0f;
        for (int c = rank + S * (threadIdx.x / kM); c < n && m < p.N; c += S * (kSplitThreads / kM)) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < S; ++i) sum += ld_cluster_s32(base[i] + (uint32_t)(c * kM * 4));
            const float v = scaled(sum, __ldg(p.sx + row0 + c), sw);
            const size_t at = (size_t)(row0 + c) * p.N + m;
            if (FP32) static_cast<float *>(p.y)[at] = v;
            else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
        }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kNMax) : "memory");
    }
}

// Token codes and scales into sorted-route order, one warp per row.
__global__ void __launch_bounds__(256) k_gather_i8(const int8_t *__restrict__ xq, const float *__restrict__ sx,
                                                   const int32_t *__restrict__ sorted_route,
                                                   const int32_t *__restrict__ offsets, int E, int k, int H, int R,
                                                   int8_t *__restrict__ xs, float *__restrict__ ss) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, per = H / 16;
    const int n = min(__ldg(offsets + E), R);
    const int warps = (int)(gridDim.x * (blockDim.x >> 5));
    for (int s = (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)); s < n; s += warps) {
        const int route = __ldg(sorted_route + s);
        if (route < 0 || route >= R) {
            if (lane == 0) record_error(0x2009u, (unsigned)s);
            continue;
        }
        const int t = route / k;
        const uint4 *src = reinterpret_cast<const uint4 *>(xq + (size_t)t * H);
        uint4 *dst = reinterpret_cast<uint4 *>(xs + (size_t)s * H);
        for (int c0 = lane; c0 < per; c0 += 32 * 6) {
            uint4 u[6];
#pragma unroll
            for (int j = 0; j < 6; ++j)
                if (c0 + 32 * j < per) u[j] = __ldg(src + c0 + 32 * j);
#pragma unroll
            for (int j = 0; j < 6; ++j)
                if (c0 + 32 * j < per) dst[c0 + 32 * j] = u[j];
        }
        if (lane == 0) ss[s] = __ldg(sx + t);
    }
}

// Codes and scale of each row of h, one warp per row; V > 0: rows of at most 128 V
// values, held in registers; V = 0: read twice.
template <int V>
__global__ void __launch_bounds__(256) k_codes_h(const float *__restrict__ h, const int32_t *__restrict__ offsets, int E,
                                                 int I, int R, int8_t *__restrict__ hq, float *__restrict__ sh) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, n = min(__ldg(offsets + E), R), per = I / 4;
    const int s = (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5));
    if (s >= n) return;
    const float4 *src = reinterpret_cast<const float4 *>(h + (size_t)s * I);
    uint32_t *dst = reinterpret_cast<uint32_t *>(hq + (size_t)s * I);
    float4 v[V > 0 ? V : 1];
    float amax = 0.0f;
    auto grow = [&](float4 u) {
        amax = max_nan(amax, max_nan(max_nan(fabsf(u.x), fabsf(u.y)), max_nan(fabsf(u.z), fabsf(u.w))));
    };
    if (V > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = lane + 32 * i < per ? src[lane + 32 * i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) grow(v[i]);
    } else {
        for (int c = lane; c < per; c += 32) grow(src[c]);
    }
    amax = warp_max(amax);
    const CodeScale sc = code_scale(amax);
    if (V > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < per) dst[lane + 32 * i] = sc.code4(v[i]);
    } else {
        for (int c = lane; c < per; c += 32) dst[c] = sc.code4(src[c]);
    }
    if (lane == 0) sh[s] = sc.s;
}

// ------------------------------------------------------------------ host side
constexpr size_t kDynSmem = 1024 + kRing;
static_assert(kDynSmem + 4 * (3 * kMaxE + 1) + 4 * kMaxE + 4 * kEpiWarps * kNMax + 768 <= 232448, "int8 tensor-core kernel exceeds shared memory");

// W13 codes of every blob: {K, 16 rows, blocks of 16 rows, gate or up, blob},
// box = 16 gate rows and their 16 up rows.
bool encode_w13(CUtensorMap *m, const void *base, uint64_t H, uint64_t I, uint64_t blobs, uint64_t stride) {
    cuuint64_t dims[5] = {H, 16, I / 16, 2, blobs};
    cuuint64_t strides[4] = {H, 16 * H, I * H, stride};
    cuuint32_t box[5] = {(cuuint32_t)kKB, 16, 1, 2, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int ATOMS, int CG>
cudaError_t launch_tc(const CUtensorMap &mh, const CUtensorMap &mp, const void *b, const TcI8Params &p, int n_sm,
                      cudaStream_t s) {
    TokenMaps mb;
    for (int i = 0; i < 4; ++i) {
        if (i > 0 && (MODE < kPhase1 || (8 << i) >= p.R)) {  // a box that no block of R rows needs: not read
            mb.m[i] = mb.m[i - 1];
            continue;
        }
        if (!encode_2d(&mb.m[i], b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)p.K, (uint64_t)p.R, kKB,
                       MODE < kPhase1 ? (uint32_t)block_rows<CG>(p.R) / CG : 16u << i, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    auto kern = k_i8_tc<MODE, ATOMS, CG>;
    static bool attr[kMaxDevices] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!attr[dev]) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDynSmem);
        if (err != cudaSuccess) return err;
        attr[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n_sm / CG * CG));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kDynSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CG;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, mh, mp, mb, p);
}

template <int S, bool FP32>
cudaError_t launch_split(const LinearArgs &a, const CUtensorMap &mw, cudaStream_t s) {
    SplitParams p{a.sx, a.sw, a.T, a.N, a.K, block_rows<1>(a.T), (a.N + kM - 1) / kM, 0, a.y};
    CUtensorMap mb;
    if (!encode_2d(&mb, a.xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.K, (uint64_t)a.T, kKB, (uint32_t)p.blk,
                   CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    p.stages = std::min(kSplitStages, kRing / ((int)kABytes + p.blk * kKB));
    auto kern = k_i8_split<S, FP32>;
    static bool attr[kMaxDevices] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!attr[dev]) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDynSmem);
        if (err != cudaSuccess) return err;
        attr[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.m_tiles * blocks_of(a.T) * S));
    cfg.blockDim = dim3(kSplitThreads);
    // the ring, or the sums of a block's columns
    cfg.dynamicSmemBytes = 1024 + (size_t)std::max(p.stages * ((int)kABytes + p.blk * kKB), p.blk * kM * 4);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = S;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, mw, mb, p);
}
template <int S>
cudaError_t launch_split(const LinearArgs &a, const CUtensorMap &mw, cudaStream_t s) {
    return a.fp32 ? launch_split<S, true>(a, mw, s) : launch_split<S, false>(a, mw, s);
}

size_t a256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

cudaError_t launch_linear_i8_tc(const LinearArgs &a, cudaStream_t s) {
    cudaError_t err = get_encoder();
    int n_sm = 0;
    if (err != cudaSuccess || (err = sm_count(&n_sm)) != cudaSuccess) return err;
    CUtensorMap mw;
    if (!encode_3d(&mw, a.wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.K, (uint64_t)a.N, 1,
                   (uint64_t)a.K, kKB, kM, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    // Few tiles: a cluster each, where the GPU holds four CTAs a tile or more and K has a
    // pair of atoms for each, up to 128 tokens.  Measured on B200, split / not, 2816
    // long: 2816 rows, 16 tokens 5.3 / 8.5 us, 77 tokens 7.2 / 9.2, 200 tokens 11.3 / 10.9;
    // 1409 rows, 77 tokens 6.1 / 9.1; over two CTAs, 8192 rows, 64 tokens 10.2 / 8.9
    const int64_t tiles = (int64_t)((a.N + kM - 1) / kM) * blocks_of(a.T);
    const int share = (int)std::min<int64_t>(n_sm / tiles, (a.K + kKB - 1) / kKB / 2);
    if (a.T <= kSplitTokens && share >= 8) return launch_split<8>(a, mw, s);
    if (a.T <= kSplitTokens && share >= 4) return launch_split<4>(a, mw, s);
    TcI8Params p{};
    p.E = 1;
    p.R = a.T;
    p.K = a.K;
    p.M = a.N;
    p.brow = a.sx;
    p.wscale = a.sw;
    p.out = a.y;
    // a pair's tiles (256 rows by up to 256 tokens) where they fill the GPU
    const bool pairs = (int64_t)((a.N + 2 * kM - 1) / (2 * kM)) * blocks_of(a.T) >= n_sm / 2;
    if (pairs)
        return a.fp32 ? launch_tc<kLinearF32, 1, 2>(mw, mw, a.xq, p, n_sm, s)
                      : launch_tc<kLinear, 1, 2>(mw, mw, a.xq, p, n_sm, s);
    return a.fp32 ? launch_tc<kLinearF32, 1, 1>(mw, mw, a.xq, p, n_sm, s)
                  : launch_tc<kLinear, 1, 1>(mw, mw, a.xq, p, n_sm, s);
}

// h fp32 | codes of h | scales of h | gathered codes | gathered scales
size_t ffn_i8_tc_workspace(int H, int I, int T, int k) {
    const size_t R = (size_t)T * k;
    return a256(R * I * 4) + a256(R * I) + a256(R * 4) + a256(R * H) + a256(R * 4);
}

cudaError_t launch_ffn_i8_tc(const FfnI8Args &a, cudaStream_t s) {
    cudaError_t err = get_encoder();
    int n_sm = 0;
    if (err != cudaSuccess || (err = sm_count(&n_sm)) != cudaSuccess) return err;
    const int R = a.T * a.k, H = a.L.H, I = a.L.I, E = a.L.E;
    char *at = static_cast<char *>(a.ws);
    float *h = reinterpret_cast<float *>(at);
    at += a256((size_t)R * I * 4);
    int8_t *hq = reinterpret_cast<int8_t *>(at);
    at += a256((size_t)R * I);
    float *sh = reinterpret_cast<float *>(at);
    at += a256((size_t)R * 4);
    int8_t *xs = reinterpret_cast<int8_t *>(at);
    at += a256((size_t)R * H);
    float *ss = reinterpret_cast<float *>(at);

    const bool slotted = a.L.slot_table != nullptr;
    CUtensorMap h1, p1, h2, p2;
    if (!encode_w13(&h1, a.L.home + a.L.off.q13, H, I, E, a.L.stride) ||
        !encode_3d(&h2, a.L.home + a.L.off.q2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, I, H, E, a.L.stride, kKB, kM,
                   CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (!slotted) {
        p1 = h1;  // not read
        p2 = h2;
    } else if (!encode_w13(&p1, a.L.pool + a.L.off.q13, H, I, (uint64_t)a.L.pool_slots, a.L.stride) ||
               !encode_3d(&p2, a.L.pool + a.L.off.q2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, I, H,
                          (uint64_t)a.L.pool_slots, a.L.stride, kKB, kM, CU_TENSOR_MAP_SWIZZLE_128B)) {
        return cudaErrorInvalidValue;
    }

    const int blocks = (int)std::min<int64_t>(((int64_t)R + 7) / 8, (int64_t)n_sm * 8);
    err = launch_pdl(k_gather_i8, dim3((unsigned)blocks), dim3(256), 0, s, a.xq, a.sx, a.sorted_route, a.offsets, E, a.k,
                     H, R, xs, ss);
    if (err != cudaSuccess) return err;
    TcI8Params p{};
    p.L = a.L;
    p.counts = a.counts;
    p.offsets = a.offsets;
    p.E = E;
    p.R = R;
    p.K = H;
    p.M = I;
    p.brow = ss;
    p.out = h;
    const bool few = (int64_t)R <= (int64_t)E * kFewRoutes;
    err = few ? launch_tc<kPhase1, 2, 1>(h1, p1, xs, p, n_sm, s) : launch_tc<kPhase1, 1, 1>(h1, p1, xs, p, n_sm, s);
    if (err != cudaSuccess) return err;
    const dim3 rows8((unsigned)((R + 7) / 8));
    if (I <= 768) err = launch_pdl(k_codes_h<6>, rows8, dim3(256), 0, s, (const float *)h, a.offsets, E, I, R, hq, sh);
    else err = launch_pdl(k_codes_h<0>, rows8, dim3(256), 0, s, (const float *)h, a.offsets, E, I, R, hq, sh);
    if (err != cudaSuccess) return err;
    p.K = I;
    p.M = H;
    p.brow = sh;
    p.out = a.rows;
    return few ? launch_tc<kPhase2, 2, 1>(h2, p2, hq, p, n_sm, s) : launch_tc<kPhase2, 1, 1>(h2, p2, hq, p, n_sm, s);
}

cudaError_t i8tc_take_error(unsigned *code, unsigned *info) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_i8tc_error, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(info, g_i8tc_error_info, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i8tc_error, &zero, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i8tc_error_info, &zero, sizeof(unsigned));
    return e;
}

}  // namespace moe
