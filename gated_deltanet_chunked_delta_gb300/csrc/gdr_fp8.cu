// gdr_fp8.cu -- product of 8-bit activations with 8-bit weights, one scale for
// each 128 k of a token and for each 128 x 128 block of weights:
//
//   out[m, n] = sum_kb sa[kb, m] sb[n / 128, kb] P_kb[m, n],  P_kb = sum_{k in kb} a[m, k] b[n, k]
//
// Large products are bound by the tensor cores, products of a few tokens by
// reading the weights.  The scales are plain fp32, so a block's product P_kb is
// formed by four tcgen05 MMAs (fp32 accumulators in tensor memory) and then
// taken into registers with its scale, in fp32: accumulators alternate, so that
// the MMAs of one block run while another is read.  Warp 0 feeds the operand
// ring by TMA (128-byte swizzled K-major tiles, zeros past the edges), warp 2
// each block's scales by asynchronous copies (scales read by the accumulating
// warps themselves, one block ahead, cost 1.6 times the whole product's time: a
// block lasts less than such a read), warp 1 issues the MMAs, the warps from 4
// on take the accumulators.
//
// The operand whose rows lie along the MMA's 128 rows (X) is the activations,
// except for few tokens (kSwap): there it is the weights, so that no MMA row is
// wasted and a tile's columns are the tokens; where its tiles leave SMs idle,
// the CTAs of a cluster share a tile's k blocks and add their parts through
// distributed shared memory, in rank order.  With many tokens two CTAs form a
// pair (kPair, cta_group::2): 256 x 256 tiles, 128 rows of X and half of Y in
// each CTA's shared memory, one MMA over both.  A single CTA with a 128 x 256
// tile moves 96 KiB a block through its shared memory (in and out), 768 cycles
// at 128 bytes a cycle against 512 of MMAs; a pair's CTA moves 64 KiB.
//
// 8192 x 8192 x 4096 takes 228 us (2.41 PFLOP/s); MMAs and copies alone take
// 137 us of it, the rest is the round trip from a block's MMAs to its
// accumulator's being free again (two of 256 columns fill tensor memory).
// 16 x 8192 x 4096 takes 10.4 us where the weights lie in L2, 12.3 from HBM
// (2.7 TB/s).
#include <cuda.h>

#include "gdr_layer.h"

namespace {

__device__ unsigned g_fp8_status;

constexpr long long kSpins = 1LL << 22, kDrain = 1LL << 24;

struct Fp8P {
    const float *sx, *sy;  // scales of X's and Y's rows (see below)
    void *out;
    long long M, N;
    int nk, tx, ty, split, f32;  // split: CTAs on one tile's k
};

__device__ __forceinline__ uint32_t su32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// The place of a shared-memory address in the pair's first CTA.
__device__ __forceinline__ uint32_t in_leader(const void *p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(su32(p)));
    return r;
}
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
// What the arrival reports (accumulators read) is ordered by the tcgen05 fence
// before it, not by memory: a release at cluster scope waits for a memory
// barrier, which tripled the product's time.
__device__ __forceinline__ void bar_arrive_at(uint32_t b) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok;
}
// Bounded wait of a whole warp; false once the CTA gives up.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, volatile int *abort) {
    bool ok = false;
    for (long long i = 0;; ++i) {
        if (bar_try(b, parity)) { ok = true; break; }
        if (*abort) break;
        if (i >= kSpins) {
            *abort = 1;
            atomicOr(&g_fp8_status, kStatusTimeout);
            break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void bar_drain(uint64_t *b, uint32_t parity) {
    for (long long i = 0; i < kDrain; ++i)
        if (bar_try(b, parity)) return;
}
// Into this CTA's memory, counted on the leader's barrier.
__device__ __forceinline__ void tma2d_pair(void *dst, const CUtensorMap *m, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(su32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma2d(void *dst, const CUtensorMap *m, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(su32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(su32(bar))
        : "memory");
}
// K-major operand tile of 128-byte rows, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// Four MMAs over the 128 bytes of k of one tile pair (32 a step), from a zero
// accumulator; one elected lane issues.
#define MMA_BLOCK(GROUP)                                                                    \
    asm volatile(                                                                           \
        "{\n\t.reg .pred p, q, e;\n\t.reg .b64 x, y;\n\t"                                 \
        "setp.ne.b32 p, %3, %3;\n\t"                                                        \
        "setp.eq.b32 q, %3, %3;\n\t"                                                        \
        "elect.sync _|e, 0xffffffff;\n\t"                                                   \
        "@e tcgen05.mma." GROUP ".kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"                     \
        "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"                                       \
        "@e tcgen05.mma." GROUP ".kind::f8f6f4 [%0], x, y, %3, q;\n\t"                       \
        "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"                                         \
        "@e tcgen05.mma." GROUP ".kind::f8f6f4 [%0], x, y, %3, q;\n\t"                       \
        "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"                                         \
        "@e tcgen05.mma." GROUP ".kind::f8f6f4 [%0], x, y, %3, q;\n\t}" ::"r"(d),            \
        "l"(a), "l"(b), "r"(idesc)                                                          \
        : "memory")
template <bool kPair>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    if (kPair) MMA_BLOCK("cta_group::2");
    else MMA_BLOCK("cta_group::1");
}
#undef MMA_BLOCK
// Arrives on the barrier (of both CTAs of a pair) when the MMAs so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    if (kPair)
        asm volatile(
            "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(su32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(su32(bar))
            : "memory");
}
// kW consecutive accumulator columns of this warp's 32 lanes: issue only; the
// values are there after take_wait of the same registers.
#define R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
              "=r"(r[i + 6]), "=r"(r[i + 7])
#define W8(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
              "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void take_issue(uint32_t ta, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : R8(0), R8(8)
        : "r"(ta));
}
__device__ __forceinline__ void take_issue(uint32_t ta, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : R8(0), R8(8), R8(16), R8(24)
        : "r"(ta));
}
__device__ __forceinline__ void take_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : W8(0), W8(8)::"memory");
}
__device__ __forceinline__ void take_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : W8(0), W8(8), W8(16), W8(24)::"memory");
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 remote_f32x4(uint32_t saddr, int rank) {
    float4 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(saddr), "r"(rank)
                 : "memory");
    return v;
}

// Scales of a block: X's rows, Y's rows (or the block of them) as far as they
// are needed, zeros past the edges.  The ring is sixteen deep: when the operand
// ring (at most six deep) lets block i in, block i - 6's MMAs are done, so (with
// at most four accumulators) block i - 10 has been taken, and block i - 11's
// scales have been read.  A stage of the operand ring is free once its MMAs are
// done and the scales' warp has passed it, so neither ring overtakes the other.
constexpr int kScaleSlots = 16, kScaleRow = 132;
// Asynchronous copy of one float, zero if it does not exist.
__device__ __forceinline__ void copy_f32(float *to, const float *from, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(su32(to)), "l"(from), "r"(real ? 4 : 0) : "memory");
}

template <int kTN, bool kPair>
struct Cfg {
    static constexpr int kStages = kPair || kTN == 128 ? 6 : kTN == 64 ? 3 : kTN == 32 ? 4 : 5;
    static constexpr int kRowsY = kPair ? kTN / 2 : kTN;  // rows of Y in a CTA
    static constexpr int kBytes = 16384 + kRowsY * 128;   // one stage of the ring
    static constexpr int kTake = kTN >= 128 ? 8 : 4;      // warps that take the accumulators
    static constexpr int kBufs = kTN >= 128 ? 512 / kTN : 2;  // accumulators
    static constexpr int kThreads = 128 + 32 * kTake;     // whole warpgroups: the feeding one, the accumulating ones
    static constexpr int kOut = kTake * 2048;             // 32 rows x 64 bytes an accumulating warp, for coalesced stores
    static constexpr int kSmem = kStages * kBytes + 1024 + kOut;
};

template <int kTN, bool kSwap, bool kPair>
__global__ void __launch_bounds__(Cfg<kTN, kPair>::kThreads, 1)
    k_fp8_matmul(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my, const Fp8P p) {
    using G = Cfg<kTN, kPair>;
    constexpr int kStages = G::kStages, kBytes = G::kBytes, kTake = G::kTake;
    constexpr int kCols = kTake == 8 ? kTN / 2 : kTN;  // columns of an accumulating warp
    constexpr int kBufs = G::kBufs;
    constexpr uint32_t kTmem = kTN * kBufs;
    constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kTN >> 3) << 17) | ((kPair ? 16u : 8u) << 24);  // e4m3 x e4m3 -> fp32, 128 (256) x kTN
    extern __shared__ char raw[];
    __shared__ __align__(16) float scales[kScaleSlots][kScaleRow];
    __shared__ uint64_t full[kStages], empty[kStages], tfull[kBufs], tempty[kBufs], sfull[kScaleSlots], done;
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    char *ring = raw + ((1024u - (su32(raw) & 1023u)) & 1023u);
    volatile int *abort = &abort_flag;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // kPair: p.split is 2, the CTAs of a cluster share a tile's rows; else they share its k blocks.
    const int rank = blockIdx.x % p.split, first = blockIdx.x / p.split, step = gridDim.x / p.split, tiles = p.tx * p.ty;
    constexpr int kRowsX = kPair ? 256 : 128;
    const int xr = kPair ? 128 * rank : 0;  // this CTA's rows of a tile
    const int kb0 = kPair ? 0 : (int)((long long)p.nk * rank / p.split), kb1 = kPair ? p.nk : (int)((long long)p.nk * (rank + 1) / p.split);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&full[i], 1);
            bar_init(&empty[i], 2);  // the MMAs, and warp 2
        }
        for (int i = 0; i < kBufs; ++i) {
            bar_init(&tfull[i], 1);
            bar_init(&tempty[i], kPair ? 2 * kTake : kTake);
        }
        for (int i = 0; i < kScaleSlots; ++i) bar_init(&sfull[i], 32);
        bar_init(&done, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_at)), "r"(kTmem) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_at)), "r"(kTmem) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (kPair) cluster_barrier();  // both CTAs' barriers and tensor memory are there
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_at;

    // 384 threads are launched with 168 registers each: 128 x 56 + 256 x 224 of them
    if (kTN == 256 && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
        int it = 0;
        bool ok = true;
        const uint32_t leader_full = kPair ? in_leader(&full[0]) : 0;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const int x0 = tile % p.tx * kRowsX + xr, y0 = tile / p.tx * kTN;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % kStages;
                if (it >= kStages && !(ok = bar_wait(&empty[s], (it / kStages - 1) & 1, abort))) break;
                if (lane == 0) {
                    char *to = ring + s * kBytes;
                    if (kPair) {
                        const uint32_t bar = leader_full + s * 8;
                        if (rank == 0) bar_expect(&full[s], 2 * kBytes);
                        tma2d_pair(to, &mx, kb * 128, x0, bar);
                        tma2d_pair(to + 16384, &my, kb * 128, y0 + rank * G::kRowsY, bar);
                    } else {
                        bar_expect(&full[s], kBytes);
                        tma2d(to, &mx, kb * 128, x0, &full[s]);
                        tma2d(to + 16384, &my, kb * 128, y0, &full[s]);
                    }
                }
            }
        }
        // every copy (of a pair: of both CTAs) has landed before it leaves
        if (!kPair || rank == 0)
            for (int i = it > kStages ? it - kStages : 0; i < it; ++i) bar_drain(&full[i % kStages], (i / kStages) & 1);
    } else if (warp == 2) {
        // The scales, at the pace of the operand ring (a slot is free by then, as above).
        int it = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const int x0 = tile % p.tx * kRowsX + xr, y0 = tile / p.tx * kTN;
            constexpr int kEach = kSwap ? (kTN + 31) / 32 : 4;  // token scales a lane copies
            const long long m0 = kSwap ? y0 : x0;
            const float *tok = (kSwap ? p.sy : p.sx) + (long long)kb0 * p.M + m0 + lane;
            int bytes[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) bytes[i] = m0 + 32 * i + lane < p.M && (!kSwap || 32 * i + lane < kTN) ? 4 : 0;
            const long long nb = (kSwap ? x0 : y0) / 128 + lane;  // weight blocks: one, or two by the first lanes
            const bool wide = lane < (kSwap ? 1 : (kTN + 127) / 128), there = wide && nb * 128 < p.N;
            const float *wt = (kSwap ? p.sx : p.sy) + (there ? nb * p.nk + kb0 : 0);
            for (int kb = kb0; kb < kb1; ++kb, ++it, tok += p.M, wt += there) {
                if (it >= kStages && !(ok = bar_wait(&empty[it % kStages], (it / kStages - 1) & 1, abort))) break;
                // Nothing but this arrival keeps the stage from being emptied again before this warp has looked:
                // block it's MMAs need the scales of block it - kBufs only, and a second turn would undo the parity.
                if (lane == 0) bar_arrive(&empty[it % kStages]);
                float *sc = scales[it % kScaleSlots];
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (!kSwap || 32 * i + lane < kTN) copy_f32(&sc[32 * i + lane], bytes[i] ? tok + 32 * i : p.sx, bytes[i]);
                if (wide) copy_f32(&sc[128 + lane], wt, there);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(su32(&sfull[it % kScaleSlots])) : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 1 && (!kPair || rank == 0)) {
        int it = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += step) {
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % kStages, a = it % kBufs;
                if (!(ok = bar_wait(&full[s], (it / kStages) & 1, abort))) break;
                if (it >= kBufs && !(ok = bar_wait(&tempty[a], (it / kBufs - 1) & 1, abort))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = su32(ring + s * kBytes);
                mma_block<kPair>(tmem + a * kTN, tile_desc(at), tile_desc(at + 16384), kIdesc);
                mma_commit<kPair>(&empty[s]);
                mma_commit<kPair>(&tfull[a]);
            }
        }
        mma_commit<kPair>(&done);
        bar_drain(&done, 0);
    } else if (warp >= 4) {
        if (kTN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int quad = warp & 3, half = (warp - 4) / 4;
        const int row = 32 * quad + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + half * kCols;
        const uint32_t leader_tempty = kPair ? in_leader(&tempty[0]) : 0;
        int it = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const int x0 = tile % p.tx * kRowsX + xr, y0 = tile / p.tx * kTN;
            f32x2 acc[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = 0ull;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int a = it % kBufs;
                const float *sc = scales[it % kScaleSlots];
                if (!(ok = bar_wait(&tfull[a], (it / kBufs) & 1, abort))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                // one piece is on its way while the piece before it is scaled and added
                constexpr int kW = kCols < 32 || kCols > 64 ? 16 : 32, kPieces = kCols / kW;
                uint32_t r[2][kW];
                take_issue(lanes + a * kTN, r[0]);
                ok = bar_wait(&sfull[it % kScaleSlots], (it / kScaleSlots) & 1, abort);
                const float s1 = kSwap ? sc[128] : sc[row] * sc[128 + half * kCols / 128];
                const f32x2 s2 = mk2(s1, s1);
#pragma unroll
                for (int c = 0; c < kPieces; ++c) {
                    take_wait(r[c & 1]);
                    if (c + 1 < kPieces) {
                        take_issue(lanes + a * kTN + (c + 1) * kW, r[(c + 1) & 1]);
                    } else {  // all of it is in registers
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            if (kPair) bar_arrive_at(leader_tempty + a * 8);
                            else bar_arrive(&tempty[a]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kW; j += 2) {
                        const int col = c * kW + j;
                        // by columns where the tokens are: a pair of scales, the same for all lanes
                        const f32x2 k2 = kSwap ? mul2(s2, *reinterpret_cast<const f32x2 *>(&sc[col])) : s2;
                        acc[col / 2] = fma2(mk2(__uint_as_float(r[c & 1][j]), __uint_as_float(r[c & 1][j + 1])), k2, acc[col / 2]);
                    }
                }
            }
            if (!ok) break;
            if (kSwap && p.split > 1) {  // this CTA's part of the tile: [kTN][128] in the ring, which is idle by now
                float *part = reinterpret_cast<float *>(ring);
#pragma unroll
                for (int j = 0; j < kCols / 2; ++j) {
                    float lo, hi;
                    un2(acc[j], lo, hi);
                    part[(half * kCols + 2 * j) * 128 + row] = lo;
                    part[(half * kCols + 2 * j + 1) * 128 + row] = hi;
                }
                break;
            }
            if (kSwap) {
                const long long n = x0 + row;
                if (n < p.N)
#pragma unroll
                    for (int j = 0; j < kCols / 2; ++j) {
                        float v[2];
                        un2(acc[j], v[0], v[1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const long long m = y0 + 2 * j + k;
                            if (m >= p.M) continue;
                            if (p.f32) static_cast<float *>(p.out)[m * p.N + n] = v[k];
                            else from_f(static_cast<bf16_t *>(p.out)[m * p.N + n], v[k]);
                        }
                    }
            } else {
                // 32 rows x 64 bytes at a time through shared memory: a store
                // instruction then writes 64 bytes each of eight rows.
                const long long n0 = y0 + half * kCols;
                const int mrows = (int)min(32LL, p.M - x0 - 32 * quad);  // rows of this warp that exist
                char *out = ring + kStages * kBytes + (warp - 4) * 2048;
                const bool vec = p.N % 8 == 0;
                if (mrows > 0)
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        if (!p.f32 && c % 32) continue;  // 16 columns of fp32 or 32 of bf16
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // 16-byte chunk i of a row lies at i ^ (row / 2 % 4)
                            uint4 w;
                            if (p.f32) {
                                const f32x2 v0 = acc[c / 2 + 2 * i], v1 = acc[c / 2 + 2 * i + 1];
                                w = make_uint4((uint32_t)v0, (uint32_t)(v0 >> 32), (uint32_t)v1, (uint32_t)(v1 >> 32));
                            } else {
                                float v[8];
#pragma unroll
                                for (int k = 0; k < 4; ++k) un2(acc[(c / 2 + 4 * i + k) % (kCols / 2)], v[2 * k], v[2 * k + 1]);
                                w = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                            }
                            *reinterpret_cast<uint4 *>(out + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) = w;
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + lane / 4, ch = lane % 4;
                            const long long n = n0 + c + ch * (p.f32 ? 4 : 8), m = x0 + 32 * quad + r;
                            if (r >= mrows || n >= p.N) continue;
                            const uint4 w = *reinterpret_cast<const uint4 *>(out + r * 64 + ((ch ^ (r >> 1 & 3)) << 4));
                            char *o = static_cast<char *>(p.out) + (m * p.N + n) * (p.f32 ? 4 : 2);
                            if (vec) {
                                *reinterpret_cast<uint4 *>(o) = w;
                            } else {
                                const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if (p.f32) {
                                        if (n + k < p.N) reinterpret_cast<uint32_t *>(o)[k] = q[k];
                                    } else {
                                        if (n + 2 * k < p.N) reinterpret_cast<uint16_t *>(o)[2 * k] = (uint16_t)q[k];
                                        if (n + 2 * k + 1 < p.N) reinterpret_cast<uint16_t *>(o)[2 * k + 1] = (uint16_t)(q[k] >> 16);
                                    }
                                }
                            }
                        }
                    }
            }
        }
    }
    if (kPair) {  // neither CTA leaves while the other's MMAs, copies or arrivals reach it
        __syncwarp();
        cluster_barrier();
    } else if (kSwap && p.split > 1) {
        __syncwarp();
        cluster_barrier();
        if (kSwap && warp >= 4) {  // this CTA adds up its share of the tile's tokens, four weight rows a thread
            const int t = threadIdx.x - 128, row = t % 32 * 4;
            const int x0 = first % p.tx * 128, y0 = first / p.tx * kTN;
            const int c1 = kTN * (rank + 1) / p.split;
            for (int c = kTN * rank / p.split + t / 32; c < c1; c += kTake) {
                const uint32_t at = su32(ring) + (c * 128 + row) * 4;
                float4 part[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < p.split) part[k] = remote_f32x4(at, k);
                float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < p.split) {
                        v[0] += part[k].x; v[1] += part[k].y; v[2] += part[k].z; v[3] += part[k].w;
                    }
                const long long m = y0 + c, n = x0 + row;
                if (m >= p.M) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (n + k >= p.N) break;
                    if (p.f32) static_cast<float *>(p.out)[m * p.N + n + k] = v[k];
                    else from_f(static_cast<bf16_t *>(p.out)[m * p.N + n + k], v[k]);
                }
            }
        }
        __syncwarp();
        cluster_barrier();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
    }
}

// ---- host ------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static EncodeFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<EncodeFn>(ptr);
    }();
    return fn;
}

// [rows, K] bytes in tiles of box rows x 128; zeros past the edges.
bool tile_map(CUtensorMap *m, const void *base, long long rows, long long K, int box) {
    const cuuint64_t d[2] = {(cuuint64_t)K, (cuuint64_t)rows}, s[1] = {(cuuint64_t)K};
    const cuuint32_t b[2] = {128, (cuuint32_t)box}, es[2] = {1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Fp8Plan {
    int tn, split;
    bool swap, pair;
};

// Up to 64 tokens: weights as rows, one tile of tokens, and clusters of up to 8
// on a tile's k blocks where tiles are few.  Otherwise the tile that finishes
// first by waves x time a block, as measured (ns a block: pairs of CTAs on
// 256 x 256 500, 128 x 128 405, 128 x 64 400 alone on an SM and 800 two on
// one; splitting k there cost more than it gave, 28.7 against 17.7 us for
// 128 x 8192 x 4096).
Fp8Plan fp8_plan(long long M, long long N, int nk) {
    const long long sms = layer_sms();
    Fp8Plan pl{0, 1, M <= 64, false};
    if (pl.swap) {
        pl.tn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
        const long long tiles = (N + 127) / 128;
        // two CTAs an SM, one where a tile has 64 tokens (64 x 8192 x 4096: 14.4 us, 18.4 with two)
        const long long room = pl.tn == 64 ? sms : 2 * sms;
        while (pl.split < 8 && tiles * pl.split * 2 <= room && nk >= pl.split * 2 * 2) pl.split *= 2;
        return pl;
    }
    auto waves = [](long long t, long long at) { return (double)((t + at - 1) / at); };
    const long long mt = (M + 127) / 128, t128 = mt * ((N + 127) / 128), t64 = mt * ((N + 63) / 64);
    const long long t256 = ((M + 255) / 256) * ((N + 255) / 256);
    const double c256 = waves(t256, sms / 2) * 500, c128 = waves(t128, sms) * 405, c64 = t64 <= sms ? 400 : waves(t64, 2 * sms) * 800;
    pl.pair = c256 <= c128 && c256 <= c64;
    pl.tn = pl.pair ? 256 : c128 < c64 ? 128 : 64;
    if (pl.pair) pl.split = 2;
    return pl;
}

template <int kTN, bool kSwap, bool kPair>
int launch(const CUtensorMap &mx, const CUtensorMap &my, const Fp8P &p, cudaStream_t st) {
    constexpr int kSmem = Cfg<kTN, kPair>::kSmem;
    const long long tiles = (long long)p.tx * p.ty;
    cudaError_t e = cudaFuncSetAttribute(k_fp8_matmul<kTN, kSwap, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "matmul: %s", cudaGetErrorString(e));
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(Cfg<kTN, kPair>::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    long long ctas = (long long)layer_sms() * (kTN <= 64 ? 2 : 1);
    if (kPair) {  // pairs that run at a time (asked once a device): one more would take the whole time again
        static gdr::OncePerDevice pairs;
        const int n = pairs.get(layer_device(), 1, [&] {
            int most = 0;
            cfg.gridDim = dim3((unsigned)(ctas & ~1LL));
            if (cudaOccupancyMaxActiveClusters(&most, k_fp8_matmul<kTN, kSwap, kPair>, &cfg) == cudaSuccess) return most;
            cudaGetLastError();
            return 0;
        });
        ctas = std::min(ctas, 2LL * n);
    }
    cfg.gridDim = dim3((unsigned)(kPair ? std::min(tiles, ctas / 2) * 2 : p.split > 1 ? tiles * p.split : std::min(tiles, ctas)));
    e = cudaLaunchKernelEx(&cfg, k_fp8_matmul<kTN, kSwap, kPair>, mx, my, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return layer_fail(GDR_ERR_CUDA, "matmul launch failed: %s", cudaGetErrorString(e));
    }
    return GDR_OK;
}

}  // namespace

namespace gdr {
unsigned fp8_take_status(cudaStream_t st) {
    unsigned v = 0, z = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_fp8_status, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return 0x80000000u;
    cudaMemcpyToSymbolAsync(g_fp8_status, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    if (cudaStreamSynchronize(st) != cudaSuccess) return 0x80000000u;
    return v;
}
}  // namespace gdr

extern "C" int gdr_fp8_matmul(const gdr_fp8_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    if (a->M < 0 || a->N < 1 || a->K < 16 || a->K % 16)
        return layer_fail(GDR_ERR_SHAPE, "matmul: M >= 0, N >= 1 and K a positive multiple of 16 (got %lld, %lld, %lld)", a->M, a->N, a->K);
    if (a->M >= (1LL << 30) || a->N >= (1LL << 30) || a->K >= (1LL << 30) || ((a->M + 127) / 128) * ((a->N + 15) / 16) >= (1LL << 30))
        return layer_fail(GDR_ERR_SHAPE, "matmul: problem too large");
    if (a->out_dtype != GDR_BF16 && a->out_dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "matmul: unknown dtype %d", a->out_dtype);
    const bool any = a->M > 0;
    int rc;
    if ((rc = layer_ptr("a", a->a, any, 16)) || (rc = layer_ptr("b", a->b, true, 16)) || (rc = layer_ptr("a_scales", a->a_scales, any, 4)) ||
        (rc = layer_ptr("b_scales", a->b_scales, true, 4)) || (rc = layer_ptr("out", a->out, any, 16)))
        return rc;
    if (!any) return GDR_OK;
    if (!encoder()) return layer_fail(GDR_ERR_CUDA, "matmul: the driver has no cuTensorMapEncodeTiled");
    const int nk = (int)((a->K + 127) / 128);
    const Fp8Plan pl = fp8_plan(a->M, a->N, nk);
    Fp8P p{};
    p.M = a->M; p.N = a->N; p.nk = nk; p.split = pl.split; p.out = a->out; p.f32 = a->out_dtype == GDR_F32;
    CUtensorMap ma, mb;
    if (!tile_map(&ma, a->a, a->M, a->K, pl.swap ? pl.tn : 128) || !tile_map(&mb, a->b, a->N, a->K, pl.swap || pl.pair ? 128 : pl.tn))
        return layer_fail(GDR_ERR_CUDA, "matmul: tensor map refused");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl.swap) {
        p.sx = a->b_scales; p.sy = a->a_scales;
        p.tx = (int)((a->N + 127) / 128); p.ty = (int)((a->M + pl.tn - 1) / pl.tn);
        return pl.tn == 16   ? launch<16, true, false>(mb, ma, p, st)
               : pl.tn == 32 ? launch<32, true, false>(mb, ma, p, st)
                             : launch<64, true, false>(mb, ma, p, st);
    }
    p.sx = a->a_scales; p.sy = a->b_scales;
    p.tx = (int)(pl.pair ? (a->M + 255) / 256 : (a->M + 127) / 128); p.ty = (int)((a->N + pl.tn - 1) / pl.tn);
    return pl.pair        ? launch<256, false, true>(ma, mb, p, st)
           : pl.tn == 128 ? launch<128, false, false>(ma, mb, p, st)
                          : launch<64, false, false>(ma, mb, p, st);
}
