// gdr_fp8.cu -- product of 8-bit activations with 8-bit weights, one scale for
// each 128 k of a token and for each 128 x 128 block of weights:
//
//   out[m, n] = sum_kb sa[kb, m] sb[n / 128, kb] P_kb[m, n],  P_kb = sum_{k in kb} a[m, k] b[n, k]
//
// Large products are bound by the tensor cores, products of a few tokens by
// reading the weights.  The scales are plain fp32, so a block's product P_kb is
// formed by four tcgen05 MMAs (fp32 accumulators in tensor memory) and then
// taken into registers with its scale, in fp32: two accumulators alternate, so
// that the MMAs of one block run while the other is read.  Warp 0 feeds the
// operand ring by TMA (128-byte swizzled K-major tiles, zeros past the edges),
// warp 1 issues the MMAs, the others take the accumulators.
//
// The operand whose rows lie along the MMA's 128 rows (X) is the activations,
// except for few tokens (kSwap): there it is the weights, so that no MMA row is
// wasted and a tile's columns are the tokens.  Where the tiles leave SMs idle,
// the CTAs of a cluster share a tile's k blocks and add their parts through
// distributed shared memory, in rank order.
#include <cuda.h>

#include "gdr_layer.h"

namespace {

__device__ unsigned g_fp8_status;

constexpr long long kSpins = 1LL << 22, kDrain = 1LL << 24;

struct Fp8P {
    const float *sx, *sy;  // scales of X's and Y's rows (see below)
    void *out;
    long long M, N;
    int nk, tx, ty, split, f32;
};

__device__ __forceinline__ uint32_t su32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
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
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q, e;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %3, %3;\n\t"
        "setp.eq.b32 q, %3, %3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, q;\n\t"
        "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, q;\n\t"
        "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(su32(bar))
        : "memory");
}
#define R4(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define W4(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])
__device__ __forceinline__ void tmem_ld16(uint32_t ta, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : R4(0), R4(4), R4(8), R4(12)
        : "r"(ta));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : W4(0), W4(4), W4(8), W4(12)::"memory");
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float remote_f32(uint32_t saddr, int rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(saddr), "r"(rank)
                 : "memory");
    return v;
}

template <int kTN>
struct Cfg {
    static constexpr int kStages = kTN == 256 ? 4 : kTN == 128 ? 6 : kTN == 64 ? 4 : kTN == 32 ? 5 : 6;
    static constexpr int kBytes = 16384 + kTN * 128;      // one stage of the ring
    static constexpr int kTake = kTN >= 128 ? 8 : 4;      // warps that take the accumulators
    static constexpr int kThreads = 64 + 32 * kTake;
    static constexpr int kSmem = kStages * kBytes + 1024;
};

template <int kTN, bool kSwap>
__global__ void __launch_bounds__(Cfg<kTN>::kThreads, 1)
    k_fp8_matmul(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my, const Fp8P p) {
    constexpr int kStages = Cfg<kTN>::kStages, kBytes = Cfg<kTN>::kBytes, kTake = Cfg<kTN>::kTake;
    constexpr int kCols = kTake == 8 ? kTN / 2 : kTN;  // columns of an accumulating warp
    constexpr uint32_t kTmem = kTN * 2 < 32 ? 32 : kTN * 2;
    constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kTN >> 3) << 17) | (8u << 24);  // e4m3 x e4m3 -> fp32, 128 x kTN
    extern __shared__ char raw[];
    __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], done;
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    char *ring = raw + ((1024u - (su32(raw) & 1023u)) & 1023u);
    volatile int *abort = &abort_flag;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % p.split, step = gridDim.x / p.split, tiles = p.tx * p.ty;
    const int kb0 = (int)((long long)p.nk * rank / p.split), kb1 = (int)((long long)p.nk * (rank + 1) / p.split);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&full[i], 1);
            bar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&tfull[i], 1);
            bar_init(&tempty[i], kTake);
        }
        bar_init(&done, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_at)), "r"(kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_at;

    if (warp == 0) {
        int it = 0;
        bool ok = true;
        for (int tile = blockIdx.x / p.split; ok && tile < tiles; tile += step) {
            const int x0 = (tile % p.tx) * 128, y0 = (tile / p.tx) * kTN;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % kStages;
                if (it >= kStages && !(ok = bar_wait(&empty[s], (it / kStages - 1) & 1, abort))) break;
                if (lane == 0) {
                    char *to = ring + s * kBytes;
                    bar_expect(&full[s], kBytes);
                    tma2d(to, &mx, kb * 128, x0, &full[s]);
                    tma2d(to + 16384, &my, kb * 128, y0, &full[s]);
                }
            }
        }
        // every copy of this CTA has landed before it leaves
        for (int i = it > kStages ? it - kStages : 0; i < it; ++i) bar_drain(&full[i % kStages], (i / kStages) & 1);
    } else if (warp == 1) {
        int it = 0;
        bool ok = true;
        for (int tile = blockIdx.x / p.split; ok && tile < tiles; tile += step) {
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % kStages, a = it & 1;
                if (!(ok = bar_wait(&full[s], (it / kStages) & 1, abort))) break;
                if (it >= 2 && !(ok = bar_wait(&tempty[a], (it / 2 - 1) & 1, abort))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = su32(ring + s * kBytes);
                mma_block(tmem + a * kTN, tile_desc(at), tile_desc(at + 16384), kIdesc);
                mma_commit(&empty[s]);
                mma_commit(&tfull[a]);
            }
        }
        mma_commit(&done);
        bar_drain(&done, 0);
    } else {
        const int quad = warp & 3, half = (warp - 2) / 4;
        const int row = 32 * quad + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + half * kCols;
        int it = 0;
        bool ok = true;
        for (int tile = blockIdx.x / p.split; ok && tile < tiles; tile += step) {
            const int x0 = (tile % p.tx) * 128, y0 = (tile / p.tx) * kTN;
            f32x2 acc[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = 0ull;
            // Scales of block kb.  Activations as rows: one factor a thread.
            // Activations as columns (kSwap): lane l holds those of columns l, l + 32.
            constexpr int kS = kSwap ? (kTN + 31) / 32 : 1;
            float sc[kS], nx[kS];
            auto scales = [&](int kb, float (&v)[kS]) {
                if (kSwap) {
                    const float sb = p.sx[(long long)(x0 / 128) * p.nk + kb];
#pragma unroll
                    for (int i = 0; i < kS; ++i) {
                        const long long m = y0 + 32 * i + lane;
                        v[i] = 32 * i + lane < kTN && m < p.M ? sb * p.sy[(long long)kb * p.M + m] : 0.f;
                    }
                } else {
                    const long long m = x0 + row, nb = (y0 + half * kCols) / 128;
                    v[0] = m < p.M && nb * 128 < p.N ? p.sx[(long long)kb * p.M + m] * p.sy[nb * p.nk + kb] : 0.f;
                }
            };
            if (kb0 < kb1) scales(kb0, nx);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int a = it & 1;
#pragma unroll
                for (int i = 0; i < kS; ++i) sc[i] = nx[i];
                if (kb + 1 < kb1) scales(kb + 1, nx);
                if (!(ok = bar_wait(&tfull[a], (it / 2) & 1, abort))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(lanes + a * kTN + c, r);
                    tmem_wait16(r);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        f32x2 s2;
                        if (kSwap) {
                            const float lo = __shfl_sync(0xffffffffu, sc[(c + j) / 32], (c + j) % 32);
                            const float hi = __shfl_sync(0xffffffffu, sc[(c + j) / 32], (c + j) % 32 + 1);
                            s2 = mk2(lo, hi);
                        } else {
                            s2 = mk2(sc[0], sc[0]);
                        }
                        acc[(c + j) / 2] = fma2(mk2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), s2, acc[(c + j) / 2]);
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(&tempty[a]);
            }
            if (!ok) break;
            if (p.split > 1) {  // this CTA's part of the tile: [kTN][128] in the ring, which is idle by now
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
                const long long m = x0 + row, n0 = y0 + half * kCols;
                const bool vec = p.N % 8 == 0;
                if (m < p.M)
#pragma unroll
                    for (int j = 0; j < kCols / 2; j += 4) {
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) un2(acc[j + k], v[2 * k], v[2 * k + 1]);
                        const long long n = n0 + 2 * j;
                        const int nv = (int)min(8LL, p.N - n);
                        if (nv <= 0) continue;
                        if (p.f32) {
                            float *o = static_cast<float *>(p.out) + m * p.N + n;
                            if (vec) store8<float, true>(o, v, nv); else store8<float, false>(o, v, nv);
                        } else {
                            bf16_t *o = static_cast<bf16_t *>(p.out) + m * p.N + n;
                            if (vec) store8<bf16_t, true>(o, v, nv); else store8<bf16_t, false>(o, v, nv);
                        }
                    }
            }
        }
    }
    if (p.split > 1) {
        __syncwarp();
        cluster_barrier();
        if (warp >= 2) {  // this CTA adds up its share of the tile's columns
            const int t = threadIdx.x - 64, row = t % 128, tile = blockIdx.x / p.split;
            const int x0 = (tile % p.tx) * 128, y0 = (tile / p.tx) * kTN;
            const uint32_t part = su32(ring);
            const int c0 = kTN * rank / p.split, c1 = kTN * (rank + 1) / p.split;
            for (int c = c0 + t / 128; c < c1; c += kTake / 4) {
                float v = 0.f;
                for (int k = 0; k < p.split; ++k) v += remote_f32(part + (c * 128 + row) * 4, k);
                const long long m = kSwap ? y0 + c : x0 + row, n = kSwap ? x0 + row : y0 + c;
                if (m >= p.M || n >= p.N) continue;
                if (p.f32) static_cast<float *>(p.out)[m * p.N + n] = v;
                else from_f(static_cast<bf16_t *>(p.out)[m * p.N + n], v);
            }
        }
        __syncwarp();
        cluster_barrier();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
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
    bool swap;
};

// Up to 64 tokens: weights as rows, one tile of tokens.  Otherwise the tile
// width that finishes first by waves x time a block (in cycles, from the MMA
// rates and the ring's copies), and clusters of up to 8 where tiles are few.
Fp8Plan fp8_plan(long long M, long long N, int nk) {
    const long long sms = layer_sms();
    Fp8Plan pl{0, 1, M <= 64};
    long long tiles, room;
    if (pl.swap) {
        pl.tn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
        tiles = (N + 127) / 128;
        room = 2 * sms;
    } else {
        double best = 1e300;
        const int tn[3] = {256, 128, 64};
        const double cost[3] = {560, 300, 190};
        for (int i = 0; i < 3; ++i) {
            const long long t = ((M + 127) / 128) * ((N + tn[i] - 1) / tn[i]);
            const double c = (double)((t + sms - 1) / sms) * cost[i];
            if (c < best * 0.99) {
                best = c;
                pl.tn = tn[i];
            }
        }
        tiles = ((M + 127) / 128) * ((N + pl.tn - 1) / pl.tn);
        room = sms;
    }
    while (pl.split < 8 && pl.tn <= 128 && tiles * pl.split * 2 <= room && nk >= pl.split * 2 * 2) pl.split *= 2;
    return pl;
}

template <int kTN, bool kSwap>
int launch(const CUtensorMap &mx, const CUtensorMap &my, const Fp8P &p, cudaStream_t st) {
    constexpr int kSmem = Cfg<kTN>::kSmem;
    const long long tiles = (long long)p.tx * p.ty;
    cudaError_t e = cudaFuncSetAttribute(k_fp8_matmul<kTN, kSwap>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "matmul: %s", cudaGetErrorString(e));
    const long long grid = p.split > 1 ? tiles * p.split : std::min<long long>(tiles, (long long)layer_sms() * (kTN <= 64 ? 2 : 1));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Cfg<kTN>::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_fp8_matmul<kTN, kSwap>, mx, my, p);
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
    if (!tile_map(&ma, a->a, a->M, a->K, pl.swap ? pl.tn : 128) || !tile_map(&mb, a->b, a->N, a->K, pl.swap ? 128 : pl.tn))
        return layer_fail(GDR_ERR_CUDA, "matmul: tensor map refused");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl.swap) {
        p.sx = a->b_scales; p.sy = a->a_scales;
        p.tx = (int)((a->N + 127) / 128); p.ty = (int)((a->M + pl.tn - 1) / pl.tn);
        return pl.tn == 16 ? launch<16, true>(mb, ma, p, st) : pl.tn == 32 ? launch<32, true>(mb, ma, p, st) : launch<64, true>(mb, ma, p, st);
    }
    p.sx = a->a_scales; p.sy = a->b_scales;
    p.tx = (int)((a->M + 127) / 128); p.ty = (int)((a->N + pl.tn - 1) / pl.tn);
    return pl.tn == 256 ? launch<256, false>(ma, mb, p, st) : pl.tn == 128 ? launch<128, false>(ma, mb, p, st) : launch<64, false>(ma, mb, p, st);
}
