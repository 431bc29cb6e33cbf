// gdr_norm.cu -- root-mean-square norm of a residual stream, in the input's
// type or in 8 bits with scales, and its gradient.
//
//   r = x + residual (rounded to the stored type), y = r rstd w,  rstd = (mean r^2 + eps)^-1/2
//   dr = rstd (w dy - r rstd^2 mean(w dy r)) + dsum,  dw = sum over rows of dy r rstd
//
// Bound by memory: a row is read once into the registers of one CTA, reduced
// once, and written once.  The norm is taken of r as it is stored, so that
// the gradient, which reads the stored r, is that of what was computed.
#include "gdr_layer.h"

namespace {

constexpr int kMaxThreads = 512, kMaxIter = 4;  // 8 x 512 x 4 channels a row

struct NormP {
    const void *x, *residual;
    const float *weight;
    void *sum, *y;
    uint8_t *q;
    float *scales;
    long long M, x_row, r_row;
    int D;
    float eps;
};

// Sum of (up to two) values over the CTA; `buf` alternates between calls so
// that one barrier a call is enough.
__device__ __forceinline__ float2 cta_sum(float a, float b, float2 *buf) {
#pragma unroll
    for (int m = 16; m >= 1; m /= 2) {
        a += __shfl_xor_sync(0xffffffffu, a, m);
        b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = make_float2(a, b);
    __syncthreads();
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
    const float2 v = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
    a = v.x;
    b = v.y;
#pragma unroll
    for (int m = 8; m >= 1; m /= 2) {
        a += __shfl_xor_sync(0xffffffffu, a, m);
        b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    return make_float2(__shfl_sync(0xffffffffu, a, 0), __shfl_sync(0xffffffffu, b, 0));
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <typename T, int kIter, bool kVec, bool kQuant>
__global__ void __launch_bounds__(kMaxThreads) k_norm_fwd(const NormP p) {
    __shared__ float2 buf[32];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.x_row;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + row * p.r_row : nullptr;
    const long long out = row * p.D;
    Raw8<T> rx[kIter], rr[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = min(8, p.D - c);
        rx[i] = load8<T, kVec>(x + c, n);
        if (res) rr[i] = load8<T, kVec>(res + c, n);
    }
    float v[kIter][8], sq = 0.f;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = min(8, p.D - c);
        unpack8(rx[i], v[i]);
        if (res) {
            float f[8];
            unpack8(rr[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] += f[e];
            store8<T, kVec>(static_cast<T *>(p.sum) + out + c, v[i], n);
            Raw8<T> stored;
            pack8(v[i], stored);
            unpack8(stored, v[i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(v[i][e], v[i][e], sq);
    }
    const float rstd = 1.f / sqrtf(cta_sum(sq, 0.f, buf).x / (float)p.D + p.eps);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8, n = min(8, p.D - c);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = e < n ? v[i][e] * rstd * p.weight[c + e] : 0.f;
        if (!kQuant) {
            store8<T, kVec>(static_cast<T *>(p.y) + out + c, v[i], n);
            continue;
        }
        // 16 neighbouring threads hold a block of 128 channels
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(v[i][e]));
#pragma unroll
        for (int m = 8; m >= 1; m /= 2) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
        const float scale = max_nan(top, 1e-30f) / 448.f, inv = 1.f / scale;
        if (n <= 0) continue;
        if (threadIdx.x % 16 == 0) p.scales[(long long)(c / 128) * p.M + row] = scale;
        const uint32_t lo = e4m3x4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
        const uint32_t hi = e4m3x4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv);
        if (kVec) {
            *reinterpret_cast<uint2 *>(p.q + out + c) = make_uint2(lo, hi);
        } else {
            for (int e = 0; e < n; ++e) p.q[out + c + e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
        }
    }
}

struct NormBwdP {
    const void *r, *dy, *dsum;
    const float *weight;
    void *dr;
    float *part, *dweight;  // part: [CTAs, D]
    long long M;
    int D;
    float eps;
};

// A CTA takes every gridDim-th row and keeps its part of dweight in registers.
template <typename T, int kIter, bool kVec>
__global__ void __launch_bounds__(kMaxThreads) k_norm_bwd(const NormBwdP p) {
    __shared__ float2 buf[2][32];
    float gw[kIter][8];
#pragma unroll
    for (int i = 0; i < kIter; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[i][e] = 0.f;
    int turn = 0;
    for (long long row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
        const long long at = row * p.D;
        Raw8<T> rr[kIter], rg[kIter], rs[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8, n = min(8, p.D - c);
            rr[i] = load8<T, kVec>(static_cast<const T *>(p.r) + at + c, n);
            rg[i] = load8<T, kVec>(static_cast<const T *>(p.dy) + at + c, n);
            if (p.dsum) rs[i] = load8<T, kVec>(static_cast<const T *>(p.dsum) + at + c, n);
        }
        float sq = 0.f, gr = 0.f;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8, n = min(8, p.D - c);
            float r[8], g[8];
            unpack8(rr[i], r);
            unpack8(rg[i], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sq = fmaf(r[e], r[e], sq);
                gr = fmaf(e < n ? g[e] * p.weight[c + e] : 0.f, r[e], gr);
            }
        }
        const float2 s = cta_sum(sq, gr, buf[turn]);
        const float rstd = 1.f / sqrtf(s.x / (float)p.D + p.eps), k = rstd * rstd * s.y / (float)p.D;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8, n = min(8, p.D - c);
            float r[8], g[8], o[8];
            unpack8(rr[i], r);
            unpack8(rg[i], g);
            if (p.dsum) unpack8(rs[i], o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gv = e < n ? g[e] * p.weight[c + e] : 0.f;
                o[e] = fmaf(rstd, gv - r[e] * k, p.dsum ? o[e] : 0.f);
                gw[i][e] = fmaf(g[e], r[e] * rstd, gw[i][e]);
            }
            store8<T, kVec>(static_cast<T *>(p.dr) + at + c, o, n);
        }
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < p.D) p.part[(long long)blockIdx.x * p.D + c + e] = gw[i][e];
    }
}

// dweight: the CTAs' parts in a fixed order, 32 channels a CTA.
__global__ void __launch_bounds__(1024) k_norm_bwd_sum(const float *part, int rows, int D, float *dweight) {
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < D)
        for (int r = threadIdx.y; r < rows; r += 32) a += part[(long long)r * D + c];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    a = red[threadIdx.x][threadIdx.y];  // warp y adds the 32 parts of channel y
#pragma unroll
    for (int m = 16; m >= 1; m /= 2) a += __shfl_xor_sync(0xffffffffu, a, m);
    if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < D) dweight[blockIdx.x * 32 + threadIdx.y] = a;
}

int norm_sizes(long long M, long long D, int dtype) {
    if (M < 0 || D < 1) return layer_fail(GDR_ERR_SHAPE, "norm: M must be >= 0 and D >= 1 (got %lld, %lld)", M, D);
    if (D > 8LL * kMaxThreads * kMaxIter) return layer_fail(GDR_ERR_SHAPE, "norm: D must be at most %d (got %lld)", 8 * kMaxThreads * kMaxIter, D);
    if (M >= (1LL << 31)) return layer_fail(GDR_ERR_SHAPE, "norm: too many rows");
    if (dtype != GDR_BF16 && dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "norm: unknown dtype %d", dtype);
    return GDR_OK;
}

// Two or more 8-channel vectors a thread where a row has them: the row's loads
// are in flight together.
void shape_of(long long D, int *threads, int *iter) {
    const int vecs = (int)((D + 7) / 8);
    int t = std::min(kMaxThreads, std::max(32, ((vecs + 1) / 2 + 31) / 32 * 32));
    *threads = t;
    const int need = (vecs + t - 1) / t;
    *iter = need <= 1 ? 1 : need <= 2 ? 2 : 4;
}

int bwd_ctas(long long M, long long D) {
    int threads, iter;
    shape_of(D, &threads, &iter);
    const long long per_sm = std::max(1, std::min(16, 1024 / threads));
    return (int)std::max(1LL, std::min(M, per_sm * layer_sms()));
}

template <typename F>
void norm_by_type(int dtype, int iter, bool vec, F f) {
    auto w = [&](auto t) {
        auto v = [&](auto l) {
            if (vec) f(t, l, std::true_type{}); else f(t, l, std::false_type{});
        };
        if (iter == 1) v(std::integral_constant<int, 1>{});
        else if (iter == 2) v(std::integral_constant<int, 2>{});
        else v(std::integral_constant<int, 4>{});
    };
    if (dtype == GDR_BF16) w(bf16_t{}); else w(float{});
}

}  // namespace

extern "C" {

int gdr_norm_fwd(const gdr_norm_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    if ((rc = norm_sizes(a->M, a->D, a->dtype))) return rc;
    if (a->M > 0 && !a->y == !a->q) return layer_fail(GDR_ERR_ARG, "norm: one of y and q is written");
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->M > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("weight", a->weight, true, 4)) ||
        (rc = layer_ptr("residual", a->residual, false, e)) || (rc = layer_ptr("sum", a->sum, any && a->residual, e)) ||
        (rc = layer_ptr("y", a->y, false, e)) || (rc = layer_ptr("scales", a->scales, any && a->q, 4)))
        return rc;
    if (!any) return GDR_OK;
    NormP p{a->x, a->residual, a->weight, a->sum, a->y, static_cast<uint8_t *>(a->q), a->scales, a->M, a->x_row, a->r_row, (int)a->D, a->eps};
    const long long q = a->dtype == GDR_BF16 ? 8 : 4;
    const bool vec = a->D % 8 == 0 && a->x_row % q == 0 && (!a->residual || a->r_row % q == 0) && multiple16(a->x) &&
                     multiple16(a->residual) && multiple16(a->sum) && multiple16(a->y) && multiple16(a->q);
    int threads, iter;
    shape_of(a->D, &threads, &iter);
    norm_by_type(a->dtype, iter, vec, [&](auto t, auto l, auto v) {
        using E = decltype(t);
        constexpr int I = decltype(l)::value;
        constexpr bool V = decltype(v)::value;
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (a->q) k_norm_fwd<E, I, V, true><<<(unsigned)a->M, threads, 0, st>>>(p);
        else k_norm_fwd<E, I, V, false><<<(unsigned)a->M, threads, 0, st>>>(p);
    });
    return layer_launched("norm forward");
}

size_t gdr_norm_bwd_workspace_size(long long M, long long D) {
    if (norm_sizes(M, D, GDR_BF16)) return 0;
    return (size_t)bwd_ctas(M, D) * D * 4;
}

int gdr_norm_bwd(const gdr_norm_bwd_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    if ((rc = norm_sizes(a->M, a->D, a->dtype))) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->M > 0;
    if ((rc = layer_ptr("r", a->r, any, e)) || (rc = layer_ptr("dy", a->dy, any, e)) || (rc = layer_ptr("dsum", a->dsum, false, e)) ||
        (rc = layer_ptr("weight", a->weight, true, 4)) || (rc = layer_ptr("dr", a->dr, any, e)) ||
        (rc = layer_ptr("dweight", a->dweight, true, 4)))
        return rc;
    if (!a->workspace) return layer_fail(GDR_ERR_WORKSPACE, "norm backward: workspace is null");
    if (!multiple16(a->workspace)) return layer_fail(GDR_ERR_ALIGN, "norm backward: workspace must be 16-byte aligned");
    if (a->workspace_bytes < gdr_norm_bwd_workspace_size(a->M, a->D))
        return layer_fail(GDR_ERR_WORKSPACE, "norm backward: workspace too small");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    NormBwdP p{a->r, a->dy, a->dsum, a->weight, a->dr, static_cast<float *>(a->workspace), a->dweight, a->M, (int)a->D, a->eps};
    const bool vec = a->D % 8 == 0 && multiple16(a->r) && multiple16(a->dy) && multiple16(a->dsum) && multiple16(a->dr);
    int threads, iter;
    shape_of(a->D, &threads, &iter);
    const int ctas = bwd_ctas(a->M, a->D);
    norm_by_type(a->dtype, iter, vec, [&](auto t, auto l, auto v) {
        k_norm_bwd<decltype(t), decltype(l)::value, decltype(v)::value><<<ctas, threads, 0, st>>>(p);
    });
    k_norm_bwd_sum<<<(unsigned)((a->D + 31) / 32), dim3(32, 32), 0, st>>>(p.part, ctas, (int)a->D, a->dweight);
    return layer_launched("norm backward");
}

}  // extern "C"
