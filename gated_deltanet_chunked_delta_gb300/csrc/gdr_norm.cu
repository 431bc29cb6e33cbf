// gdr_norm.cu -- root-mean-square norm of a residual stream, in the input's
// type or in 8 bits with scales, and its gradient.
//
//   r = x + residual (rounded to the stored type), y = r rstd w,  rstd = (mean r^2 + eps)^-1/2
//   dr = rstd (w dy - r rstd^2 mean(w dy r)) + dsum,  dw = sum over rows of dy r rstd
//
// Bound by memory: a row is read once into the registers of one CTA, reduced
// once, and written once (16384 x 4096 in 8 bits: 74 us, 6.4 TB/s).  The
// gradient of 8192 x 4096 takes 70 us with its sums, 3.8 TB/s: a CTA reads a row
// only after the row before it has been reduced and written, so that nothing is
// on its way meanwhile.  The norm is taken of r as it is stored, so that
// the gradient, which reads the stored r, is that of what was computed.
//
// Accesses are of eight elements.  Where a row's length is not a multiple of
// eight, rows begin inside one; there (kShift) a thread's eight channels are
// those of an aligned piece of memory.  A row's first and last piece then
// reaches into its neighbours: it is read whole all the same where it lies
// inside the tensor and cut in registers (element by element in the first and
// last rows of a tensor that begins or ends in it), and written element by
// element.
#include "gdr_layer.h"
#include "gdr_piece.h"

namespace {

constexpr int kMaxThreads = 512, kMaxIter = 4;
constexpr int kMaxD = 8 * kMaxThreads * kMaxIter;
// A shifted row of more than kMaxD - 7 channels may lie in one piece more than
// kMaxThreads x kMaxIter: it takes five pieces a thread (kIter = 5).
constexpr int kWideThreads = 416;
static_assert(8 * kWideThreads * (kMaxIter + 1) >= kMaxD + 7, "the widest row");
constexpr int max_threads(int iter) { return iter > kMaxIter ? kWideThreads : kMaxThreads; }

struct NormP {
    const void *x, *residual;
    const float *weight;
    void *sum, *y;
    uint8_t *q;
    float *scales;
    long long M, x_row, r_row;
    int D;
    float eps;
    bool x_vec, r_vec, o_vec;  // kShift: pieces of x, residual and the outputs are aligned
};

// Channels c .. c + 7 of a row of D, of which [lo, hi) exist.
struct Piece {
    int c, lo, hi;
    __device__ __forceinline__ Piece(int c_, int D) : c(c_), lo(max(0, -c_)), hi(min(8, D - c_)) {}
    __device__ __forceinline__ bool whole() const { return lo == 0 && hi == 8; }
};
// A piece of the i-th of M rows from base, `stride` elements apart (vec: pieces are aligned).
template <typename T, bool kShift>
__device__ __forceinline__ Raw8<T> load_piece(const T *base, long long i, long long M, int D, long long stride, const Piece &k, bool vec) {
    const T *row = base + i * stride;
    if (!kShift) return load8<T>(row + k.c, k.hi);
    if (vec && (k.whole() || (k.hi > 0 && gdr::piece_inside(i, k.c, M, D, stride)))) return load8<T>(row + k.c, 8);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e >= k.lo && e < k.hi ? to_f(row[k.c + e]) : 0.f;
    Raw8<T> r;
    pack8(f, r);
    return r;
}
template <bool kShift, typename R>
__device__ __forceinline__ void unpack_piece(const R &r, const Piece &k, float (&f)[8]) {
    unpack8(r, f);
    if (kShift && !k.whole())
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < k.lo || e >= k.hi) f[e] = 0.f;
}
template <typename T, bool kShift>
__device__ __forceinline__ void store_piece(T *row, const Piece &k, const float (&f)[8], bool vec) {
    if (!kShift) {
        store8<T, true>(row + k.c, f, k.hi);
    } else if (k.whole() && vec) {
        store8<T, true>(row + k.c, f, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= k.lo && e < k.hi) from_f(row[k.c + e], f[e]);
    }
}
template <int kBy>
__device__ __forceinline__ void pick8(const float (&win)[16], float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = win[8 - kBy + e];
}
// The weights of a piece.  Shifted ones are cut from sixteen aligned ones (the
// shift is the row's, the same for all threads): eight scalar reads a thread
// touch eight times the lines.
template <bool kShift>
__device__ __forceinline__ void load_weight(const float *w, const Piece &k, int D, float (&f)[8]) {
    const int base = (k.c + 7) & ~7, shift = base - k.c;  // a multiple of eight
    if (!kShift && k.hi > 0) {
        *reinterpret_cast<float4 *>(f) = *reinterpret_cast<const float4 *>(w + k.c);
        *reinterpret_cast<float4 *>(f + 4) = *reinterpret_cast<const float4 *>(w + k.c + 4);
    } else if (kShift && base >= 8 && base + 8 <= D && !(reinterpret_cast<uintptr_t>(w) & 15u)) {
        float win[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(win + 4 * i) = *reinterpret_cast<const float4 *>(w + base - 8 + 4 * i);
        switch (shift) {
            case 0: pick8<0>(win, f); break;
            case 1: pick8<1>(win, f); break;
            case 2: pick8<2>(win, f); break;
            case 3: pick8<3>(win, f); break;
            case 4: pick8<4>(win, f); break;
            case 5: pick8<5>(win, f); break;
            case 6: pick8<6>(win, f); break;
            default: pick8<7>(win, f); break;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = kShift && e >= k.lo && e < k.hi ? w[k.c + e] : 0.f;
    }
}

// Sum of (up to two) values over the CTA; `buf` alternates between calls so
// that one barrier a call is enough.
static_assert(kMaxThreads <= 16 * 32, "cta_sum adds the sums of 16 warps");
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

// y / scale, rounded once: the product with the rounded reciprocal and one
// correction by its remainder, which is exact (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  Without
// the correction values on the border of two 8-bit ones can take the wrong
// side; a division in its place takes 84 us for 16384 x 4096, this 74.  (Shifted
// rows keep two scales a thread: at three CTAs of 512 threads an SM, 40 registers,
// that spills and costs 7 %.)
struct Divisor {
    float inv, neg;
    __device__ __forceinline__ explicit Divisor(float scale) : inv(1.f / scale) {
        neg = inv > 0.f ? -scale : 0.f;  // an infinite scale has no remainder: finite / inf is 0
    }
};
__device__ __forceinline__ void divide2(float &a, float &b, const Divisor &by_a, const Divisor &by_b) {
    const f32x2 y = mk2(a, b), inv = mk2(by_a.inv, by_b.inv), q = mul2(y, inv);
    un2(fma2(fma2(q, mk2(by_a.neg, by_b.neg), y), inv, q), a, b);
}

template <typename T, int kIter, bool kShift, bool kQuant>
__global__ void __launch_bounds__(max_threads(kIter), kIter >= 4 ? 1 : kShift && kQuant ? 2 : 3) k_norm_fwd(const NormP p) {
    __shared__ float2 buf[32];
    __shared__ unsigned tops[kShift && kQuant ? 128 : 1];  // greatest magnitudes of the row's blocks, as ordered bits
    const long long row = blockIdx.x, out = row * p.D;
    const int shift = kShift ? (int)(out & 7) : 0;
    const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.residual);
    if (kShift && kQuant)
        for (int i = threadIdx.x; i < 128; i += blockDim.x) tops[i] = 0;
    auto piece = [&](int i) { return Piece((int)(threadIdx.x + i * blockDim.x) * 8 - shift, p.D); };
    Raw8<T> rx[kIter], rr[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const Piece k = piece(i);
        rx[i] = load_piece<T, kShift>(x, row, p.M, p.D, p.x_row, k, p.x_vec);
        if (res) rr[i] = load_piece<T, kShift>(res, row, p.M, p.D, p.r_row, k, p.r_vec);
    }
    float v[kIter][8], sq = 0.f;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        unpack_piece<kShift>(rx[i], piece(i), v[i]);
        if (res) {
            float f[8];
            unpack_piece<kShift>(rr[i], piece(i), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] += f[e];
            store_piece<T, kShift>(static_cast<T *>(p.sum) + out, piece(i), v[i], p.o_vec);
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
        const Piece k = piece(i);
        float w[8];
        load_weight<kShift>(p.weight, k, p.D, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = e >= k.lo && e < k.hi ? v[i][e] * rstd * w[e] : 0.f;
        if (!kQuant) {
            store_piece<T, kShift>(static_cast<T *>(p.y) + out, k, v[i], p.o_vec);
        } else if (kShift) {
            // a piece may lie in two blocks of 128, a warp's pieces in three
            const int b0 = max(k.c, 0) / 128;
            unsigned mine[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned bits = __float_as_uint(fabsf(v[i][e]));  // NaN above all
                if ((k.c + e) / 128 == b0 || k.c + e < 0) mine[0] = max(mine[0], bits);
                else mine[1] = max(mine[1], bits);
            }
            const int first = max(__shfl_sync(0xffffffffu, k.c, 0), 0) / 128;
#pragma unroll
            for (int b = 0; b < 3; ++b) {
                const unsigned top = __reduce_max_sync(0xffffffffu, first + b == b0 ? mine[0] : first + b == b0 + 1 ? mine[1] : 0u);
                if (threadIdx.x % 32 == 0 && top && first + b < 128) atomicMax(&tops[first + b], top);
            }
        } else {
            // 16 neighbouring threads hold a block of 128 channels
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(v[i][e]));
#pragma unroll
            for (int m = 8; m >= 1; m /= 2) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
            const float scale = max_nan(top, 1e-30f) / 448.f;
            if (k.hi <= 0) continue;
            if (threadIdx.x % 16 == 0) p.scales[(long long)(k.c / 128) * p.M + row] = scale;
            const Divisor by(scale);
#pragma unroll
            for (int e = 0; e < 8; e += 2) divide2(v[i][e], v[i][e + 1], by, by);
            *reinterpret_cast<uint2 *>(p.q + out + k.c) =
                make_uint2(e4m3x4(v[i][0], v[i][1], v[i][2], v[i][3]), e4m3x4(v[i][4], v[i][5], v[i][6], v[i][7]));
        }
    }
    if (!kShift || !kQuant) return;
    __syncthreads();
    auto scale_of = [&](int b) { return max_nan(__uint_as_float(tops[b]), 1e-30f) / 448.f; };
    for (int b = threadIdx.x; b < (p.D + 127) / 128; b += blockDim.x) p.scales[(long long)b * p.M + row] = scale_of(b);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const Piece k = piece(i);
        if (k.hi <= 0) continue;
        const int b0 = max(k.c, 0) / 128, b1 = min(k.c + 7, p.D - 1) / 128;
        const Divisor by0(scale_of(b0)), by1(scale_of(b1));
        const int cut = b1 * 128 - k.c;  // the first channel of the second block
#pragma unroll
        for (int e = 0; e < 8; e += 2) divide2(v[i][e], v[i][e + 1], e >= cut ? by1 : by0, e + 1 >= cut ? by1 : by0);
        const uint32_t lo = e4m3x4(v[i][0], v[i][1], v[i][2], v[i][3]), hi = e4m3x4(v[i][4], v[i][5], v[i][6], v[i][7]);
        if (k.whole() && p.o_vec) {
            *reinterpret_cast<uint2 *>(p.q + out + k.c) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= k.lo && e < k.hi) p.q[out + k.c + e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
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
    bool vec;  // kShift: pieces are aligned
};

// A CTA takes every gridDim-th row and keeps its part of dweight in registers
// (kShift: gridDim is a multiple of eight, so that its rows begin alike).
template <typename T, int kIter, bool kShift>
__global__ void __launch_bounds__(max_threads(kIter)) k_norm_bwd(const NormBwdP p) {
    __shared__ float2 buf[2][32];
    const int shift = kShift ? (int)(((long long)blockIdx.x * p.D) & 7) : 0;
    auto piece = [&](int i) { return Piece((int)(threadIdx.x + i * blockDim.x) * 8 - shift, p.D); };
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
            const Piece k = piece(i);
            rr[i] = load_piece<T, kShift>(static_cast<const T *>(p.r), row, p.M, p.D, p.D, k, p.vec);
            rg[i] = load_piece<T, kShift>(static_cast<const T *>(p.dy), row, p.M, p.D, p.D, k, p.vec);
            if (p.dsum) rs[i] = load_piece<T, kShift>(static_cast<const T *>(p.dsum), row, p.M, p.D, p.D, k, p.vec);
        }
        float sq = 0.f, gr = 0.f;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            float r[8], g[8], w[8];
            unpack_piece<kShift>(rr[i], piece(i), r);
            unpack_piece<kShift>(rg[i], piece(i), g);
            load_weight<kShift>(p.weight, piece(i), p.D, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sq = fmaf(r[e], r[e], sq);
                gr = fmaf(g[e] * w[e], r[e], gr);
            }
        }
        const float2 s = cta_sum(sq, gr, buf[turn]);
        const float rstd = 1.f / sqrtf(s.x / (float)p.D + p.eps), m = rstd * rstd * s.y / (float)p.D;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const Piece k = piece(i);
            float r[8], g[8], o[8], w[8];
            unpack_piece<kShift>(rr[i], k, r);
            unpack_piece<kShift>(rg[i], k, g);
            if (p.dsum) unpack8(rs[i], o);
            load_weight<kShift>(p.weight, k, p.D, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = fmaf(rstd, g[e] * w[e] - r[e] * m, p.dsum ? o[e] : 0.f);
                gw[i][e] = fmaf(g[e], r[e] * rstd, gw[i][e]);
            }
            store_piece<T, kShift>(static_cast<T *>(p.dr) + at, k, o, p.vec);
        }
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const Piece k = piece(i);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= k.lo && e < k.hi) p.part[(long long)blockIdx.x * p.D + k.c + e] = gw[i][e];
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
    if (D > kMaxD) return layer_fail(GDR_ERR_SHAPE, "norm: D must be at most %d (got %lld)", kMaxD, D);
    if (M >= (1LL << 31)) return layer_fail(GDR_ERR_SHAPE, "norm: too many rows");
    if (dtype != GDR_BF16 && dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "norm: unknown dtype %d", dtype);
    return GDR_OK;
}

// Two or more 8-channel vectors a thread where a row has them: the row's loads
// are in flight together.
void shape_of(long long D, bool shift, int *threads, int *iter) {
    const int vecs = (int)((D + (shift ? 14 : 7)) / 8);  // a shifted row may need a piece more
    const int t = std::min(kMaxThreads, std::max(32, ((vecs + 1) / 2 + 31) / 32 * 32)), need = (vecs + t - 1) / t;
    *threads = need > kMaxIter ? kWideThreads : t;
    *iter = need <= 1 ? 1 : need <= 2 ? 2 : need <= kMaxIter ? 4 : 5;
}

int bwd_ctas(long long M, long long D) {
    int threads, iter;
    shape_of(D, true, &threads, &iter);
    const long long per_sm = std::max(1, std::min(16, 768 / threads));
    return (int)((std::max(1LL, std::min(M, per_sm * layer_sms())) + 7) / 8 * 8);
}

template <typename F>
void norm_by_type(int dtype, int iter, bool shift, F f) {
    auto w = [&](auto t) {
        auto v = [&](auto l) {
            if (shift) f(t, l, std::true_type{}); else f(t, l, std::false_type{});
        };
        if (iter == 5) return f(t, std::integral_constant<int, 5>{}, std::true_type{});  // shifted rows only
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
    NormP p{a->x, a->residual, a->weight, a->sum, a->y, static_cast<uint8_t *>(a->q), a->scales, a->M, a->x_row, a->r_row, (int)a->D, a->eps, true, true, true};
    // rows of a tensor begin as the outputs' do
    auto alike = [&](const void *t, long long row) { return !t || (multiple16(t) && (row - a->D) % 8 == 0); };
    p.x_vec = alike(a->x, a->x_row);
    p.r_vec = alike(a->residual, a->r_row);
    p.o_vec = multiple16(a->sum) && multiple16(a->y) && multiple16(a->q);
    const bool shift = a->D % 8 || !p.x_vec || !p.r_vec || !p.o_vec || !multiple16(a->weight);
    int threads, iter;
    shape_of(a->D, shift, &threads, &iter);
    norm_by_type(a->dtype, iter, shift, [&](auto t, auto l, auto v) {
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
    NormBwdP p{a->r, a->dy, a->dsum, a->weight, a->dr, static_cast<float *>(a->workspace), a->dweight, a->M, (int)a->D, a->eps, true};
    p.vec = multiple16(a->r) && multiple16(a->dy) && multiple16(a->dsum) && multiple16(a->dr);
    const bool shift = a->D % 8 || !p.vec || !multiple16(a->weight);
    int threads, iter;
    shape_of(a->D, shift, &threads, &iter);
    const int ctas = bwd_ctas(a->M, a->D);
    norm_by_type(a->dtype, iter, shift, [&](auto t, auto l, auto v) {
        k_norm_bwd<decltype(t), decltype(l)::value, decltype(v)::value><<<ctas, threads, 0, st>>>(p);
    });
    k_norm_bwd_sum<<<(unsigned)((a->D + 31) / 32), dim3(32, 32), 0, st>>>(p.part, ctas, (int)a->D, a->dweight);
    return layer_launched("norm backward");
}

}  // extern "C"
