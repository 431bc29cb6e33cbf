// gdr_block.cu -- the norm after a block, with the block's gate, the residual
// stream and the norm before the next block; and its gradient.
//
//   n = x rx,  u = n w silu(g),  r = residual + scale u,  y = r rr w',
//   rx = (mean x^2 + eps)^-1/2,  rr = (mean r^2 + eps)^-1/2
// and backwards, with f = dy w' and du = scale dr_total:
//   dr_total = dr + rr (f - r rr^2 mean(f r)),  dresidual = dr_total,
//   b = du w silu(g),  dx = rx (b - n mean(b n)),  dg = du n w silu'(g),
//   dw = sum over rows of du n silu(g),  dw' = sum over rows of dy r rr.
// mean(b n) needs dr_total, which needs mean(f r) first; but with c = w silu(g) n
//   sum b n = scale (sum (dr + rr f) c - rr^3 mean(f r) sum r c),
// so that one round of three sums a row is enough (the forward keeps rx and rr).
//
// Bound by memory: a row is read once into the registers of its threads, reduced
// there, and written once.  Short rows (the heads of a mixer's output) share a
// warp: 16 or 32 lanes a row and shuffles alone; longer ones have a CTA.
#include "gdr_layer.h"

namespace {

constexpr int kMaxD = 16384, kWide = 1024, kNarrow = 512, kShort = 256;  // greatest row; threads of a CTA

struct BlockP {
    const void *x, *gate, *residual, *dr, *dy;
    const float *weight, *next;
    void *r, *y, *dx, *dgate, *dres;
    float *stats, *part;  // part: [CTAs, 2, D], the sums of dw and dw'
    long long M, x_row, x_outer, gate_row, gate_outer, res_row, res_outer;
    int D, lanes, inner;  // lanes: threads of a row
    float scale, eps;
};

// Where a row of x, gate and residual begins: `inner` heads of a token have a stride of their own.
struct Row {
    long long outer, head;
    __device__ __forceinline__ Row(long long row, int inner) {
        const unsigned r = (unsigned)row, n = (unsigned)inner, o = r / n;  // fewer than 2^31 rows
        outer = o;
        head = r - o * n;
    }
    __device__ __forceinline__ long long at(long long row_stride, long long outer_stride) const { return outer * outer_stride + head * row_stride; }
};

// A thread's kN elements of a row: vectors of eight (kV = 8: rows begin on
// 16-byte boundaries and hold whole vectors) or single elements, neighbouring
// ones in neighbouring threads.
template <typename T, int kV, int kN>
struct Part {
    struct Raw {
        Raw8<T> v[kV == 8 ? kN / 8 : 1];
        T s[kV == 8 ? 1 : kN];
    };
    static __device__ __forceinline__ int at(int i, int tid, int lanes) { return (i / kV * lanes + tid) * kV + i % kV; }
    static __device__ __forceinline__ void load(const T *row, int D, int tid, int lanes, Raw &raw) {
        if (kV == 8) {
#pragma unroll
            for (int i = 0; i < kN / 8; ++i) raw.v[i] = load8<T>(row + at(8 * i, tid, lanes), D - at(8 * i, tid, lanes));
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int c = at(i, tid, lanes);
                if (c < D) raw.s[i] = row[c]; else from_f(raw.s[i], 0.f);
            }
        }
    }
    static __device__ __forceinline__ void get(const Raw &raw, float (&f)[kN]) {
#pragma unroll
        for (int i = 0; i < kN; i += kV) {
            if (kV == 8) {
                float e[8];
                unpack8(raw.v[i / 8], e);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[i + k < kN ? i + k : 0] = e[k];
            } else {
                f[i] = to_f(raw.s[kV == 8 ? 0 : i]);
            }
        }
    }
    static __device__ __forceinline__ void store(T *row, int D, int tid, int lanes, const float (&f)[kN]) {
        if (kV == 8) {
#pragma unroll
            for (int i = 0; i < kN / 8; ++i) {
                float e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] = f[8 * i + k];
                store8<T, true>(row + at(8 * i, tid, lanes), e, D - at(8 * i, tid, lanes));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int c = at(i, tid, lanes);
                if (c < D) from_f(row[c], f[i]);
            }
        }
    }
};

// Sums over the threads of a row, each kept by all of them.  `buf` alternates
// between calls, so that one barrier a call is enough.
template <int kS, bool kCta>
__device__ __forceinline__ void row_sum(float (&v)[kS], int lanes, float (*buf)[32]) {
#pragma unroll
    for (int m = 16; m >= 1; m /= 2)
        if (kCta || m < lanes)
#pragma unroll
            for (int s = 0; s < kS; ++s) v[s] += __shfl_xor_sync(0xffffffffu, v[s], m);
    if (!kCta) return;
    const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0)
#pragma unroll
        for (int s = 0; s < kS; ++s) buf[s][threadIdx.x / 32] = v[s];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kS; ++s) v[s] = lane < warps ? buf[s][lane] : 0.f;
#pragma unroll
    for (int m = 16; m >= 1; m /= 2)
#pragma unroll
        for (int s = 0; s < kS; ++s) v[s] += __shfl_xor_sync(0xffffffffu, v[s], m);
}

// silu(v) and its derivative.
__device__ __forceinline__ float silu(float v) { return v * sigmoidf(v); }
__device__ __forceinline__ void silu_both(float v, float &f, float &df) {
    const float g = sigmoidf(v);
    f = v * g;
    df = g * fmaf(v, 1.f - g, 1.f);
}

// kCta: a row has the CTA, else `lanes` lanes of a warp.
template <typename T, int kV, int kN, int kThreads, bool kCta>
__global__ void __launch_bounds__(kThreads) k_block_fwd(const BlockP p) {
    using P = Part<T, kV, kN>;
    __shared__ float buf[2][1][32];
    const int tid = kCta ? threadIdx.x : threadIdx.x % p.lanes, D = p.D;
    const long long row = kCta ? blockIdx.x : (long long)blockIdx.x * (blockDim.x / p.lanes) + threadIdx.x / p.lanes;
    const bool on = row < p.M;  // lanes of rows past the last only join the shuffles
    typename P::Raw rx, rg, rr;
    const int len = on ? D : 0;
    const Row from(row, p.inner);
    P::load(static_cast<const T *>(p.x) + from.at(p.x_row, p.x_outer), len, tid, p.lanes, rx);
    if (p.gate) P::load(static_cast<const T *>(p.gate) + from.at(p.gate_row, p.gate_outer), len, tid, p.lanes, rg);
    if (p.residual) P::load(static_cast<const T *>(p.residual) + from.at(p.res_row, p.res_outer), len, tid, p.lanes, rr);
    float v[kN], sum[1] = {0.f};
    P::get(rx, v);
#pragma unroll
    for (int i = 0; i < kN; ++i) sum[0] = fmaf(v[i], v[i], sum[0]);
    row_sum<1, kCta>(sum, p.lanes, buf[0]);
    const float inv_x = 1.f / sqrtf(sum[0] / (float)D + p.eps);
    float g[kN], w[kN];
    typename Part<float, kV, kN>::Raw rw;
    Part<float, kV, kN>::load(p.weight, D, tid, p.lanes, rw);
    Part<float, kV, kN>::get(rw, w);
    if (p.gate) {
        P::get(rg, g);
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] *= silu(g[i]);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = p.scale * (v[i] * inv_x * w[i]);
    if (p.residual) {
        P::get(rr, g);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] += g[i];
    }
    P::store(static_cast<T *>(p.r) + row * D, len, tid, p.lanes, v);
    float inv_r = 0.f;
    if (p.next) {
        sum[0] = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (P::at(i, tid, p.lanes) < D) sum[0] = fmaf(v[i], v[i], sum[0]);
        row_sum<1, kCta>(sum, p.lanes, buf[1]);
        inv_r = 1.f / sqrtf(sum[0] / (float)D + p.eps);
        Part<float, kV, kN>::load(p.next, D, tid, p.lanes, rw);
        Part<float, kV, kN>::get(rw, w);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = v[i] * inv_r * w[i];
        P::store(static_cast<T *>(p.y) + row * D, len, tid, p.lanes, v);
    }
    if (p.stats && on && tid == 0) *reinterpret_cast<float2 *>(p.stats + 2 * row) = make_float2(inv_x, inv_r);
}

// A CTA takes every gridDim-th group of rows and keeps its part of the weights'
// gradients in registers.
template <typename T, int kV, int kN, int kThreads, bool kCta>
__global__ void __launch_bounds__(kThreads) k_block_bwd(const BlockP p) {
    using P = Part<T, kV, kN>;
    using W = Part<float, kV, kN>;
    __shared__ float buf[2][3][32];
    const int tid = kCta ? threadIdx.x : threadIdx.x % p.lanes, D = p.D;
    const int group = kCta ? 1 : blockDim.x / p.lanes;
    float gw[kN], gn[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) gw[i] = gn[i] = 0.f;
    int turn = 0;
    for (long long first = (long long)blockIdx.x * group; first < p.M; first += (long long)gridDim.x * group, turn ^= 1) {
        const long long row = first + (kCta ? 0 : threadIdx.x / p.lanes);
        const int len = row < p.M ? D : 0;
        typename P::Raw rx, rg, rr, ru, ry;
        const Row from(row, p.inner);
        P::load(static_cast<const T *>(p.x) + from.at(p.x_row, p.x_outer), len, tid, p.lanes, rx);
        if (p.gate) P::load(static_cast<const T *>(p.gate) + from.at(p.gate_row, p.gate_outer), len, tid, p.lanes, rg);
        if (p.dr) P::load(static_cast<const T *>(p.dr) + row * D, len, tid, p.lanes, ru);
        if (p.next) {
            if (p.residual) P::load(static_cast<const T *>(p.residual) + from.at(p.res_row, p.res_outer), len, tid, p.lanes, rr);
            if (p.dy) P::load(static_cast<const T *>(p.dy) + row * D, len, tid, p.lanes, ry);
        }
        const float2 inv = len ? *reinterpret_cast<const float2 *>(p.stats + 2 * row) : make_float2(0.f, 0.f);
        float n[kN], c[kN], u[kN], f[kN], r[kN];  // c: n w silu(gate)
        P::get(rx, n);
        typename W::Raw rw;
        W::load(p.weight, D, tid, p.lanes, rw);
        W::get(rw, c);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            n[i] *= inv.x;
            u[i] = 0.f;
        }
        if (p.gate) {
            P::get(rg, r);
#pragma unroll
            for (int i = 0; i < kN; ++i) c[i] *= silu(r[i]);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) c[i] *= n[i];
        if (p.dr) P::get(ru, u);
        float s[3] = {0.f, 0.f, 0.f};
        if (p.next) {
#pragma unroll
            for (int i = 0; i < kN; ++i) r[i] = 0.f;
            if (p.residual) P::get(rr, r);
            if (p.dy) {
                P::get(ry, f);
            } else {
#pragma unroll
                for (int i = 0; i < kN; ++i) f[i] = 0.f;
            }
            typename W::Raw rn;
            W::load(p.next, D, tid, p.lanes, rn);
            float w2[kN];
            W::get(rn, w2);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                r[i] = fmaf(p.scale, c[i], r[i]);
                gn[i] = fmaf(f[i], r[i] * inv.y, gn[i]);
                f[i] *= w2[i];
                s[0] = fmaf(f[i], r[i], s[0]);
                u[i] = fmaf(inv.y, f[i], u[i]);
                s[2] = fmaf(r[i], c[i], s[2]);
            }
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) s[1] = fmaf(u[i], c[i], s[1]);
        row_sum<3, kCta>(s, p.lanes, buf[turn]);
        const float k = p.next ? inv.y * inv.y * inv.y * s[0] / (float)D : 0.f;
        const float mean = p.scale * (s[1] - k * s[2]) / (float)D;  // of b n
        if (p.next) {
#pragma unroll
            for (int i = 0; i < kN; ++i) u[i] = fmaf(-k, r[i], u[i]);
            if (p.dres) P::store(static_cast<T *>(p.dres) + row * D, len, tid, p.lanes, u);
        }
        W::load(p.weight, D, tid, p.lanes, rw);
        float w[kN];
        W::get(rw, w);
        if (p.gate) {
            float g[kN];
            P::get(rg, g);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                float sl, ds;
                silu_both(g[i], sl, ds);
                u[i] *= p.scale;
                gw[i] = fmaf(u[i] * n[i], sl, gw[i]);
                f[i] = inv.x * fmaf(u[i] * w[i], sl, -n[i] * mean);
                g[i] = u[i] * n[i] * w[i] * ds;
            }
            P::store(static_cast<T *>(p.dgate) + row * D, len, tid, p.lanes, g);
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                u[i] *= p.scale;
                gw[i] = fmaf(u[i], n[i], gw[i]);
                f[i] = inv.x * (u[i] * w[i] - n[i] * mean);
            }
        }
        P::store(static_cast<T *>(p.dx) + row * D, len, tid, p.lanes, f);
    }
    float *to = p.part + (long long)blockIdx.x * 2 * D;
    if (kCta) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int c = P::at(i, tid, p.lanes);
            if (c < D) {
                to[c] = gw[i];
                to[D + c] = gn[i];
            }
        }
    } else {
        // the groups' parts in order
        __shared__ float sums[2][kCta ? 1 : 32 * kN];
        for (int v = 0; v < group; ++v) {
            if ((int)threadIdx.x / p.lanes == v)
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const int c = P::at(i, tid, p.lanes);
                    sums[0][c] = v ? sums[0][c] + gw[i] : gw[i];
                    sums[1][c] = v ? sums[1][c] + gn[i] : gn[i];
                }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            to[c] = sums[0][c];
            to[D + c] = sums[1][c];
        }
    }
}

// dw and dw' (blockIdx.y): the CTAs' parts in a fixed order, 32 channels a CTA.
__global__ void __launch_bounds__(1024) k_block_sum(const float *part, int rows, int D, float *dweight, float *dnext) {
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float *to = blockIdx.y ? dnext : dweight;
    float a = 0.f;
    if (c < D)
        for (int r = threadIdx.y; r < rows; r += 32) a += part[((long long)r * 2 + blockIdx.y) * D + c];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    a = red[threadIdx.x][threadIdx.y];  // warp y adds the 32 parts of channel y
#pragma unroll
    for (int m = 16; m >= 1; m /= 2) a += __shfl_xor_sync(0xffffffffu, a, m);
    if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < D) to[blockIdx.x * 32 + threadIdx.y] = a;
}

// ---- host ------------------------------------------------------------------

struct BlockPlan {
    int n, lanes, threads;  // elements a thread, threads a row, threads a CTA
    bool cta;
    int rows() const { return cta ? 1 : threads / lanes; }
};
// Eight elements a thread for short rows, sixteen (two vectors on their way) for others.
BlockPlan block_plan(long long D) {
    if (D <= 128) return {8, 16, kShort, false};
    if (D <= 256) return {8, 32, kShort, false};
    if (D <= 512) return {16, 32, kShort, false};
    const int t = (int)((D + 511) / 512 * 32);
    return {16, t, t, true};
}

int block_ctas(long long M, long long D) {
    const BlockPlan pl = block_plan(D);
    const long long per_sm = std::max(1, std::min(8, 768 / pl.threads)), need = (M + pl.rows() - 1) / pl.rows();
    return (int)std::max(1LL, std::min(need, per_sm * layer_sms()));
}

int block_common(const gdr_block_norm_args *a, bool bwd) {
    int rc;
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    if (a->M < 0 || a->D < 1) return layer_fail(GDR_ERR_SHAPE, "block norm: M must be >= 0 and D >= 1 (got %lld, %lld)", a->M, a->D);
    if (a->D > kMaxD) return layer_fail(GDR_ERR_SHAPE, "block norm: D must be at most %d (got %lld)", kMaxD, a->D);
    if (a->M >= (1LL << 31)) return layer_fail(GDR_ERR_SHAPE, "block norm: too many rows");
    if (a->inner < 1 || a->inner >= (1LL << 31) || a->M % a->inner)
        return layer_fail(GDR_ERR_SHAPE, "block norm: M (%lld) must be a multiple of inner (%lld), which is at least 1", a->M, a->inner);
    if (a->dtype != GDR_BF16 && a->dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "block norm: unknown dtype %d", a->dtype);
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->M > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("gate", a->gate, false, e)) || (rc = layer_ptr("residual", a->residual, false, e)) ||
        (rc = layer_ptr("weight", a->weight, true, 4)) || (rc = layer_ptr("next_weight", a->next_weight, false, 4)))
        return rc;
    if (bwd)
        return (rc = layer_ptr("dr", a->dr, false, e)) || (rc = layer_ptr("dy", a->dy, false, e)) || (rc = layer_ptr("stats", a->stats, any, 8)) ||
               (rc = layer_ptr("dx", a->dx, any, e)) || (rc = layer_ptr("dgate", a->dgate, any && a->gate, e)) ||
               (rc = layer_ptr("dresidual", a->dresidual, any && a->residual && a->next_weight, e)) || (rc = layer_ptr("dweight", a->dweight, true, 4)) ||
               (rc = layer_ptr("dnext_weight", a->dnext_weight, a->next_weight != nullptr, 4)) ? rc : GDR_OK;
    return (rc = layer_ptr("r", a->r, any, e)) || (rc = layer_ptr("y", a->y, any && a->next_weight, e)) || (rc = layer_ptr("stats", a->stats, false, 8)) ? rc : GDR_OK;
}

// Whether rows of every tensor are whole vectors on 16-byte boundaries.
bool block_vec(const gdr_block_norm_args *a) {
    for (long long v : {a->D, a->x_row, a->x_outer, a->gate ? a->gate_row : 0, a->gate ? a->gate_outer : 0, a->residual ? a->residual_row : 0,
                        a->residual ? a->residual_outer : 0})
        if (v % 8) return false;
    for (const void *p : {a->x, a->gate, a->residual, a->dr, a->dy, static_cast<const void *>(a->weight), static_cast<const void *>(a->next_weight),
                          static_cast<const void *>(a->r), static_cast<const void *>(a->y), static_cast<const void *>(a->dx),
                          static_cast<const void *>(a->dgate), static_cast<const void *>(a->dresidual)})
        if (!multiple16(p)) return false;
    return true;
}

BlockP block_fill(const gdr_block_norm_args *a, const BlockPlan &pl) {
    BlockP p{};
    p.x = a->x; p.gate = a->gate; p.residual = a->residual; p.dr = a->dr; p.dy = a->dy;
    p.weight = a->weight; p.next = a->next_weight;
    p.r = a->r; p.y = a->y; p.dx = a->dx; p.dgate = a->dgate; p.dres = a->next_weight ? a->dresidual : nullptr;
    p.stats = a->stats; p.part = static_cast<float *>(a->workspace);
    p.M = a->M; p.x_row = a->x_row; p.gate_row = a->gate_row; p.res_row = a->residual_row;
    p.x_outer = a->x_outer; p.gate_outer = a->gate_outer; p.res_outer = a->residual_outer;
    p.D = (int)a->D; p.lanes = pl.lanes; p.inner = (int)a->inner;
    p.scale = a->scale; p.eps = a->eps;
    return p;
}

// f(type, vector, elements, most threads, a CTA a row)
template <typename F>
void block_by_type(int dtype, bool vec, const BlockPlan &pl, F f) {
    auto w = [&](auto t, auto v) {
        using std::integral_constant;
        if (!pl.cta && pl.n == 8) f(t, v, integral_constant<int, 8>{}, integral_constant<int, kShort>{}, std::false_type{});
        else if (!pl.cta) f(t, v, integral_constant<int, 16>{}, integral_constant<int, kShort>{}, std::false_type{});
        else if (pl.threads <= kNarrow) f(t, v, integral_constant<int, 16>{}, integral_constant<int, kNarrow>{}, std::true_type{});
        else f(t, v, integral_constant<int, 16>{}, integral_constant<int, kWide>{}, std::true_type{});
    };
    auto k = [&](auto t) {
        if (vec) w(t, std::integral_constant<int, 8>{}); else w(t, std::integral_constant<int, 1>{});
    };
    if (dtype == GDR_BF16) k(bf16_t{}); else k(float{});
}

}  // namespace

extern "C" {

int gdr_block_norm_fwd(const gdr_block_norm_args *a, void *stream) {
    const int rc = block_common(a, false);
    if (rc || a->M == 0) return rc;
    const BlockPlan pl = block_plan(a->D);
    const BlockP p = block_fill(a, pl);
    const unsigned ctas = (unsigned)((a->M + pl.rows() - 1) / pl.rows());
    block_by_type(a->dtype, block_vec(a), pl, [&](auto t, auto v, auto n, auto th, auto cta) {
        k_block_fwd<decltype(t), decltype(v)::value, decltype(n)::value, decltype(th)::value, decltype(cta)::value>
            <<<ctas, pl.threads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return layer_launched("block norm forward");
}

size_t gdr_block_norm_bwd_workspace_size(long long M, long long D) {
    if (M < 0 || D < 1 || D > kMaxD || M >= (1LL << 31)) return 0;
    return ((size_t)block_ctas(M, D) * 2 * D * 4 + 15) & ~size_t(15);
}

int gdr_block_norm_bwd(const gdr_block_norm_args *a, void *stream) {
    const int rc = block_common(a, true);
    if (rc) return rc;
    if (!a->workspace) return layer_fail(GDR_ERR_WORKSPACE, "block norm backward: workspace is null");
    if (!multiple16(a->workspace)) return layer_fail(GDR_ERR_ALIGN, "block norm backward: workspace must be 16-byte aligned");
    if (a->workspace_bytes < gdr_block_norm_bwd_workspace_size(a->M, a->D))
        return layer_fail(GDR_ERR_WORKSPACE, "block norm backward: workspace too small");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const BlockPlan pl = block_plan(a->D);
    const BlockP p = block_fill(a, pl);
    const int ctas = block_ctas(a->M, a->D);
    block_by_type(a->dtype, block_vec(a), pl, [&](auto t, auto v, auto n, auto th, auto cta) {
        k_block_bwd<decltype(t), decltype(v)::value, decltype(n)::value, decltype(th)::value, decltype(cta)::value><<<ctas, pl.threads, 0, st>>>(p);
    });
    k_block_sum<<<dim3((unsigned)((a->D + 31) / 32), a->next_weight ? 2 : 1), dim3(32, 32), 0, st>>>(p.part, ctas, p.D, a->dweight, a->dnext_weight);
    return layer_launched("block norm backward");
}

}  // extern "C"
