// gdr_conv.cu -- short causal depthwise convolution along the tokens, forward,
// backward and single-token step.
//
//   pre_t = bias + sum_j w_j x_{t-W+1+j},  y = silu(pre)
//   dp_t = dy_t silu'(pre_t);  dx_s = sum_j w_j dp_{s+W-1-j} (same sequence);
//   dw_j = sum_t dp_t x_{t-W+1+j};  dbias = sum_t dp_t
//
// Bound by memory: the forward reads x and writes y once, the backward reads x
// and dy and writes dx.  A thread owns kE neighbouring channels and walks a run
// of tokens with the last W - 1 inputs in registers, so an input is read from
// memory once per run plus the W - 1 tokens of overlap between runs, which
// neighbouring threads' lines cover.  kE is 4 where rows allow it, else 2 or 1:
// neighbouring lanes always read neighbouring channels.  (Eight channels a
// thread cost the occupancy that hides the reads; as eight scalar reads a
// thread, for odd widths, they took 2.3 times as long.)  8192 x 4096, bf16,
// packed: forward 45 us (3.0 TB/s), backward 99 us with its sums (2.0 TB/s).
#include <cstring>
#include <initializer_list>

#include "gdr_layer.h"

namespace {

__device__ unsigned g_conv_status;

constexpr int kCols = 32;   // columns of kE channels of a CTA (one warp)
constexpr int kRuns = 8;    // token runs of a CTA (its warps), forward
constexpr int kRunsB = 4;   // and backward
constexpr int kAheadF = 8, kAheadB = 4;  // tokens read at a time (backward of 8192 x 4096: 99 us with 4, 121 with 8)

struct ConvP {
    const void *x, *h0, *dy, *dht;
    const float *weight, *bias;
    void *y, *ht, *dx, *dh0;
    float *part;  // [blocks along tokens][W + 1][D]
    Seqs seqs;
    long long x_row, x_batch;
    int T, D, silu, run;  // run: tokens of a thread
};

// kE neighbouring elements as they lie in memory, none where a thread has no channel.
template <typename T, int kE>
struct Raw;
template <>
struct Raw<bf16_t, 4> {
    uint2 r;
};
template <>
struct Raw<float, 4> {
    uint4 r;
};
template <>
struct Raw<bf16_t, 2> {
    uint32_t r;
};
template <>
struct Raw<float, 2> {
    uint2 r;
};
template <typename T>
struct Raw<T, 1> {
    T r;
};
template <typename T, int kE>
__device__ __forceinline__ Raw<T, kE> load_e(const T *p, bool on) {
    Raw<T, kE> v;
    memset(&v, 0, sizeof(v));
    if (on) v = *reinterpret_cast<const Raw<T, kE> *>(p);
    return v;
}
template <typename T, int kE>
__device__ __forceinline__ void unpack_e(const Raw<T, kE> &v, float (&f)[kE]) {
    if constexpr (kE == 1) {
        f[0] = to_f(v.r);
    } else {
        uint32_t w[sizeof(v) / 4];
        memcpy(w, &v, sizeof(v));
#pragma unroll
        for (int i = 0; i < (int)(sizeof(v) / 4); ++i) {
            if constexpr (sizeof(T) == 2) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                f[i] = __uint_as_float(w[i]);
            }
        }
    }
}
template <typename T, int kE>
__device__ __forceinline__ void store_e(T *p, const float (&f)[kE], bool on) {
    if (!on) return;
    if constexpr (kE == 1) {
        from_f(p[0], f[0]);
    } else {
        Raw<T, kE> v;
        uint32_t w[sizeof(v) / 4];
#pragma unroll
        for (int i = 0; i < (int)(sizeof(v) / 4); ++i) {
            if constexpr (sizeof(T) == 2) w[i] = pack2(f[2 * i], f[2 * i + 1]);
            else w[i] = __float_as_uint(f[i]);
        }
        memcpy(&v, w, sizeof(v));
        *reinterpret_cast<Raw<T, kE> *>(p) = v;
    }
}

// Inputs of a sequence before its first token: row i of its initial state.
template <typename T, int W, int kE>
__device__ __forceinline__ void init_row(const ConvP &p, int seq, int i, int ch, bool on, float (&f)[kE]) {
    if (!p.h0 || i < 0 || i >= W - 1) {
#pragma unroll
        for (int e = 0; e < kE; ++e) f[e] = 0.f;
        return;
    }
    unpack_e<T, kE>(load_e<T, kE>(static_cast<const T *>(p.h0) + ((long long)seq * (W - 1) + i) * p.D + ch, on), f);
}

// The input of token t (of the sequence starting at s0), t - s0 may be negative.
template <typename T, int W, int kE>
__device__ __forceinline__ void input_at(const ConvP &p, const T *x, int seq, int s0, int t, int ch, bool on, float (&f)[kE]) {
    if (t >= s0 && t >= 0) unpack_e<T, kE>(load_e<T, kE>(x + (long long)t * p.x_row + ch, on), f);
    else init_row<T, W, kE>(p, seq, t - s0 + W - 1, ch, on, f);
}

// The state that a sequence without tokens hands on is the one it got.
template <typename T, int W, int kE>
__device__ __forceinline__ void pass_on(const ConvP &p, int seq, int ch, bool on) {
    if (!p.ht) return;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        float f[kE];
        init_row<T, W, kE>(p, seq, i, ch, on, f);
        store_e<T, kE>(static_cast<T *>(p.ht) + ((long long)seq * (W - 1) + i) * p.D + ch, f, on);
    }
}

template <int W, int kE>
__device__ __forceinline__ void load_weights(const float *weight, const float *bias, int ch, bool on, float (&w)[W][kE],
                                             float (&b)[kE]) {
    if constexpr (kE >= 4) {  // the channels' taps are one aligned run of 4 kE W bytes
        float f[kE * W];
#pragma unroll
        for (int i = 0; i < kE * W / 4; ++i)
            *reinterpret_cast<float4 *>(f + 4 * i) = on ? reinterpret_cast<const float4 *>(weight + (long long)ch * W)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < kE; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = on ? weight[(long long)(ch + e) * W + j] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) b[e] = on && bias ? bias[ch + e] : 0.f;
}

template <typename T, int W, int kE>
__global__ void __launch_bounds__(kCols *kRuns) k_conv_fwd(const ConvP p) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_conv_status);
    const int ch = (blockIdx.x * kCols + threadIdx.x % kCols) * kE;
    const bool on = ch < p.D;
    if (!on) return;
    const int bz = blockIdx.z;
    const T *x = static_cast<const T *>(p.x) + bz * p.x_batch;
    T *y = static_cast<T *>(p.y) + (long long)bz * p.T * p.D;
    const int t0 = (blockIdx.y * kRuns + threadIdx.x / kCols) * p.run, t1 = min(t0 + p.run, p.T);
    const int sbase = p.seqs.cu ? 0 : bz;  // index of this row's first sequence
    if (t0 == 0 && p.seqs.cu)              // leading sequences without tokens
        for (int n = 0; n < p.seqs.n && p.seqs.bound(n + 1) <= 0; ++n) pass_on<T, W, kE>(p, n, ch, on);
    if (t0 >= t1) return;
    float w[W][kE], b[kE];
    load_weights<W, kE>(p.weight, p.bias, ch, on, w, b);
    int n = p.seqs.find(t0), s0 = p.seqs.bound(n), s1 = p.seqs.bound(n + 1);
    float hist[W - 1][kE];  // inputs of t - W + 1 .. t - 1
#pragma unroll
    for (int j = 0; j < W - 1; ++j) input_at<T, W, kE>(p, x, sbase + n, s0, t0 - (W - 1) + j, ch, on, hist[j]);
    for (int tb = t0; tb < t1; tb += kAheadF) {
        Raw<T, kE> raw[kAheadF];
#pragma unroll
        for (int i = 0; i < kAheadF; ++i)
            raw[i] = load_e<T, kE>(x + (long long)min(tb + i, p.T - 1) * p.x_row + ch, tb + i < t1);
#pragma unroll
        for (int i = 0; i < kAheadF; ++i) {
            const int t = tb + i;
            if (t >= t1) break;
            if (t >= s1 && n + 1 < p.seqs.count()) {  // the next sequence with tokens
                do {
                    ++n;
                    s0 = s1;
                    s1 = p.seqs.bound(n + 1);
                } while (s1 <= t && n + 1 < p.seqs.count());
#pragma unroll
                for (int j = 0; j < W - 1; ++j) init_row<T, W, kE>(p, sbase + n, j, ch, on, hist[j]);
            }
            float cur[kE], o[kE];
            unpack_e<T, kE>(raw[i], cur);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                float a = fmaf(w[W - 1][e], cur[e], b[e]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], hist[j][e], a);
                o[e] = p.silu ? a * sigmoidf(a) : a;
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) hist[j][e] = hist[j + 1][e];
                hist[W - 2][e] = cur[e];
            }
            store_e<T, kE>(y + (long long)t * p.D + ch, o, on);
            if (p.ht && t == s1 - 1) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    store_e<T, kE>(static_cast<T *>(p.ht) + ((long long)(sbase + n) * (W - 1) + j) * p.D + ch, hist[j], on);
                // the sequences without tokens that follow
                if (p.seqs.cu)
                    for (int m = n + 1; m < p.seqs.n && p.seqs.bound(m + 1) <= s1; ++m) pass_on<T, W, kE>(p, m, ch, on);
            }
        }
    }
}

// Walks the tokens of a run and the W - 1 after it.  Token t's dp belongs to
// the weights' gradient if t is in the run; it is added to the gradients of the
// W - 1 tokens before it (as far as they are of its sequence), which wait in
// registers, and completes that of token t - W + 1.  The CTA's runs are added
// through shared memory in order.
template <typename T, int W, int kE>
__global__ void __launch_bounds__(kCols *kRunsB) k_conv_bwd(const ConvP p) {
    __shared__ float red[kRunsB][kCols][kE];
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_conv_status);
    const int col = threadIdx.x % kCols, rn = threadIdx.x / kCols;
    const int ch = (blockIdx.x * kCols + col) * kE;
    const bool on = ch < p.D;
    const int bz = blockIdx.z;
    const T *x = static_cast<const T *>(p.x) + bz * p.x_batch;
    const T *dy = static_cast<const T *>(p.dy) + (long long)bz * p.T * p.D;
    T *dx = static_cast<T *>(p.dx) + (long long)bz * p.T * p.D;
    const int t0 = (blockIdx.y * kRunsB + rn) * p.run, t1 = min(t0 + p.run, p.T);
    const int sbase = p.seqs.cu ? 0 : bz;
    float dw[W + 1][kE];  // taps, bias
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < kE; ++e) dw[j][e] = 0.f;
    if (on && t0 < t1) {
        float w[W][kE], b[kE], hist[W - 1][kE], wait[W - 1][kE];  // wait[i]: gradient of token t - W + 1 + i
        load_weights<W, kE>(p.weight, p.bias, ch, on, w, b);
        int n = p.seqs.find(t0), s0 = p.seqs.bound(n), s1 = p.seqs.bound(n + 1);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            input_at<T, W, kE>(p, x, sbase + n, s0, t0 - (W - 1) + j, ch, on, hist[j]);
#pragma unroll
            for (int e = 0; e < kE; ++e) wait[j][e] = 0.f;
        }
        for (int tb = t0; tb < t1 + W - 1; tb += kAheadB) {
            Raw<T, kE> rx[kAheadB], rg[kAheadB];
#pragma unroll
            for (int i = 0; i < kAheadB; ++i) {
                const int t = min(tb + i, p.T - 1);
                const bool nl = tb + i < min(t1 + W - 1, p.T);
                rx[i] = load_e<T, kE>(x + (long long)t * p.x_row + ch, nl);
                rg[i] = load_e<T, kE>(dy + (long long)t * p.D + ch, nl);
            }
#pragma unroll
            for (int i = 0; i < kAheadB; ++i) {
                const int t = tb + i;
                if (t >= t1 + W - 1) break;
                float dp[kE];
                if (t < p.T) {
                    if (t >= s1 && n + 1 < p.seqs.count()) {
                        do {
                            ++n;
                            s0 = s1;
                            s1 = p.seqs.bound(n + 1);
                        } while (s1 <= t && n + 1 < p.seqs.count());
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) init_row<T, W, kE>(p, sbase + n, j, ch, on, hist[j]);
                    }
                    float cur[kE], g[kE];
                    unpack_e<T, kE>(rx[i], cur);
                    unpack_e<T, kE>(rg[i], g);
                    const bool mine = t < t1;
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        float a = fmaf(w[W - 1][e], cur[e], b[e]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], hist[j][e], a);
                        float d = g[e];
                        if (p.silu) {
                            const float s = sigmoidf(a);
                            d *= s * fmaf(a, 1.f - s, 1.f);
                        }
                        dp[e] = d;
                        if (mine) {
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(d, hist[j][e], dw[j][e]);
                            dw[W - 1][e] = fmaf(d, cur[e], dw[W - 1][e]);
                            dw[W][e] += d;
                        }
#pragma unroll
                        for (int j = 0; j + 1 < W - 1; ++j) hist[j][e] = hist[j + 1][e];
                        hist[W - 2][e] = cur[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < kE; ++e) dp[e] = 0.f;
                }
                const int old = t < p.T ? t - s0 : -1;  // tokens of this one's sequence before it
                float o[kE];
#pragma unroll
                for (int j = 0; j < W; ++j) {  // to the token W - 1 - j before this one
                    const bool same = W - 1 - j <= old;
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        // not the weight: another sequence's dp may be NaN or infinite
                        const float v = fmaf(w[j][e], same ? dp[e] : 0.f, j < W - 1 ? wait[j < W - 1 ? j : 0][e] : 0.f);
                        if (j == 0) o[e] = v;
                        else wait[j - 1 < 0 ? 0 : j - 1][e] = v;
                    }
                }
                const int k = W - 1 - (s1 - t);  // row of the final state that holds token t
                if (p.dht && t < p.T && k >= 0 && k < W - 1) {
                    float f[kE];
                    unpack_e<T, kE>(load_e<T, kE>(static_cast<const T *>(p.dht) + ((long long)(sbase + n) * (W - 1) + k) * p.D + ch, on), f);
#pragma unroll
                    for (int e = 0; e < kE; ++e) wait[W - 2][e] += f[e];
                }
                const int s = t - (W - 1);
                if (s >= t0 && s < t1) store_e<T, kE>(dx + (long long)s * p.D + ch, o, on);
            }
        }
    }
    float *part = p.part + ((long long)blockIdx.z * gridDim.y + blockIdx.y) * (W + 1) * p.D;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kE; ++e) red[rn][col][e] = dw[j][e];
        __syncthreads();
        for (int i = threadIdx.x; i < kCols * kE; i += kCols * kRunsB) {
            const int d = blockIdx.x * kCols * kE + i;
            if (d >= p.D) break;
            float a = 0.f;
#pragma unroll
            for (int r = 0; r < kRunsB; ++r) a += red[r][i / kE][i % kE];
            part[(long long)j * p.D + d] = a;
        }
    }
}

// Adds the blocks' partial sums in order.
template <int W>
__global__ void k_conv_bwd_sum(const float *part, int blocks, int D, float *dweight, float *dbias) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x, j = blockIdx.y;
    if (d >= D) return;
    float a = 0.f;
    for (int b = 0; b < blocks; ++b) a += part[((long long)b * (W + 1) + j) * D + d];
    if (j < W) dweight[(long long)d * W + j] = a;
    else if (dbias) dbias[d] = a;
}

// Gradient of the initial state: row i feeds the outputs of tokens 0 .. i
// (token u through tap i - u), and the final state of a sequence shorter than
// W - 1 tokens.
template <typename T, int W>
__global__ void k_conv_bwd_init(const ConvP p, int n_seqs) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    const int sq = blockIdx.y;
    if (d >= p.D) return;
    const int bz = p.seqs.cu ? 0 : sq, n = p.seqs.cu ? sq : 0;
    const int s0 = p.seqs.bound(n), len = max(0, p.seqs.bound(n + 1) - s0);
    const T *x = static_cast<const T *>(p.x) + bz * p.x_batch;
    const T *dy = static_cast<const T *>(p.dy) + (long long)bz * p.T * p.D;
    float in[2 * (W - 1)], g[W - 1], w[W];  // the initial inputs and the first tokens'
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = p.weight[(long long)d * W + j];
    const float b = p.bias ? p.bias[d] : 0.f;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        in[i] = p.h0 ? to_f(static_cast<const T *>(p.h0)[((long long)sq * (W - 1) + i) * p.D + d]) : 0.f;
        in[W - 1 + i] = i < len ? to_f(x[(long long)(s0 + i) * p.x_row + d]) : 0.f;
        g[i] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < W - 1; ++u) {
        if (u >= len) break;
        float a = b;
#pragma unroll
        for (int j = 0; j < W; ++j) a = fmaf(w[j], in[u + j], a);
        float dp = to_f(dy[(long long)(s0 + u) * p.D + d]);
        if (p.silu) {
            const float s = sigmoidf(a);
            dp *= s * fmaf(a, 1.f - s, 1.f);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            if (i >= u) g[i] = fmaf(w[i - u], dp, g[i]);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        if (p.dht && i >= len) g[i] += to_f(static_cast<const T *>(p.dht)[((long long)sq * (W - 1) + i - len) * p.D + d]);
        from_f(static_cast<T *>(p.dh0)[((long long)sq * (W - 1) + i) * p.D + d], g[i]);
    }
}

struct StepP {
    const void *x;
    const float *weight, *bias;
    void *state, *y;
    const int32_t *slots;
    long long x_row, n_slots;
    int rows, D, silu;
};

template <typename T, int W, int kE>
__global__ void k_conv_step(const StepP p) {
    const int ch = (blockIdx.x * blockDim.x + threadIdx.x) * kE, r = blockIdx.y;
    const bool on = ch < p.D;
    if (!on) return;
    const long long slot = p.slots ? p.slots[r] : r;
    T *y = static_cast<T *>(p.y) + (long long)r * p.D + ch;
    float o[kE];
    if (slot < 0 || slot >= p.n_slots) {
        if (slot >= 0 && threadIdx.x == 0) atomicOr(&g_conv_status, kStatusIndex);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = 0.f;
        store_e<T, kE>(y, o, on);
        return;
    }
    T *st = static_cast<T *>(p.state) + slot * (W - 1) * p.D + ch;
    Raw<T, kE> raw[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j] = load_e<T, kE>(st + (long long)j * p.D, on);
    raw[W - 1] = load_e<T, kE>(static_cast<const T *>(p.x) + r * p.x_row + ch, on);
    float w[W][kE];
    load_weights<W, kE>(p.weight, p.bias, ch, on, w, o);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float f[kE];
        unpack_e<T, kE>(raw[j], f);
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = fmaf(w[j][e], f[e], o[e]);
        if (j > 0) store_e<T, kE>(st + (long long)(j - 1) * p.D, f, on);
    }
    if (p.silu)
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] *= sigmoidf(o[e]);
    store_e<T, kE>(y, o, on);
}

// ---- host ------------------------------------------------------------------

int conv_sizes(long long B, long long T, long long D, int W, int dtype) {
    if (B < 1 || T < 0 || D < 1) return layer_fail(GDR_ERR_SHAPE, "conv: B and D must be >= 1 and T >= 0 (got %lld, %lld, %lld)", B, D, T);
    if (W < 2 || W > 4) return layer_fail(GDR_ERR_SHAPE, "conv: W must be 2, 3 or 4 (got %d)", W);
    if (T >= (1LL << 30) || D >= (1LL << 24) || B > 65535) return layer_fail(GDR_ERR_SHAPE, "conv: problem too large");
    if (dtype != GDR_BF16 && dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "conv: unknown dtype %d", dtype);
    return GDR_OK;
}

int conv_seqs(const gdr_conv_args *a, Seqs *s) {
    if (a->cu_seqlens ? (a->B != 1 || a->n_seqs < 1) : a->n_seqs != a->B)
        return layer_fail(GDR_ERR_SHAPE, "conv: packed sequences need B == 1 and n_seqs >= 1, a batch n_seqs == B");
    if (a->n_seqs > (1 << 24)) return layer_fail(GDR_ERR_SHAPE, "conv: too many sequences");
    s->cu = a->cu_seqlens;
    s->n = (int)a->n_seqs;
    s->T = (int)a->T;
    return GDR_OK;
}

// Channels of a thread: as many as rows and pointers allow to be moved at once.
int channels(long long D, std::initializer_list<long long> strides, int dtype, const float *weight,
             std::initializer_list<const void *> ptrs) {
    const int size = dtype == GDR_BF16 ? 2 : 4;
    auto ok = [&](int e) {
        if (D % e) return false;
        for (long long v : strides)
            if (v % e) return false;
        for (const void *p : ptrs)
            if (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(e * size - 1)) return false;
        return true;
    };
    return ok(4) && multiple16(weight) ? 4 : ok(2) ? 2 : 1;
}

// Tokens of a thread: long runs read less twice, short ones fill the SMs.
int run_length(long long B, long long T, long long D, int e, bool bwd) {
    const long long cols = (D + e * kCols - 1) / (e * kCols), runs = bwd ? kRunsB : kRuns;
    int run = bwd ? 64 : 32;
    auto blocks = [&] { return (T + run * runs - 1) / (run * runs); };
    while (run > 4 && cols * B * blocks() < 3LL * layer_sms()) run /= 2;
    while (blocks() > 65535) run *= 2;
    return run;
}

void fill(const gdr_conv_args *a, const Seqs &s, ConvP *p) {
    *p = ConvP{};
    p->x = a->x; p->h0 = a->h0; p->weight = a->weight; p->bias = a->bias; p->seqs = s;
    p->x_row = a->x_row; p->x_batch = a->x_batch; p->T = (int)a->T; p->D = (int)a->D; p->silu = a->silu;
}

template <typename F>
void by_type(int dtype, int W, int e, F f) {
    auto w = [&](auto t) {
        auto v = [&](auto c) {
            if (e == 4) f(t, c, std::integral_constant<int, 4>{});
            else if (e == 2) f(t, c, std::integral_constant<int, 2>{});
            else f(t, c, std::integral_constant<int, 1>{});
        };
        if (W == 2) v(std::integral_constant<int, 2>{});
        else if (W == 3) v(std::integral_constant<int, 3>{});
        else v(std::integral_constant<int, 4>{});
    };
    if (dtype == GDR_BF16) w(bf16_t{}); else w(float{});
}

long long bwd_blocks(long long B, long long T, long long D, int e) {
    const long long span = (long long)run_length(B, T, D, e, true) * kRunsB;
    return B * ((T + span - 1) / span);
}

}  // namespace

namespace gdr {
unsigned conv_take_status(cudaStream_t st) {
    unsigned v = 0, z = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_conv_status, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return 0x80000000u;
    cudaMemcpyToSymbolAsync(g_conv_status, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    if (cudaStreamSynchronize(st) != cudaSuccess) return 0x80000000u;
    return v;
}
}  // namespace gdr

extern "C" {

int gdr_conv_fwd(const gdr_conv_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    Seqs s;
    if ((rc = conv_sizes(a->B, a->T, a->D, a->W, a->dtype)) || (rc = conv_seqs(a, &s))) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->T > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("weight", a->weight, true, 4)) ||
        (rc = layer_ptr("bias", a->bias, false, 4)) || (rc = layer_ptr("h0", a->h0, false, e)) ||
        (rc = layer_ptr("y", a->y, any, e)) || (rc = layer_ptr("ht", a->ht, false, e)))
        return rc;
    if (!any && !a->ht) return GDR_OK;
    ConvP p;
    fill(a, s, &p);
    p.y = a->y;
    p.ht = a->ht;
    if (!any && !a->cu_seqlens) {  // a batch without tokens: treated as packed sequences without tokens
        const size_t bytes = (size_t)a->n_seqs * (a->W - 1) * a->D * e;
        const cudaError_t err = a->h0 ? cudaMemcpyAsync(a->ht, a->h0, bytes, cudaMemcpyDeviceToDevice, static_cast<cudaStream_t>(stream))
                                      : cudaMemsetAsync(a->ht, 0, bytes, static_cast<cudaStream_t>(stream));
        return err == cudaSuccess ? GDR_OK : layer_fail(GDR_ERR_CUDA, "conv: %s", cudaGetErrorString(err));
    }
    const int vec = channels(a->D, {a->x_row, a->x_batch}, a->dtype, a->weight, {a->x, a->y, a->h0, a->ht});
    p.run = run_length(a->B, a->T, a->D, vec, false);
    const long long span = (long long)p.run * kRuns;
    const dim3 grid((unsigned)((a->D + vec * kCols - 1) / (vec * kCols)), (unsigned)(any ? (a->T + span - 1) / span : 1), (unsigned)a->B);
    by_type(a->dtype, a->W, vec, [&](auto t, auto w, auto v) {
        k_conv_fwd<decltype(t), decltype(w)::value, decltype(v)::value><<<grid, kCols * kRuns, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return layer_launched("conv forward");
}

size_t gdr_conv_bwd_workspace_size(long long B, long long T, long long D, int W) {
    if (conv_sizes(B, T, D, W, GDR_BF16)) return 0;
    long long blocks = 0;  // whichever way the call's rows can be read
    for (int e : {4, 2, 1}) blocks = std::max(blocks, bwd_blocks(B, T, D, e));
    return (size_t)(blocks * (W + 1) * D * 4 + 16);
}

int gdr_conv_bwd(const gdr_conv_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    Seqs s;
    if ((rc = conv_sizes(a->B, a->T, a->D, a->W, a->dtype)) || (rc = conv_seqs(a, &s))) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->T > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("weight", a->weight, true, 4)) ||
        (rc = layer_ptr("bias", a->bias, false, 4)) || (rc = layer_ptr("h0", a->h0, false, e)) ||
        (rc = layer_ptr("dy", a->dy, any, e)) || (rc = layer_ptr("dht", a->dht, false, e)) ||
        (rc = layer_ptr("dx", a->dx, any, e)) || (rc = layer_ptr("dweight", a->dweight, true, 4)) ||
        (rc = layer_ptr("dbias", a->dbias, false, 4)) || (rc = layer_ptr("dh0", a->dh0, false, e)))
        return rc;
    if (!a->workspace) return layer_fail(GDR_ERR_WORKSPACE, "conv backward: workspace is null");
    if (!multiple16(a->workspace)) return layer_fail(GDR_ERR_ALIGN, "conv backward: workspace must be 16-byte aligned");
    if (a->workspace_bytes < gdr_conv_bwd_workspace_size(a->B, a->T, a->D, a->W))
        return layer_fail(GDR_ERR_WORKSPACE, "conv backward: workspace too small");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    ConvP p;
    fill(a, s, &p);
    p.dy = a->dy; p.dht = a->dht; p.dx = a->dx; p.dh0 = a->dh0;
    p.part = static_cast<float *>(a->workspace);
    const int vec = channels(a->D, {a->x_row, a->x_batch}, a->dtype, a->weight, {a->x, a->dy, a->dx, a->h0, a->dht});
    p.run = run_length(a->B, a->T, a->D, vec, true);
    const long long span = (long long)p.run * kRunsB;
    const dim3 grid((unsigned)((a->D + vec * kCols - 1) / (vec * kCols)), (unsigned)((a->T + span - 1) / span), (unsigned)a->B);
    const long long blocks = bwd_blocks(a->B, a->T, a->D, vec);
    if (a->dh0 && (a->n_seqs > 65535)) return layer_fail(GDR_ERR_SHAPE, "conv backward: dh0 of more than 65535 sequences");
    by_type(a->dtype, a->W, vec, [&](auto t, auto w, auto v) {
        using E = decltype(t);
        constexpr int W = decltype(w)::value;
        if (any) k_conv_bwd<E, W, decltype(v)::value><<<grid, kCols * kRunsB, 0, st>>>(p);
        k_conv_bwd_sum<W><<<dim3((unsigned)((a->D + 255) / 256), W + 1), 256, 0, st>>>(p.part, (int)blocks, (int)a->D, a->dweight, a->dbias);
        if (a->dh0) k_conv_bwd_init<E, W><<<dim3((unsigned)((a->D + 255) / 256), (unsigned)a->n_seqs), 256, 0, st>>>(p, (int)a->n_seqs);
    });
    return layer_launched("conv backward");
}

int gdr_conv_step(const gdr_conv_step_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    if ((rc = conv_sizes(1, a->rows, a->D, a->W, a->dtype))) return rc;
    if (a->rows > 65535) return layer_fail(GDR_ERR_SHAPE, "conv step: at most 65535 rows");
    if (a->n_slots < 0 || (!a->slots && a->n_slots < a->rows))
        return layer_fail(GDR_ERR_SHAPE, "conv step: %lld state slots for %lld rows", a->n_slots, a->rows);
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->rows > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("weight", a->weight, true, 4)) ||
        (rc = layer_ptr("bias", a->bias, false, 4)) || (rc = layer_ptr("state", a->state, any && a->n_slots > 0, e)) ||
        (rc = layer_ptr("slots", a->slots, false, 4)) || (rc = layer_ptr("y", a->y, any, e)))
        return rc;
    if (!any) return GDR_OK;
    StepP p{a->x, a->weight, a->bias, a->state, a->y, a->slots, a->x_row, a->n_slots, (int)a->rows, (int)a->D, a->silu};
    const int vec = channels(a->D, {a->x_row}, a->dtype, a->weight, {a->x, a->state, a->y});
    const int cols = (int)((a->D + vec - 1) / vec), threads = cols >= 128 ? 128 : (cols + 31) / 32 * 32;
    const dim3 grid((unsigned)((cols + threads - 1) / threads), (unsigned)a->rows);
    by_type(a->dtype, a->W, vec, [&](auto t, auto w, auto v) {
        k_conv_step<decltype(t), decltype(w)::value, decltype(v)::value><<<grid, threads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return layer_launched("conv step");
}

}  // extern "C"
