// gdr_conv.cu -- short causal depthwise convolution along the tokens, forward,
// backward and single-token step.
//
//   pre_t = bias + sum_j w_j x_{t-W+1+j},  y = silu(pre)
//   dp_t = dy_t silu'(pre_t);  dx_s = sum_j w_j dp_{s+W-1-j} (same sequence);
//   dw_j = sum_t dp_t x_{t-W+1+j};  dbias = sum_t dp_t
//
// Bound by memory: the forward reads x and writes y once, the backward reads x
// and dy and writes dx.  A thread owns eight neighbouring channels (16-byte
// accesses in bf16) and walks a run of tokens with the last W - 1 inputs in
// registers, so an input is read from memory once per run plus the W - 1
// tokens of overlap between runs, which neighbouring threads' lines cover.
#include "gdr_layer.h"

namespace {

__device__ unsigned g_conv_status;

constexpr int kCols = 32;   // 8-channel columns of a CTA (one warp)
constexpr int kRuns = 8;    // token runs of a CTA (its warps)

struct ConvP {
    const void *x, *h0, *dy, *dht;
    const float *weight, *bias;
    void *y, *ht, *dx, *dh0;
    float *part;  // [blocks along tokens][W + 1][D]
    Seqs seqs;
    long long x_row, x_batch;
    int T, D, silu, run;  // run: tokens of a thread
};

// Inputs of a sequence before its first token: row i of its initial state.
template <typename T, int W, bool kVec>
__device__ __forceinline__ void init_row(const ConvP &p, int seq, int i, int ch, int nv, float (&f)[8]) {
    if (!p.h0 || i < 0 || i >= W - 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
        return;
    }
    unpack8(load8<T, kVec>(static_cast<const T *>(p.h0) + ((long long)seq * (W - 1) + i) * p.D + ch, nv), f);
}

// The input of token t (of the sequence starting at s0), t - s0 may be negative.
template <typename T, int W, bool kVec>
__device__ __forceinline__ void input_at(const ConvP &p, const T *x, int seq, int s0, int t, int ch, int nv, float (&f)[8]) {
    if (t >= s0 && t >= 0) unpack8(load8<T, kVec>(x + (long long)t * p.x_row + ch, nv), f);
    else init_row<T, W, kVec>(p, seq, t - s0 + W - 1, ch, nv, f);
}

// The state that a sequence without tokens hands on is the one it got.
template <typename T, int W, bool kVec>
__device__ __forceinline__ void pass_on(const ConvP &p, int seq, int ch, int nv) {
    if (!p.ht) return;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        float f[8];
        init_row<T, W, kVec>(p, seq, i, ch, nv, f);
        store8<T, kVec>(static_cast<T *>(p.ht) + ((long long)seq * (W - 1) + i) * p.D + ch, f, nv);
    }
}

template <int W, bool kVec>
__device__ __forceinline__ void load_weights(const float *weight, const float *bias, int ch, int nv, float (&w)[W][8],
                                             float (&b)[8]) {
    if constexpr (kVec) {  // eight channels' taps are one aligned run of 32 W bytes
        float f[8 * W];
#pragma unroll
        for (int i = 0; i < 2 * W; ++i)
            *reinterpret_cast<float4 *>(f + 4 * i) = reinterpret_cast<const float4 *>(weight + (long long)ch * W)[i];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            b[e] = bias ? bias[ch + e] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
        }
    } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        b[e] = e < nv && bias ? bias[ch + e] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = e < nv ? weight[(long long)(ch + e) * W + j] : 0.f;
    }
    }
}

template <typename T, int W, bool kVec>
__global__ void __launch_bounds__(kCols *kRuns) k_conv_fwd(const ConvP p) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_conv_status);
    const int ch = (blockIdx.x * kCols + threadIdx.x % kCols) * 8, nv = min(8, p.D - ch);
    if (nv <= 0) return;
    const int bz = blockIdx.z;
    const T *x = static_cast<const T *>(p.x) + bz * p.x_batch;
    T *y = static_cast<T *>(p.y) + (long long)bz * p.T * p.D;
    const int t0 = (blockIdx.y * kRuns + threadIdx.x / kCols) * p.run, t1 = min(t0 + p.run, p.T);
    const int sbase = p.seqs.cu ? 0 : bz;  // index of this row's first sequence
    if (t0 == 0 && p.seqs.cu)              // leading sequences without tokens
        for (int n = 0; n < p.seqs.n && p.seqs.bound(n + 1) <= 0; ++n) pass_on<T, W, kVec>(p, n, ch, nv);
    if (t0 >= t1) return;
    float w[W][8], b[8];
    load_weights<W, kVec>(p.weight, p.bias, ch, nv, w, b);
    int n = p.seqs.find(t0), s0 = p.seqs.bound(n), s1 = p.seqs.bound(n + 1);
    float hist[W - 1][8];  // inputs of t - W + 1 .. t - 1
#pragma unroll
    for (int j = 0; j < W - 1; ++j) input_at<T, W, kVec>(p, x, sbase + n, s0, t0 - (W - 1) + j, ch, nv, hist[j]);
    constexpr int kAhead = 4;
    for (int tb = t0; tb < t1; tb += kAhead) {
        Raw8<T> raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            raw[i] = load8<T, kVec>(x + (long long)min(tb + i, p.T - 1) * p.x_row + ch, tb + i < t1 ? nv : 0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = tb + i;
            if (t >= t1) break;
            if (t >= s1 && n + 1 < p.seqs.count()) {  // the next sequence with tokens
                do {
                    ++n;
                    s0 = s1;
                    s1 = p.seqs.bound(n + 1);
                } while (s1 <= t && n + 1 < p.seqs.count());
#pragma unroll
                for (int j = 0; j < W - 1; ++j) init_row<T, W, kVec>(p, sbase + n, j, ch, nv, hist[j]);
            }
            float cur[8], o[8];
            unpack8(raw[i], cur);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a = fmaf(w[W - 1][e], cur[e], b[e]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], hist[j][e], a);
                o[e] = p.silu ? a * sigmoidf(a) : a;
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) hist[j][e] = hist[j + 1][e];
                hist[W - 2][e] = cur[e];
            }
            store8<T, kVec>(y + (long long)t * p.D + ch, o, nv);
            if (p.ht && t == s1 - 1) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    store8<T, kVec>(static_cast<T *>(p.ht) + ((long long)(sbase + n) * (W - 1) + j) * p.D + ch, hist[j], nv);
                // the sequences without tokens that follow
                if (p.seqs.cu)
                    for (int m = n + 1; m < p.seqs.n && p.seqs.bound(m + 1) <= s1; ++m) pass_on<T, W, kVec>(p, m, ch, nv);
            }
        }
    }
}

// Walks the tokens of a run and the W - 1 after it: token t's dp belongs to
// the weights' gradient if t is in the run, and the W-th last token's dx is
// then complete.  The CTA's runs are added through shared memory in order.
template <typename T, int W, bool kVec>
__global__ void __launch_bounds__(kCols *kRuns) k_conv_bwd(const ConvP p) {
    __shared__ float red[kRuns][kCols][8];
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_conv_status);
    const int col = threadIdx.x % kCols, rn = threadIdx.x / kCols;
    const int ch = (blockIdx.x * kCols + col) * 8, nv = min(8, p.D - ch);
    const int bz = blockIdx.z;
    const T *x = static_cast<const T *>(p.x) + bz * p.x_batch;
    const T *dy = static_cast<const T *>(p.dy) + (long long)bz * p.T * p.D;
    T *dx = static_cast<T *>(p.dx) + (long long)bz * p.T * p.D;
    const int t0 = (blockIdx.y * kRuns + rn) * p.run, t1 = min(t0 + p.run, p.T);
    const int sbase = p.seqs.cu ? 0 : bz;
    float dw[W + 1][8];  // taps, bias
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.f;
    if (nv > 0 && t0 < t1) {
        float w[W][8], b[8], hist[W - 1][8], dps[W][8];  // dps[i]: dp of token t - W + 1 + i
        int seq_of[W], end_of[W];
        load_weights<W, kVec>(p.weight, p.bias, ch, nv, w, b);
        int n = p.seqs.find(t0), s0 = p.seqs.bound(n), s1 = p.seqs.bound(n + 1);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<T, W, kVec>(p, x, sbase + n, s0, t0 - (W - 1) + j, ch, nv, hist[j]);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            seq_of[j] = end_of[j] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) dps[j][e] = 0.f;
        }
        for (int t = t0; t < t1 + W - 1; ++t) {
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) {
                seq_of[j] = seq_of[j + 1];
                end_of[j] = end_of[j + 1];
#pragma unroll
                for (int e = 0; e < 8; ++e) dps[j][e] = dps[j + 1][e];
            }
            if (t < p.T) {
                float cur[8], g[8];
                unpack8(load8<T, kVec>(x + (long long)t * p.x_row + ch, nv), cur);
                unpack8(load8<T, kVec>(dy + (long long)t * p.D + ch, nv), g);
                if (t >= s1 && n + 1 < p.seqs.count()) {
                    do {
                        ++n;
                        s0 = s1;
                        s1 = p.seqs.bound(n + 1);
                    } while (s1 <= t && n + 1 < p.seqs.count());
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) init_row<T, W, kVec>(p, sbase + n, j, ch, nv, hist[j]);
                }
                seq_of[W - 1] = sbase + n;
                end_of[W - 1] = s1;
                const bool mine = t < t1;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float a = fmaf(w[W - 1][e], cur[e], b[e]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], hist[j][e], a);
                    float d = g[e];
                    if (p.silu) {
                        const float s = sigmoidf(a);
                        d *= s * fmaf(a, 1.f - s, 1.f);
                    }
                    dps[W - 1][e] = d;
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
                for (int e = 0; e < 8; ++e) dps[W - 1][e] = 0.f;
            }
            const int s = t - (W - 1);
            if (s >= t0 && s < t1) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i)  // dp of token s + i times tap W - 1 - i
                    if (s + i < end_of[0])
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = fmaf(w[W - 1 - i][e], dps[i][e], o[e]);
                const int k = W - 1 - (end_of[0] - s);  // row of the final state that holds token s
                if (p.dht && k >= 0 && k < W - 1) {
                    float f[8];
                    unpack8(load8<T, kVec>(static_cast<const T *>(p.dht) + ((long long)seq_of[0] * (W - 1) + k) * p.D + ch, nv), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += f[e];
                }
                store8<T, kVec>(dx + (long long)s * p.D + ch, o, nv);
            }
        }
    }
    float *part = p.part + ((long long)blockIdx.z * gridDim.y + blockIdx.y) * (W + 1) * p.D;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[rn][col][e] = dw[j][e];
        __syncthreads();
        const int c = threadIdx.x >> 3, e = threadIdx.x & 7;  // 256 threads, 256 channels
        const int d = (blockIdx.x * kCols + c) * 8 + e;
        if (d < p.D) {
            float a = 0.f;
#pragma unroll
            for (int r = 0; r < kRuns; ++r) a += red[r][c][e];
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

template <typename T, int W, bool kVec>
__global__ void k_conv_step(const StepP p) {
    const int ch = (blockIdx.x * blockDim.x + threadIdx.x) * 8, nv = min(8, p.D - ch), r = blockIdx.y;
    if (nv <= 0) return;
    const long long slot = p.slots ? p.slots[r] : r;
    T *y = static_cast<T *>(p.y) + (long long)r * p.D + ch;
    float o[8];
    if (slot < 0 || slot >= p.n_slots) {
        if (slot >= 0 && threadIdx.x == 0) atomicOr(&g_conv_status, kStatusIndex);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
        store8<T, kVec>(y, o, nv);
        return;
    }
    T *st = static_cast<T *>(p.state) + slot * (W - 1) * p.D + ch;
    Raw8<T> raw[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j] = load8<T, kVec>(st + (long long)j * p.D, nv);
    raw[W - 1] = load8<T, kVec>(static_cast<const T *>(p.x) + r * p.x_row + ch, nv);
    float w[W][8];
    load_weights<W, kVec>(p.weight, p.bias, ch, nv, w, o);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float f[8];
        unpack8(raw[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(w[j][e], f[e], o[e]);
        if (j > 0) store8<T, kVec>(st + (long long)(j - 1) * p.D, f, nv);
    }
    if (p.silu)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= sigmoidf(o[e]);
    store8<T, kVec>(y, o, nv);
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

// Tokens of a thread: long runs read less twice, short ones fill the SMs.
int run_length(long long B, long long T, long long D, bool bwd) {
    const long long cols = (D + 8 * kCols - 1) / (8 * kCols);
    int run = bwd ? 64 : 16;
    while (run > 4 && cols * B * ((T + (long long)run * kRuns - 1) / ((long long)run * kRuns)) < 2LL * layer_sms()) run /= 2;
    while ((T + (long long)run * kRuns - 1) / ((long long)run * kRuns) > 65535) run *= 2;
    return run;
}

bool vec_ok(long long D, long long row, long long batch, int dtype) {
    const long long q = dtype == GDR_BF16 ? 8 : 4;
    return D % 8 == 0 && row % q == 0 && batch % q == 0;
}

void fill(const gdr_conv_args *a, const Seqs &s, ConvP *p) {
    *p = ConvP{};
    p->x = a->x; p->h0 = a->h0; p->weight = a->weight; p->bias = a->bias; p->seqs = s;
    p->x_row = a->x_row; p->x_batch = a->x_batch; p->T = (int)a->T; p->D = (int)a->D; p->silu = a->silu;
}

template <typename F>
void by_type(int dtype, int W, bool vec, F f) {
    auto w = [&](auto t) {
        auto v = [&](auto c) {
            if (vec) f(t, c, std::true_type{}); else f(t, c, std::false_type{});
        };
        if (W == 2) v(std::integral_constant<int, 2>{});
        else if (W == 3) v(std::integral_constant<int, 3>{});
        else v(std::integral_constant<int, 4>{});
    };
    if (dtype == GDR_BF16) w(bf16_t{}); else w(float{});
}

long long bwd_blocks(long long B, long long T, long long D) {
    const long long span = (long long)run_length(B, T, D, true) * kRuns;
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
    p.run = run_length(a->B, a->T, a->D, false);
    const bool vec = vec_ok(a->D, a->x_row, a->x_batch, a->dtype) && multiple16(a->x) && multiple16(a->weight) && multiple16(a->y) &&
                     multiple16(a->h0) && multiple16(a->ht);
    const long long span = (long long)p.run * kRuns;
    const dim3 grid((unsigned)((a->D + 8 * kCols - 1) / (8 * kCols)), (unsigned)(any ? (a->T + span - 1) / span : 1), (unsigned)a->B);
    by_type(a->dtype, a->W, vec, [&](auto t, auto w, auto v) {
        k_conv_fwd<decltype(t), decltype(w)::value, decltype(v)::value><<<grid, kCols * kRuns, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return layer_launched("conv forward");
}

size_t gdr_conv_bwd_workspace_size(long long B, long long T, long long D, int W) {
    if (conv_sizes(B, T, D, W, GDR_BF16)) return 0;
    return (size_t)(bwd_blocks(B, T, D) * (W + 1) * D * 4 + 16);
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
    p.run = run_length(a->B, a->T, a->D, true);
    const bool vec = vec_ok(a->D, a->x_row, a->x_batch, a->dtype) && multiple16(a->x) && multiple16(a->weight) && multiple16(a->dy) &&
                     multiple16(a->dx) && multiple16(a->h0) && multiple16(a->dht);
    const long long span = (long long)p.run * kRuns;
    const dim3 grid((unsigned)((a->D + 8 * kCols - 1) / (8 * kCols)), (unsigned)((a->T + span - 1) / span), (unsigned)a->B);
    const long long blocks = bwd_blocks(a->B, a->T, a->D);
    if (a->dh0 && (a->n_seqs > 65535)) return layer_fail(GDR_ERR_SHAPE, "conv backward: dh0 of more than 65535 sequences");
    by_type(a->dtype, a->W, vec, [&](auto t, auto w, auto v) {
        using E = decltype(t);
        constexpr int W = decltype(w)::value;
        if (any) k_conv_bwd<E, W, decltype(v)::value><<<grid, kCols * kRuns, 0, st>>>(p);
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
    const bool vec = vec_ok(a->D, a->x_row, 0, a->dtype) && multiple16(a->x) && multiple16(a->weight) && multiple16(a->state) && multiple16(a->y);
    const int cols = (int)((a->D + 7) / 8), threads = cols >= 128 ? 128 : (cols + 31) / 32 * 32;
    const dim3 grid((unsigned)((cols + threads - 1) / threads), (unsigned)a->rows);
    by_type(a->dtype, a->W, vec, [&](auto t, auto w, auto v) {
        k_conv_step<decltype(t), decltype(w)::value, decltype(v)::value><<<grid, threads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return layer_launched("conv step");
}

}  // extern "C"
