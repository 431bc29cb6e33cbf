// gdr_ssm.cu -- selective state space scan (diagonal transition), forward,
// backward and single-token step.
//
// Per sequence, channel d and state n (s = softplus(dt + dt_bias)):
//     h_t = e^{s_t A} h_{t-1} + s_t x_t B_t,  u_t = C_t . h_t + skip x_t,  y_t = u_t silu(z_t)
// and backwards, with du = dy silu(z) and e_t the gradient of h_t:
//     e_t = C_t du_t + e^{s_{t+1} A} e_{t+1},  f_t = e_t h_{t-1} e^{s_t A},
//     dx = s (e . B) + skip du,  ds = x (e . B) + f . A,  dA = sum f s,
//     dB = sum_d e s x,  dC = sum_d h du,  dz = dy u silu'(z).
//
// Bound by arithmetic: T D N exponentials a pass (the special-function units)
// and about five fp32 operations beside each, against 8 bytes of bf16 a (t, d).
// So a state stays in registers (four neighbouring states of a channel a
// thread, pairs in packed fp32 instructions), the per-(t, d) functions
// (softplus, silu) are evaluated once, by the thread that loads the element,
// and the sums over a channel's lanes are transposed (each lane ends with one
// token's sum) instead of repeated in every lane.
//
// Where sequences x channels leave SMs idle the tokens are cut into segments:
// a summary pass gives each segment's end state from a zero start, and as the
// transition over a segment is e^{A sum s}, a segment's start state follows
// from the summaries before it (back to the last sequence start) in the main
// pass itself.  The backward does the same from the other end; it takes its
// states from the forward's checkpoints, one before every 16th token.
#include "gdr_layer.h"

namespace {

__device__ unsigned g_ssm_status;

constexpr int kThreads = 128;
constexpr int kTile = 32;              // tokens staged at a time (forward)
constexpr int kBack = GDR_SSM_STRIDE;  // tokens of a backward tile, and between checkpoints

struct SsmP {
    const void *x, *dt, *z, *Bm, *Cm, *dy;
    const float *A, *skip, *dt_bias, *h0, *dht;
    void *y, *dx, *ddt, *dz, *dB, *dC;
    float *ht, *states, *dA, *dskip, *ddt_bias, *dh0;
    float *sum_h, *sum_s;  // segment summaries [B, S, D, N], [B, S, D]
    float *pB, *pC, *pA, *pD;  // partial gradients: [tiles, B T, N] twice, [B S, D, N], [B S, 2, D]
    Seqs seqs;
    long long x_row, x_batch, dt_row, dt_batch, z_row, z_batch, b_row, b_batch, c_row, c_batch;
    int B, T, D, G, Dg, tiles, S, seg_len, softplus;  // tiles: channel tiles of a group
};

// Sum over the lanes of a channel of kL values each: lane q ends with the sum of value q.
template <int kL>
__device__ __forceinline__ float lane_sums(float (&v)[kL], int q) {
#pragma unroll
    for (int step = kL / 2; step >= 1; step /= 2) {
        const bool up = q & step;
#pragma unroll
        for (int i = 0; i < step; ++i) {
            const float keep = up ? v[i + step] : v[i], send = up ? v[i] : v[i + step];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
        }
    }
    return v[0];
}
// Sum over the kC channels of a warp (lanes kL apart) of four states at kC
// tokens: the lanes of channel c end with token c's sums in v[0].
template <int kL, int kC>
__device__ __forceinline__ void channel_sums(float (&v)[kC][4], int c) {
#pragma unroll
    for (int step = kC / 2; step >= 1; step /= 2) {
        const bool up = c & step;
#pragma unroll
        for (int i = 0; i < step; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float keep = up ? v[i + step][k] : v[i][k], send = up ? v[i][k] : v[i + step][k];
                v[i][k] = keep + __shfl_xor_sync(0xffffffffu, send, step * kL);
            }
    }
}

struct State {  // four neighbouring states
    f32x2 a, b;
};
__device__ __forceinline__ State zero_state() { return State{mk2(0.f, 0.f), mk2(0.f, 0.f)}; }
__device__ __forceinline__ State load_state(const float *p) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    return State{mk2(v.x, v.y), mk2(v.z, v.w)};
}
__device__ __forceinline__ void store_state(float *p, const State &s) {
    float4 v;
    un2(s.a, v.x, v.y);
    un2(s.b, v.z, v.w);
    *reinterpret_cast<float4 *>(p) = v;
}
__device__ __forceinline__ float dot(const State &x, const State &y) {
    float lo, hi;
    un2(fma2(x.a, y.a, mul2(x.b, y.b)), lo, hi);
    return lo + hi;
}
// e^{s A} of four states, A2 = A log2 e
__device__ __forceinline__ State decay(const State &A2, float s) {
    const f32x2 s2 = mk2(s, s);
    float a, b, c, d;
    un2(mul2(A2.a, s2), a, b);
    un2(mul2(A2.b, s2), c, d);
    return State{mk2(ex2f(a), ex2f(b)), mk2(ex2f(c), ex2f(d))};
}
__device__ __forceinline__ State advance(const State &a, const State &h, float in, const State &Bt) {
    const f32x2 i2 = mk2(in, in);
    return State{fma2(a.a, h.a, mul2(i2, Bt.a)), fma2(a.b, h.b, mul2(i2, Bt.b))};
}

// Where a thread works: channel d (states n0 .. n0 + 3), whether it exists.
template <int kL>
struct Place {
    static constexpr int kCh = kThreads / kL, kN = 4 * kL;
    int g, gt, c0, nch, ch, q, d, n0;
    bool on;
    __device__ __forceinline__ explicit Place(const SsmP &p) {
        gt = blockIdx.x;
        g = gt / p.tiles;
        c0 = g * p.Dg + (gt % p.tiles) * kCh;
        nch = min(kCh, (g + 1) * p.Dg - c0);
        ch = threadIdx.x / kL;
        q = threadIdx.x % kL;
        on = ch < nch;
        d = c0 + (on ? ch : 0);
        n0 = 4 * q;
    }
    __device__ __forceinline__ long long at(long long row, const SsmP &p) const { return (row * p.D + d) * kN + n0; }
};

template <int kL>
__device__ __forceinline__ State start_state(const SsmP &p, const Place<kL> &w, int seq) {
    return p.h0 && w.on ? load_state(p.h0 + w.at(seq, p)) : zero_state();
}
// The state (or its gradient) that a sequence without tokens hands on.
template <int kL>
__device__ __forceinline__ void pass_state(const SsmP &p, const Place<kL> &w, const float *from, float *to, int seq) {
    if (to && w.on) store_state(to + w.at(seq, p), from ? load_state(from + w.at(seq, p)) : zero_state());
}

// Segment boundary state from the summaries of segments j0, j0 + step, ..
// up to (not including) seg: v <- e^{A sum s_j} v + summary_j.
template <int kL>
__device__ __forceinline__ State chain(const SsmP &p, const Place<kL> &w, const State &A2, int b, int j0, int seg, int step) {
    State v = zero_state();
    if (!w.on) return v;
    for (int j = j0; j != seg; j += step) {
        const long long row = (long long)b * p.S + j;
        const State a = decay(A2, p.sum_s[row * p.D + w.d]);
        const State e = load_state(p.sum_h + w.at(row, p));
        v = State{fma2(a.a, v.a, e.a), fma2(a.b, v.b, e.b)};
    }
    return v;
}

template <int kL>
__device__ __forceinline__ State load_A2(const SsmP &p, const Place<kL> &w, State *A) {
    State a = w.on ? load_state(p.A + w.at(0, p)) : zero_state();
    if (A) *A = a;
    const f32x2 k = mk2(kLog2e, kLog2e);
    return State{mul2(a.a, k), mul2(a.b, k)};
}

// Forward, or (kSum) the segments' summaries.
template <typename T, int kL, bool kVec, bool kSum>
__global__ void __launch_bounds__(kThreads) k_ssm_fwd(const SsmP p) {
    using W = Place<kL>;
    constexpr int kCh = W::kCh, kN = W::kN;
    constexpr int kVecs = kTile * kCh / 8, kNV = (kVecs + kThreads - 1) / kThreads;
    constexpr int kBV = kTile * kN / 8, kNB = ((kSum ? 1 : 2) * kBV + kThreads - 1) / kThreads;
    constexpr int kPad = 32 / kL < 4 ? 4 : 32 / kL;
    __shared__ __align__(16) float2 s_in[kTile][kCh];  // s, s x
    __shared__ __align__(16) float s_B[kTile][kN], s_C[kSum ? 1 : kTile][kN];
    __shared__ __align__(16) float s_y[kSum ? 1 : kTile][kCh + kPad];
    __shared__ __align__(16) float s_bias[kCh], s_skip[kCh];
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_ssm_status);
    const W w(p);
    const int tid = threadIdx.x, seg = blockIdx.y, b = blockIdx.z;
    const int ts = seg * p.seg_len, te = min(ts + p.seg_len, p.T);
    const int sbase = p.seqs.cu ? 0 : b;
    const T *x = static_cast<const T *>(p.x) + b * p.x_batch + w.c0;
    const T *dt = static_cast<const T *>(p.dt) + b * p.dt_batch + w.c0;
    const T *z = p.z ? static_cast<const T *>(p.z) + b * p.z_batch + w.c0 : nullptr;
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.b_batch + (long long)w.g * kN;
    const T *Cm = static_cast<const T *>(p.Cm) + b * p.c_batch + (long long)w.g * kN;
    T *y = static_cast<T *>(p.y) + (long long)b * p.T * p.D + w.c0;
    for (int i = tid; i < kCh; i += kThreads) {
        s_bias[i] = p.dt_bias && i < w.nch ? p.dt_bias[w.c0 + i] : 0.f;
        s_skip[i] = p.skip && i < w.nch ? p.skip[w.c0 + i] : 0.f;
    }
    __syncthreads();  // the first tile is staged with them
    const State A2 = load_A2<kL>(p, w, nullptr);

    int n = p.seqs.find(ts), s0 = p.seqs.bound(n), s1 = p.seqs.bound(n + 1);
    State h;
    if (ts <= s0) h = start_state<kL>(p, w, sbase + n);
    else h = kSum ? zero_state() : chain<kL>(p, w, A2, b, s0 / p.seg_len, seg, 1);
    if (!kSum && seg == 0 && p.seqs.cu)
        for (int m = 0; m < p.seqs.n && p.seqs.bound(m + 1) <= 0; ++m) pass_state<kL>(p, w, p.h0, p.ht, m);
    float total = 0.f;

    Raw8<T> rx[kNV], rd[kNV], rz[kNV], rb[kNB], cx[kNV], cz[kNV];
    auto fetch = [&](int tb) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int v = tid + i * kThreads, row = tb + v / (kCh / 8), col = (v % (kCh / 8)) * 8;
            const int nv = v < kVecs && row < te ? min(8, w.nch - col) : 0;
            rx[i] = load8<T, kVec>(x + row * p.x_row + col, nv);
            rd[i] = load8<T, kVec>(dt + row * p.dt_row + col, nv);
            if (!kSum && z) rz[i] = load8<T, kVec>(z + row * p.z_row + col, nv);
        }
#pragma unroll
        for (int i = 0; i < kNB; ++i) {
            const int v = tid + i * kThreads, r = v % kBV, row = tb + r / (kN / 8), col = (r % (kN / 8)) * 8;
            const bool is_c = v >= kBV;
            rb[i] = load8<T, kVec>(is_c ? Cm + row * p.c_row + col : Bm + row * p.b_row + col,
                                   v < (kSum ? 1 : 2) * kBV && row < te ? 8 : 0);
        }
    };
    fetch(ts);
    for (int tb = ts; tb < te; tb += kTile) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int v = tid + i * kThreads, row = v / (kCh / 8), col = (v % (kCh / 8)) * 8;
            cx[i] = rx[i];
            if (!kSum && z) cz[i] = rz[i];
            if (v >= kVecs) continue;
            float fx[8], fd[8];
            unpack8(rx[i], fx);
            unpack8(rd[i], fd);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float s[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float raw = fd[e + k] + s_bias[col + e + k];
                    s[k] = p.softplus ? softplusf(raw) : raw;
                }
                *reinterpret_cast<float4 *>(&s_in[row][col + e]) = make_float4(s[0], s[0] * fx[e], s[1], s[1] * fx[e + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < kNB; ++i) {
            const int v = tid + i * kThreads, r = v % kBV, row = r / (kN / 8), col = (r % (kN / 8)) * 8;
            if (v >= (kSum ? 1 : 2) * kBV) continue;
            float f[8];
            unpack8(rb[i], f);
            float *to = !kSum && v >= kBV ? &s_C[kSum ? 0 : row][col] : &s_B[row][col];
            *reinterpret_cast<float4 *>(to) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
        __syncthreads();
        if (tb + kTile < te) fetch(tb + kTile);

        const int tend = min(tb + kTile, te);
        auto keep = [&](int t) {  // the checkpoint before token t
            if (!kSum && p.states && (t & (kBack - 1)) == 0 && w.on)
                store_state(p.states + w.at((long long)b * ((p.T + kBack - 1) / kBack) + t / kBack, p), h);
        };
        auto token = [&](int i) {
            const float2 in = s_in[i][w.ch];
            h = advance(decay(A2, in.x), h, in.y, load_state(&s_B[i][w.n0]));
            total += in.x;
            return kSum ? 0.f : dot(h, load_state(&s_C[kSum ? 0 : i][w.n0]));
        };
        auto single = [&](int t) {
            keep(t);
            float u = token(t - tb);
            if (kSum) return;
#pragma unroll
            for (int m = kL / 2; m >= 1; m /= 2) u += __shfl_xor_sync(0xffffffffu, u, m);
            if (w.q == 0) s_y[kSum ? 0 : t - tb][w.ch] = u;
        };
        for (int t = tb; t < tend;) {
            if (t >= s1 && n + 1 < p.seqs.count()) {
                do {
                    ++n;
                    s0 = s1;
                    s1 = p.seqs.bound(n + 1);
                } while (s1 <= t && n + 1 < p.seqs.count());
                h = start_state<kL>(p, w, sbase + n);
            }
            const int to = s1 > t ? min(tend, s1) : tend;
            while (t < to && t % kL) single(t++);
            for (; t + kL <= to; t += kL) {
                keep(t);
                float u[kL];
#pragma unroll
                for (int i = 0; i < kL; ++i) u[i] = token(t - tb + i);
                if (!kSum) {
                    const float mine = lane_sums<kL>(u, w.q);
                    s_y[kSum ? 0 : t - tb + w.q][w.ch] = mine;
                }
            }
            while (t < to) single(t++);
            if (!kSum && t == s1) {
                if (p.ht && w.on) store_state(p.ht + w.at(sbase + n, p), h);
                if (p.seqs.cu)
                    for (int m = n + 1; m < p.seqs.n && p.seqs.bound(m + 1) <= s1; ++m)
                        pass_state<kL>(p, w, p.h0, p.ht, m);
            }
        }
        __syncthreads();
        if (!kSum) {
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                const int v = tid + i * kThreads, row = v / (kCh / 8), col = (v % (kCh / 8)) * 8;
                if (v >= kVecs || tb + row >= te || col >= w.nch) continue;
                float fx[8], fz[8], o[8];
                unpack8(cx[i], fx);
                if (z) unpack8(cz[i], fz);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    o[e] = fmaf(s_skip[col + e], fx[e], s_y[kSum ? 0 : row][col + e]);
                    if (z) o[e] *= fz[e] * sigmoidf(fz[e]);
                }
                store8<T, kVec>(y + (long long)(tb + row) * p.D + col, o, min(8, w.nch - col));
            }
        }
    }
    if (kSum && w.on) {
        const long long row = (long long)b * p.S + seg;
        store_state(p.sum_h + w.at(row, p), h);
        if (w.q == 0) p.sum_s[row * p.D + w.d] = total;
    }
}

// Backward, or (kSum) the segments' reverse summaries.  Tiles of kBack tokens
// from the segment's end: the states of a tile are recomputed from its
// checkpoint and kept in registers with their decays, then the gradient runs
// back over them.
template <typename T, int kL, bool kVec, bool kSum>
__global__ void __launch_bounds__(kThreads) k_ssm_bwd(const SsmP p) {
    using W = Place<kL>;
    constexpr int kCh = W::kCh, kN = W::kN, kC = 32 / kL;  // kC: channels of a warp
    constexpr int kVecs = kBack * kCh / 8;                 // of x and dt; as many of z and dy
    constexpr int kNV = (2 * kVecs + kThreads - 1) / kThreads;
    constexpr int kBV = kBack * kN / 8, kNB = (2 * kBV + kThreads - 1) / kThreads;
    constexpr int kPad = 32 / kL < 4 ? 4 : 32 / kL;
    constexpr int kWarps = kThreads / 32;
    __shared__ __align__(16) float4 s_in[kBack][kCh];  // s, s x, du, x
    __shared__ __align__(16) float s_B[kBack][kN], s_C[kBack][kN];
    __shared__ __align__(16) float s_u[kSum ? 1 : kBack][kCh + kPad], s_eb[kSum ? 1 : kBack][kCh + kPad],
        s_fa[kSum ? 1 : kBack][kCh + kPad];
    __shared__ __align__(16) float s_dB[kSum ? 1 : kWarps][kBack][kN], s_dC[kSum ? 1 : kWarps][kBack][kN];
    __shared__ __align__(16) float s_bias[kCh], s_skip[kCh];
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_ssm_status);
    const W w(p);
    const int tid = threadIdx.x, b = blockIdx.z, warp = tid / 32, cw = (tid % 32) / kL;
    const int seg = kSum ? blockIdx.y + 1 : blockIdx.y;  // nothing follows from the first segment's summary
    const int ts = seg * p.seg_len, te = min(ts + p.seg_len, p.T);
    const int sbase = p.seqs.cu ? 0 : b;
    const T *x = static_cast<const T *>(p.x) + b * p.x_batch + w.c0;
    const T *dt = static_cast<const T *>(p.dt) + b * p.dt_batch + w.c0;
    const T *z = p.z ? static_cast<const T *>(p.z) + b * p.z_batch + w.c0 : nullptr;
    const long long own = (long long)b * p.T * p.D + w.c0;
    const T *dy = static_cast<const T *>(p.dy) + own;
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.b_batch + (long long)w.g * kN;
    const T *Cm = static_cast<const T *>(p.Cm) + b * p.c_batch + (long long)w.g * kN;
    for (int i = tid; i < kCh; i += kThreads) {
        s_bias[i] = p.dt_bias && i < w.nch ? p.dt_bias[w.c0 + i] : 0.f;
        s_skip[i] = p.skip && i < w.nch ? p.skip[w.c0 + i] : 0.f;
    }
    __syncthreads();  // the first tile is staged with them
    State A;
    const State A2 = load_A2<kL>(p, w, &A);
    const long long ck0 = (long long)b * ((p.T + kBack - 1) / kBack);

    // The gradient that flows into the segment's last token from behind.
    int n = p.seqs.find(te - 1), s0 = p.seqs.bound(n), s1 = p.seqs.bound(n + 1);
    auto end_grad = [&](int seq) { return p.dht && w.on ? load_state(p.dht + w.at(sbase + seq, p)) : zero_state(); };
    State e;
    if (s1 <= te) e = end_grad(n);
    else e = kSum ? zero_state() : chain<kL>(p, w, A2, b, min((s1 - 1) / p.seg_len, p.S - 1), seg, -1);
    if (!kSum && te == p.T && p.seqs.cu && p.dh0)
        for (int m = n + 1; m < p.seqs.n; ++m) pass_state<kL>(p, w, p.dht, p.dh0, m);
    float total = 0.f;
    State gA = zero_state();
    float gskip[8], gbias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) gskip[i] = gbias[i] = 0.f;

    Raw8<T> r1[kNV], r2[kNV], rb[kNB];
    auto fetch = [&](int tb) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int v = tid + i * kThreads, r = v % kVecs, row = tb + r / (kCh / 8), col = (r % (kCh / 8)) * 8;
            const int nv = v < 2 * kVecs && row < te ? min(8, w.nch - col) : 0;
            if (v < kVecs) {
                r1[i] = load8<T, kVec>(x + row * p.x_row + col, nv);
                r2[i] = load8<T, kVec>(dt + row * p.dt_row + col, nv);
            } else {
                r1[i] = load8<T, kVec>(dy + (long long)row * p.D + col, nv);
                if (z) r2[i] = load8<T, kVec>(z + row * p.z_row + col, nv);
            }
        }
#pragma unroll
        for (int i = 0; i < kNB; ++i) {
            const int v = tid + i * kThreads, r = v % kBV, row = tb + r / (kN / 8), col = (r % (kN / 8)) * 8;
            rb[i] = load8<T, kVec>(v >= kBV ? Cm + row * p.c_row + col : Bm + row * p.b_row + col,
                                   v < 2 * kBV && row < te ? 8 : 0);
        }
    };
    const int last = ts + (te - ts - 1) / kBack * kBack;
    fetch(last);
    State ck_next = zero_state();
    if (!kSum && w.on) ck_next = load_state(p.states + w.at(ck0 + last / kBack, p));
    for (int tb = last; tb >= ts; tb -= kBack) {
        Raw8<T> c1[kNV], c2[kNV];
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int v = tid + i * kThreads, r = v % kVecs, row = r / (kCh / 8), col = (r % (kCh / 8)) * 8;
            c1[i] = r1[i];
            c2[i] = r2[i];
            if (v >= 2 * kVecs) continue;
            const bool real = tb + row < te;  // a row past the end changes nothing: s = 0, du = 0
            float f1[8], f2[8];
            unpack8(r1[i], f1);
            unpack8(r2[i], f2);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float4 *to = &s_in[row][col + k];
                if (v < kVecs) {
                    const float raw = f2[k] + s_bias[col + k];
                    const float s = !real ? 0.f : p.softplus ? softplusf(raw) : raw;
                    to->x = s;
                    to->y = s * f1[k];
                    to->w = f1[k];
                } else {
                    to->z = z ? f1[k] * f2[k] * sigmoidf(f2[k]) : f1[k];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kNB; ++i) {
            const int v = tid + i * kThreads, r = v % kBV, row = r / (kN / 8), col = (r % (kN / 8)) * 8;
            if (v >= 2 * kBV) continue;
            float f[8];
            unpack8(rb[i], f);
            float *to = v >= kBV ? &s_C[row][col] : &s_B[row][col];
            *reinterpret_cast<float4 *>(to) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
        __syncthreads();
        const State ck = ck_next;
        if (tb - kBack >= ts) {
            fetch(tb - kBack);
            if (!kSum && w.on) ck_next = load_state(p.states + w.at(ck0 + tb / kBack - 1, p));
        }
        auto turn = [&](int t) {  // token t opens sequence n: e is its start state's gradient
            if (!kSum && p.dh0 && w.on) store_state(p.dh0 + w.at(sbase + n, p), e);
            e = zero_state();
            if (!p.seqs.cu) return;
            while (n > 0) {
                --n;
                s1 = s0;
                s0 = p.seqs.bound(n);
                if (s0 < s1) break;
                if (!kSum && p.dh0) pass_state<kL>(p, w, p.dht, p.dh0, n);
            }
            if (s0 < t) e = end_grad(n);
        };
        if (kSum) {
            for (int i = min(kBack, te - tb) - 1; i >= 0; --i) {
                const float4 in = s_in[i][w.ch];
                const State C = load_state(&s_C[i][w.n0]), a = decay(A2, in.x);
                const f32x2 du = mk2(in.z, in.z);
                e = State{mul2(a.a, fma2(du, C.a, e.a)), mul2(a.b, fma2(du, C.b, e.b))};
                total += in.x;
                if (tb + i == s0) turn(tb + i);
            }
            __syncthreads();
            continue;
        }
        State H[kBack], E[kBack];
        {
            int m = 0, next = p.T;  // the next sequence to open inside the tile
            if (p.seqs.cu) {
                m = p.seqs.find(tb);
                next = p.seqs.bound(m + 1);
            }
            State h = ck;
            float u[kL], v[kC][4];
#pragma unroll
            for (int i = 0; i < kBack; ++i) {
                if (p.seqs.cu && tb + i >= next && tb + i < te) {
                    while (next <= tb + i && m + 1 < p.seqs.n) next = p.seqs.bound(++m + 1);
                    h = start_state<kL>(p, w, m);
                    if (next <= tb + i) next = p.T;
                }
                const float4 in = s_in[i][w.ch];
                E[i] = decay(A2, in.x);
                h = advance(E[i], h, in.y, load_state(&s_B[i][w.n0]));
                H[i] = h;
                if (z) {
                    u[i % kL] = dot(h, load_state(&s_C[i][w.n0]));
                    if (i % kL == kL - 1) s_u[kSum ? 0 : i - kL + 1 + w.q][w.ch] = lane_sums<kL>(u, w.q);
                }
                const f32x2 du = mk2(in.z, in.z);
                un2(mul2(du, h.a), v[i % kC][0], v[i % kC][1]);
                un2(mul2(du, h.b), v[i % kC][2], v[i % kC][3]);
                if (i % kC == kC - 1) {
                    channel_sums<kL, kC>(v, cw);
                    *reinterpret_cast<float4 *>(&s_dC[kSum ? 0 : warp][i - kC + 1 + cw][w.n0]) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
                }
            }
        }
        {
            float ub[kL], ua[kL], v[kC][4];
#pragma unroll
            for (int i = kBack - 1; i >= 0; --i) {
                const float4 in = s_in[i][w.ch];
                const State C = load_state(&s_C[i][w.n0]), Bt = load_state(&s_B[i][w.n0]);
                const bool opens = tb + i == s0 && tb + i < te;
                const f32x2 du = mk2(in.z, in.z), sx = mk2(in.y, in.y), s2 = mk2(in.x, in.x);
                e = State{fma2(du, C.a, e.a), fma2(du, C.b, e.b)};
                ub[i % kL] = dot(e, Bt);
                un2(mul2(e.a, sx), v[i % kC][0], v[i % kC][1]);
                un2(mul2(e.b, sx), v[i % kC][2], v[i % kC][3]);
                State before = i ? H[i ? i - 1 : 0] : ck;
                if (opens && i) before = start_state<kL>(p, w, sbase + n);
                e = State{mul2(e.a, E[i].a), mul2(e.b, E[i].b)};
                const State f = State{mul2(e.a, before.a), mul2(e.b, before.b)};
                ua[i % kL] = dot(f, A);
                gA = State{fma2(f.a, s2, gA.a), fma2(f.b, s2, gA.b)};
                if (opens) turn(tb + i);
                if (i % kL == 0) {
                    s_eb[kSum ? 0 : i + w.q][w.ch] = lane_sums<kL>(ub, w.q);
                    s_fa[kSum ? 0 : i + w.q][w.ch] = lane_sums<kL>(ua, w.q);
                }
                if (i % kC == 0) {
                    channel_sums<kL, kC>(v, cw);
                    *reinterpret_cast<float4 *>(&s_dB[kSum ? 0 : warp][i + cw][w.n0]) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int v = tid + i * kThreads, r = v % kVecs, row = r / (kCh / 8), col = (r % (kCh / 8)) * 8;
            if (v >= 2 * kVecs || tb + row >= te || col >= w.nch) continue;
            const int nv = min(8, w.nch - col);
            const long long at = own + (long long)(tb + row) * p.D + col;
            float f1[8], f2[8], o1[8], o2[8];
            unpack8(c1[i], f1);
            unpack8(c2[i], f2);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 in = s_in[row][col + k];
                const float sk = s_skip[col + k];
                if (v < kVecs) {
                    const float eb = s_eb[kSum ? 0 : row][col + k];
                    o1[k] = fmaf(in.x, eb, sk * in.z);
                    o2[k] = fmaf(in.w, eb, s_fa[kSum ? 0 : row][col + k]);
                    if (p.softplus) o2[k] *= sigmoidf(f2[k] + s_bias[col + k]);
                    gskip[k] = fmaf(in.z, in.w, gskip[k]);
                    gbias[k] += o2[k];
                } else {
                    const float g = sigmoidf(f2[k]), u = fmaf(sk, in.w, s_u[kSum ? 0 : row][col + k]);
                    o1[k] = f1[k] * u * g * fmaf(f2[k], 1.f - g, 1.f);
                }
            }
            if (v < kVecs) {
                store8<T, kVec>(static_cast<T *>(p.dx) + at, o1, nv);
                store8<T, kVec>(static_cast<T *>(p.ddt) + at, o2, nv);
            } else if (z) {
                store8<T, kVec>(static_cast<T *>(p.dz) + at, o1, nv);
            }
        }
        for (int i = tid; i < 2 * kBack * kN / 4; i += kThreads) {  // the warps' channels, in order
            const bool is_c = i >= kBack * kN / 4;
            const int r = i % (kBack * kN / 4), row = r / (kN / 4), col = (r % (kN / 4)) * 4;
            if (tb + row >= te) continue;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 v = *reinterpret_cast<const float4 *>(is_c ? &s_dC[kSum ? 0 : k][row][col] : &s_dB[kSum ? 0 : k][row][col]);
                a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
            }
            float *to = (is_c ? p.pC : p.pB) + (((long long)w.gt * p.B + b) * p.T + tb + row) * kN + col;
            *reinterpret_cast<float4 *>(to) = a;
        }
        __syncthreads();
    }
    const long long row = (long long)b * p.S + seg;
    if (kSum) {
        if (w.on) {
            store_state(p.sum_h + w.at(row, p), e);
            if (w.q == 0) p.sum_s[row * p.D + w.d] = total;
        }
        return;
    }
    if (w.on) store_state(p.pA + w.at(row, p), gA);
    // dskip and ddt_bias: the tile rows' sums, in order
    float *acc = &s_in[0][0].x;  // [2][kBack][kCh]
    static_assert(sizeof(s_in) >= 2 * kBack * kCh * sizeof(float), "");
    if (tid < kVecs) {
        const int rr = tid / (kCh / 8), col = (tid % (kCh / 8)) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            acc[rr * kCh + col + k] = gskip[k];
            acc[(kBack + rr) * kCh + col + k] = gbias[k];
        }
    }
    __syncthreads();
    for (int i = tid; i < 2 * kCh; i += kThreads) {
        const int which = i / kCh, c = i % kCh;
        if (c >= w.nch) continue;
        float a = 0.f;
        for (int k = 0; k < kBack; ++k) a += acc[(which * kBack + k) * kCh + c];
        p.pD[(row * 2 + which) * p.D + w.c0 + c] = a;
    }
}

// Adds the partial gradients in order: dB and dC over a group's channel tiles,
// dA, dskip and ddt_bias over batch rows and segments.
template <typename T>
__global__ void k_ssm_bwd_sum(const SsmP p, int N) {
    const long long bc = (long long)p.B * p.T * p.G * N, da = (long long)p.D * N;
    const long long rows = (long long)p.B * p.S;
    long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < 2 * bc) {
        const bool is_c = i >= bc;
        if (is_c) i -= bc;
        const int nn = i % N, g = (i / N) % p.G;
        const long long bt = i / N / p.G, plane = (long long)p.B * p.T * N;
        const float *from = (is_c ? p.pC : p.pB) + (long long)g * p.tiles * plane + bt * N + nn;
        float a = 0.f;
        for (int k = 0; k < p.tiles; ++k) a += from[k * plane];
        from_f(static_cast<T *>(is_c ? p.dC : p.dB)[i], a);
        return;
    }
    i -= 2 * bc;
    if (i < da) {
        float a = 0.f;
        for (long long k = 0; k < rows; ++k) a += p.pA[k * da + i];
        p.dA[i] = a;
        return;
    }
    i -= da;
    if (i < 2 * p.D) {
        float *to = i < p.D ? p.dskip : p.ddt_bias;
        if (!to) return;
        float a = 0.f;
        for (long long k = 0; k < rows; ++k) a += p.pD[k * 2 * p.D + i];
        to[i % p.D] = a;
    }
}

struct StepP {
    const void *x, *dt, *z, *Bm, *Cm;
    const float *A, *skip, *dt_bias;
    float *state;
    const int32_t *slots;
    void *y;
    long long x_row, dt_row, z_row, b_row, c_row, n_slots;
    int D, Dg, softplus;
};

template <typename T>
__device__ __forceinline__ State four(const T *p) {
    return State{mk2(to_f(p[0]), to_f(p[1])), mk2(to_f(p[2]), to_f(p[3]))};
}

// Bound by memory: the states of the rows are read and written once.
template <typename T, int kL>
__global__ void __launch_bounds__(kThreads) k_ssm_step(const StepP p) {
    constexpr int kCh = kThreads / kL, kN = 4 * kL;
    const int r = blockIdx.y, d = blockIdx.x * kCh + threadIdx.x / kL, q = threadIdx.x % kL;
    const long long slot = p.slots ? p.slots[r] : r;
    const bool known = slot >= 0 && slot < p.n_slots, on = d < p.D;
    if (slot >= p.n_slots && threadIdx.x == 0) atomicOr(&g_ssm_status, kStatusIndex);
    float u = 0.f, xv = 0.f;
    if (on && known) {
        float *st = p.state + (slot * p.D + d) * kN + 4 * q;
        const State h0 = load_state(st), A = load_state(p.A + (long long)d * kN + 4 * q);
        const int g = d / p.Dg;
        const State Bt = four(static_cast<const T *>(p.Bm) + r * p.b_row + g * kN + 4 * q);
        const State Ct = four(static_cast<const T *>(p.Cm) + r * p.c_row + g * kN + 4 * q);
        xv = to_f(static_cast<const T *>(p.x)[r * p.x_row + d]);
        const float raw = to_f(static_cast<const T *>(p.dt)[r * p.dt_row + d]) + (p.dt_bias ? p.dt_bias[d] : 0.f);
        const float s = p.softplus ? softplusf(raw) : raw;
        const f32x2 k = mk2(kLog2e, kLog2e);
        const State h = advance(decay(State{mul2(A.a, k), mul2(A.b, k)}, s), h0, s * xv, Bt);
        store_state(st, h);
        u = dot(h, Ct);
    }
#pragma unroll
    for (int m = kL / 2; m >= 1; m /= 2) u += __shfl_xor_sync(0xffffffffu, u, m);
    if (on && q == 0) {
        if (known) {
            if (p.skip) u = fmaf(p.skip[d], xv, u);
            if (p.z) {
                const float zv = to_f(static_cast<const T *>(p.z)[r * p.z_row + d]);
                u *= zv * sigmoidf(zv);
            }
        }
        from_f(static_cast<T *>(p.y)[(long long)r * p.D + d], u);
    }
}

// ---- host ------------------------------------------------------------------

int ssm_sizes(long long B, long long T, long long D, long long G, int N, int dtype) {
    if (B < 1 || T < 0 || D < 1 || G < 1)
        return layer_fail(GDR_ERR_SHAPE, "scan: B, D and G must be >= 1 and T >= 0 (got %lld, %lld, %lld, %lld)", B, D, G, T);
    if (D % G) return layer_fail(GDR_ERR_SHAPE, "scan: D (%lld) must be a multiple of G (%lld)", D, G);
    if (N != 8 && N != 16 && N != 32 && N != 64) return layer_fail(GDR_ERR_SHAPE, "scan: N must be 8, 16, 32 or 64 (got %d)", N);
    if (T >= (1LL << 30) || D >= (1LL << 24) || B > 65535) return layer_fail(GDR_ERR_SHAPE, "scan: problem too large");
    if (dtype != GDR_BF16 && dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "scan: unknown dtype %d", dtype);
    return GDR_OK;
}

struct SsmPlan {
    int tiles, S, seg_len;
};

// Segments: an estimate in cycles a token of a CTA.  A CTA alone on an SM
// advances a token in about kLat cycles (its four warps wait on the chain of
// decays); k of them share the SM's issue slots at about kThr each.
SsmPlan ssm_plan(long long B, long long T, long long D, long long G, int N, bool bwd) {
    const int ch = kThreads / (N / 4);
    const long long tiles = (D / G + ch - 1) / ch, ctas = tiles * G * B, sms = layer_sms();
    const double kLat = bwd ? 140 : 45, kThr = bwd ? 100 : 25, kSum = bwd ? 0.35 : 0.6;
    double best = 1e300;
    int S = 1;
    for (int s = 1; s <= 64; ++s) {
        if (s > 1 && (T / s < 64)) break;
        const double tok = (double)((T + s - 1) / s);
        const double per = std::max(kLat, kThr * (double)((ctas * s + sms - 1) / sms));
        const double sum = s == 1 ? 0 : kSum * std::max(kLat, kThr * (double)((ctas * (s - 1) + sms - 1) / sms));
        const double t = tok * (per + sum) + (s > 1 ? 6000 + 200.0 * s : 0);
        if (t < best * 0.999) {
            best = t;
            S = s;
        }
    }
    long long len = (T + S - 1) / S;
    len = std::max(32LL, (len + 31) / 32 * 32);
    return SsmPlan{(int)tiles, (int)std::max(1LL, (T + len - 1) / len), (int)len};
}

size_t up16(size_t v) { return (v + 15) & ~size_t(15); }

struct SsmSpace {
    size_t sum_h, sum_s, pB, pC, pA, pD, total;
};
SsmSpace ssm_space(const gdr_ssm_args *a, const SsmPlan &pl, bool bwd) {
    SsmSpace s{};
    size_t off = 0;
    auto take = [&](size_t n) { size_t r = off; off += up16(n * 4); return r; };
    const size_t seg = (size_t)a->B * pl.S, D = a->D, N = a->N;
    if (pl.S > 1) {
        s.sum_h = take(seg * D * N);
        s.sum_s = take(seg * D);
    }
    if (bwd) {
        const size_t plane = (size_t)a->B * a->T * N * pl.tiles * a->G;
        s.pB = take(plane);
        s.pC = take(plane);
        s.pA = take(seg * D * N);
        s.pD = take(seg * 2 * D);
    }
    s.total = off;
    return s;
}

bool ssm_vec(const gdr_ssm_args *a) {
    const long long q = a->dtype == GDR_BF16 ? 8 : 4;
    for (long long v : {a->x_row, a->x_batch, a->dt_row, a->dt_batch, a->z ? a->z_row : 0, a->z ? a->z_batch : 0,
                        a->b_row, a->b_batch, a->c_row, a->c_batch})
        if (v % q) return false;
    return (a->D / a->G) % 8 == 0 && multiple16(a->x) && multiple16(a->dt) && multiple16(a->z) && multiple16(a->Bm) &&
           multiple16(a->Cm);
}

int ssm_common(const gdr_ssm_args *a, Seqs *s) {
    int rc;
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    if ((rc = ssm_sizes(a->B, a->T, a->D, a->G, a->N, a->dtype))) return rc;
    if (a->cu_seqlens ? (a->B != 1 || a->n_seqs < 1) : a->n_seqs != a->B)
        return layer_fail(GDR_ERR_SHAPE, "scan: packed sequences need B == 1 and n_seqs >= 1, a batch n_seqs == B");
    if (a->n_seqs > (1 << 24)) return layer_fail(GDR_ERR_SHAPE, "scan: too many sequences");
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->T > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("dt", a->dt, any, e)) || (rc = layer_ptr("z", a->z, false, e)) ||
        (rc = layer_ptr("B", a->Bm, any, e)) || (rc = layer_ptr("C", a->Cm, any, e)) || (rc = layer_ptr("A", a->A, true, 16)) ||
        (rc = layer_ptr("D", a->skip, false, 4)) || (rc = layer_ptr("dt_bias", a->dt_bias, false, 4)) ||
        (rc = layer_ptr("h0", a->h0, false, 16)) || (rc = layer_ptr("states", a->states, false, 16)))
        return rc;
    s->cu = a->cu_seqlens;
    s->n = (int)a->n_seqs;
    s->T = (int)a->T;
    return GDR_OK;
}

void ssm_fill(const gdr_ssm_args *a, const Seqs &s, const SsmPlan &pl, const SsmSpace &sp, SsmP *p) {
    *p = SsmP{};
    p->x = a->x; p->dt = a->dt; p->z = a->z; p->Bm = a->Bm; p->Cm = a->Cm; p->dy = a->dy;
    p->A = a->A; p->skip = a->skip; p->dt_bias = a->dt_bias; p->h0 = a->h0; p->dht = a->dht;
    p->y = a->y; p->dx = a->dx; p->ddt = a->ddt; p->dz = a->dz; p->dB = a->dB; p->dC = a->dC;
    p->ht = a->ht; p->states = a->states; p->dA = a->dA; p->dskip = a->dskip; p->ddt_bias = a->ddt_bias; p->dh0 = a->dh0;
    char *ws = static_cast<char *>(a->workspace);
    auto f = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    p->sum_h = f(sp.sum_h); p->sum_s = f(sp.sum_s);
    p->pB = f(sp.pB); p->pC = f(sp.pC); p->pA = f(sp.pA); p->pD = f(sp.pD);
    p->seqs = s;
    p->x_row = a->x_row; p->x_batch = a->x_batch; p->dt_row = a->dt_row; p->dt_batch = a->dt_batch;
    p->z_row = a->z_row; p->z_batch = a->z_batch; p->b_row = a->b_row; p->b_batch = a->b_batch;
    p->c_row = a->c_row; p->c_batch = a->c_batch;
    p->B = (int)a->B; p->T = (int)a->T; p->D = (int)a->D; p->G = (int)a->G; p->Dg = (int)(a->D / a->G);
    p->tiles = pl.tiles; p->S = pl.S; p->seg_len = pl.seg_len; p->softplus = a->softplus;
}

template <typename F>
void ssm_by_type(int dtype, int N, bool vec, F f) {
    auto w = [&](auto t) {
        auto v = [&](auto l) {
            if (vec) f(t, l, std::true_type{}); else f(t, l, std::false_type{});
        };
        if (N == 8) v(std::integral_constant<int, 2>{});
        else if (N == 16) v(std::integral_constant<int, 4>{});
        else if (N == 32) v(std::integral_constant<int, 8>{});
        else v(std::integral_constant<int, 16>{});
    };
    if (dtype == GDR_BF16) w(bf16_t{}); else w(float{});
}

int ssm_workspace(const gdr_ssm_args *a, size_t need, const char *what) {
    if (!need) return GDR_OK;
    if (!a->workspace) return layer_fail(GDR_ERR_WORKSPACE, "%s: workspace is null", what);
    if (!multiple16(a->workspace)) return layer_fail(GDR_ERR_ALIGN, "%s: workspace must be 16-byte aligned", what);
    if (a->workspace_bytes < need)
        return layer_fail(GDR_ERR_WORKSPACE, "%s: workspace too small: %zu < %zu bytes", what, a->workspace_bytes, need);
    return GDR_OK;
}

// A call without tokens hands the states through.
int ssm_hand_on(const float *from, float *to, size_t n, cudaStream_t st) {
    if (!to) return GDR_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, n * 4, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, n * 4, st);
    return e == cudaSuccess ? GDR_OK : layer_fail(GDR_ERR_CUDA, "scan: %s", cudaGetErrorString(e));
}

}  // namespace

namespace gdr {
unsigned ssm_take_status(cudaStream_t st) {
    unsigned v = 0, z = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_ssm_status, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return 0x80000000u;
    cudaMemcpyToSymbolAsync(g_ssm_status, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    if (cudaStreamSynchronize(st) != cudaSuccess) return 0x80000000u;
    return v;
}
}  // namespace gdr

extern "C" {

size_t gdr_ssm_fwd_workspace_size(const gdr_ssm_args *a) {
    if (!a || ssm_sizes(a->B, a->T, a->D, a->G, a->N, a->dtype)) return 0;
    return ssm_space(a, ssm_plan(a->B, a->T, a->D, a->G, a->N, false), false).total;
}

size_t gdr_ssm_bwd_workspace_size(const gdr_ssm_args *a) {
    if (!a || ssm_sizes(a->B, a->T, a->D, a->G, a->N, a->dtype)) return 0;
    return ssm_space(a, ssm_plan(a->B, a->T, a->D, a->G, a->N, true), true).total;
}

int gdr_ssm_fwd(const gdr_ssm_args *a, void *stream) {
    Seqs s;
    int rc = ssm_common(a, &s);
    if (rc) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    if ((rc = layer_ptr("y", a->y, a->T > 0, e)) || (rc = layer_ptr("ht", a->ht, false, 16))) return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->T == 0) return ssm_hand_on(a->h0, a->ht, (size_t)a->n_seqs * a->D * a->N, st);
    const SsmPlan pl = ssm_plan(a->B, a->T, a->D, a->G, a->N, false);
    const SsmSpace sp = ssm_space(a, pl, false);
    if ((rc = ssm_workspace(a, sp.total, "scan forward"))) return rc;
    SsmP p;
    ssm_fill(a, s, pl, sp, &p);
    const bool vec = ssm_vec(a) && multiple16(a->y);
    ssm_by_type(a->dtype, a->N, vec, [&](auto t, auto l, auto v) {
        using E = decltype(t);
        constexpr int L = decltype(l)::value;
        constexpr bool V = decltype(v)::value;
        const unsigned gx = (unsigned)(pl.tiles * a->G), gz = (unsigned)a->B;
        if (pl.S > 1) k_ssm_fwd<E, L, V, true><<<dim3(gx, pl.S - 1, gz), kThreads, 0, st>>>(p);
        k_ssm_fwd<E, L, V, false><<<dim3(gx, pl.S, gz), kThreads, 0, st>>>(p);
    });
    return layer_launched("scan forward");
}

int gdr_ssm_bwd(const gdr_ssm_args *a, void *stream) {
    Seqs s;
    int rc = ssm_common(a, &s);
    if (rc) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->T > 0;
    if ((rc = layer_ptr("dy", a->dy, any, e)) || (rc = layer_ptr("states", a->states, any, 16)) ||
        (rc = layer_ptr("dht", a->dht, false, 16)) || (rc = layer_ptr("dx", a->dx, any, e)) ||
        (rc = layer_ptr("ddt", a->ddt, any, e)) || (rc = layer_ptr("dz", a->dz, any && a->z, e)) ||
        (rc = layer_ptr("dB", a->dB, any, e)) || (rc = layer_ptr("dC", a->dC, any, e)) ||
        (rc = layer_ptr("dA", a->dA, true, 4)) || (rc = layer_ptr("dD", a->dskip, a->skip != nullptr, 4)) ||
        (rc = layer_ptr("ddt_bias", a->ddt_bias, a->dt_bias != nullptr, 4)) || (rc = layer_ptr("dh0", a->dh0, false, 16)))
        return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!any) {
        if ((rc = ssm_hand_on(nullptr, a->dA, (size_t)a->D * a->N, st)) || (rc = ssm_hand_on(nullptr, a->dskip, a->D, st)) ||
            (rc = ssm_hand_on(nullptr, a->ddt_bias, a->D, st)))
            return rc;
        return ssm_hand_on(a->dht, a->dh0, (size_t)a->n_seqs * a->D * a->N, st);
    }
    const SsmPlan pl = ssm_plan(a->B, a->T, a->D, a->G, a->N, true);
    const SsmSpace sp = ssm_space(a, pl, true);
    if ((rc = ssm_workspace(a, sp.total, "scan backward"))) return rc;
    SsmP p;
    ssm_fill(a, s, pl, sp, &p);
    const bool vec = ssm_vec(a) && multiple16(a->dy) && multiple16(a->dx) && multiple16(a->ddt) && multiple16(a->dz);
    const long long outs = 2 * a->B * a->T * a->G * a->N + a->D * a->N + 2 * a->D;
    ssm_by_type(a->dtype, a->N, vec, [&](auto t, auto l, auto v) {
        using E = decltype(t);
        constexpr int L = decltype(l)::value;
        constexpr bool V = decltype(v)::value;
        const unsigned gx = (unsigned)(pl.tiles * a->G), gz = (unsigned)a->B;
        if (pl.S > 1) k_ssm_bwd<E, L, V, true><<<dim3(gx, pl.S - 1, gz), kThreads, 0, st>>>(p);
        k_ssm_bwd<E, L, V, false><<<dim3(gx, pl.S, gz), kThreads, 0, st>>>(p);
        k_ssm_bwd_sum<E><<<(unsigned)((outs + 255) / 256), 256, 0, st>>>(p, a->N);
    });
    return layer_launched("scan backward");
}

int gdr_ssm_step(const gdr_ssm_step_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    if ((rc = ssm_sizes(1, a->rows, a->D, a->G, a->N, a->dtype))) return rc;
    if (a->rows > 65535) return layer_fail(GDR_ERR_SHAPE, "scan step: at most 65535 rows");
    if (a->n_slots < 0 || (!a->slots && a->n_slots < a->rows))
        return layer_fail(GDR_ERR_SHAPE, "scan step: %lld state slots for %lld rows", a->n_slots, a->rows);
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->rows > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("dt", a->dt, any, e)) || (rc = layer_ptr("z", a->z, false, e)) ||
        (rc = layer_ptr("B", a->Bm, any, e)) || (rc = layer_ptr("C", a->Cm, any, e)) || (rc = layer_ptr("A", a->A, true, 16)) ||
        (rc = layer_ptr("D", a->skip, false, 4)) || (rc = layer_ptr("dt_bias", a->dt_bias, false, 4)) ||
        (rc = layer_ptr("state", a->state, any && a->n_slots > 0, 16)) || (rc = layer_ptr("slots", a->slots, false, 4)) ||
        (rc = layer_ptr("y", a->y, any, e)))
        return rc;
    if (!any) return GDR_OK;
    StepP p{a->x, a->dt, a->z, a->Bm, a->Cm, a->A, a->skip, a->dt_bias, a->state, a->slots, a->y,
            a->x_row, a->dt_row, a->z_row, a->b_row, a->c_row, a->n_slots, (int)a->D, (int)(a->D / a->G), a->softplus};
    ssm_by_type(a->dtype, a->N, true, [&](auto t, auto l, auto) {
        constexpr int L = decltype(l)::value;
        const int ch = kThreads / L;
        k_ssm_step<decltype(t), L><<<dim3((unsigned)((a->D + ch - 1) / ch), (unsigned)a->rows), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return layer_launched("scan step");
}

}  // extern "C"
