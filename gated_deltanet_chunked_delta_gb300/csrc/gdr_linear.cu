// gdr_linear.cu -- gated linear recurrence (one state a channel), forward,
// backward and single-token step.
//
// Per sequence and channel, with s = c softplus(decay), L_t = -s sigmoid(r_t),
// a_t = e^{L_t}, m_t = sqrt(1 - a_t^2) and u_t = sigmoid(i_t) x_t:
//     h_t = a_t h_{t-1} + m_t u_t,   y_t = h_t silu(z_t) (or h_t),
// and backwards, with e_t the gradient of h_t and din_t = dy_t silu(z_t):
//     e_t = din_t + a_{t+1} e_{t+1},  dx = e m sigmoid(i),  di = e m u (1 - sigmoid(i)),
//     G = dL L = L a e h_{t-1} + e u a^2 (-L / m),  dr = G (1 - sigmoid(r)),
//     ddecay = sigmoid(decay) / softplus(decay) sum G,  dz = dy h silu'(z).
// G takes the place of dL because dm/dL = -a^2 / m has no bound as L goes to
// zero, while -L / m goes to sqrt(-L / 2).
//
// Bound by memory (8 bytes of bf16 an element forward, 14 backward), so the
// data is read once: the tokens are cut into chunks, a CTA holds a chunk of 32
// or 64 channels in registers (a warp a run of neighbouring tokens, a lane one or
// two neighbouring channels), and the state is handed from chunk to chunk
// between CTAs.  A chunk acts on the state before it as h -> A h + B; its CTA
// publishes (A, B) as soon as it has read its data, then looks back for the
// nearest chunk whose own state is known, goes forward from there over the
// (A, B) between, and publishes the state after itself.  Going forward in
// order, whatever the place it starts from, makes every result independent of
// the CTAs' timing, bit for bit.  CTAs take their chunks from a counter, all
// channels of the first chunk before the second: a CTA waits only for ones that
// run already.
#include "gdr_layer.h"

namespace {

__device__ unsigned g_linear_status;

constexpr int kStride = GDR_LINEAR_STRIDE;  // tokens between the states kept for the backward
constexpr int kFwdRun = 16, kBwdRun = 8;    // tokens of a warp
constexpr int kMaxWarps = 8;
constexpr int kWindow = 4;                  // chunks looked back at once
constexpr int kPolls = 1 << 20;             // of the records before a chunk, before its wait is given up

struct LinP {
    const void *x, *i, *r, *z, *dy;
    const float *decay, *h0, *dht;
    void *y, *dx, *di, *dr, *dz;
    float *ht, *states, *dh0, *part;  // part: [B chunks, D] sums of G
    float4 *rec;                      // [columns, chunks, 32 kC] of {A, B, state, flag}
    unsigned *ticket;
    Seqs seqs;
    long long x_row, x_batch, i_row, i_batch, r_row, r_batch, z_row, z_batch;
    long long tiles;
    int B, T, D, nd, chunks;  // nd: channel tiles
    float scale;
};

// kC neighbouring channels of a token as they lie in memory.
template <typename T, int kC>
struct Ch;
template <>
struct Ch<bf16_t, 2> {
    uint32_t w;
    __device__ __forceinline__ void load(const bf16_t *p) { w = *reinterpret_cast<const uint32_t *>(p); }
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void get(float (&f)[2]) const {
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(bf16_t *p, const float (&f)[2]) { *reinterpret_cast<uint32_t *>(p) = pack2(f[0], f[1]); }
};
template <typename T>
struct Ch<T, 1> {
    T w;
    __device__ __forceinline__ void load(const T *p) { w = *p; }
    __device__ __forceinline__ void zero() { from_f(w, 0.f); }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f(w); }
    static __device__ __forceinline__ void store(T *p, const float (&f)[1]) { from_f(*p, f[0]); }
};

// sigmoid(v) and 1 - sigmoid(v), both to full relative precision; NaN stays.
__device__ __forceinline__ void sigmoids(float v, float &on, float &off) {
    float t;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(t) : "f"(-kLog2e * v), "f"(126.f));
    const float e = ex2f(t);
    on = rcpf(1.f + e);
    off = e * on;
}
__device__ __forceinline__ float sqrt_of(float v) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
// The decay of a step: log2 a, a, 1 - a^2.  s2 is s log2 e, sig sigmoid(r).
// a: the argument of ex2.approx is moved up by 1.5e-8 of the result, which it
// lies low by on average (a slow state multiplies hundreds of decays).
// 1 - a^2 = 1 - e^{-v}, v = 2 s sig: by its series below 1/2 (the remainder is
// v^8 / 9! < 2^-26 of it), where the difference would lose its leading digits.
__device__ __forceinline__ void decay_of(float s2, float sig, float &l2, float &a, float &w) {
    l2 = -s2 * sig;
    a = ex2f(fmaf(-s2, sig, 2.2e-8f));
    const float v = -1.3862943611198906f * l2;
    float q = fmaf(v, 1.f / 40320, -1.f / 5040);
    q = fmaf(v, -q, -1.f / 720);
    q = fmaf(v, -q, -1.f / 120);
    q = fmaf(v, -q, -1.f / 24);
    q = fmaf(v, -q, -1.f / 6);
    q = fmaf(v, -q, -1.f / 2);
    q = fmaf(v, q, 1.f);
    w = v < 0.5f ? v * q : fmaf(-a, a, 1.f);
}

// How tokens act on the state before them: h -> a h + b, or h -> b (a < 0)
// where a sequence starts on the way: what lies before it, NaN and infinities
// included, is left out, not multiplied by zero.
template <bool kPacked>
__device__ __forceinline__ float act(float a, float b, float h) {
    return kPacked && a < 0.f ? b : fmaf(a, h, b);
}
template <bool kPacked>
__device__ __forceinline__ float join(float a, float next) {  // the product, negative once one is
    return kPacked && (a < 0.f || next < 0.f) ? -1.f : a * next;
}

struct Rec {
    float a, b, h;
    uint32_t flag;  // 0 nothing yet, 1: a and b, 2: the state after the chunk too
};
// A record is written and read in one piece, so that its flag vouches for it.
__device__ __forceinline__ void write_rec(float4 *p, float a, float b, float h, uint32_t flag) {
    const unsigned long long lo = (unsigned long long)__float_as_uint(a) | (unsigned long long)__float_as_uint(b) << 32;
    const unsigned long long hi = (unsigned long long)__float_as_uint(h) | (unsigned long long)flag << 32;
    asm volatile("{\n.reg .b128 v;\nmov.b128 v, {%1, %2};\nst.relaxed.gpu.global.b128 [%0], v;\n}" ::"l"(p), "l"(lo), "l"(hi) : "memory");
}
__device__ __forceinline__ Rec read_rec(const float4 *p) {
    unsigned long long lo, hi;
    asm volatile("{\n.reg .b128 v;\nld.relaxed.gpu.global.b128 v, [%2];\nmov.b128 {%0, %1}, v;\n}" : "=l"(lo), "=l"(hi) : "l"(p) : "memory");
    return Rec{__uint_as_float((uint32_t)lo), __uint_as_float((uint32_t)(lo >> 32)), __uint_as_float((uint32_t)hi), (uint32_t)(hi >> 32)};
}

// One warp: the state before its chunk, the `ordinal`-th, from the records of
// the ones before it (`mine`: this lane's own record, `step` from chunk to
// chunk).  False when the wait was given up.
template <int kC, bool kPacked>
__device__ __forceinline__ bool look_back(const float4 *mine, long long step, int ordinal, float (&h)[kC]) {
    const int reach = min(kWindow, ordinal);
    for (int polls = 0; polls < kPolls; ++polls) {
        Rec rec[kWindow][kC];
#pragma unroll
        for (int j = 0; j < kWindow; ++j)
#pragma unroll
            for (int c = 0; c < kC; ++c) rec[j][c] = j < reach ? read_rec(mine - (j + 1) * step + c) : Rec{0.f, 0.f, 0.f, 0};
        int from = -1;
        bool open = true;  // every chunk nearer than j has its a and b
#pragma unroll
        for (int j = 0; j < kWindow; ++j) {
            uint32_t flag = rec[j][0].flag;
#pragma unroll
            for (int c = 1; c < kC; ++c) flag = min(flag, rec[j][c].flag);
            if (open && from < 0 && __all_sync(0xffffffffu, flag == 2)) from = j;
            open = open && __all_sync(0xffffffffu, flag >= 1);
        }
        if (from >= 0) {
#pragma unroll
            for (int j = kWindow - 1; j >= 0; --j)
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    if (j == from) h[c] = rec[j][c].h;
                    else if (j < from) h[c] = act<kPacked>(rec[j][c].a, rec[j][c].b, h[c]);
                }
            return true;
        }
    }
    return false;
}

// What the CTAs of both directions share.
template <int kC, int kRun>
struct LinSmem {
    float sub[kMaxWarps][2][kC][32];  // the warps' a and b
    float carry[kC][32];              // the state that comes into the chunk
    int start_of[kMaxWarps * kRun], end_of[kMaxWarps * kRun];  // sequence whose first / last token this is, or -1
    unsigned tile;
};

// Where a CTA works.
template <int kC, int kRun>
struct Where {
    int lane, warp, warps, b, d, chunk, ordinal, t0, n;  // t0, n: the warp's tokens
    long long col;
    bool on;
    __device__ __forceinline__ Where(const LinP &p, LinSmem<kC, kRun> &s, bool backward) {
        lane = threadIdx.x;
        warp = threadIdx.y;
        warps = blockDim.y;
        long long tile = blockIdx.x;
        if (p.chunks > 1) {
            if (lane == 0 && warp == 0) s.tile = atomicAdd(p.ticket, 1u);
            __syncthreads();
            tile = s.tile;
        }
        const long long cols = (long long)p.B * p.nd;
        ordinal = (int)(tile / cols);
        col = tile % cols;
        chunk = backward ? p.chunks - 1 - ordinal : ordinal;
        b = (int)(col / p.nd);
        d = (int)(col % p.nd) * 32 * kC + lane * kC;
        on = d < p.D;
        t0 = (chunk * warps + warp) * kRun;
        n = max(0, min(kRun, p.T - t0));
    }
    __device__ __forceinline__ float4 *rec(const LinP &p, int ord) const {
        return p.rec + ((col * p.chunks + ord) * 32 + lane) * kC;
    }
    // Which of the chunk's tokens start and end sequences.
    __device__ __forceinline__ void mark(const LinP &p, LinSmem<kC, kRun> &s) const {
        const int base = chunk * warps * kRun;
        for (int k = warp * 32 + lane; k < warps * kRun; k += warps * 32) {
            const int t = base + k;
            int first = -1, last = -1;
            if (t < p.T) {
                const int q = p.seqs.find(t);
                if (p.seqs.bound(q) == t) first = q;
                if (p.seqs.bound(q + 1) == t + 1) last = q;
            }
            s.start_of[k] = first;
            s.end_of[k] = last;
        }
    }
    // The bounds are meant to rise from 0 to T: one CTA looks them over.
    __device__ __forceinline__ void check(const LinP &p) const {
        if (ordinal != 0 || col != 0) return;
        for (int q = warp * 32 + lane; q <= p.seqs.n; q += warps * 32) {
            const int v = p.seqs.cu[q];
            if ((q == 0 && v != 0) || (q == p.seqs.n && v != p.T) || (q > 0 && v < p.seqs.cu[q - 1])) atomicOr(&g_linear_status, kStatusIndex);
        }
    }
    // What a sequence without tokens hands on (one CTA a column of chunks).
    __device__ __forceinline__ void pass_empty(const LinP &p, const float *from, float *to) const {
        if (!to || ordinal != 0) return;
        for (int q0 = warp * 32; q0 < p.seqs.n; q0 += warps * 32) {
            const int q = q0 + lane;
            unsigned empty = __ballot_sync(0xffffffffu, q < p.seqs.n && p.seqs.bound(q) == p.seqs.bound(q + 1));
            for (; empty; empty &= empty - 1) {
                const long long at = (long long)(q0 + __ffs(empty) - 1) * p.D + d;
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    if (on) to[at + c] = from ? from[at + c] : 0.f;
            }
        }
    }
};

// The state that comes into the chunk, for all warps (s.carry); `first` is the
// one before the chunk with ordinal 0.  The warps' (a, b) lie in s.sub; kBack:
// the last warp acts first.  Called by warp 0.
template <int kC, int kRun, bool kPacked, bool kBack>
__device__ __forceinline__ void hand_over(const LinP &p, LinSmem<kC, kRun> &s, const Where<kC, kRun> &w, const float (&first)[kC]) {
    float a[kC], b[kC], h[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        a[c] = 1.f;
        b[c] = 0.f;
        h[c] = first[c];
    }
    if (p.chunks > 1) {
        for (int k = 0; k < w.warps; ++k) {
            const int v = kBack ? w.warps - 1 - k : k;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const float av = s.sub[v][0][c][w.lane];
                b[c] = act<kPacked>(av, s.sub[v][1][c][w.lane], b[c]);
                a[c] = join<kPacked>(a[c], av);
            }
        }
        float4 *mine = w.rec(p, w.ordinal);
        if (w.ordinal > 0) {
#pragma unroll
            for (int c = 0; c < kC; ++c) write_rec(mine + c, a[c], b[c], 0.f, 1);
            if (!look_back<kC, kPacked>(mine, 32 * kC, w.ordinal, h) && w.lane == 0) atomicOr(&g_linear_status, kStatusTimeout);
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) write_rec(mine + c, a[c], b[c], act<kPacked>(a[c], b[c], h[c]), 2);
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) s.carry[c][w.lane] = h[c];
}

template <typename T, int kC, bool kZ, bool kPacked>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) k_linear_fwd(const LinP p) {
    using V = Ch<T, kC>;
    constexpr int kRun = kFwdRun;
    __shared__ LinSmem<kC, kRun> s;
    const Where<kC, kRun> w(p, s, false);
    V x[kRun], gi[kRun], gr[kRun], gz[kZ ? kRun : 1];
    {
        const T *px = static_cast<const T *>(p.x) + w.b * p.x_batch + w.t0 * p.x_row + w.d;
        const T *pi = static_cast<const T *>(p.i) + w.b * p.i_batch + w.t0 * p.i_row + w.d;
        const T *pr = static_cast<const T *>(p.r) + w.b * p.r_batch + w.t0 * p.r_row + w.d;
        const T *pz = kZ ? static_cast<const T *>(p.z) + w.b * p.z_batch + w.t0 * p.z_row + w.d : nullptr;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            x[j].zero();
            gi[j].zero();
            gr[j].zero();
            if (kZ) gz[j].zero();
            if (w.on && j < w.n) {
                gr[j].load(pr + j * p.r_row);
                gi[j].load(pi + j * p.i_row);
                x[j].load(px + j * p.x_row);
                if (kZ) gz[j].load(pz + j * p.z_row);
            }
        }
    }
    if (kPacked) {
        w.mark(p, s);
        __syncthreads();
    }
    float s2[kC], first[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        s2[c] = w.on ? p.scale * kLog2e * softplusf(p.decay[w.d + c]) : 0.f;
        first[c] = !kPacked && p.h0 && w.on ? p.h0[(long long)w.b * p.D + w.d + c] : 0.f;
    }
    float a[kRun][kC], b[kRun][kC], A[kC], B[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        A[c] = 1.f;
        B[c] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        float fx[kC], fi[kC], fr[kC];
        x[j].get(fx);
        gi[j].get(fi);
        gr[j].get(fr);
        const int start = kPacked ? s.start_of[w.warp * kRun + j] : -1;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float l2, wt;
            decay_of(s2[c], sigmoidf(fr[c]), l2, a[j][c], wt);
            b[j][c] = sqrt_of(wt) * (sigmoidf(fi[c]) * fx[c]);
            if (kPacked && start >= 0) {
                if (p.h0 && w.on) b[j][c] = fmaf(a[j][c], p.h0[(long long)start * p.D + w.d + c], b[j][c]);
                a[j][c] = -1.f;
            }
            if (j < w.n) {
                B[c] = act<kPacked>(a[j][c], b[j][c], B[c]);
                A[c] = join<kPacked>(A[c], a[j][c]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        s.sub[w.warp][0][c][w.lane] = A[c];
        s.sub[w.warp][1][c][w.lane] = B[c];
    }
    __syncthreads();
    if (w.warp == 0) hand_over<kC, kRun, kPacked, false>(p, s, w, first);
    __syncthreads();
    float h[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) h[c] = s.carry[c][w.lane];
    for (int k = 0; k < w.warp; ++k)
#pragma unroll
        for (int c = 0; c < kC; ++c) h[c] = act<kPacked>(s.sub[k][0][c][w.lane], s.sub[k][1][c][w.lane], h[c]);
    if (p.states && w.on && w.n > 0 && w.t0 % kStride == 0) {
        float *to = p.states + ((long long)w.b * ((p.T + kStride - 1) / kStride) + w.t0 / kStride) * p.D + w.d;
#pragma unroll
        for (int c = 0; c < kC; ++c) to[c] = h[c];
    }
    T *py = static_cast<T *>(p.y) + ((long long)w.b * p.T + w.t0) * p.D + w.d;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        if (j < w.n && w.on) {
            float out[kC], fz[kC];
            if (kZ) gz[j].get(fz);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                h[c] = act<kPacked>(a[j][c], b[j][c], h[c]);
                out[c] = kZ ? h[c] * (fz[c] * sigmoidf(fz[c])) : h[c];
            }
            V::store(py + (long long)j * p.D, out);
            const int last = kPacked ? s.end_of[w.warp * kRun + j] : w.t0 + j == p.T - 1 ? w.b : -1;
            if (last >= 0 && p.ht)
#pragma unroll
                for (int c = 0; c < kC; ++c) p.ht[(long long)last * p.D + w.d + c] = h[c];
        }
    }
    if (kPacked) {
        w.pass_empty(p, p.h0, p.ht);
        w.check(p);
    }
}

template <typename T, int kC, bool kZ, bool kPacked>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) k_linear_bwd(const LinP p) {
    using V = Ch<T, kC>;
    constexpr int kRun = kBwdRun;
    __shared__ LinSmem<kC, kRun> s;
    __shared__ float fwd[kMaxWarps][2][kC][32];  // the warps' (a, b) from the first token on
    const Where<kC, kRun> w(p, s, true);
    const long long out = ((long long)w.b * p.T + w.t0) * p.D + w.d;
    V x[kRun], gi[kRun], gr[kRun], gz[kZ ? kRun : 1], gy[kRun];
    {
        const T *px = static_cast<const T *>(p.x) + w.b * p.x_batch + w.t0 * p.x_row + w.d;
        const T *pi = static_cast<const T *>(p.i) + w.b * p.i_batch + w.t0 * p.i_row + w.d;
        const T *pr = static_cast<const T *>(p.r) + w.b * p.r_batch + w.t0 * p.r_row + w.d;
        const T *pz = kZ ? static_cast<const T *>(p.z) + w.b * p.z_batch + w.t0 * p.z_row + w.d : nullptr;
        const T *py = static_cast<const T *>(p.dy) + out;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            x[j].zero();
            gi[j].zero();
            gr[j].zero();
            gy[j].zero();
            if (kZ) gz[j].zero();
            if (w.on && j < w.n) {
                gr[j].load(pr + j * p.r_row);
                gi[j].load(pi + j * p.i_row);
                x[j].load(px + j * p.x_row);
                gy[j].load(py + (long long)j * p.D);
                if (kZ) gz[j].load(pz + j * p.z_row);
            }
        }
    }
    if (kPacked) {
        w.mark(p, s);
        __syncthreads();
    }
    float sl[kC], first[kC], h[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        sl[c] = w.on ? p.scale * softplusf(p.decay[w.d + c]) : 0.f;
        first[c] = !kPacked && p.dht && w.on ? p.dht[(long long)w.b * p.D + w.d + c] : 0.f;
        h[c] = w.on ? p.states[((long long)w.b * ((p.T + kStride - 1) / kStride) + w.chunk * w.warps * kRun / kStride) * p.D + w.d + c] : 0.f;
    }
    auto starts = [&](int j) { return kPacked ? s.start_of[w.warp * kRun + j] : -1; };
    auto ends = [&](int j) { return kPacked ? s.end_of[w.warp * kRun + j] : -1; };
    auto given = [&](const float *t, int q, int c) { return t && w.on ? t[(long long)q * p.D + w.d + c] : 0.f; };
    float a[kRun][kC], m[kRun][kC], si[kRun][kC], sr[kRun][kC];
    float A[kC], B[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        A[c] = 1.f;
        B[c] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        float fx[kC], fi[kC], fr[kC];
        x[j].get(fx);
        gi[j].get(fi);
        gr[j].get(fr);
        const int start = starts(j);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float l2, wt;
            sr[j][c] = sigmoidf(fr[c]);
            si[j][c] = sigmoidf(fi[c]);
            decay_of(sl[c] * kLog2e, sr[j][c], l2, a[j][c], wt);
            m[j][c] = sqrt_of(wt);
            if (j < w.n) {
                const float b = m[j][c] * (si[j][c] * fx[c]);
                if (kPacked && start >= 0) {
                    B[c] = fmaf(a[j][c], given(p.h0, start, c), b);
                    A[c] = -1.f;
                } else {
                    B[c] = fmaf(a[j][c], B[c], b);
                    A[c] = join<kPacked>(A[c], a[j][c]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        fwd[w.warp][0][c][w.lane] = A[c];
        fwd[w.warp][1][c][w.lane] = B[c];
        A[c] = 1.f;
        B[c] = 0.f;
    }
    auto gradient = [&](int j, float (&din)[kC]) {
        gy[j].get(din);
        if (kZ) {
            float fz[kC];
            gz[j].get(fz);
#pragma unroll
            for (int c = 0; c < kC; ++c) din[c] *= fz[c] * sigmoidf(fz[c]);
        }
    };
#pragma unroll
    for (int j = kRun - 1; j >= 0; --j) {
        if (j < w.n) {
            float din[kC];
            gradient(j, din);
            const int last = ends(j);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                if (kPacked && last >= 0) {
                    B[c] = given(p.dht, last, c);
                    A[c] = -1.f;
                } else {
                    A[c] = join<kPacked>(A[c], a[j][c]);
                }
                B[c] = a[j][c] * (din[c] + B[c]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        s.sub[w.warp][0][c][w.lane] = A[c];
        s.sub[w.warp][1][c][w.lane] = B[c];
    }
    __syncthreads();
    if (w.warp == 0) hand_over<kC, kRun, kPacked, true>(p, s, w, first);
    for (int k = 0; k < w.warp; ++k)
#pragma unroll
        for (int c = 0; c < kC; ++c) h[c] = act<kPacked>(fwd[k][0][c][w.lane], fwd[k][1][c][w.lane], h[c]);
    float before[kRun][kC];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        float fx[kC];
        x[j].get(fx);
        const int start = starts(j);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            before[j][c] = kPacked && start >= 0 ? given(p.h0, start, c) : h[c];
            h[c] = fmaf(a[j][c], before[j][c], m[j][c] * (si[j][c] * fx[c]));
        }
    }
    __syncthreads();
    float e[kC], sum[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        e[c] = s.carry[c][w.lane];
        sum[c] = 0.f;
    }
    for (int k = w.warps - 1; k > w.warp; --k)
#pragma unroll
        for (int c = 0; c < kC; ++c) e[c] = act<kPacked>(s.sub[k][0][c][w.lane], s.sub[k][1][c][w.lane], e[c]);
#pragma unroll
    for (int j = kRun - 1; j >= 0; --j) {
        if (j < w.n && w.on) {
            float fx[kC], din[kC], dx[kC], di[kC], dr[kC];
            x[j].get(fx);
            gradient(j, din);
            const int last = ends(j);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                if (kPacked && last >= 0) e[c] = given(p.dht, last, c);
                e[c] += din[c];
                const float u = si[j][c] * fx[c], L = -sl[c] * sr[j][c], aj = a[j][c];
                const float rho = m[j][c] > 0.f ? -L * rcpf(m[j][c]) : 0.f;
                const float g = e[c] * fmaf(L * aj, before[j][c], u * (aj * aj) * rho);
                dx[c] = e[c] * m[j][c] * si[j][c];
                di[c] = dx[c] * (fx[c] * (1.f - si[j][c]));
                dr[c] = g * (1.f - sr[j][c]);
                sum[c] += g;
            }
            const long long at = out + (long long)j * p.D;
            V::store(static_cast<T *>(p.dx) + at, dx);
            V::store(static_cast<T *>(p.di) + at, di);
            V::store(static_cast<T *>(p.dr) + at, dr);
            if (kZ) {
                float dz[kC], fz[kC], fy[kC];
                gz[j].get(fz);
                gy[j].get(fy);
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const float hj = fmaf(a[j][c], before[j][c], m[j][c] * (si[j][c] * fx[c]));
                    float on, off;
                    sigmoids(fz[c], on, off);
                    dz[c] = fy[c] * hj * on * fmaf(fz[c], off, 1.f);
                }
                V::store(static_cast<T *>(p.dz) + at, dz);
            }
            const int start = kPacked ? starts(j) : w.t0 + j == 0 ? w.b : -1;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                e[c] *= a[j][c];
                if (start >= 0 && p.dh0) p.dh0[(long long)start * p.D + w.d + c] = e[c];
            }
        }
    }
    __syncthreads();  // fwd has been read
#pragma unroll
    for (int c = 0; c < kC; ++c) fwd[w.warp][0][c][w.lane] = sum[c];
    __syncthreads();
    if (w.warp == 0 && w.on) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float g = 0.f;
            for (int k = 0; k < w.warps; ++k) g += fwd[k][0][c][w.lane];
            p.part[((long long)w.b * p.chunks + w.chunk) * p.D + w.d + c] = g;
        }
    }
    if (kPacked) {
        w.pass_empty(p, p.dht, p.dh0);
        w.check(p);
    }
}

// ddecay from the chunks' sums in a fixed order, 32 channels a CTA.
__global__ void __launch_bounds__(1024) k_linear_ddecay(const float *part, long long rows, int D, const float *decay, float *ddecay) {
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < D)
        for (long long r = threadIdx.y; r < rows; r += 32) a += part[r * D + c];
    red[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    a = red[threadIdx.x][threadIdx.y];  // warp y adds the 32 parts of channel y
#pragma unroll
    for (int m = 16; m >= 1; m /= 2) a += __shfl_xor_sync(0xffffffffu, a, m);
    const int d = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && d < D) {
        // sigmoid(v) / softplus(v) goes to 1 - e^v / 2 for small e^v, where both may vanish
        const float v = decay[d];
        ddecay[d] = a * (v < -20.f ? 1.f : sigmoidf(v) / softplusf(v));
    }
}

struct LinStepP {
    const void *x, *i, *r, *z;
    const float *decay;
    float *state;
    const int32_t *slots;
    void *y;
    long long x_row, i_row, r_row, z_row, n_slots;
    int D;
    float scale;
};

constexpr int kStepThreads = 128;

template <typename T, int kC>
__global__ void __launch_bounds__(kStepThreads) k_linear_step(const LinStepP p) {
    using V = Ch<T, kC>;
    const long long row = blockIdx.y;
    const int d = (blockIdx.x * kStepThreads + threadIdx.x) * kC;
    const long long slot = p.slots ? p.slots[row] : row;
    const bool known = slot >= 0 && slot < p.n_slots;
    if (slot >= p.n_slots && threadIdx.x == 0) atomicOr(&g_linear_status, kStatusIndex);
    if (d >= p.D) return;
    float y[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) y[c] = 0.f;
    if (known) {
        V x, i, r, z;
        x.load(static_cast<const T *>(p.x) + row * p.x_row + d);
        i.load(static_cast<const T *>(p.i) + row * p.i_row + d);
        r.load(static_cast<const T *>(p.r) + row * p.r_row + d);
        if (p.z) z.load(static_cast<const T *>(p.z) + row * p.z_row + d);
        float *st = p.state + slot * p.D + d;
        float fx[kC], fi[kC], fr[kC], fz[kC];
        x.get(fx);
        i.get(fi);
        r.get(fr);
        if (p.z) z.get(fz);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float l2, a, wt;
            decay_of(p.scale * kLog2e * softplusf(p.decay[d + c]), sigmoidf(fr[c]), l2, a, wt);
            const float h = fmaf(a, st[c], sqrt_of(wt) * (sigmoidf(fi[c]) * fx[c]));
            st[c] = h;
            y[c] = p.z ? h * (fz[c] * sigmoidf(fz[c])) : h;
        }
    }
    V::store(static_cast<T *>(p.y) + row * p.D + d, y);
}

// ---- host ------------------------------------------------------------------

int linear_sizes(long long B, long long T, long long D, int dtype) {
    if (B < 1 || T < 0 || D < 1) return layer_fail(GDR_ERR_SHAPE, "linear scan: B and D must be >= 1 and T >= 0 (got %lld, %lld, %lld)", B, D, T);
    if (T >= (1LL << 30) || D >= (1LL << 24) || B > 65535) return layer_fail(GDR_ERR_SHAPE, "linear scan: problem too large");
    if (dtype != GDR_BF16 && dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "linear scan: unknown dtype %d", dtype);
    return GDR_OK;
}

struct LinPlan {
    int warps;
    long long chunks;
};
LinPlan linear_plan(long long T, bool bwd) {
    const int run = bwd ? kBwdRun : kFwdRun;
    const int warps = (int)std::max(1LL, std::min<long long>(kMaxWarps, (T + run - 1) / run));
    return LinPlan{warps, std::max(1LL, (T + warps * run - 1) / (warps * run))};
}

// The workspace: the counter, the records (where there is more than one chunk),
// the backward's sums.
struct LinSpace {
    size_t rec, part, total, zeroed;
};
LinSpace linear_space(long long B, long long T, long long D, bool bwd) {
    const LinPlan pl = linear_plan(T, bwd);
    LinSpace s{};
    size_t off = 0;
    if (pl.chunks > 1) {
        s.rec = 16;
        off = s.zeroed = 16 + (size_t)B * pl.chunks * ((D + 63) / 64 * 64) * sizeof(float4);
    }
    s.part = off;
    if (bwd) off += (size_t)B * pl.chunks * D * 4;
    s.total = (off + 15) & ~size_t(15);
    return s;
}

int linear_common(const gdr_linear_args *a, Seqs *s) {
    int rc;
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    if ((rc = linear_sizes(a->B, a->T, a->D, a->dtype))) return rc;
    if (a->cu_seqlens ? (a->B != 1 || a->n_seqs < 1) : a->n_seqs != a->B)
        return layer_fail(GDR_ERR_SHAPE, "linear scan: packed sequences need B == 1 and n_seqs >= 1, a batch n_seqs == B");
    if (a->n_seqs > (1 << 24)) return layer_fail(GDR_ERR_SHAPE, "linear scan: too many sequences");
    if (!(a->decay_scale > 0.f) || a->decay_scale > 3e38f) return layer_fail(GDR_ERR_ARG, "linear scan: decay_scale must be positive and finite");
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->T > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("input_gate", a->input_gate, any, e)) ||
        (rc = layer_ptr("decay_gate", a->decay_gate, any, e)) || (rc = layer_ptr("z", a->z, false, e)) ||
        (rc = layer_ptr("decay", a->decay, true, 4)) || (rc = layer_ptr("h0", a->h0, false, 4)) ||
        (rc = layer_ptr("states", a->states, false, 4)) || (rc = layer_ptr("cu_seqlens", a->cu_seqlens, false, 4)))
        return rc;
    s->cu = a->cu_seqlens;
    s->n = (int)a->n_seqs;
    s->T = (int)a->T;
    return GDR_OK;
}

int linear_workspace(const gdr_linear_args *a, const LinSpace &sp, const char *what) {
    if (!sp.total) return GDR_OK;
    if (!a->workspace) return layer_fail(GDR_ERR_WORKSPACE, "%s: workspace is null", what);
    if (!multiple16(a->workspace)) return layer_fail(GDR_ERR_ALIGN, "%s: workspace must be 16-byte aligned", what);
    if (a->workspace_bytes < sp.total)
        return layer_fail(GDR_ERR_WORKSPACE, "%s: workspace too small: %zu < %zu bytes", what, a->workspace_bytes, sp.total);
    return GDR_OK;
}

// Two bf16 channels a lane where pairs lie on 4-byte boundaries.
bool linear_pairs(const gdr_linear_args *a) {
    if (a->dtype != GDR_BF16 || a->D % 2) return false;
    for (long long v : {a->x_row, a->x_batch, a->i_row, a->i_batch, a->r_row, a->r_batch, a->z ? a->z_row : 0, a->z ? a->z_batch : 0})
        if (v % 2) return false;
    for (const void *p : {a->x, a->input_gate, a->decay_gate, a->z, a->dy, static_cast<const void *>(a->y), static_cast<const void *>(a->dx),
                          static_cast<const void *>(a->di), static_cast<const void *>(a->dr), static_cast<const void *>(a->dz)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return false;
    return true;
}

int linear_fill(const gdr_linear_args *a, const Seqs &s, bool bwd, const LinSpace &sp, bool pairs, LinP *p, LinPlan *pl, cudaStream_t st) {
    *p = LinP{};
    *pl = linear_plan(a->T, bwd);
    p->x = a->x; p->i = a->input_gate; p->r = a->decay_gate; p->z = a->z; p->dy = a->dy;
    p->decay = a->decay; p->h0 = a->h0; p->dht = a->dht;
    p->y = a->y; p->dx = a->dx; p->di = a->di; p->dr = a->dr; p->dz = a->dz;
    p->ht = a->ht; p->states = a->states; p->dh0 = a->dh0;
    char *ws = static_cast<char *>(a->workspace);
    p->ticket = reinterpret_cast<unsigned *>(ws);
    p->rec = reinterpret_cast<float4 *>(ws + sp.rec);
    p->part = reinterpret_cast<float *>(ws + sp.part);
    p->seqs = s;
    p->x_row = a->x_row; p->x_batch = a->x_batch; p->i_row = a->i_row; p->i_batch = a->i_batch;
    p->r_row = a->r_row; p->r_batch = a->r_batch; p->z_row = a->z_row; p->z_batch = a->z_batch;
    p->B = (int)a->B; p->T = (int)a->T; p->D = (int)a->D;
    const int ch = pairs ? 64 : 32;
    p->nd = (int)((a->D + ch - 1) / ch);
    p->chunks = (int)pl->chunks;
    p->tiles = (long long)p->B * p->nd * p->chunks;
    p->scale = a->decay_scale;
    if (p->tiles >= (1LL << 31)) return layer_fail(GDR_ERR_SHAPE, "linear scan: problem too large");
    if (sp.zeroed) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sp.zeroed, st);
        if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "linear scan: %s", cudaGetErrorString(e));
    }
    return GDR_OK;
}

template <typename F>
void linear_by_type(const gdr_linear_args *a, bool pairs, F f) {
    auto w = [&](auto t, auto c) {
        auto v = [&](auto z) {
            if (a->cu_seqlens) f(t, c, z, std::true_type{}); else f(t, c, z, std::false_type{});
        };
        if (a->z) v(std::true_type{}); else v(std::false_type{});
    };
    using One = std::integral_constant<int, 1>;
    if (a->dtype == GDR_F32) w(float{}, One{});
    else if (pairs) w(bf16_t{}, std::integral_constant<int, 2>{});
    else w(bf16_t{}, One{});
}

// A call without tokens hands the states through.
int linear_hand_on(const float *from, float *to, size_t n, cudaStream_t st) {
    if (!to) return GDR_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, n * 4, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, n * 4, st);
    return e == cudaSuccess ? GDR_OK : layer_fail(GDR_ERR_CUDA, "linear scan: %s", cudaGetErrorString(e));
}

}  // namespace

namespace gdr {
unsigned linear_take_status(cudaStream_t st) {
    unsigned v = 0, z = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_linear_status, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return 0x80000000u;
    cudaMemcpyToSymbolAsync(g_linear_status, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    if (cudaStreamSynchronize(st) != cudaSuccess) return 0x80000000u;
    return v;
}
}  // namespace gdr

extern "C" {

size_t gdr_linear_fwd_workspace_size(long long B, long long T, long long D) {
    return linear_sizes(B, T, D, GDR_BF16) ? 0 : linear_space(B, T, D, false).total;
}

size_t gdr_linear_bwd_workspace_size(long long B, long long T, long long D) {
    return linear_sizes(B, T, D, GDR_BF16) ? 0 : linear_space(B, T, D, true).total;
}

int gdr_linear_fwd(const gdr_linear_args *a, void *stream) {
    Seqs s;
    int rc = linear_common(a, &s);
    if (rc) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    if ((rc = layer_ptr("y", a->y, a->T > 0, e)) || (rc = layer_ptr("ht", a->ht, false, 4))) return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->T == 0) return linear_hand_on(a->h0, a->ht, (size_t)a->n_seqs * a->D, st);
    const LinSpace sp = linear_space(a->B, a->T, a->D, false);
    if ((rc = linear_workspace(a, sp, "linear scan forward"))) return rc;
    const bool pairs = linear_pairs(a);
    LinP p;
    LinPlan pl;
    if ((rc = linear_fill(a, s, false, sp, pairs, &p, &pl, st))) return rc;
    linear_by_type(a, pairs, [&](auto t, auto c, auto z, auto k) {
        k_linear_fwd<decltype(t), decltype(c)::value, decltype(z)::value, decltype(k)::value><<<(unsigned)p.tiles, dim3(32, pl.warps), 0, st>>>(p);
    });
    return layer_launched("linear scan forward");
}

int gdr_linear_bwd(const gdr_linear_args *a, void *stream) {
    Seqs s;
    int rc = linear_common(a, &s);
    if (rc) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->T > 0;
    if ((rc = layer_ptr("dy", a->dy, any, e)) || (rc = layer_ptr("states", a->states, any, 4)) || (rc = layer_ptr("dht", a->dht, false, 4)) ||
        (rc = layer_ptr("dx", a->dx, any, e)) || (rc = layer_ptr("di", a->di, any, e)) || (rc = layer_ptr("dr", a->dr, any, e)) ||
        (rc = layer_ptr("dz", a->dz, any && a->z, e)) || (rc = layer_ptr("ddecay", a->ddecay, true, 4)) || (rc = layer_ptr("dh0", a->dh0, false, 4)))
        return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!any) {
        if ((rc = linear_hand_on(nullptr, a->ddecay, a->D, st))) return rc;
        return linear_hand_on(a->dht, a->dh0, (size_t)a->n_seqs * a->D, st);
    }
    const LinSpace sp = linear_space(a->B, a->T, a->D, true);
    if ((rc = linear_workspace(a, sp, "linear scan backward"))) return rc;
    const bool pairs = linear_pairs(a);
    LinP p;
    LinPlan pl;
    if ((rc = linear_fill(a, s, true, sp, pairs, &p, &pl, st))) return rc;
    linear_by_type(a, pairs, [&](auto t, auto c, auto z, auto k) {
        k_linear_bwd<decltype(t), decltype(c)::value, decltype(z)::value, decltype(k)::value><<<(unsigned)p.tiles, dim3(32, pl.warps), 0, st>>>(p);
    });
    k_linear_ddecay<<<(unsigned)((a->D + 31) / 32), dim3(32, 32), 0, st>>>(p.part, (long long)p.B * p.chunks, p.D, a->decay, a->ddecay);
    return layer_launched("linear scan backward");
}

int gdr_linear_step(const gdr_linear_step_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    if ((rc = linear_sizes(1, a->rows, a->D, a->dtype))) return rc;
    if (a->rows > 65535) return layer_fail(GDR_ERR_SHAPE, "linear step: at most 65535 rows");
    if (a->n_slots < 0 || (!a->slots && a->n_slots < a->rows))
        return layer_fail(GDR_ERR_SHAPE, "linear step: %lld state slots for %lld rows", a->n_slots, a->rows);
    if (!(a->decay_scale > 0.f) || a->decay_scale > 3e38f) return layer_fail(GDR_ERR_ARG, "linear step: decay_scale must be positive and finite");
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->rows > 0;
    if ((rc = layer_ptr("x", a->x, any, e)) || (rc = layer_ptr("input_gate", a->input_gate, any, e)) ||
        (rc = layer_ptr("decay_gate", a->decay_gate, any, e)) || (rc = layer_ptr("z", a->z, false, e)) ||
        (rc = layer_ptr("decay", a->decay, true, 4)) || (rc = layer_ptr("state", a->state, any && a->n_slots > 0, 4)) ||
        (rc = layer_ptr("slots", a->slots, false, 4)) || (rc = layer_ptr("y", a->y, any, e)))
        return rc;
    if (!any) return GDR_OK;
    LinStepP p{a->x, a->input_gate, a->decay_gate, a->z, a->decay, a->state, a->slots, a->y,
               a->x_row, a->i_row, a->r_row, a->z_row, a->n_slots, (int)a->D, a->decay_scale};
    bool pairs = a->dtype == GDR_BF16 && a->D % 2 == 0;
    for (long long v : {a->x_row, a->i_row, a->r_row, a->z ? a->z_row : 0}) pairs = pairs && v % 2 == 0;
    for (const void *q : {a->x, a->input_gate, a->decay_gate, a->z, static_cast<const void *>(a->y)})
        pairs = pairs && !(reinterpret_cast<uintptr_t>(q) & 3u);
    const long long per = kStepThreads * (pairs ? 2 : 1);
    const dim3 grid((unsigned)((a->D + per - 1) / per), (unsigned)a->rows);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->dtype == GDR_F32) k_linear_step<float, 1><<<grid, kStepThreads, 0, st>>>(p);
    else if (pairs) k_linear_step<bf16_t, 2><<<grid, kStepThreads, 0, st>>>(p);
    else k_linear_step<bf16_t, 1><<<grid, kStepThreads, 0, st>>>(p);
    return layer_launched("linear step");
}

}  // extern "C"
