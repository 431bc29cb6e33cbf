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
// Bound by arithmetic: T D N exponentials a pass (the special-function units
// take 4 cycles for a warp's, packed fp32 pairs 2, both measured) and about
// five fp32 operations beside each, against 8 bytes of bf16 a (t, d).  So a
// state stays in registers (four neighbouring states of a channel a lane, pairs
// in packed fp32 instructions), and a CTA's warps are split by role: four scan,
// one an SM quarter, and do nothing else; four more read the next tile of
// tokens (softplus and silu are evaluated there, once a (t, d)) and finish the
// tile before (sums over a channel's lanes, skip, gate).  The roles meet at one
// barrier a tile, over double buffers.
//
// Where sequences x channels leave SMs idle the tokens are cut into segments:
// a summary pass gives each segment's end state from a zero start, and as the
// transition over a segment is e^{A sum s}, a segment's start state follows
// from the summaries before it (back to the last sequence start) in the main
// pass itself.  The backward does the same from the other end; it takes its
// states from the forward's checkpoints, one before every 16th token.
//
// 8192 tokens x 4096 channels x 16 states, bf16: 230 us (first form, one role
// a thread: 402); 2 x 2048 tokens forward 113 us, backward 493 (1180).  What
// bounds them is the shared-memory pipe (28 and about 140 cycles a token of a
// CTA) and, with one CTA an SM, the roles' own latencies.
#include "gdr_layer.h"

namespace {

__device__ unsigned g_ssm_status;

constexpr int kThreads = 128;          // scanning threads of a CTA
constexpr int kBack = GDR_SSM_STRIDE;  // tokens of a backward tile, and between checkpoints
constexpr int kGroup = 8;              // tokens of a backward tile whose latencies overlap

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

__device__ __forceinline__ f32x2 dup(float v) { return mk2(v, v); }

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
// e^{s A} of four states, A2 = A log2 e.  ex2.approx lies low by 1.8e-8 to 2.7e-8
// on average for arguments between -1/4 and -2^-8, by 5e-9 to 8e-9 nearer to zero
// (measured; single values within 1.2e-7), and a slow state multiplies hundreds of
// decays: the argument is moved up by what makes 1.5e-8 of the result, in the same
// instruction.  ex2.approx(2.2e-8) is 1 (measured), so that tokens without a step
// change nothing.
__device__ __forceinline__ State decay(const State &A2, f32x2 s2) {
    const f32x2 low = dup(2.2e-8f);  // 1.5e-8 log2 e
    float a, b, c, d;
    un2(fma2(A2.a, s2, low), a, b);
    un2(fma2(A2.b, s2, low), c, d);
    return State{mk2(ex2f(a), ex2f(b)), mk2(ex2f(c), ex2f(d))};
}
__device__ __forceinline__ State advance(const State &a, const State &h, f32x2 i2, const State &Bt) {
    return State{fma2(a.a, h.a, mul2(i2, Bt.a)), fma2(a.b, h.b, mul2(i2, Bt.b))};
}

// Where a thread works: channel d (states n0 .. n0 + 3), whether it exists.
// Neighbouring lanes are neighbouring channels and share their states' place:
// 16-byte reads of B and C then cost 2 cycles of the shared-memory pipe; 4 with
// the states' places across neighbouring lanes (both measured).
template <int kL>
struct Place {
    static constexpr int kCh = kThreads / kL, kN = 4 * kL, kC = 32 / kL;  // kC: channels of a warp
    int g, gt, c0, nch, ch, q, d, n0;
    bool on;
    __device__ __forceinline__ explicit Place(const SsmP &p) {
        gt = blockIdx.x;
        g = gt / p.tiles;
        c0 = g * p.Dg + (gt % p.tiles) * kCh;
        nch = min(kCh, (g + 1) * p.Dg - c0);
        ch = threadIdx.x % kThreads / 32 * kC + threadIdx.x % kC;
        q = threadIdx.x % 32 / kC;
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
// up to (not including) seg: v <- e^{A sum s_j} v + summary_j.  Nothing comes
// before the first of them, in which the sequence starts (or, backwards, ends);
// its sum of s is left out, for it holds other sequences' tokens too, and 0
// times the infinity or NaN that they can make of it is not 0.
template <int kL>
__device__ __forceinline__ State chain(const SsmP &p, const Place<kL> &w, const State &A2, int b, int j0, int seg, int step) {
    State v = zero_state();
    if (!w.on) return v;
    for (int j = j0; j != seg; j += step) {
        const long long row = (long long)b * p.S + j;
        const State e = load_state(p.sum_h + w.at(row, p));
        if (j == j0) {
            v = e;
            continue;
        }
        const State a = decay(A2, dup(p.sum_s[row * p.D + w.d]));
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

// Eight neighbouring elements on their way.  Where rows are not 16-byte
// aligned (odd widths), bf16 elements come in the aligned 16-byte pieces that
// hold them (each holds at least one of them, so none leaves the tensor's
// memory) and are cut out once they have arrived; fp32 ones come one by one
// (three pieces for eight of them cost registers: 77 against 62 us for packed
// prompts of 3001 x 1031).
template <typename T, bool kVec>
struct Flight {
    static constexpr bool kCut = !kVec && sizeof(T) == 2;
    static constexpr int kPieces = sizeof(T) / 2 + (kCut ? 1 : 0);
    uint4 w[kPieces];
    int off, n;
    __device__ __forceinline__ void fetch(const T *p, int count) {  // count elements exist, at most eight
        if (kVec) {
            const Raw8<T> r = load8<T>(p, count);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) w[i] = r.w[i];
            return;
        }
        if (!kCut) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < count ? reinterpret_cast<const uint32_t *>(p)[i] : 0u;
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            return;
        }
        n = min(count, 8);
        off = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
        const uint4 *base = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            w[i] = 16 * i < off + n * (int)sizeof(T) && n > 0 ? base[i] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ Raw8<T> land() const {
        Raw8<T> r;
        if constexpr (!kCut) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) r.w[i] = w[i];
        } else {
            uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 6; ++i) v[i] = off & 8 ? v[i + 2] : v[i];
#pragma unroll
            for (int i = 0; i < 5; ++i) v[i] = off & 4 ? v[i + 1] : v[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = off & 2 ? __funnelshift_r(v[i], v[i + 1], 16) : v[i];
            if (n < 8)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= n) v[e / 2] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
            r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
        }
        return r;
    }
};

// Eight neighbouring channels of one token as packed pairs.
template <typename T>
__device__ __forceinline__ void get8(const Raw8<T> &r, f32x2 (&v)[4]) {
    float f[8];
    unpack8(r, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = mk2(f[2 * k], f[2 * k + 1]);
}
template <typename T, bool kVec>
__device__ __forceinline__ void put8(T *p, const f32x2 (&v)[4], int n) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) un2(v[k], f[2 * k], f[2 * k + 1]);
    store8<T, kVec>(p, f, n);
}
// Parameters of eight channels, zeros where there are none.
__device__ __forceinline__ void param8(const float *p, int n, f32x2 (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = mk2(p && 2 * k < n ? p[2 * k] : 0.f, p && 2 * k + 1 < n ? p[2 * k + 1] : 0.f);
}
// A helper owns eight channels of a token, 128 bytes of 16-byte entries, and
// its neighbours the next ones: entry e of them lies at place e ^ place_key, so
// that eight threads' accesses to their e-th entries fall into eight different
// bank groups.
template <int kCh>
__device__ __forceinline__ int place_key(int row, int ch) { return (row * (kCh / 8) + ch / 8) & 7; }
template <int kCh>
__device__ __forceinline__ int place(int row, int ch) { return ch ^ place_key<kCh>(row, ch); }
// The same for 8-byte entries, moved two at a time.
template <int kCh>
__device__ __forceinline__ int pair_key(int row, int ch) { return (row * (kCh / 8) + ch / 8) & 6; }
template <int kCh>
__device__ __forceinline__ int pair_place(int row, int ch) { return ch ^ pair_key<kCh>(row, ch); }
// The scalar functions of gdr_layer.h for two values at once.
__device__ __forceinline__ f32x2 softplus2(f32x2 v) {
    float a, b;
    un2(v, a, b);
    const float ua = ex2f(-kLog2e * fabsf(a)), ub = ex2f(-kLog2e * fabsf(b));
    float da, db;
    un2(add2(mk2(ua, ub), dup(2.f)), da, db);
    const f32x2 s = mul2(mk2(ua, ub), mk2(rcpf(da), rcpf(db))), s2 = mul2(s, s);
    f32x2 p = fma2(s2, dup(1.f / 13), dup(1.f / 11));
    p = fma2(s2, p, dup(1.f / 9));
    p = fma2(s2, p, dup(1.f / 7));
    p = fma2(s2, p, dup(1.f / 5));
    p = fma2(s2, p, dup(1.f / 3));
    p = fma2(s2, p, dup(1.f));
    return fma2(add2(s, s), p, mk2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
__device__ __forceinline__ f32x2 sigmoid2(f32x2 v) {
    float a, b;
    un2(mul2(v, dup(-kLog2e)), a, b);
    un2(add2(mk2(ex2f(a), ex2f(b)), dup(1.f)), a, b);
    return mk2(rcpf(a), rcpf(b));
}
// Sum of a channel's kL partial sums, which lie together.
template <int kL>
__device__ __forceinline__ float lane_sum(const float *p) {
    if (kL == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        return v.x + v.y;
    }
    float4 v = *reinterpret_cast<const float4 *>(p);
#pragma unroll
    for (int i = 4; i < kL; i += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(p + i);
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    return (v.x + v.y) + (v.z + v.w);
}

// Forward, or (kSum) the segments' summaries.  kHelp: groups of 128 helping
// threads.  One where two CTAs share an SM; two (and tiles of 64 tokens) where
// a CTA has an SM to itself: the helpers of 32 tokens take 0.84 us there, the
// scan 0.75 us, each waiting on its own latencies.
template <int kL, bool kSum, int kHelp>
struct FwdSmem {
    static constexpr int kTile = 32 * kHelp, kCh = kThreads / kL, kN = 4 * kL;
    float2 in[2][kTile][kCh];  // s, s x
    float B[2][kTile][kN];
    float C[kSum ? 1 : 2][kTile][kN];
    float part[kSum ? 1 : 2][kTile][kCh][kL];  // C . h, a lane's part
};

template <typename T, int kL, bool kVec, bool kSum, int kHelp>
__global__ void __launch_bounds__((1 + kHelp) * kThreads, kHelp == 1 ? 2 : 1) k_ssm_fwd(const SsmP p) {
    using W = Place<kL>;
    using S = FwdSmem<kL, kSum, kHelp>;
    constexpr int kCh = W::kCh, kN = W::kN, kTile = S::kTile, kHelpers = kHelp * kThreads;
    extern __shared__ __align__(16) char smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_ssm_status);
    const W w(p);
    const int seg = blockIdx.y, b = blockIdx.z;
    const int ts = seg * p.seg_len, te = min(ts + p.seg_len, p.T), tiles = (te - ts + kTile - 1) / kTile;

    if (threadIdx.x >= kThreads) {  // ---- the helpers
        constexpr int kItems = kTile * kCh / 8, kNI = (kItems + kHelpers - 1) / kHelpers;  // 8 channels of a token each
        constexpr int kBV = kTile * kN / 8, kNB = ((kSum ? 1 : 2) * kBV + kHelpers - 1) / kHelpers;
        constexpr int kRows = kHelpers / (kCh / 8);  // tokens from a thread's item to its next
        const int ht = threadIdx.x - kThreads;
        const int c = ht % (kCh / 8) * 8, row0 = ht / (kCh / 8), nv = min(8, w.nch - c);
        const T *x = static_cast<const T *>(p.x) + b * p.x_batch + w.c0 + c;
        const T *dt = static_cast<const T *>(p.dt) + b * p.dt_batch + w.c0 + c;
        const T *z = p.z ? static_cast<const T *>(p.z) + b * p.z_batch + w.c0 + c : nullptr;
        const T *Bm = static_cast<const T *>(p.Bm) + b * p.b_batch + (long long)w.g * kN;
        const T *Cm = static_cast<const T *>(p.Cm) + b * p.c_batch + (long long)w.g * kN;
        T *y = static_cast<T *>(p.y) + (long long)b * p.T * p.D + w.c0 + c;
        f32x2 bias[4], skip[4];
        param8(p.dt_bias ? p.dt_bias + w.c0 + c : nullptr, nv, bias);
        param8(p.skip ? p.skip + w.c0 + c : nullptr, nv, skip);
        struct Fetched {
            Raw8<T> x[kNI], dt[kNI], z[kNI], bc[kNB];
        };
        struct Flying {
            Flight<T, kVec> x[kNI], dt[kNI], z[kNI], bc[kNB];
        };
        auto land = [&](const Flying &f) {
            Fetched g;
#pragma unroll
            for (int i = 0; i < kNI; ++i) {
                g.x[i] = f.x[i].land();
                g.dt[i] = f.dt[i].land();
                if (!kSum && z) g.z[i] = f.z[i].land();
            }
#pragma unroll
            for (int i = 0; i < kNB; ++i) g.bc[i] = f.bc[i].land();
            return g;
        };
        auto fetch = [&](int tb, Flying &f) {
#pragma unroll
            for (int i = 0; i < kNI; ++i) {
                const int row = tb + row0 + i * kRows, n = ht + i * kHelpers < kItems && row < te ? nv : 0;
                f.x[i].fetch(x + row * p.x_row, n);
                f.dt[i].fetch(dt + row * p.dt_row, n);
                if (!kSum && z) f.z[i].fetch(z + row * p.z_row, n);
            }
#pragma unroll
            for (int i = 0; i < kNB; ++i) {
                const int v = ht + i * kHelpers, r = v % kBV, row = tb + r / (kN / 8), col = (r % (kN / 8)) * 8;
                const int n = v < (kSum ? 1 : 2) * kBV && row < te ? 8 : 0;
                f.bc[i].fetch(v >= kBV ? Cm + row * p.c_row + col : Bm + row * p.b_row + col, n);
            }
        };
        auto stage = [&](int tb, int buf, const Fetched &f) {
#pragma unroll
            for (int i = 0; i < kNI; ++i) {
                if (ht + i * kHelpers >= kItems) continue;
                const int row = row0 + i * kRows, key = pair_key<kCh>(row, c);
                const bool real = tb + row < te;  // past the end: no decay, no input
                f32x2 xv[4], dv[4];
                get8(f.x[i], xv);
                get8(f.dt[i], dv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f32x2 st = add2(dv[k], bias[k]);
                    if (p.softplus) st = softplus2(st);
                    if (!real) st = dup(0.f);
                    float s0, s1, i0, i1;
                    un2(st, s0, s1);
                    un2(mul2(st, xv[k]), i0, i1);
                    *reinterpret_cast<float4 *>(&sm.in[buf][row][c + ((2 * k) ^ key)]) = make_float4(s0, i0, s1, i1);
                }
            }
#pragma unroll
            for (int i = 0; i < kNB; ++i) {
                const int v = ht + i * kHelpers, r = v % kBV, row = r / (kN / 8), col = (r % (kN / 8)) * 8;
                if (v >= (kSum ? 1 : 2) * kBV) continue;
                float g[8];
                unpack8(f.bc[i], g);
                float *to = !kSum && v >= kBV ? &sm.C[kSum ? 0 : buf][row][col] : &sm.B[buf][row][col];
                *reinterpret_cast<float4 *>(to) = make_float4(g[0], g[1], g[2], g[3]);
                *reinterpret_cast<float4 *>(to + 4) = make_float4(g[4], g[5], g[6], g[7]);
            }
        };
        // Tiles in flight: the one to finish, the one being scanned, the one to
        // stage, and the one being fetched.
        Fetched done, now, next;
        Flying then;
        fetch(ts, then);
        now = land(then);
        if (tiles > 1) fetch(ts + kTile, then);
        stage(ts, 0, now);
        next = land(then);
        __syncthreads();
        for (int i = 0; i <= tiles; ++i) {
            if (i + 2 < tiles) fetch(ts + (i + 2) * kTile, then);
            if (i + 1 < tiles) stage(ts + (i + 1) * kTile, (i + 1) & 1, next);
            if (!kSum && i > 0) {
                const int tp = ts + (i - 1) * kTile;
#pragma unroll
                for (int j = 0; j < kNI; ++j) {
                    const int row = row0 + j * kRows, key = place_key<kCh>(row, c);
                    if (ht + j * kHelpers >= kItems || tp + row >= te || nv <= 0) continue;
                    f32x2 xv[4], zv[4], u[4];
                    get8(done.x[j], xv);
                    if (z) get8(done.z[j], zv);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float(*part)[kL] = &sm.part[kSum ? 0 : (i - 1) & 1][row][c];
                        u[k] = fma2(skip[k], xv[k], mk2(lane_sum<kL>(part[(2 * k) ^ key]), lane_sum<kL>(part[(2 * k + 1) ^ key])));
                        if (z) u[k] = mul2(u[k], mul2(zv[k], sigmoid2(zv[k])));
                    }
                    put8<T, kVec>(y + (long long)(tp + row) * p.D, u, nv);
                }
            }
            done = now;
            now = next;
            next = land(then);
            if (i < tiles) __syncthreads();
        }
        return;
    }

    // ---- the scan
    const int sbase = p.seqs.cu ? 0 : b;
    const State A2 = load_A2<kL>(p, w, nullptr);
    int n = p.seqs.find(ts), s0 = p.seqs.bound(n), s1 = p.seqs.bound(n + 1);
    State h;
    if (ts <= s0) h = start_state<kL>(p, w, sbase + n);
    else h = kSum ? zero_state() : chain<kL>(p, w, A2, b, s0 / p.seg_len, seg, 1);
    if (!kSum && seg == 0 && p.seqs.cu)
        for (int m = 0; m < p.seqs.n && p.seqs.bound(m + 1) <= 0; ++m) pass_state<kL>(p, w, p.h0, p.ht, m);
    float total = 0.f;
    const long long ck0 = (long long)b * ((p.T + kBack - 1) / kBack);
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const int tb = ts + i * kTile, buf = i & 1;
        auto keep = [&](int t) {  // the checkpoint before token t
            if (!kSum && p.states && w.on) store_state(p.states + w.at(ck0 + t / kBack, p), h);
        };
        auto one = [&](int r) {
            const float2 in = sm.in[buf][r][pair_place<kCh>(r, w.ch)];
            h = advance(decay(A2, dup(in.x)), h, dup(in.y), load_state(&sm.B[buf][r][w.n0]));
            if (kSum) total += in.x;
            return kSum ? 0.f : dot(h, load_state(&sm.C[kSum ? 0 : buf][r][w.n0]));
        };
        auto put = [&](int r, float u) {
            if (!kSum) sm.part[kSum ? 0 : buf][r][place<kCh>(r, w.ch)][w.q] = u;
        };
        const int tend = min(tb + kTile, te);
        if (p.seqs.cu && s1 < tend) {  // a sequence ends inside the tile, or ended before it
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
                for (; t < to; ++t) {
                    if (t % kBack == 0) keep(t);
                    put(t - tb, one(t - tb));
                }
                if (!kSum && t == s1) {
                    if (p.ht && w.on) store_state(p.ht + w.at(sbase + n, p), h);
                    for (int m = n + 1; m < p.seqs.n && p.seqs.bound(m + 1) <= s1; ++m) pass_state<kL>(p, w, p.h0, p.ht, m);
                }
            }
        } else {  // tokens past the end change nothing
#pragma unroll 1
            for (int g = 0; g < kTile; g += kBack) {
                if (tb + g < te) keep(tb + g);
                float u[kBack];  // stored after the last load: a store would hold back the loads behind it
#pragma unroll
                for (int r = 0; r < kBack; ++r) u[r] = one(g + r);
#pragma unroll
                for (int r = 0; r < kBack; ++r) put(g + r, u[r]);
            }
            if (!kSum && p.ht && tend == s1 && w.on) {
                store_state(p.ht + w.at(sbase + n, p), h);
                if (p.seqs.cu)
                    for (int m = n + 1; m < p.seqs.n && p.seqs.bound(m + 1) <= s1; ++m) pass_state<kL>(p, w, p.h0, p.ht, m);
            }
        }
        __syncthreads();
    }
    if (kSum && w.on) {
        const long long row = (long long)b * p.S + seg;
        store_state(p.sum_h + w.at(row, p), h);
        if (w.q == 0) p.sum_s[row * p.D + w.d] = total;
    }
}

// Backward, or (kSum) the segments' reverse summaries.  Tiles of kBack tokens
// from the segment's end: a scanning lane recomputes the states of a tile from
// its checkpoint, keeps them in registers, and runs the gradient back over
// them (the decays are formed again: the special-function units have room, the
// registers have not).
//
// dB and dC are sums over channels, which lie across lanes: two exchanges leave
// every lane with one state's sum over four channels, the helpers add the rest.
template <int kL, bool kSum>
struct BwdSmem {
    static constexpr int kCh = kThreads / kL, kN = 4 * kL, kC = 32 / kL;  // kC: channels of a warp
    static constexpr int kFold = kC < 4 ? kC : 4, kParts = kThreads / 32 * (kC / kFold);
    float2 in[2][kBack][kCh];  // s, s x
    float du[2][kBack][kCh];
    float B[2][kBack][kN], C[2][kBack][kN];
    float u[kSum ? 1 : 2][kBack][kCh][kL], eb[kSum ? 1 : 2][kBack][kCh][kL], fa[kSum ? 1 : 2][kBack][kCh][kL];
    float dB[kSum ? 1 : 2][kBack][kParts][kN], dC[kSum ? 1 : 2][kBack][kParts][kN];
};

// The sum over kFold neighbouring lanes of four states: lane m of them ends
// with state m's (of two lanes, lane m with states 2 m and 2 m + 1).
template <int kL>
__device__ __forceinline__ float2 fold_channels(State v) {
    constexpr int kC = 32 / kL, kFirst = kC >= 4 ? 2 : 1;
    const bool up = threadIdx.x & kFirst;
    float lo, hi;
    un2(up ? v.a : v.b, lo, hi);
    un2(add2(up ? v.b : v.a, mk2(__shfl_xor_sync(0xffffffffu, lo, kFirst), __shfl_xor_sync(0xffffffffu, hi, kFirst))), lo, hi);
    if (kC >= 4) {
        const bool odd = threadIdx.x & 1;
        return make_float2((odd ? hi : lo) + __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1), 0.f);
    }
    return make_float2(lo, hi);
}
template <int kL>
__device__ __forceinline__ void put_fold(float *to, float2 v) {
    if (32 / kL >= 4) *to = v.x;
    else *reinterpret_cast<float2 *>(to) = v;
}

template <typename T, int kL, bool kVec, bool kSum>
__global__ void __launch_bounds__(2 * kThreads, sizeof(T) == 2 ? 2 : 1) k_ssm_bwd(const SsmP p) {
    using W = Place<kL>;
    using S = BwdSmem<kL, kSum>;
    constexpr int kCh = W::kCh, kN = W::kN;
    extern __shared__ __align__(16) char smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_bounds(p.seqs, &g_ssm_status);
    const W w(p);
    const int b = blockIdx.z, seg = kSum ? blockIdx.y + 1 : blockIdx.y;  // nothing follows from the first segment's summary
    const int ts = seg * p.seg_len, te = min(ts + p.seg_len, p.T), tiles = (te - ts + kBack - 1) / kBack;
    const long long srow = (long long)b * p.S + seg;

    if (threadIdx.x >= kThreads) {  // ---- the helpers
        // An item is eight channels of a token: of x and dt (items below kPer: s, dx, ddt) or of dy and z (du, dz).
        constexpr int kPer = kBack * kCh / 8, kNI = (2 * kPer + kThreads - 1) / kThreads;
        constexpr int kBV = kBack * kN / 8, kNB = (2 * kBV + kThreads - 1) / kThreads;
        const int ht = threadIdx.x - kThreads;
        const int c = ht % (kCh / 8) * 8, row = ht % kPer / (kCh / 8), nv = min(8, w.nch - c);
        const int key = place_key<kCh>(row, c), key2 = pair_key<kCh>(row, c);
        const T *x = static_cast<const T *>(p.x) + b * p.x_batch + w.c0 + c;
        const T *dt = static_cast<const T *>(p.dt) + b * p.dt_batch + w.c0 + c;
        const T *z = p.z ? static_cast<const T *>(p.z) + b * p.z_batch + w.c0 + c : nullptr;
        const long long own = (long long)b * p.T * p.D + w.c0 + c;
        const T *dy = static_cast<const T *>(p.dy) + own;
        const T *Bm = static_cast<const T *>(p.Bm) + b * p.b_batch + (long long)w.g * kN;
        const T *Cm = static_cast<const T *>(p.Cm) + b * p.c_batch + (long long)w.g * kN;
        f32x2 bias[4], skip[4], gskip[4], gbias[4];
        param8(p.dt_bias ? p.dt_bias + w.c0 + c : nullptr, nv, bias);
        param8(p.skip ? p.skip + w.c0 + c : nullptr, nv, skip);
#pragma unroll
        for (int k = 0; k < 4; ++k) gskip[k] = gbias[k] = dup(0.f);
        struct Fetched {
            Raw8<T> x[kNI], g[kNI], z[kNI], bc[kNB];  // g: dt, or dy
        };
        struct Flying {
            Flight<T, kVec> x[kNI], g[kNI], z[kNI], bc[kNB];
        };
        auto land = [&](const Flying &f) {
            Fetched r;
#pragma unroll
            for (int i = 0; i < kNI; ++i) {
                r.x[i] = f.x[i].land();
                r.g[i] = f.g[i].land();
                if (z) r.z[i] = f.z[i].land();
            }
#pragma unroll
            for (int i = 0; i < kNB; ++i) r.bc[i] = f.bc[i].land();
            return r;
        };
        auto fetch = [&](int tb, Flying &f) {
#pragma unroll
            for (int i = 0; i < kNI; ++i) {
                const int v = ht + i * kThreads, t = tb + row, n = v < 2 * kPer && t < te ? nv : 0;
                f.x[i].fetch(x + t * p.x_row, n);
                f.g[i].fetch(v < kPer ? dt + t * p.dt_row : dy + (long long)t * p.D, n);
                if (z) f.z[i].fetch(z + t * p.z_row, v >= kPer ? n : 0);
            }
#pragma unroll
            for (int i = 0; i < kNB; ++i) {
                const int v = ht + i * kThreads, r = v % kBV, t = tb + r / (kN / 8), col = (r % (kN / 8)) * 8;
                const int n = v < 2 * kBV && t < te ? 8 : 0;
                f.bc[i].fetch(v >= kBV ? Cm + t * p.c_row + col : Bm + t * p.b_row + col, n);
            }
        };
        auto stage = [&](int tb, int buf, const Fetched &f) {
#pragma unroll
            for (int i = 0; i < kNI; ++i) {
                const int v = ht + i * kThreads;
                if (v >= 2 * kPer) continue;
                f32x2 g[4];
                get8(f.g[i], g);
                if (v < kPer) {
                    const bool real = tb + row < te;  // past the end: no decay, no input
                    f32x2 xv[4];
                    get8(f.x[i], xv);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f32x2 st = add2(g[k], bias[k]);
                        if (p.softplus) st = softplus2(st);
                        if (!real) st = dup(0.f);
                        float s0, s1, i0, i1;
                        un2(st, s0, s1);
                        un2(mul2(st, xv[k]), i0, i1);
                        *reinterpret_cast<float4 *>(&sm.in[buf][row][c + ((2 * k) ^ key2)]) = make_float4(s0, i0, s1, i1);
                    }
                } else {
                    if (z) {
                        f32x2 zv[4];
                        get8(f.z[i], zv);
#pragma unroll
                        for (int k = 0; k < 4; ++k) g[k] = mul2(g[k], mul2(zv[k], sigmoid2(zv[k])));
                    }
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        float4 u;
                        un2(g[k], u.x, u.y);
                        un2(g[k + 1], u.z, u.w);
                        *reinterpret_cast<float4 *>(&sm.du[buf][row][c + 2 * k]) = u;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kNB; ++i) {
                const int v = ht + i * kThreads, r = v % kBV, rr = r / (kN / 8), col = (r % (kN / 8)) * 8;
                if (v >= 2 * kBV) continue;
                float g[8];
                unpack8(f.bc[i], g);
                float *to = v >= kBV ? &sm.C[buf][rr][col] : &sm.B[buf][rr][col];
                *reinterpret_cast<float4 *>(to) = make_float4(g[0], g[1], g[2], g[3]);
                *reinterpret_cast<float4 *>(to + 4) = make_float4(g[4], g[5], g[6], g[7]);
            }
        };
        const int last = ts + (tiles - 1) * kBack;
        Fetched done, now, next;  // as in the forward
        Flying then;
        fetch(last, then);
        now = land(then);
        if (tiles > 1) fetch(last - kBack, then);
        stage(last, 0, now);
        next = land(then);
        __syncthreads();
        for (int i = 0; i <= tiles; ++i) {
            if (i + 2 < tiles) fetch(last - (i + 2) * kBack, then);
            const int tp = last - (i - 1) * kBack, pb = (i - 1) & 1;  // the tile to finish
            if (!kSum && i > 0) {
#pragma unroll
                for (int j = 0; j < kNI; ++j) {
                    const int v = ht + j * kThreads;
                    if (v >= 2 * kPer || tp + row >= te || nv <= 0) continue;
                    const long long at = own + (long long)(tp + row) * p.D;
                    f32x2 xv[4], g[4], o[4];
                    get8(done.x[j], xv);
                    get8(done.g[j], g);
                    if (v < kPer) {
                        f32x2 dd[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int e0 = c + ((2 * k) ^ key), e1 = c + ((2 * k + 1) ^ key);
                            const float4 in = *reinterpret_cast<const float4 *>(&sm.in[pb][row][c + ((2 * k) ^ key2)]);
                            const float2 u2 = *reinterpret_cast<const float2 *>(&sm.du[pb][row][c + 2 * k]);
                            const f32x2 st = mk2(in.x, in.z), du = mk2(u2.x, u2.y);
                            const auto &eb = sm.eb[kSum ? 0 : pb][row];
                            const auto &fa = sm.fa[kSum ? 0 : pb][row];
                            const f32x2 ev = mk2(lane_sum<kL>(eb[e0]), lane_sum<kL>(eb[e1]));
                            o[k] = fma2(st, ev, mul2(skip[k], du));
                            dd[k] = fma2(xv[k], ev, mk2(lane_sum<kL>(fa[e0]), lane_sum<kL>(fa[e1])));
                            if (p.softplus) dd[k] = mul2(dd[k], sigmoid2(add2(g[k], bias[k])));
                            gskip[k] = fma2(du, xv[k], gskip[k]);
                            gbias[k] = add2(gbias[k], dd[k]);
                        }
                        put8<T, kVec>(static_cast<T *>(p.dx) + at, o, nv);
                        put8<T, kVec>(static_cast<T *>(p.ddt) + at, dd, nv);
                    } else if (z) {
                        f32x2 zv[4];
                        get8(done.z[j], zv);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const auto &up = sm.u[kSum ? 0 : pb][row];
                            const f32x2 u = fma2(skip[k], xv[k], mk2(lane_sum<kL>(up[c + ((2 * k) ^ key)]), lane_sum<kL>(up[c + ((2 * k + 1) ^ key)])));
                            const f32x2 sg = sigmoid2(zv[k]);  // silu' = sg (1 + z (1 - sg))
                            const f32x2 ds = mul2(sg, fma2(zv[k], fma2(sg, dup(-1.f), dup(1.f)), dup(1.f)));
                            o[k] = mul2(g[k], mul2(u, ds));
                        }
                        put8<T, kVec>(static_cast<T *>(p.dz) + at, o, nv);
                    }
                }
                for (int j = ht; j < 2 * kBack * kN / 4; j += kThreads) {  // the warps' channels, in order
                    const bool is_c = j >= kBack * kN / 4;
                    const int r = j % (kBack * kN / 4), rr = r / (kN / 4), col = (r % (kN / 4)) * 4;
                    if (tp + rr >= te) continue;
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < S::kParts; ++k) {
                        const float4 v = *reinterpret_cast<const float4 *>(is_c ? &sm.dC[kSum ? 0 : pb][rr][k][col] : &sm.dB[kSum ? 0 : pb][rr][k][col]);
                        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
                    }
                    float *to = (is_c ? p.pC : p.pB) + (((long long)w.gt * p.B + b) * p.T + tp + rr) * kN + col;
                    *reinterpret_cast<float4 *>(to) = a;
                }
                // other threads' elements of this tile are read above (du) before the next tile takes their place
                asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
            }
            if (i + 1 < tiles) stage(last - (i + 1) * kBack, (i + 1) & 1, next);
            done = now;
            now = next;
            next = land(then);
            if (i < tiles) __syncthreads();
        }
        if (kSum) return;
        // dskip and ddt_bias: the tile rows' sums, in order (only the helpers are left)
    float *acc = &sm.eb[0][0][0][0];  // [2][kBack][kCh], one buffer of parts
        if (ht < kPer) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                un2(gskip[k], lo, hi);
                *reinterpret_cast<float2 *>(&acc[row * kCh + c + 2 * k]) = make_float2(lo, hi);
                un2(gbias[k], lo, hi);
                *reinterpret_cast<float2 *>(&acc[(kBack + row) * kCh + c + 2 * k]) = make_float2(lo, hi);
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        for (int i = ht; i < 2 * kCh; i += kThreads) {
            const int which = i / kCh, cc = i % kCh;
            if (cc >= w.nch) continue;
            float a = 0.f;
            for (int k = 0; k < kBack; ++k) a += acc[(which * kBack + k) * kCh + cc];
            p.pD[(srow * 2 + which) * p.D + w.c0 + cc] = a;
        }
        return;
    }

    // ---- the scan
    const int sbase = p.seqs.cu ? 0 : b, warp = threadIdx.x / 32, cw = threadIdx.x % W::kC;  // cw: channel of the warp
    const int part = warp * (S::kC / S::kFold) + cw / S::kFold;             // whose sums of dB and dC this lane has
    const int at = w.n0 + (S::kFold == 2 ? 2 * (cw & 1) : cw & 3);          // and of which state
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
        for (int j = n + 1; j < p.seqs.n; ++j) pass_state<kL>(p, w, p.dht, p.dh0, j);
    float total = 0.f;
    State gA = zero_state();
    const int last = ts + (tiles - 1) * kBack;
    State ck_next = zero_state();
    if (!kSum && w.on) ck_next = load_state(p.states + w.at(ck0 + last / kBack, p));
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const int tb = last - i * kBack, buf = i & 1;
        const State ck = ck_next;
        if (!kSum && i + 1 < tiles && w.on) ck_next = load_state(p.states + w.at(ck0 + tb / kBack - 1, p));
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
        const int end = min(kBack, te - tb);
        const bool opening = s0 > tb && s0 < tb + end;  // a sequence opens after the tile's first token
        if (kSum) {
            auto token = [&](int r) {
                const float2 in = sm.in[buf][r][pair_place<kCh>(r, w.ch)];
                const State C = load_state(&sm.C[buf][r][w.n0]), a = decay(A2, dup(in.x));
                const f32x2 d2 = dup(sm.du[buf][r][w.ch]);
                e = State{mul2(a.a, fma2(d2, C.a, e.a)), mul2(a.b, fma2(d2, C.b, e.b))};
                total += in.x;
            };
            if (opening) {
                for (int r = end - 1; r >= 0; --r) {
                    token(r);
                    if (tb + r == s0) turn(tb + r);
                }
            } else {
#pragma unroll
                for (int r = kBack - 1; r >= 0; --r) token(r);
                if (tb == s0) turn(tb);
            }
            __syncthreads();
            continue;
        }
        State H[kBack];
        State A2r = A2;  // opaque, or the compiler keeps the forward's decays (and spills them)
        asm volatile("" : "+l"(A2r.a), "+l"(A2r.b));
        // Tokens lo .. hi - 1 of the tile, all of one sequence, from state h.
        // kPart: the others change nothing (s, du, B and C are taken as 0, not
        // multiplied by it: they may be NaN or infinite) and leave no result.
        auto tile = [&](auto some, State h, int lo, int hi) {
            constexpr bool kPart = decltype(some)::value;
            const State hs = h;
            auto mine = [&](int r) { return !kPart || (r >= lo && r < hi); };
            auto load = [&](const float(&from)[kBack][kN], int r) { return mine(r) ? load_state(&from[r][w.n0]) : zero_state(); };
            auto factors = [&](int r, f32x2 &s2, f32x2 &i2, f32x2 &d2) {
                const float2 in = sm.in[buf][r][pair_place<kCh>(r, w.ch)];
                const float du = sm.du[buf][r][w.ch];
                s2 = dup(mine(r) ? in.x : 0.f);
                i2 = dup(mine(r) ? in.y : 0.f);
                d2 = dup(mine(r) ? du : 0.f);
            };
            // Results are stored a group of tokens at a time: a store would
            // hold back the loads behind it.
#pragma unroll
            for (int g = 0; g < kBack; g += kGroup) {
                float u[kGroup];
                float2 c[kGroup];
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    const int r = g + k;
                    f32x2 s2, i2, d2;
                    factors(r, s2, i2, d2);
                    h = advance(decay(A2, s2), h, i2, load(sm.B[buf], r));
                    H[r] = h;
                    u[k] = dot(h, load(sm.C[buf], r));
                    c[k] = fold_channels<kL>(State{mul2(d2, h.a), mul2(d2, h.b)});
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    if (!mine(g + k)) continue;
                    sm.u[kSum ? 0 : buf][g + k][place<kCh>(g + k, w.ch)][w.q] = u[k];
                    put_fold<kL>(&sm.dC[kSum ? 0 : buf][g + k][part][at], c[k]);
                }
            }
            asm volatile("" ::: "memory");  // read the factors again rather than keep (and spill) sixteen tokens'
            // dA is summed by tiles: one running sum over thousands of tokens loses 9e-7 of it, a tile's first 3e-7
            State gT = zero_state();
#pragma unroll
            for (int g = kBack - kGroup; g >= 0; g -= kGroup) {
                float eb[kGroup], fa[kGroup];
                float2 c[kGroup];
#pragma unroll
                for (int k = kGroup - 1; k >= 0; --k) {
                    const int r = g + k;
                    f32x2 s2, i2, d2;
                    factors(r, s2, i2, d2);
                    const State C = load(sm.C[buf], r), Bt = load(sm.B[buf], r);
                    e = State{fma2(d2, C.a, e.a), fma2(d2, C.b, e.b)};
                    eb[k] = dot(e, Bt);
                    c[k] = fold_channels<kL>(State{mul2(i2, e.a), mul2(i2, e.b)});
                    const State before = r ? H[r ? r - 1 : 0] : hs, E = decay(A2r, s2);
                    e = State{mul2(e.a, E.a), mul2(e.b, E.b)};
                    const State f = State{mul2(e.a, before.a), mul2(e.b, before.b)};
                    fa[k] = dot(f, A);
                    gT = State{fma2(f.a, s2, gT.a), fma2(f.b, s2, gT.b)};
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    if (!mine(g + k)) continue;
                    const int e = place<kCh>(g + k, w.ch);
                    sm.eb[kSum ? 0 : buf][g + k][e][w.q] = eb[k];
                    sm.fa[kSum ? 0 : buf][g + k][e][w.q] = fa[k];
                    put_fold<kL>(&sm.dB[kSum ? 0 : buf][g + k][part][at], c[k]);
                }
            }
            gA = State{add2(gA.a, gT.a), add2(gA.b, gT.b)};
        };
        if (!opening) {
            tile(std::false_type{}, ck, 0, kBack);
            if (tb == s0) turn(tb);
        } else {
            for (int hi = end; hi > 0;) {  // the sequences in the tile, from the last
                const int lo = max(s0 - tb, 0);
                if (lo >= hi) break;
                tile(std::true_type{}, lo ? start_state<kL>(p, w, sbase + n) : ck, lo, hi);
                if (tb + lo != s0) break;
                turn(s0);
                hi = lo;
            }
        }
        __syncthreads();
    }
    if (kSum) {
        if (w.on) {
            store_state(p.sum_h + w.at(srow, p), e);
            if (w.q == 0) p.sum_s[srow * p.D + w.d] = total;
        }
        return;
    }
    if (w.on) store_state(p.pA + w.at(srow, p), gA);
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

// The states of the rows are read and written once: 71 MB for 128 rows x 4096 x
// 16 in bf16, 20.6 us (20.5 to 20.6 in nine runs of 24) where the states come from
// HBM, 18.5 where a cache of 34 MB stays in L2; 3.5 TB/s.  A CTA waits for its
// row's slot, then for its states, and ends: latencies rather than bandwidth.
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
        const State h = advance(decay(State{mul2(A.a, k), mul2(A.b, k)}, dup(s)), h0, dup(s * xv), Bt);
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

// Segments: an estimate from measured times a token of a CTA (ns, N = 16):
// forward 28 alone on an SM, else 26 times the CTAs of an SM; backward 160 and
// 115; a summary pass 19 and 50 times the CTAs of an SM; and 6 us for the pass.
SsmPlan ssm_plan(long long B, long long T, long long D, long long G, int N, bool bwd) {
    const int ch = kThreads / (N / 4);
    const long long tiles = (D / G + ch - 1) / ch, ctas = tiles * G * B, sms = layer_sms();
    const double one = bwd ? 160 : 28, more = bwd ? 115 : 26, sum = bwd ? 50 : 19;
    auto load = [&](long long n) { return (double)((n + sms - 1) / sms); };
    double best = 1e300;
    int S = 1;
    for (int s = 1; s <= 64; ++s) {
        if (s > 1 && T / s < 64) break;
        const double tok = (double)((T + s - 1) / s), k = load(ctas * s);
        const double t = tok * (std::max(one, more * k) + (s > 1 ? sum * load(ctas * (s - 1)) : 0)) + (s > 1 ? 6000 + 100.0 * s : 0);
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

// Whether eight channels are always there and 16-byte aligned.
bool ssm_vec(const gdr_ssm_args *a) {
    const long long q = a->dtype == GDR_BF16 ? 8 : 4;
    for (long long v : {a->x_row, a->x_batch, a->dt_row, a->dt_batch, a->z ? a->z_row : 0, a->z ? a->z_batch : 0,
                        a->b_row, a->b_batch, a->c_row, a->c_batch})
        if (v % q) return false;
    for (const void *p : {a->x, a->dt, a->z, a->Bm, a->Cm, a->dy, static_cast<const void *>(a->y), static_cast<const void *>(a->dx),
                          static_cast<const void *>(a->ddt), static_cast<const void *>(a->dz)})
        if (!multiple16(p)) return false;
    return (a->D / a->G) % 8 == 0;
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

template <typename K>
int ssm_launch(K *kernel, size_t smem, int threads, dim3 grid, const SsmP &p, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "scan: %s", cudaGetErrorString(e));
    kernel<<<grid, threads, smem, st>>>(p);
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
    const bool vec = ssm_vec(a);
    ssm_by_type(a->dtype, a->N, vec, [&](auto t, auto l, auto v) {
        using E = decltype(t);
        constexpr int L = decltype(l)::value;
        constexpr bool V = decltype(v)::value;
        const unsigned gx = (unsigned)(pl.tiles * a->G), gz = (unsigned)a->B;
        rc = GDR_OK;
        if (pl.S > 1) rc = ssm_launch(k_ssm_fwd<E, L, V, true, 1>, sizeof(FwdSmem<L, true, 1>), 2 * kThreads, dim3(gx, pl.S - 1, gz), p, st);
        if (rc) return;
        if ((long long)gx * pl.S * gz <= layer_sms())
            rc = ssm_launch(k_ssm_fwd<E, L, V, false, 2>, sizeof(FwdSmem<L, false, 2>), 3 * kThreads, dim3(gx, pl.S, gz), p, st);
        else
            rc = ssm_launch(k_ssm_fwd<E, L, V, false, 1>, sizeof(FwdSmem<L, false, 1>), 2 * kThreads, dim3(gx, pl.S, gz), p, st);
    });
    return rc ? rc : layer_launched("scan forward");
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
    const bool vec = ssm_vec(a);
    const long long outs = 2 * a->B * a->T * a->G * a->N + a->D * a->N + 2 * a->D;
    ssm_by_type(a->dtype, a->N, vec, [&](auto t, auto l, auto v) {
        using E = decltype(t);
        constexpr int L = decltype(l)::value;
        constexpr bool V = decltype(v)::value;
        const unsigned gx = (unsigned)(pl.tiles * a->G), gz = (unsigned)a->B;
        rc = GDR_OK;
        if (pl.S > 1) rc = ssm_launch(k_ssm_bwd<E, L, V, true>, sizeof(BwdSmem<L, true>), 2 * kThreads, dim3(gx, pl.S - 1, gz), p, st);
        if (!rc) rc = ssm_launch(k_ssm_bwd<E, L, V, false>, sizeof(BwdSmem<L, false>), 2 * kThreads, dim3(gx, pl.S, gz), p, st);
        if (!rc) k_ssm_bwd_sum<E><<<(unsigned)((outs + 255) / 256), 256, 0, st>>>(p, a->N);
    });
    return rc ? rc : layer_launched("scan backward");
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
