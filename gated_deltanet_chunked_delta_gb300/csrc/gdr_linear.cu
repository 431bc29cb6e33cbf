// gdr_linear.cu -- gated linear recurrence (one state a channel), forward,
// backward and single-token step.
//
// Per sequence and channel, with s = c softplus(decay), L_t = -s sigmoid(r_t),
// a_t = e^{L_t}, m_t = sqrt(1 - a_t^2) and u_t = sigmoid(i_t) x_t:
//     h_t = a_t h_{t-1} + m_t u_t,   y_t = h_t silu(z_t) (or h_t),
// and backwards, with e_t the gradient of h_t and din_t = dy_t silu(z_t):
//     e_t = din_t + a_{t+1} e_{t+1},  dx = e m sigmoid(i),  di = dx x (1 - sigmoid(i)),
//     G = dL L = e (L a h_{t-1} + u a^2 (-L / m)),  dr = G (1 - sigmoid(r)),
//     ddecay = sigmoid(decay) / softplus(decay) sum G,  dz = dy h silu'(z).
// G takes the place of dL because dm/dL = -a^2 / m has no bound as L goes to
// zero, while -L / m goes to sqrt(-L / 2).
//
// Bound by memory (8 bytes of bf16 an element forward, 14 backward) and, next to
// it, by instructions, so the data is read once: the tokens are cut into
// chunks, a CTA takes a chunk of 64 channels at a time (a warp a run of
// neighbouring tokens, a lane two neighbouring channels, which share packed fp32
// instructions), and the state is handed from chunk to chunk between CTAs.  A
// chunk acts on the state before it as h -> A h + B.  Its CTA publishes (A, B) as
// soon as it has them; another of its warps meanwhile looks back for the nearest
// chunk whose own state is known and goes forward from there over the (A, B)
// between.  Going forward in order, whatever the place it starts from, makes
// every result independent of the CTAs' timing, bit for bit.  CTAs take chunks
// from a counter, all channels of the first chunk before the second, and work
// them off in that order: a chunk waits only for ones that are being worked on.
// While a chunk is worked on the next one's data is copied to shared memory.
#include "gdr_layer.h"

namespace {

__device__ unsigned g_linear_status;

constexpr int kTile = 64;     // channels of a CTA
constexpr int kWindow = 4;    // chunks looked back at once
constexpr int kPolls = 1 << 20;  // of the records before a chunk, before its wait is given up
constexpr int kHelpers = 2;   // warps beside those with tokens: one publishes, one looks back

// Tokens of a warp and the warps with tokens of a full chunk.  Two CTAs an SM,
// each with the tile that it works on and the next one in shared memory.  Long
// runs: what a warp does once a tile costs as much as two tokens.
template <typename T, bool kBack>
struct Shape {
    static constexpr bool kHalf = sizeof(T) == 2;
    static constexpr int kRun = kBack ? (kHalf ? 8 : 4) : (kHalf ? 16 : 8);
    static constexpr int kWarps = 6, kChunk = kRun * kWarps;
    static constexpr int kThreads = 32 * (kWarps + kHelpers), kCtas = 2;
    static constexpr int kStride = kHalf ? GDR_LINEAR_STRIDE_BF16 : GDR_LINEAR_STRIDE_F32;  // tokens between the states kept
    static_assert(!kBack || kChunk == kStride, "the backward's chunks begin at kept states");
    static_assert(kBack || kStride % kRun == 0, "a run of the forward begins at every one");
};

struct LinP {
    const void *x, *i, *r, *z, *dy;
    const float *decay, *h0, *dht;
    void *y, *dx, *di, *dr, *dz;
    float *ht, *states, *dh0, *part;  // part: [B chunks, D] sums of G
    float4 *rec;                      // [columns, chunks, kTile] of {A, B, state, flag}
    unsigned *ticket;
    Seqs seqs;
    long long x_row, x_batch, i_row, i_batch, r_row, r_batch, z_row, z_batch;
    int tiles, B, T, D, nd, chunks;  // nd: channel tiles
    float scale;
    // Pairs of constants, read from the parameters: packed instructions take no
    // immediate operand, and the compiler would make a pair of one at each use.
    f32x2 neg_log2e, one, minus, low, poly[5];
};

__host__ __device__ __forceinline__ f32x2 pair_of(float v) {
    union {
        float f[2];
        f32x2 p;
    } u;
    u.f[0] = u.f[1] = v;
    return u.p;
}
__device__ __forceinline__ f32x2 dup(float v) { return mk2(v, v); }
template <typename F>
__device__ __forceinline__ f32x2 each(f32x2 v, F f) {
    float a, b;
    un2(v, a, b);
    return mk2(f(a), f(b));
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 v) { return each(v, [](float x) { return ex2f(x); }); }
__device__ __forceinline__ f32x2 sqrt_2(f32x2 v) {
    return each(v, [](float x) {
        float y;
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
        return y;
    });
}
__device__ __forceinline__ f32x2 rsqrt_2(f32x2 v) {
    return each(v, [](float x) {
        float y;
        asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
        return y;
    });
}
__device__ __forceinline__ f32x2 sigmoid2(const LinP &p, f32x2 v) {
    return each(add2(ex2_2(mul2(v, p.neg_log2e)), p.one), [](float x) { return rcpf(x); });
}
// a = e^{-s sig}.  The argument of ex2.approx is moved up by 1.5e-8 of the result,
// which it lies low by on average (a slow state multiplies hundreds of decays);
// ex2.approx(2.2e-8) is 1 (measured), so that a closed gate changes nothing.
__device__ __forceinline__ f32x2 decay2(const LinP &p, f32x2 sig, f32x2 neg_s2) { return ex2_2(fma2(sig, neg_s2, p.low)); }
// 1 - a^2 = 1 - e^-v, v = 2 s sig.  The difference loses its
// leading digits for small v: below 1/2 by a polynomial of (1 - e^-v) / v
// (interpolated at the Chebyshev points of [0, 1/2], off by at most 1.5e-9 of
// it).  kSmall: no v of the call's channel tile reaches 1/2.
template <bool kSmall>
__device__ __forceinline__ f32x2 rest2(const LinP &p, f32x2 v, f32x2 a) {
    f32x2 q = fma2(v, p.poly[4], p.poly[3]);
    q = fma2(v, q, p.poly[2]);
    q = fma2(v, q, p.poly[1]);
    q = fma2(v, q, p.poly[0]);
    q = fma2(v, q, p.one);
    q = mul2(v, q);
    if (kSmall) return q;
    float v0, v1, a0, a1, q0, q1;
    un2(v, v0, v1);
    un2(a, a0, a1);
    un2(q, q0, q1);
    return mk2(v0 < 0.5f ? q0 : fmaf(-a0, a0, 1.f), v1 < 0.5f ? q1 : fmaf(-a1, a1, 1.f));
}

// How tokens act on the state before them: h -> a h + b, or h -> b (a < 0)
// where a sequence starts on the way: what lies before it, NaN and infinities
// included, is left out, not multiplied by zero.
template <bool kPacked>
__device__ __forceinline__ float act(float a, float b, float h) {
    return kPacked && a < 0.f ? b : fmaf(a, h, b);
}
template <bool kPacked>
__device__ __forceinline__ f32x2 act2(float2 a, float2 b, f32x2 h) {
    if (!kPacked) return fma2(mk2(a.x, a.y), h, mk2(b.x, b.y));
    float h0, h1;
    un2(h, h0, h1);
    return mk2(act<true>(a.x, b.x, h0), act<true>(a.y, b.y, h1));
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
// the ones before it (`mine`: this lane's own records of two channels).  False
// when the wait was given up.
template <bool kPacked>
__device__ __forceinline__ bool look_back(const float4 *mine, int ordinal, float (&h)[2]) {
    const int reach = min(kWindow, ordinal);
    for (int polls = 0; polls < kPolls; ++polls) {
        Rec rec[kWindow][2];
        rec[0][0] = read_rec(mine - kTile);
        rec[0][1] = read_rec(mine - kTile + 1);
        const uint32_t near = min(rec[0][0].flag, rec[0][1].flag);
        if (__all_sync(0xffffffffu, near == 2)) {
            h[0] = rec[0][0].h;
            h[1] = rec[0][1].h;
            return true;
        }
        if (!__all_sync(0xffffffffu, near >= 1)) {
            __nanosleep(60);
            continue;
        }
#pragma unroll
        for (int j = 1; j < kWindow; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) rec[j][c] = j < reach ? read_rec(mine - (j + 1) * kTile + c) : Rec{0.f, 0.f, 0.f, 0};
        int from = -1;
        bool open = true;  // every chunk nearer than j has its a and b
#pragma unroll
        for (int j = 1; j < kWindow; ++j) {
            const uint32_t flag = min(rec[j][0].flag, rec[j][1].flag);
            if (open && from < 0 && __all_sync(0xffffffffu, flag == 2)) from = j;
            open = open && __all_sync(0xffffffffu, flag >= 1);
        }
        if (from < 0) continue;
#pragma unroll
        for (int j = kWindow - 1; j >= 0; --j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (j == from) h[c] = rec[j][c].h;
                else if (j < from) h[c] = act<kPacked>(rec[j][c].a, rec[j][c].b, h[c]);
            }
        return true;
    }
    return false;
}

// ---- tiles -------------------------------------------------------------------

// The access width kAcc of a call in bytes: 16 where every row of 64 channels
// begins on a 16-byte boundary and holds whole pieces, else 4 (words; bf16: pairs
// lie in one), else 2 (bf16 rows of any address).
template <typename T, int kAcc>
struct Mem {
    static constexpr int kRow = kTile * (int)sizeof(T) + (kAcc == 2 ? 4 : 0);  // of a staged row, in bytes

    // Copies kRun rows of 64 channels, `row` elements apart, to shared memory,
    // asynchronously: zeros behind the first `rows` of them and the first `ch`
    // channels (kWhole: all are there).  kAcc 2: the words that hold a row, which may begin inside the
    // first (`first`: the tensor's beginning, before which nothing is read).
    template <int kRun, bool kWhole>
    static __device__ __forceinline__ void stage(char *to, const T *from, const T *first, long long row, int rows, int ch) {
        const int lane = threadIdx.x % 32;
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
        if (kAcc == 16) {
            constexpr int kPer = kTile * (int)sizeof(T) / 16;
#pragma unroll
            for (int q = 0; q < kRun * kPer / 32; ++q) {
                const int j = (lane + 32 * q) / kPer, c = (lane + 32 * q) % kPer;
                const int n = kWhole ? 16 : j < rows ? max(0, min(16, ch * (int)sizeof(T) - 16 * c)) : 0;
                const char *p = kWhole || n ? reinterpret_cast<const char *>(from + j * row) + 16 * c : reinterpret_cast<const char *>(first);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + j * kRow + 16 * c), "l"(p), "r"(n) : "memory");
            }
        } else if (kAcc == 4) {
            constexpr int kPer = kTile * (int)sizeof(T) / 128;
#pragma unroll
            for (int q = 0; q < kRun * kPer; ++q) {
                const int j = q / kPer, c = lane + 32 * (q % kPer);
                const int n = kWhole ? 4 : j < rows ? max(0, min(4, ch * (int)sizeof(T) - 4 * c)) : 0;
                const char *p = kWhole || n ? reinterpret_cast<const char *>(from + j * row) + 4 * c : reinterpret_cast<const char *>(first);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at + j * kRow + 4 * c), "l"(p), "r"(n) : "memory");
            }
        } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const char *begin = reinterpret_cast<const char *>(from + j * row);
                const int shift = (int)(reinterpret_cast<uintptr_t>(begin) & 2);
                auto word = [&](int c) {
                    const char *p = begin - shift + 4 * c;
                    int n = j < rows ? max(0, min(4, ch * 2 + shift - 4 * c)) : 0;
                    if (n && p < reinterpret_cast<const char *>(first)) {  // its second half is the tensor's first element
                        *reinterpret_cast<uint32_t *>(to + j * kRow) = (uint32_t)*reinterpret_cast<const uint16_t *>(first) << 16;
                        return;
                    }
                    if (!n) p = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(first) & ~uintptr_t(3));
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at + j * kRow + 4 * c), "l"(p), "r"(n) : "memory");
                };
                word(lane);
                if (lane == 0) word(32);
            }
        }
    }
    // This lane's two channels of a staged row (kAcc 2: `begin` is where the row lies in memory).
    static __device__ __forceinline__ f32x2 get(const char *row, const T *begin) {
        const int lane = threadIdx.x % 32;
        if (sizeof(T) == 4) {
            const float2 v = *reinterpret_cast<const float2 *>(row + 8 * lane);
            return mk2(v.x, v.y);
        }
        uint32_t w;
        if (kAcc == 2) {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(row + 4 * lane + (reinterpret_cast<uintptr_t>(begin) & 2));
            w = (uint32_t)p[0] | (uint32_t)p[1] << 16;
        } else {
            w = *reinterpret_cast<const uint32_t *>(row + 4 * lane);
        }
        return mk2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    // A pair of fp32 in the place of this lane's channels of two staged rows that have been read.
    static __device__ __forceinline__ void put2(char *row0, char *row1, f32x2 v) {
        const int lane = threadIdx.x % 32;
        float a, b;
        un2(v, a, b);
        if (sizeof(T) == 4) {
            *reinterpret_cast<float2 *>(row0 + 8 * lane) = make_float2(a, b);
        } else {
            if (kAcc == 2) __syncwarp();  // a neighbour's channels may begin inside this lane's words
            *reinterpret_cast<float *>(row0 + 4 * lane) = a;
            *reinterpret_cast<float *>(row1 + 4 * lane) = b;
        }
    }
    static __device__ __forceinline__ f32x2 get2(const char *row0, const char *row1) {
        const int lane = threadIdx.x % 32;
        if (sizeof(T) == 4) {
            const float2 v = *reinterpret_cast<const float2 *>(row0 + 8 * lane);
            return mk2(v.x, v.y);
        }
        return mk2(*reinterpret_cast<const float *>(row0 + 4 * lane), *reinterpret_cast<const float *>(row1 + 4 * lane));
    }
    // Two channels of memory, of which the first n exist.
    static __device__ __forceinline__ f32x2 load(const T *p, int n) {
        if (sizeof(T) == 4 && kAcc == 16) {
            const float2 v = n > 0 ? *reinterpret_cast<const float2 *>(p) : make_float2(0.f, 0.f);
            return mk2(v.x, v.y);
        }
        if (sizeof(T) == 2 && kAcc >= 4) {
            const uint32_t w = n > 0 ? *reinterpret_cast<const uint32_t *>(p) : 0u;
            return mk2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        }
        return mk2(n > 0 ? to_f(p[0]) : 0.f, n > 1 ? to_f(p[1]) : 0.f);
    }
    static __device__ __forceinline__ void store(T *p, f32x2 v, int n) {
        float a, b;
        un2(v, a, b);
        if (sizeof(T) == 4 && kAcc == 16) {
            if (n > 0) *reinterpret_cast<float2 *>(p) = make_float2(a, b);
        } else if (sizeof(T) == 2 && kAcc >= 4) {
            if (n > 0) *reinterpret_cast<uint32_t *>(p) = pack2(a, b);
        } else {
            if (n > 0) from_f(p[0], a);
            if (n > 1) from_f(p[1], b);
        }
    }
};
// fp32 parameters and states: two channels, of which n exist.
__device__ __forceinline__ f32x2 load_f(const float *p, int n) { return mk2(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f); }
__device__ __forceinline__ void store_f(float *p, f32x2 v, int n) {
    float a, b;
    un2(v, a, b);
    if (n > 0) p[0] = a;
    if (n > 1) p[1] = b;
}

// Sequences that the kRun tokens from t0 on start and end: lane j has token t0 + j's (-1: none).
template <int kRun>
__device__ __forceinline__ void mark(const Seqs &q, int t0, int &first, int &last) {
    const int lane = threadIdx.x % 32, n = q.count();
    int lo = 0, hi = n - 1;  // the sequence of t0 is one of these
    while (hi - lo >= 32) {
        const int step = (hi - lo + 31) / 32;
        const int below = __popc(__ballot_sync(0xffffffffu, q.bound(min(lo + (lane + 1) * step, hi)) <= t0));
        const int from = lo;
        lo = min(from + below * step, hi);
        if (below < 32) hi = max(lo, min(from + (below + 1) * step, hi) - 1);
    }
    lo += max(0, __popc(__ballot_sync(0xffffffffu, lo + lane <= hi && q.bound(min(lo + lane, n)) <= t0)) - 1);
    const int bound = lo + lane < n ? q.bound(lo + lane) : 0x7fffffff;
    int mine = lo;
    bool all = false;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const int below = __popc(__ballot_sync(0xffffffffu, bound <= t0 + j));
        if (lane == j) mine = lo + max(0, below - 1);
        all = all || below == 32;
    }
    const int t = t0 + lane;
    first = last = -1;
    if (lane < kRun && t < q.T) {
        if (all) mine = q.find(t);  // 32 sequences and more start in this run (all but a few without tokens)
        if (q.bound(mine) == t) first = mine;
        if (q.bound(mine + 1) == t + 1) last = mine;
    }
}
// The bounds are meant to rise from 0 to T: one warp looks them over.
__device__ __forceinline__ void check(const Seqs &s) {
    for (int q = threadIdx.x % 32; q <= s.n; q += 32) {
        const int v = s.cu[q];
        if ((q == 0 && v != 0) || (q == s.n && v != s.T) || (q > 0 && v < s.cu[q - 1])) atomicOr(&g_linear_status, kStatusIndex);
    }
}
// What sequences without tokens hand on, 64 channels of them, by one warp.
__device__ __forceinline__ void pass_empty(const LinP &p, const float *from, float *to, int d, int nch) {
    if (!to) return;
    const int lane = threadIdx.x % 32;
    for (int q0 = 0; q0 < p.seqs.n; q0 += 32) {
        const int q = q0 + lane;
        unsigned empty = __ballot_sync(0xffffffffu, q < p.seqs.n && p.seqs.bound(q) == p.seqs.bound(q + 1));
        for (; empty; empty &= empty - 1) {
            const long long at = (long long)(q0 + __ffs(empty) - 1) * p.D + d;
            store_f(to + at, from ? load_f(from + at, nch) : dup(0.f), nch);
        }
    }
}

// Named barriers of a CTA (0 is __syncthreads'): kReady, the warps' (a, b) are
// there; kState, the state before the chunk is there; kSums, the sums of G are.
enum { kReady = 1, kState = 2, kSums = 3 };
__device__ __forceinline__ void bar_sync(int id, int warps) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int warps) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(32 * warps) : "memory"); }

// A tile as the warps work on it: laid out by the warp that looks back, two tiles
// ahead of its turn.
struct Info {
    float2 s[32];  // s of the lanes' channels (0 behind the last)
    long long rec; // of the tile's first record
    int tile, b, d0, chunk, ordinal, col, small;
};
// What the warps of a CTA tell one another; by turns, so that a warp that runs
// ahead writes where nobody reads any more.
template <int kWarps>
struct Talk {
    Info info[4];
    float2 a[2][kWarps][32], b[2][kWarps][32];  // the warps' actions, then (from the publisher) those of all warps before
    float2 carry[2][32];                        // the state that comes into the chunk
};
template <int kWarps>
struct BackTalk {
    float2 a[2][kWarps][32], b[2][kWarps][32];  // the warps' actions from the first token on
    float2 start[2][kWarps][32];                // the state before a warp's first token
    float2 sums[2][kWarps][32];                 // sums of G
};

__device__ __forceinline__ int take(const LinP &p) { return (int)min(atomicAdd(p.ticket, 1u), (unsigned)p.tiles); }

// By one warp.
template <bool kBack>
__device__ __forceinline__ void lay_out(const LinP &p, Info &to, int tile) {
    const int lane = threadIdx.x % 32;
    if (tile >= p.tiles) {
        if (lane == 0) to.tile = p.tiles;
        return;
    }
    const int cols = p.B * p.nd, ordinal = tile / cols, col = tile - ordinal * cols, b = col / p.nd, d0 = (col - b * p.nd) * kTile;
    const int d = d0 + 2 * lane, nch = p.D - d;
    const float s0 = nch > 0 ? p.scale * softplusf(p.decay[d]) : 0.f, s1 = nch > 1 ? p.scale * softplusf(p.decay[d + 1]) : 0.f;
    const bool small = __all_sync(0xffffffffu, s0 < 0.25f && s1 < 0.25f);
    to.s[lane] = make_float2(s0, s1);
    if (lane == 0) {
        to.tile = tile;
        to.b = b;
        to.d0 = d0;
        to.ordinal = ordinal;
        to.col = col;
        to.chunk = kBack ? p.chunks - 1 - ordinal : ordinal;
        to.small = small;
        to.rec = ((long long)col * p.chunks + ordinal) * kTile;
    }
}

// Whether a CTA has more than one tile: then it takes them from the counter, and
// otherwise too where chunks wait for one another.  Lays out the first two.
template <bool kBack, int kWarps>
__device__ __forceinline__ bool begin(const LinP &p, Talk<kWarps> &s, int warps) {
    const bool more = (int)gridDim.x < p.tiles;
    if ((int)threadIdx.x / 32 == warps) {
        int tile[2] = {(int)blockIdx.x, p.tiles};
        if (p.chunks > 1) {
            if (threadIdx.x % 32 == 0) {
                tile[0] = take(p);
                if (more) tile[1] = take(p);
            }
            tile[0] = __shfl_sync(0xffffffffu, tile[0], 0);
            tile[1] = __shfl_sync(0xffffffffu, tile[1], 0);
        }
        lay_out<kBack>(p, s.info[0], tile[0]);
        lay_out<kBack>(p, s.info[1], tile[1]);
    }
    __syncthreads();
    return more;
}

// The warp that publishes: the chunk's (A, B) from its warps' actions, in whose
// place it leaves those of all the warps before (kBack: the last warp acts first).
template <bool kPacked, bool kBack, int kWarps, typename F>
__device__ __forceinline__ void publish(const LinP &p, Talk<kWarps> &s, const Info &at, int turn, int warps, F meanwhile) {
    const int lane = threadIdx.x % 32;
    bar_sync(kReady, warps + 1);
    float2 a = make_float2(1.f, 1.f), b = make_float2(0.f, 0.f);
    float4 *mine = p.rec + at.rec + 2 * lane;
    for (int k = 0; k < warps; ++k) {
        const int v = kBack ? warps - 1 - k : k;
        const float2 av = s.a[turn][v][lane], bv = s.b[turn][v][lane];
        s.a[turn][v][lane] = a;
        s.b[turn][v][lane] = b;
        b = make_float2(act<kPacked>(av.x, bv.x, b.x), act<kPacked>(av.y, bv.y, b.y));
        a = make_float2(join<kPacked>(a.x, av.x), join<kPacked>(a.y, av.y));
    }
    if (at.ordinal > 0) {
        write_rec(mine, a.x, b.x, 0.f, 1);
        write_rec(mine + 1, a.y, b.y, 0.f, 1);
    }
    meanwhile();
    bar_sync(kState, warps + kHelpers);
    if (at.ordinal + 1 < p.chunks) {
        const float2 h = s.carry[turn][lane];
        write_rec(mine, a.x, b.x, act<kPacked>(a.x, b.x, h.x), 2);
        write_rec(mine + 1, a.y, b.y, act<kPacked>(a.y, b.y, h.y), 2);
    }
}
// The warp that looks back; `first` [B, D]: the state before the chunk with ordinal 0 (null: zeros).
template <bool kPacked, bool kBack, int kWarps>
__device__ __forceinline__ void receive(const LinP &p, Talk<kWarps> &s, const Info &at, const float *first, int k, int warps, bool more) {
    const int lane = threadIdx.x % 32, d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d));
    int after = p.tiles;
    if (more) {
        if (lane == 0) after = take(p);
        after = __shfl_sync(0xffffffffu, after, 0);
    }
    lay_out<kBack>(p, s.info[(k + 2) & 3], after);
    float h[2] = {0.f, 0.f};
    if (at.ordinal > 0) {
        if (!look_back<kPacked>(p.rec + at.rec + 2 * lane, at.ordinal, h) && lane == 0) atomicOr(&g_linear_status, kStatusTimeout);
    } else if (!kPacked && first) {
        un2(load_f(first + (long long)at.b * p.D + d, nch), h[0], h[1]);
    }
    s.carry[k & 1][lane] = make_float2(h[0], h[1]);
    bar_sync(kState, warps + kHelpers);
}

template <typename T, int kAcc, bool kZ, bool kPacked>
__global__ void __launch_bounds__(Shape<T, false>::kThreads, Shape<T, false>::kCtas) k_linear_fwd(const __grid_constant__ LinP p) {
    using M = Mem<T, kAcc>;
    using S = Shape<T, false>;
    constexpr int kRun = S::kRun, kWarps = S::kWarps, kStep = kRun * M::kRow;
    extern __shared__ __align__(16) char stages[];
    __shared__ Talk<kWarps> s;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32 - kHelpers;
    const bool more = begin<false>(p, s, warps);
    if (warp >= warps) {
        for (int k = 0; s.info[k & 3].tile < p.tiles; ++k) {
            const Info &at = s.info[k & 3];
            if (warp == warps) publish<kPacked, false>(p, s, at, k & 1, warps, [] {});
            else receive<kPacked, false>(p, s, at, p.h0, k, warps, more);
            if (kPacked && at.ordinal == 0) {
                const int d = at.d0 + 2 * lane;
                if (warp == warps) pass_empty(p, p.h0, p.ht, d, max(0, min(2, p.D - d)));
                else if (at.col == 0) check(p.seqs);
            }
        }
        return;
    }
    char *const own = stages + warp * 3 * kStep;
    const int other = more ? warps * 3 * kStep : 0;  // from a tile to the next one's
    const T *const tx = static_cast<const T *>(p.x), *const ti = static_cast<const T *>(p.i), *const tr = static_cast<const T *>(p.r);
    auto stage = [&](const Info &at, int turn) {
        if (at.tile < p.tiles) {
            const int t0 = (at.chunk * warps + warp) * kRun, rows = p.T - t0, ch = p.D - at.d0;
            char *to = own + turn * other;
            auto copy = [&](auto whole) {
                constexpr bool W = decltype(whole)::value;
                M::template stage<kRun, W>(to, tr + at.b * p.r_batch + t0 * p.r_row + at.d0, tr, p.r_row, rows, ch);
                M::template stage<kRun, W>(to + kStep, ti + at.b * p.i_batch + t0 * p.i_row + at.d0, ti, p.i_row, rows, ch);
                M::template stage<kRun, W>(to + 2 * kStep, tx + at.b * p.x_batch + t0 * p.x_row + at.d0, tx, p.x_row, rows, ch);
            };
            if (kAcc > 2 && rows >= kRun && ch >= kTile) copy(std::true_type{}); else copy(std::false_type{});
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int first = -1, last = -1, next_first = -1, next_last = -1;
    stage(s.info[0], 0);
    if (kPacked && s.info[0].tile < p.tiles) mark<kRun>(p.seqs, (s.info[0].chunk * warps + warp) * kRun, first, last);
    for (int k = 0; s.info[k & 3].tile < p.tiles; ++k) {
        const Info &at = s.info[k & 3], &next = s.info[(k + 1) & 3];
        const int turn = k & 1;
        stage(next, turn ^ 1);
        const int d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), t0 = (at.chunk * warps + warp) * kRun, n = min(kRun, p.T - t0);
        const f32x2 sv = mk2(at.s[lane].x, at.s[lane].y), neg_s2 = mul2(sv, p.neg_log2e), two_s = add2(sv, sv);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const char *in = own + turn * other;
        f32x2 a[kRun], b[kRun], A = p.one, B = dup(0.f);
        bool cut = false;  // a sequence starts in this run
        auto pass = [&](auto sm) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const long long tt = t0 + j;
                const f32x2 r = M::get(in + j * M::kRow, kAcc == 2 ? tr + at.b * p.r_batch + tt * p.r_row + at.d0 : nullptr);
                const f32x2 i = M::get(in + kStep + j * M::kRow, kAcc == 2 ? ti + at.b * p.i_batch + tt * p.i_row + at.d0 : nullptr);
                const f32x2 x = M::get(in + 2 * kStep + j * M::kRow, kAcc == 2 ? tx + at.b * p.x_batch + tt * p.x_row + at.d0 : nullptr);
                const f32x2 sr = sigmoid2(p, r);
                a[j] = decay2(p, sr, neg_s2);
                const f32x2 m = sqrt_2(rest2<decltype(sm)::value>(p, mul2(sr, two_s), a[j]));
                b[j] = mul2(m, mul2(sigmoid2(p, i), x));
                const int q = kPacked ? __shfl_sync(0xffffffffu, first, j) : -1;
                if (kPacked && q >= 0) {
                    if (p.h0) b[j] = fma2(a[j], load_f(p.h0 + (long long)q * p.D + d, nch), b[j]);
                    B = b[j];
                    A = p.one;
                    cut = true;
                } else {
                    B = fma2(a[j], B, b[j]);
                    A = mul2(A, a[j]);
                }
            }
        };
        if (at.small) pass(std::true_type{}); else pass(std::false_type{});
        {
            float a0, a1, b0, b1;
            un2(A, a0, a1);
            un2(B, b0, b1);
            s.a[turn][warp][lane] = cut ? make_float2(-1.f, -1.f) : make_float2(a0, a1);
            s.b[turn][warp][lane] = make_float2(b0, b1);
        }
        bar_arrive(kReady, warps + 1);
        constexpr int kAhead = kRun < 8 ? kRun : 8;  // z is read in runs of eight
        f32x2 z[kZ ? kAhead : 1];
        const T *pz = kZ ? static_cast<const T *>(p.z) + at.b * p.z_batch + t0 * p.z_row + d : nullptr;
        auto read_z = [&](int from) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) z[kZ ? j : 0] = M::load(pz + (from + j) * p.z_row, from + j < n ? nch : 0);
        };
        if (kZ) read_z(0);
        if (kPacked && next.tile < p.tiles) mark<kRun>(p.seqs, (next.chunk * warps + warp) * kRun, next_first, next_last);
        bar_sync(kState, warps + kHelpers);
        const float2 c = s.carry[turn][lane];
        f32x2 h = act2<kPacked>(s.a[turn][warp][lane], s.b[turn][warp][lane], mk2(c.x, c.y));
        T *py = static_cast<T *>(p.y) + ((long long)at.b * p.T + t0) * p.D + d;
        float *const pst = p.states + (long long)at.b * ((p.T + S::kStride - 1) / S::kStride) * p.D + d;
        auto finish = [&](auto whole) {
            constexpr bool W = decltype(whole)::value;
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                if (W || j < n) {
                    if (j == 0 && p.states && t0 % S::kStride == 0) store_f(pst + (long long)(t0 / S::kStride) * p.D, h, nch);
                    const bool start = kPacked && __shfl_sync(0xffffffffu, first, j) >= 0;
                    h = start ? b[j] : fma2(a[j], h, b[j]);
                    f32x2 y = h;
                    if (kZ) {
                        if (j && j % kAhead == 0) read_z(j);
                        y = mul2(h, mul2(z[j % kAhead], sigmoid2(p, z[j % kAhead])));
                    }
                    M::store(py + (long long)j * p.D, y, W ? 2 : nch);
                    if (kPacked) {
                        const int q = __shfl_sync(0xffffffffu, last, j);
                        if (q >= 0 && p.ht) store_f(p.ht + (long long)q * p.D + d, h, nch);
                    }
                }
            }
            if (!kPacked && p.ht && n > 0 && t0 + n == p.T) store_f(p.ht + (long long)at.b * p.D + d, h, nch);
        };
        if (n == kRun && p.D - at.d0 >= kTile) finish(std::true_type{}); else finish(std::false_type{});
        first = next_first;
        last = next_last;
    }
}

template <typename T, int kAcc, bool kZ, bool kPacked>
__global__ void __launch_bounds__(Shape<T, true>::kThreads, Shape<T, true>::kCtas) k_linear_bwd(const __grid_constant__ LinP p) {
    using M = Mem<T, kAcc>;
    using S = Shape<T, true>;
    constexpr int kRun = S::kRun, kWarps = S::kWarps, kIn = kZ ? 5 : 4, kStep = kRun * M::kRow;
    extern __shared__ __align__(16) char stages[];
    __shared__ Talk<kWarps> s;
    __shared__ BackTalk<kWarps> f;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32 - kHelpers;
    const bool more = begin<true>(p, s, warps);
    if (warp >= warps) {
        for (int k = 0; s.info[k & 3].tile < p.tiles; ++k) {
            const Info &at = s.info[k & 3];
            const int d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), turn = k & 1;
            if (warp == warps) {
                f32x2 h = load_f(p.states + ((long long)at.b * p.chunks + at.chunk) * p.D + d, nch);
                publish<kPacked, true>(p, s, at, turn, warps, [&] {
                    for (int v = 0; v < warps; ++v) {
                        float h0, h1;
                        un2(h, h0, h1);
                        f.start[turn][v][lane] = make_float2(h0, h1);
                        h = act2<kPacked>(f.a[turn][v][lane], f.b[turn][v][lane], h);
                    }
                });
                bar_sync(kSums, warps + 1);
                float2 g = make_float2(0.f, 0.f);
                for (int v = 0; v < warps; ++v) {
                    g.x += f.sums[turn][v][lane].x;
                    g.y += f.sums[turn][v][lane].y;
                }
                store_f(p.part + ((long long)at.b * p.chunks + at.chunk) * p.D + d, mk2(g.x, g.y), nch);
            } else {
                receive<kPacked, true>(p, s, at, p.dht, k, warps, more);
            }
            if (kPacked && at.ordinal == 0) {
                if (warp == warps) pass_empty(p, p.dht, p.dh0, d, nch);
                else if (at.col == 0) check(p.seqs);
            }
        }
        return;
    }
    char *const own = stages + warp * kIn * kStep;
    const int other = more ? warps * kIn * kStep : 0;  // from a tile to the next one's
    const T *const tx = static_cast<const T *>(p.x), *const ti = static_cast<const T *>(p.i), *const tr = static_cast<const T *>(p.r);
    const T *const tz = static_cast<const T *>(p.z), *const ty = static_cast<const T *>(p.dy);
    const long long y_batch = (long long)p.T * p.D;
    auto stage = [&](const Info &at, int turn) {
        if (at.tile < p.tiles) {
            const int t0 = (at.chunk * warps + warp) * kRun, rows = p.T - t0, ch = p.D - at.d0;
            char *to = own + turn * other;
            auto copy = [&](auto whole) {
                constexpr bool W = decltype(whole)::value;
                M::template stage<kRun, W>(to, tr + at.b * p.r_batch + t0 * p.r_row + at.d0, tr, p.r_row, rows, ch);
                M::template stage<kRun, W>(to + kStep, ti + at.b * p.i_batch + t0 * p.i_row + at.d0, ti, p.i_row, rows, ch);
                M::template stage<kRun, W>(to + 2 * kStep, tx + at.b * p.x_batch + t0 * p.x_row + at.d0, tx, p.x_row, rows, ch);
                M::template stage<kRun, W>(to + 3 * kStep, ty + at.b * y_batch + (long long)t0 * p.D + at.d0, ty, p.D, rows, ch);
                if (kZ) M::template stage<kRun, W>(to + 4 * kStep, tz + at.b * p.z_batch + t0 * p.z_row + at.d0, tz, p.z_row, rows, ch);
            };
            if (kAcc > 2 && rows >= kRun && ch >= kTile) copy(std::true_type{}); else copy(std::false_type{});
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int first = -1, last = -1, next_first = -1, next_last = -1;
    stage(s.info[0], 0);
    if (kPacked && s.info[0].tile < p.tiles) mark<kRun>(p.seqs, (s.info[0].chunk * warps + warp) * kRun, first, last);
    for (int k = 0; s.info[k & 3].tile < p.tiles; ++k) {
        const Info &at = s.info[k & 3], &next = s.info[(k + 1) & 3];
        const int turn = k & 1;
        __syncwarp();  // the stage has been read
        stage(next, turn ^ 1);
        const int d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), t0 = (at.chunk * warps + warp) * kRun, n = min(kRun, p.T - t0);
        const f32x2 neg_s = mul2(mk2(at.s[lane].x, at.s[lane].y), p.minus), log2e = mul2(p.neg_log2e, p.minus), neg_s2 = mul2(neg_s, log2e);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        char *in = own + turn * other;
        auto get = [&](int which, int j) {
            const long long tt = t0 + j;
            const T *from = nullptr;
            if (kAcc == 2)
                from = at.d0 + (which == 0 ? tr + at.b * p.r_batch + tt * p.r_row : which == 1 ? ti + at.b * p.i_batch + tt * p.i_row
                              : which == 2 ? tx + at.b * p.x_batch + tt * p.x_row : which == 3 ? ty + at.b * y_batch + tt * p.D
                                           : tz + at.b * p.z_batch + tt * p.z_row);
            return M::get(in + which * kStep + j * M::kRow, from);
        };
        auto starts = [&](int j) { return kPacked ? __shfl_sync(0xffffffffu, first, j) : -1; };
        auto ends = [&](int j) { return kPacked ? __shfl_sync(0xffffffffu, last, j) : -1; };
        auto given = [&](const float *t, int q) { return t ? load_f(t + (long long)q * p.D + d, nch) : dup(0.f); };
        auto din = [&](int j) {
            const f32x2 y = get(3, j);
            if (!kZ) return y;
            const f32x2 z = get(4, j);
            return mul2(y, mul2(z, sigmoid2(p, z)));
        };
        // a, m sigmoid(i), sigmoid(r); g: first sigmoid(i) a^2 (-L / m), then G / e.  sigmoid(i) waits
        // in the place of both gates.
        f32x2 a[kRun], mi[kRun], sr[kRun], g[kRun], A = p.one, B = dup(0.f);
        bool cut = false;
        auto pass = [&](auto sm) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                sr[j] = sigmoid2(p, get(0, j));
                const f32x2 si = sigmoid2(p, get(1, j));
                M::put2(in + kStep + j * M::kRow, in + j * M::kRow, si);
                a[j] = decay2(p, sr[j], neg_s2);
                const f32x2 L = mul2(sr[j], neg_s), v = mul2(add2(L, L), p.minus);
                // a gate is not quite closed here (1e-36), so that m has a reciprocal
                const f32x2 rest = add2(rest2<decltype(sm)::value>(p, v, a[j]), dup(1e-36f)), inv = rsqrt_2(rest);
                mi[j] = mul2(mul2(rest, inv), si);
                g[j] = mul2(mul2(mul2(a[j], a[j]), mul2(L, inv)), mul2(si, p.minus));
                const f32x2 b = mul2(mi[j], get(2, j));
                const int q = starts(j);
                if (kPacked && q >= 0) {
                    B = fma2(a[j], given(p.h0, q), b);
                    A = p.one;
                    cut = true;
                } else {
                    B = fma2(a[j], B, b);
                    A = mul2(A, a[j]);
                }
            }
        };
        if (at.small) pass(std::true_type{}); else pass(std::false_type{});
        auto tell = [&](float2 *ta, float2 *tb) {
            float a0, a1, b0, b1;
            un2(A, a0, a1);
            un2(B, b0, b1);
            ta[lane] = cut ? make_float2(-1.f, -1.f) : make_float2(a0, a1);
            tb[lane] = make_float2(b0, b1);
        };
        tell(f.a[turn][warp], f.b[turn][warp]);
        A = p.one;
        B = dup(0.f);
        cut = false;
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) {
            if (j < n) {
                const int q = ends(j);
                if (kPacked && q >= 0) {
                    B = given(p.dht, q);
                    A = p.one;
                    cut = true;
                }
                A = mul2(A, a[j]);
                B = mul2(a[j], add2(din(j), B));
            }
        }
        tell(s.a[turn][warp], s.b[turn][warp]);
        bar_arrive(kReady, warps + 1);
        if (kPacked && next.tile < p.tiles) mark<kRun>(p.seqs, (next.chunk * warps + warp) * kRun, next_first, next_last);
        bar_sync(kState, warps + kHelpers);
        f32x2 h = mk2(f.start[turn][warp][lane].x, f.start[turn][warp][lane].y), sum = dup(0.f);
        const float2 c = s.carry[turn][lane];
        f32x2 e = act2<kPacked>(s.a[turn][warp][lane], s.b[turn][warp][lane], mk2(c.x, c.y));
        const long long out = ((long long)at.b * p.T + t0) * p.D + d;
        T *const px = static_cast<T *>(p.dx) + out, *const pi = static_cast<T *>(p.di) + out, *const pr = static_cast<T *>(p.dr) + out;
        T *const pz = kZ ? static_cast<T *>(p.dz) + out : nullptr;
        auto finish = [&](auto whole) {
            constexpr bool W = decltype(whole)::value;
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const int q = starts(j);
                if (kPacked && q >= 0) h = given(p.h0, q);
                const f32x2 x = get(2, j), La = mul2(mul2(sr[j], neg_s), a[j]);
                g[j] = fma2(La, h, mul2(g[j], x));
                h = fma2(a[j], h, mul2(mi[j], x));
                if (kZ && (W || j < n)) {
                    const f32x2 z = get(4, j), on = sigmoid2(p, z);
                    const f32x2 slope = mul2(on, fma2(z, fma2(on, p.minus, p.one), p.one));
                    M::store(pz + (long long)j * p.D, mul2(mul2(get(3, j), h), slope), W ? 2 : nch);
                }
            }
#pragma unroll
            for (int j = kRun - 1; j >= 0; --j) {
                if (W || j < n) {
                    const int q = ends(j);
                    if (kPacked && q >= 0) e = given(p.dht, q);
                    e = add2(e, din(j));
                    const f32x2 G = mul2(e, g[j]), dx = mul2(e, mi[j]), si = M::get2(in + kStep + j * M::kRow, in + j * M::kRow);
                    sum = add2(sum, G);
                    const long long to = (long long)j * p.D;
                    M::store(px + to, dx, W ? 2 : nch);
                    M::store(pi + to, mul2(mul2(dx, get(2, j)), fma2(si, p.minus, p.one)), W ? 2 : nch);
                    M::store(pr + to, mul2(G, fma2(sr[j], p.minus, p.one)), W ? 2 : nch);
                    e = mul2(e, a[j]);
                    const int o = kPacked ? starts(j) : t0 + j == 0 ? at.b : -1;
                    if (o >= 0 && p.dh0) store_f(p.dh0 + (long long)o * p.D + d, e, nch);
                }
            }
        };
        if (n == kRun && p.D - at.d0 >= kTile) finish(std::true_type{}); else finish(std::false_type{});
        {
            float g0, g1;
            un2(sum, g0, g1);
            f.sums[turn][warp][lane] = make_float2(g0, g1);
        }
        bar_arrive(kSums, warps + 1);
        first = next_first;
        last = next_last;
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
    LinP c;  // its constants
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

// A thread has two channels of a row.
template <typename T, int kAcc>
__global__ void __launch_bounds__(kStepThreads) k_linear_step(const __grid_constant__ LinStepP p) {
    using M = Mem<T, kAcc>;
    const long long row = blockIdx.y;
    const int d = (blockIdx.x * kStepThreads + threadIdx.x) * 2, nch = max(0, min(2, p.D - d));
    const long long slot = p.slots ? p.slots[row] : row;
    if (slot >= p.n_slots && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_linear_status, kStatusIndex);
    if (!nch) return;
    f32x2 y = dup(0.f);
    if (slot >= 0 && slot < p.n_slots) {
        const f32x2 x = M::load(static_cast<const T *>(p.x) + row * p.x_row + d, nch);
        const f32x2 i = M::load(static_cast<const T *>(p.i) + row * p.i_row + d, nch);
        const f32x2 r = M::load(static_cast<const T *>(p.r) + row * p.r_row + d, nch);
        const f32x2 z = p.z ? M::load(static_cast<const T *>(p.z) + row * p.z_row + d, nch) : dup(0.f);
        float *st = p.state + slot * p.D + d;
        const f32x2 before = load_f(st, nch);
        const f32x2 s = each(load_f(p.decay + d, nch), [&](float v) { return p.scale * softplusf(v); });
        const f32x2 sr = sigmoid2(p.c, r), a = decay2(p.c, sr, mul2(s, p.c.neg_log2e));
        const f32x2 m = sqrt_2(rest2<false>(p.c, mul2(add2(s, s), sr), a));
        y = fma2(a, before, mul2(m, mul2(sigmoid2(p.c, i), x)));
        store_f(st, y, nch);
        if (p.z) y = mul2(y, mul2(z, sigmoid2(p.c, z)));
    }
    M::store(static_cast<T *>(p.y) + row * p.D + d, y, nch);
}

// ---- host ------------------------------------------------------------------

int linear_sizes(long long B, long long T, long long D, int dtype) {
    if (B < 1 || T < 0 || D < 1) return layer_fail(GDR_ERR_SHAPE, "linear scan: B and D must be >= 1 and T >= 0 (got %lld, %lld, %lld)", B, D, T);
    if (T >= (1LL << 30) || D >= (1LL << 24) || B > 65535) return layer_fail(GDR_ERR_SHAPE, "linear scan: problem too large");
    if (dtype != GDR_BF16 && dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "linear scan: unknown dtype %d", dtype);
    return GDR_OK;
}

LinP linear_constants() {
    LinP p{};
    p.neg_log2e = pair_of(-kLog2e);
    p.one = pair_of(1.f);
    p.minus = pair_of(-1.f);
    p.low = pair_of(2.2e-8f);
    const float poly[5] = {-4.9999982e-1f, 1.6666242e-1f, -4.1630073e-2f, 8.1896136e-3f, -1.1234042e-3f};
    for (int i = 0; i < 5; ++i) p.poly[i] = pair_of(poly[i]);
    return p;
}

struct LinPlan {
    int warps;  // with tokens, of a CTA
    long long chunks;
};
LinPlan linear_plan(long long T, int dtype, bool bwd) {
    auto of = [&](auto t, auto back) {
        using S = Shape<decltype(t), decltype(back)::value>;
        const int run = S::kRun, warps = (int)std::max(1LL, std::min<long long>(S::kWarps, (T + run - 1) / run));
        return LinPlan{warps, std::max(1LL, (T + warps * run - 1) / (warps * run))};
    };
    if (bwd) return dtype == GDR_BF16 ? of(bf16_t{}, std::true_type{}) : of(float{}, std::true_type{});
    return dtype == GDR_BF16 ? of(bf16_t{}, std::false_type{}) : of(float{}, std::false_type{});
}

// The workspace: the counter and the records (where there is more than one
// chunk), the backward's sums.
struct LinSpace {
    size_t rec, part, total, zeroed;
};
LinSpace linear_space(long long B, long long T, long long D, int dtype, bool bwd) {
    const LinPlan pl = linear_plan(T, dtype, bwd);
    LinSpace s{};
    size_t off = 0;
    if (pl.chunks > 1) {
        s.rec = 16;
        off = s.zeroed = 16 + (size_t)B * pl.chunks * ((D + kTile - 1) / kTile * kTile) * sizeof(float4);
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

// The access width: of tensors whose rows begin at `ptrs` and are `strides` elements apart.
int linear_access(int dtype, std::initializer_list<const void *> ptrs, std::initializer_list<long long> strides) {
    const long long e = dtype == GDR_BF16 ? 2 : 4;
    unsigned long long any = 0;
    for (const void *p : ptrs) any |= reinterpret_cast<uintptr_t>(p);
    for (long long v : strides) any |= (unsigned long long)(v * e);
    return !(any & 15) ? 16 : !(any & 3) ? 4 : 2;
}

int linear_fill(const gdr_linear_args *a, const Seqs &s, bool bwd, const LinSpace &sp, LinP *p, LinPlan *pl, cudaStream_t st) {
    *p = linear_constants();
    *pl = linear_plan(a->T, a->dtype, bwd);
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
    p->nd = (int)((a->D + kTile - 1) / kTile);
    p->chunks = (int)pl->chunks;
    p->scale = a->decay_scale;
    const long long tiles = a->B * p->nd * pl->chunks;
    if (tiles >= (1LL << 31) - (1 << 20)) return layer_fail(GDR_ERR_SHAPE, "linear scan: problem too large");
    p->tiles = (int)tiles;
    if (sp.zeroed) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sp.zeroed, st);
        if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "linear scan: %s", cudaGetErrorString(e));
    }
    return GDR_OK;
}

// As many CTAs as run at once, each with two tiles in shared memory; all tiles at
// once where they are fewer or do not hand states on.  `each`: a warp's tile.
template <typename K>
int linear_launch(K *kernel, const LinP &p, const LinPlan &pl, int ctas, size_t each, cudaStream_t st) {
    const size_t tile = each * pl.warps;
    long long grid = p.tiles;
    if (p.chunks > 1) grid = std::min(grid, (long long)layer_sms() * ctas);
    const size_t smem = grid < p.tiles ? 2 * tile : tile;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "linear scan: %s", cudaGetErrorString(e));
    kernel<<<(unsigned)grid, 32 * (pl.warps + kHelpers), smem, st>>>(p);
    return GDR_OK;
}

// f(type, access width, gated, packed)
template <typename F>
void linear_by_type(const gdr_linear_args *a, int access, F f) {
    using std::integral_constant;
    auto w = [&](auto t, auto c) {
        auto v = [&](auto z) {
            if (a->cu_seqlens) f(t, c, z, std::true_type{}); else f(t, c, z, std::false_type{});
        };
        if (a->z) v(std::true_type{}); else v(std::false_type{});
    };
    if (a->dtype == GDR_F32) {
        if (access == 16) w(float{}, integral_constant<int, 16>{}); else w(float{}, integral_constant<int, 4>{});
    } else if (access == 16) {
        w(bf16_t{}, integral_constant<int, 16>{});
    } else if (access == 4) {
        w(bf16_t{}, integral_constant<int, 4>{});
    } else {
        w(bf16_t{}, integral_constant<int, 2>{});
    }
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

size_t gdr_linear_fwd_workspace_size(long long B, long long T, long long D, int dtype) {
    return linear_sizes(B, T, D, dtype) ? 0 : linear_space(B, T, D, dtype, false).total;
}

size_t gdr_linear_bwd_workspace_size(long long B, long long T, long long D, int dtype) {
    return linear_sizes(B, T, D, dtype) ? 0 : linear_space(B, T, D, dtype, true).total;
}

int gdr_linear_fwd(const gdr_linear_args *a, void *stream) {
    Seqs s;
    int rc = linear_common(a, &s);
    if (rc) return rc;
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    if ((rc = layer_ptr("y", a->y, a->T > 0, e)) || (rc = layer_ptr("ht", a->ht, false, 4))) return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->T == 0) return linear_hand_on(a->h0, a->ht, (size_t)a->n_seqs * a->D, st);
    const LinSpace sp = linear_space(a->B, a->T, a->D, a->dtype, false);
    if ((rc = linear_workspace(a, sp, "linear scan forward"))) return rc;
    LinP p;
    LinPlan pl;
    if ((rc = linear_fill(a, s, false, sp, &p, &pl, st))) return rc;
    const int access = linear_access(a->dtype, {a->x, a->input_gate, a->decay_gate, a->z, a->y},
                                     {a->x_row, a->x_batch, a->i_row, a->i_batch, a->r_row, a->r_batch, a->z ? a->z_row : 0, a->z ? a->z_batch : 0, a->D});
    linear_by_type(a, access, [&](auto t, auto c, auto z, auto k) {
        using E = decltype(t);
        using M = Mem<E, decltype(c)::value>;
        using H = Shape<E, false>;
        static_assert(H::kCtas * (6 * H::kRun * M::kRow * H::kWarps + sizeof(Talk<H::kWarps>) + 1024) <= 228 * 1024, "CTAs of an SM");
        rc = linear_launch(k_linear_fwd<E, decltype(c)::value, decltype(z)::value, decltype(k)::value>, p, pl, H::kCtas, 3 * H::kRun * M::kRow, st);
    });
    return rc ? rc : layer_launched("linear scan forward");
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
    const LinSpace sp = linear_space(a->B, a->T, a->D, a->dtype, true);
    if ((rc = linear_workspace(a, sp, "linear scan backward"))) return rc;
    LinP p;
    LinPlan pl;
    if ((rc = linear_fill(a, s, true, sp, &p, &pl, st))) return rc;
    const int access = linear_access(a->dtype, {a->x, a->input_gate, a->decay_gate, a->z, a->dy, a->dx, a->di, a->dr, a->dz},
                                     {a->x_row, a->x_batch, a->i_row, a->i_batch, a->r_row, a->r_batch, a->z ? a->z_row : 0, a->z ? a->z_batch : 0, a->D});
    linear_by_type(a, access, [&](auto t, auto c, auto z, auto k) {
        using E = decltype(t);
        using M = Mem<E, decltype(c)::value>;
        using H = Shape<E, true>;
        constexpr int kIn = decltype(z)::value ? 5 : 4;
        static_assert(H::kCtas * (2 * kIn * H::kRun * M::kRow * H::kWarps + sizeof(Talk<H::kWarps>) + sizeof(BackTalk<H::kWarps>) + 1024) <= 228 * 1024, "CTAs of an SM");
        rc = linear_launch(k_linear_bwd<E, decltype(c)::value, decltype(z)::value, decltype(k)::value>, p, pl, H::kCtas, kIn * H::kRun * M::kRow, st);
    });
    if (rc) return rc;
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
    LinStepP p{linear_constants(), a->x, a->input_gate, a->decay_gate, a->z, a->decay, a->state, a->slots, a->y,
               a->x_row, a->i_row, a->r_row, a->z_row, a->n_slots, (int)a->D, a->decay_scale};
    const int access = linear_access(a->dtype, {a->x, a->input_gate, a->decay_gate, a->z, a->y}, {a->x_row, a->i_row, a->r_row, a->z ? a->z_row : 0, a->D});
    const dim3 grid((unsigned)((a->D + 2 * kStepThreads - 1) / (2 * kStepThreads)), (unsigned)a->rows);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->dtype == GDR_F32 && access == 16) k_linear_step<float, 16><<<grid, kStepThreads, 0, st>>>(p);
    else if (a->dtype == GDR_F32) k_linear_step<float, 4><<<grid, kStepThreads, 0, st>>>(p);
    else if (access >= 4) k_linear_step<bf16_t, 4><<<grid, kStepThreads, 0, st>>>(p);
    else k_linear_step<bf16_t, 2><<<grid, kStepThreads, 0, st>>>(p);
    return layer_launched("linear step");
}

}  // extern "C"
