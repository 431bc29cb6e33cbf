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
// A warp works out a tile's action before it finishes the tile before, whose
// state comes in meanwhile; the tile after is copied to shared memory.
//
// bf16: 16384 x 4096 128 us (4.2 TB/s, issue slots 48 % used), 2 x 4096 x 4096 67 us
// and 132 backward (54 %), packed 8192 x 2048 with the output gate 74 and 139 (issue
// slots 32 and 35 %); fp32 2 x 4096 x 2048 56 us and 86 (5.5 TB/s).  What bounds
// them: the time of a tile (2 us, packed and gated 4): three warps with tokens an
// SM quarter, whose chains of exponentials, reciprocals and roots leave half the
// issue slots empty (two tiles a warp take the registers that more warps would
// need).  Next is the special-function pipe: two ex2 (4 cycles a warp), two
// reciprocals and a root (8 each) an element are 58 us of 16384 x 4096.
// Rows off 16-byte boundaries are copied word by word: 6144 x 1026 bf16 31 us and 42
// (1024: 24 and 36), fp32 of 1031 channels 44 and 57 (1024: 31 and 41); bf16 rows off
// word boundaries also read and write two bytes at a time: 6144 x 1031 82 and 102.
// Measured against it for 16384 x 4096: a tile finished before the next is begun
// 174 us; 24 warps with tokens, one tile each at a time, states through the
// shared memory of clusters 154 us; one reciprocal for both gates, with a branch
// for gates far closed, 149 us.
#include "gdr_layer.h"

namespace {

__device__ unsigned g_linear_status;

constexpr int kTile = 64;     // channels of a CTA
constexpr int kWindow = 4;    // chunks looked back at once (eight: the packed backward 143 us, four 138)
constexpr int kPolls = 1 << 20;  // of the records before a chunk, before its wait is given up
constexpr int kHelpers = 3;   // warps beside those with tokens: one publishes, one looks back, one scouts

// The warps with tokens of a full chunk, and their tokens.
constexpr int kWarps = 12, kFwdRun = 8, kBwdRun = 4;
constexpr int kThreads = 32 * (kWarps + kHelpers), kRegs = 128;  // one full CTA an SM: 480 x 128 registers
static_assert(kWarps * kBwdRun == GDR_LINEAR_STRIDE, "the backward's chunks begin at kept states");
static_assert(GDR_LINEAR_STRIDE % kFwdRun == 0, "a run of the forward begins at every one");

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
    f32x2 neg_log2e, one, minus, poly[4];
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
// a = e^-u and 1 - a^2, u = s sig.  Below u = 1/4, where a state multiplies many
// decays and 1 - a^2 would lose its leading digits, both come from w = 1 - e^-u = u q(u),
// q a polynomial of degree 4 (least error, off by at most 3.1e-9 of it): a = 1 - w
// rounds once, to nearest, and 1 - a^2 = w (1 + a).  ex2.approx would leave every
// decay off by 0.5e-8 to 3e-8 on average (measured, by ranges of its argument),
// and more by chance: 4096 tokens' states by 1.2e-6 (norm-wise) instead of 2e-7.
// Above 1/4 a state soon forgets that.  kSmall: no u of the call's channel tile
// reaches 1/4.
template <bool kSmall>
__device__ __forceinline__ void decay2(const LinP &p, f32x2 u, f32x2 &a, f32x2 &rest) {
    f32x2 q = fma2(u, p.poly[3], p.poly[2]);
    q = fma2(u, q, p.poly[1]);
    q = fma2(u, q, p.poly[0]);
    q = fma2(u, q, p.one);
    const f32x2 w = mul2(u, q);
    a = fma2(w, p.minus, p.one);
    rest = fma2(w, a, w);
    if (kSmall) return;
    float u0, u1, a0, a1, b0, b1, r0, r1;
    un2(u, u0, u1);
    un2(a, a0, a1);
    un2(ex2_2(mul2(u, p.neg_log2e)), b0, b1);
    un2(rest, r0, r1);
    a0 = u0 < 0.25f ? a0 : b0;
    a1 = u1 < 0.25f ? a1 : b1;
    a = mk2(a0, a1);
    rest = mk2(u0 < 0.25f ? r0 : fmaf(-a0, a0, 1.f), u1 < 0.25f ? r1 : fmaf(-a1, a1, 1.f));
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
#pragma unroll
        for (int j = 0; j < kWindow; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) rec[j][c] = j < reach ? read_rec(mine - (j + 1) * kTile + c) : Rec{0.f, 0.f, 0.f, 0};
        int from = -1;
        bool open = true;  // every chunk nearer than j has its a and b
#pragma unroll
        for (int j = 0; j < kWindow; ++j)
            if (open && from < 0) {
                const uint32_t flag = min(rec[j][0].flag, rec[j][1].flag);
                if (__all_sync(0xffffffffu, flag == 2)) from = j;
                open = __all_sync(0xffffffffu, flag >= 1);
            }
        if (from < 0) {
            __nanosleep(20);
            continue;
        }
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

// Named barriers of a CTA (0 is __syncthreads'), two of each kind, for tiles by
// turns: the warps' (a, b) are there; the chunk's are; the state before the chunk
// is; the sums of G are.
enum { kReady = 1, kTotal = 3, kState = 5, kSums = 7 };
__device__ __forceinline__ void bar_sync(int id, int warps) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int warps) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(32 * warps) : "memory"); }

// A tile as the warps work on it: laid out by the warp that scouts, three tiles
// ahead.
template <int kTok>
struct Info {
    float2 s[32];                // s of the lanes' channels (0 behind the last)
    int first[kTok], last[kTok]; // packed: the sequence that a token starts, ends, or -1
    long long rec;               // of the tile's first record
    int tile, b, d0, chunk, ordinal, col, small;
};
constexpr int kInfos = 8;  // tiles k - 2 .. k + 3 are in use at once
// What the warps of a CTA tell one another.  Two of each, for tiles by turns: a
// warp begins the tile after the next only when all have the state of this one.
template <int kTok>
struct Talk {
    Info<kTok> info[kInfos];
    float2 a[2][kWarps][32], b[2][kWarps][32];  // the warps' actions, then (from the publisher) those of all warps before
    float2 total_a[2][32], total_b[2][32];      // the chunk's
    float2 carry[2][32];                        // the state that comes into the chunk
};
struct BackTalk {
    float2 a[2][kWarps][32], b[2][kWarps][32];  // the warps' actions from the first token on
    float2 start[2][kWarps][32];                // the state before a warp's first token
    float2 sums[2][kWarps][32];                 // sums of G
};

// A CTA's `k`-th tile.  Chunks that wait for one another are taken from the counter, so that what they wait for is
// being worked on; others are dealt out.  By lane 0 of a warp, each once, in order.
__device__ __forceinline__ int take(const LinP &p, int k) {
    if (p.chunks > 1) return (int)min(atomicAdd(p.ticket, 1u), (unsigned)p.tiles);
    return (int)min((long long)blockIdx.x + (long long)k * gridDim.x, (long long)p.tiles);
}
// By one warp.
template <bool kBack, bool kPacked, int kTok>
__device__ __forceinline__ void lay_out(const LinP &p, Info<kTok> &to, int k, int warps, bool more) {
    const int lane = threadIdx.x % 32;
    int tile = p.tiles;
    if (lane == 0 && (k == 0 || more)) tile = take(p, k);
    tile = __shfl_sync(0xffffffffu, tile, 0);
    if (tile >= p.tiles) {
        if (lane == 0) to.tile = p.tiles;
        return;
    }
    const int cols = p.B * p.nd, ordinal = tile / cols, col = tile - ordinal * cols, b = col / p.nd, d0 = (col - b * p.nd) * kTile;
    const int d = d0 + 2 * lane, nch = p.D - d;
    const float s0 = nch > 0 ? p.scale * softplusf(p.decay[d]) : 0.f, s1 = nch > 1 ? p.scale * softplusf(p.decay[d + 1]) : 0.f;
    const bool small = __all_sync(0xffffffffu, s0 < 0.25f && s1 < 0.25f);
    to.s[lane] = make_float2(s0, s1);
    if (kPacked) {
        const int tokens = warps * (kBack ? kBwdRun : kFwdRun), t0 = (kBack ? p.chunks - 1 - ordinal : ordinal) * tokens, t1 = min(t0 + tokens, p.T);
        for (int j = lane; j < tokens; j += 32) to.first[j] = to.last[j] = -1;
        __syncwarp();
        // the last sequence that starts at or before t0, or one before it
        int lo = 0, hi = p.seqs.n - 1;
        while (hi - lo >= 32) {
            const int step = (hi - lo + 31) / 32;
            const int below = __popc(__ballot_sync(0xffffffffu, p.seqs.bound(min(lo + (lane + 1) * step, hi)) <= t0));
            const int from = lo;
            lo = min(from + below * step, hi);
            if (below < 32) hi = max(lo, min(from + (below + 1) * step, hi) - 1);
        }
        // each lane's sequence leaves its number at its first and last token
        for (bool more = true; more; lo += 32) {
            const int q = lo + lane;
            const int start = q < p.seqs.n ? p.seqs.bound(q) : p.T, end = q < p.seqs.n ? p.seqs.bound(q + 1) : p.T;
            if (start < end) {
                if (start >= t0 && start < t1) to.first[start - t0] = q;
                if (end > t0 && end <= t1) to.last[end - 1 - t0] = q;
            }
            more = lo + 32 < p.seqs.n && __any_sync(0xffffffffu, lane == 31 && start < t1);
        }
    }
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
// Lays out the first three tiles; whether there may be more than one.
template <bool kBack, bool kPacked, int kTok>
__device__ __forceinline__ bool begin(const LinP &p, Talk<kTok> &s, int warps) {
    const bool more = (int)gridDim.x < p.tiles;
    if ((int)threadIdx.x / 32 == warps + 2)
        for (int k = 0; k < 3; ++k) lay_out<kBack, kPacked>(p, s.info[k], k, warps, more);
    __syncthreads();
    return more;
}

// The warp that publishes: the chunk's (A, B) from its warps' actions, in whose
// place it leaves those of all the warps before (kBack: the last warp acts first).
template <bool kPacked, bool kBack, int kTok>
__device__ __forceinline__ void publish(const LinP &p, Talk<kTok> &s, const Info<kTok> &at, int turn, int warps) {
    const int lane = threadIdx.x % 32;
    bar_sync(kReady + turn, warps + 1);
    float4 *mine = p.rec + at.rec + 2 * lane;
    float2 av[kWarps], bv[kWarps];  // read at once: one after another their latencies add up
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warps) {
            const int v = kBack ? warps - 1 - w : w;
            av[w] = s.a[turn][v][lane];
            bv[w] = s.b[turn][v][lane];
        }
    float2 a = make_float2(1.f, 1.f), b = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warps) {
            const float2 a0 = a, b0 = b;
            b = make_float2(act<kPacked>(av[w].x, bv[w].x, b.x), act<kPacked>(av[w].y, bv[w].y, b.y));
            a = make_float2(join<kPacked>(a.x, av[w].x), join<kPacked>(a.y, av[w].y));
            av[w] = a0;
            bv[w] = b0;
        }
    if (at.ordinal > 0 && at.ordinal + 1 < p.chunks) {
        write_rec(mine, a.x, b.x, 0.f, 1);
        write_rec(mine + 1, a.y, b.y, 0.f, 1);
    }
    s.total_a[turn][lane] = a;
    s.total_b[turn][lane] = b;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warps) {
            const int v = kBack ? warps - 1 - w : w;
            s.a[turn][v][lane] = av[w];
            s.b[turn][v][lane] = bv[w];
        }
}
// The warp that looks back; `first` [B, D]: the state before the chunk with ordinal 0 (null: zeros).
template <bool kPacked, int kTok>
__device__ __forceinline__ void receive(const LinP &p, Talk<kTok> &s, const float *first, int warps) {
    const int lane = threadIdx.x % 32;
    for (int k = 0; s.info[k % kInfos].tile < p.tiles; ++k) {
        const Info<kTok> &at = s.info[k % kInfos];
        const int turn = k & 1;
        float4 *mine = p.rec + at.rec + 2 * lane;
        float h[2] = {0.f, 0.f};
        if (at.ordinal > 0) {
            if (!look_back<kPacked>(mine, at.ordinal, h) && lane == 0) atomicOr(&g_linear_status, kStatusTimeout);
        } else if (!kPacked && first) {
            const int d = at.d0 + 2 * lane;
            un2(load_f(first + (long long)at.b * p.D + d, max(0, min(2, p.D - d))), h[0], h[1]);
        }
        bar_sync(kTotal + turn, 3);  // the tile before the last is finished: its state may go
        s.carry[turn][lane] = make_float2(h[0], h[1]);
        if (at.ordinal + 1 < p.chunks) {
            const float2 a = s.total_a[turn][lane], b = s.total_b[turn][lane];
            write_rec(mine, a.x, b.x, act<kPacked>(a.x, b.x, h[0]), 2);
            write_rec(mine + 1, a.y, b.y, act<kPacked>(a.y, b.y, h[1]), 2);
        }
        bar_arrive(kState + turn, warps + 2);
    }
}
// The warp that scouts; sequences without tokens hand on `from` to `to`.
template <bool kPacked, bool kBack, int kTok>
__device__ __forceinline__ void scout(const LinP &p, Talk<kTok> &s, const float *from, float *to, int warps, bool more) {
    for (int k = 0; s.info[k % kInfos].tile < p.tiles; ++k) {
        const Info<kTok> &at = s.info[k % kInfos];
        lay_out<kBack, kPacked>(p, s.info[(k + 3) % kInfos], k + 3, warps, more);
        bar_sync(kTotal + (k & 1), 3);  // keeps it from running further ahead
        bar_arrive(kState + (k & 1), warps + 2);
        if (kPacked && at.ordinal == 0) {
            const int d = at.d0 + 2 * (threadIdx.x % 32);
            pass_empty(p, from, to, d, max(0, min(2, p.D - d)));
            if (at.col == 0) check(p.seqs);
        }
    }
}

template <typename T, int kAcc, bool kZ, bool kPacked>
__global__ void __launch_bounds__(kThreads, 1) k_linear_fwd(const __grid_constant__ LinP p) {
    using M = Mem<T, kAcc>;
    constexpr int kRun = kFwdRun, kIn = kZ ? 4 : 3, kStep = kRun * M::kRow;
    extern __shared__ __align__(16) char stages[];
    constexpr int kTok = kPacked ? kWarps * kRun : 1;
    __shared__ Talk<kTok> s;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32 - kHelpers;
    const bool more = begin<false, kPacked>(p, s, warps);
    if (warp == warps) {
        for (int k = 0; s.info[k % kInfos].tile < p.tiles; ++k) {
            publish<kPacked, false>(p, s, s.info[k % kInfos], k & 1, warps);
            bar_arrive(kTotal + (k & 1), 3);
        }
        return;
    }
    if (warp == warps + 1) return receive<kPacked>(p, s, p.h0, warps);
    if (warp == warps + 2) return scout<kPacked, false>(p, s, p.h0, p.ht, warps, more);
    char *const own = stages + warp * kIn * kStep;
    const int other = more ? warps * kIn * kStep : 0;  // from a tile to the next one's
    const T *const tx = static_cast<const T *>(p.x), *const ti = static_cast<const T *>(p.i), *const tr = static_cast<const T *>(p.r);
    const T *const tz = static_cast<const T *>(p.z);
    // The k-th tile, and the output gates of the one before, which are read a turn later.
    auto stage = [&](int k) {
        __syncwarp();  // the stage has been read
        auto copy = [&](const Info<kTok> &at, auto f) {
            const int t0 = (at.chunk * warps + warp) * kRun, rows = p.T - t0, ch = p.D - at.d0;
            if (kAcc > 2 && rows >= kRun && ch >= kTile) f(t0, rows, ch, std::true_type{}); else f(t0, rows, ch, std::false_type{});
        };
        const Info<kTok> &at = s.info[k % kInfos];
        if (at.tile < p.tiles)
            copy(at, [&](int t0, int rows, int ch, auto whole) {
                constexpr bool W = decltype(whole)::value;
                char *to = own + (k & 1) * other;
                M::template stage<kRun, W>(to, tr + at.b * p.r_batch + t0 * p.r_row + at.d0, tr, p.r_row, rows, ch);
                M::template stage<kRun, W>(to + kStep, ti + at.b * p.i_batch + t0 * p.i_row + at.d0, ti, p.i_row, rows, ch);
                M::template stage<kRun, W>(to + 2 * kStep, tx + at.b * p.x_batch + t0 * p.x_row + at.d0, tx, p.x_row, rows, ch);
            });
        if (kZ && k > 0) {
            const Info<kTok> &before = s.info[(k - 1) % kInfos];
            if (before.tile < p.tiles)
                copy(before, [&](int t0, int rows, int ch, auto whole) {
                    M::template stage<kRun, decltype(whole)::value>(own + (k - 1 & 1) * other + 3 * kStep, tz + before.b * p.z_batch + t0 * p.z_row + before.d0,
                                                                    tz, p.z_row, rows, ch);
                });
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    struct Set {  // a tile between its two passes
        f32x2 a[kRun], b[kRun];
    };
    // Whether one of the warp's tokens is a border.
    auto border = [&](const int (&mark)[kTok]) { return __any_sync(0xffffffffu, lane < kRun && mark[kPacked ? warp * kRun + lane % kRun : 0] >= 0); };
    // The warp's action.
    auto front = [&](int k, Set &o) {
        const Info<kTok> &at = s.info[k % kInfos];
        if (at.tile >= p.tiles) return;
        const int turn = k & 1, d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), t0 = (at.chunk * warps + warp) * kRun;
        const f32x2 sv = mk2(at.s[lane].x, at.s[lane].y);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const char *in = own + turn * other;
        f32x2 A = p.one, B = dup(0.f);
        bool cut = false;  // a sequence starts in this run
        auto pass = [&](auto sm, auto borders) {
            constexpr bool C = decltype(borders)::value;
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const long long tt = t0 + j;
                const f32x2 r = M::get(in + j * M::kRow, kAcc == 2 ? tr + at.b * p.r_batch + tt * p.r_row + at.d0 : nullptr);
                const f32x2 i = M::get(in + kStep + j * M::kRow, kAcc == 2 ? ti + at.b * p.i_batch + tt * p.i_row + at.d0 : nullptr);
                const f32x2 x = M::get(in + 2 * kStep + j * M::kRow, kAcc == 2 ? tx + at.b * p.x_batch + tt * p.x_row + at.d0 : nullptr);
                const f32x2 sr = sigmoid2(p, r), si = sigmoid2(p, i);
                f32x2 rest;
                decay2<decltype(sm)::value>(p, mul2(sr, sv), o.a[j], rest);
                o.b[j] = mul2(sqrt_2(rest), mul2(si, x));
                const int q = C ? at.first[C ? warp * kRun + j : 0] : -1;
                if (C && q >= 0) {
                    if (p.h0) o.b[j] = fma2(o.a[j], load_f(p.h0 + (long long)q * p.D + d, nch), o.b[j]);
                    B = o.b[j];
                    A = p.one;
                    cut = true;
                } else {
                    B = fma2(o.a[j], B, o.b[j]);
                    A = mul2(A, o.a[j]);
                }
            }
        };
        // branches inside a run would keep its tokens' latencies from overlapping
        if (kPacked && border(at.first)) pass(std::false_type{}, std::integral_constant<bool, kPacked>{});
        else if (at.small) pass(std::true_type{}, std::false_type{});
        else pass(std::false_type{}, std::false_type{});
        float a0, a1, b0, b1;
        un2(A, a0, a1);
        un2(B, b0, b1);
        s.a[turn][warp][lane] = cut ? make_float2(-1.f, -1.f) : make_float2(a0, a1);
        s.b[turn][warp][lane] = make_float2(b0, b1);
        bar_arrive(kReady + turn, warps + 1);
    };
    // Its states and outputs.
    auto rear = [&](int k, const Set &o) {
        const Info<kTok> &at = s.info[k % kInfos];
        const int turn = k & 1, d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), t0 = (at.chunk * warps + warp) * kRun, n = min(kRun, p.T - t0);
        // the output gates are of the group before the last; where no next tile's action has waited for it, this does
        if (kZ) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
        }
        bar_sync(kState + turn, warps + 2);
        const float2 c = s.carry[turn][lane];
        f32x2 h = act2<kPacked>(s.a[turn][warp][lane], s.b[turn][warp][lane], mk2(c.x, c.y));
        T *py = static_cast<T *>(p.y) + ((long long)at.b * p.T + t0) * p.D + d;
        if (p.states && n > 0 && t0 % GDR_LINEAR_STRIDE == 0)
            store_f(p.states + ((long long)at.b * ((p.T + GDR_LINEAR_STRIDE - 1) / GDR_LINEAR_STRIDE) + t0 / GDR_LINEAR_STRIDE) * p.D + d, h, nch);
        auto finish = [&](auto whole, auto borders) {
            constexpr bool W = decltype(whole)::value, C = decltype(borders)::value;
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                if (W || j < n) {
                    const bool start = C && at.first[C ? warp * kRun + j : 0] >= 0;
                    h = start ? o.b[j] : fma2(o.a[j], h, o.b[j]);
                    f32x2 y = h;
                    if (kZ) {
                        const f32x2 z = M::get(own + turn * other + 3 * kStep + j * M::kRow,
                                               kAcc == 2 ? tz + at.b * p.z_batch + (long long)(t0 + j) * p.z_row + at.d0 : nullptr);
                        y = mul2(h, mul2(z, sigmoid2(p, z)));
                    }
                    M::store(py + (long long)j * p.D, y, W ? 2 : nch);
                    if (C) {
                        const int q = at.last[C ? warp * kRun + j : 0];
                        if (q >= 0 && p.ht) store_f(p.ht + (long long)q * p.D + d, h, nch);
                    }
                }
            }
            if (!kPacked && p.ht && n > 0 && t0 + n == p.T) store_f(p.ht + (long long)at.b * p.D + d, h, nch);
        };
        if (kPacked && (border(at.first) || border(at.last))) finish(std::false_type{}, std::integral_constant<bool, kPacked>{});
        else if (n == kRun && p.D - at.d0 >= kTile) finish(std::true_type{}, std::false_type{});
        else finish(std::false_type{}, std::false_type{});
    };
    // A tile's action is published before the one before it is finished: the state
    // comes in meanwhile.
    Set even, odd;
    stage(0);
    stage(1);
    front(0, even);
    for (int k = 0; s.info[k % kInfos].tile < p.tiles; k += 2) {
        stage(k + 2);
        front(k + 1, odd);
        rear(k, even);
        if (s.info[(k + 1) % kInfos].tile >= p.tiles) break;
        stage(k + 3);
        front(k + 2, even);
        rear(k + 1, odd);
    }
}

template <typename T, int kAcc, bool kZ, bool kPacked>
__global__ void __launch_bounds__(kThreads, 1) k_linear_bwd(const __grid_constant__ LinP p) {
    using M = Mem<T, kAcc>;
    constexpr int kRun = kBwdRun, kIn = kZ ? 5 : 4, kStep = kRun * M::kRow;
    extern __shared__ __align__(16) char stages[];
    constexpr int kTok = kPacked ? kWarps * kRun : 1;
    __shared__ Talk<kTok> s;
    __shared__ BackTalk f;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32 - kHelpers;
    const bool more = begin<true, kPacked>(p, s, warps);
    if (warp == warps) {
        auto sum = [&](int k) {
            const Info<kTok> &at = s.info[k % kInfos];
            const int turn = k & 1, d = at.d0 + 2 * lane;
            bar_sync(kSums + turn, warps + 1);
            f32x2 g = dup(0.f);
            for (int v = 0; v < warps; ++v) g = add2(g, mk2(f.sums[turn][v][lane].x, f.sums[turn][v][lane].y));
            store_f(p.part + ((long long)at.b * p.chunks + at.chunk) * p.D + d, g, max(0, min(2, p.D - d)));
        };
        int k = 0;
        for (; s.info[k % kInfos].tile < p.tiles; ++k) {
            const Info<kTok> &at = s.info[k % kInfos];
            const int d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), turn = k & 1;
            f32x2 h = load_f(p.states + ((long long)at.b * p.chunks + at.chunk) * p.D + d, nch);
            publish<kPacked, true>(p, s, at, turn, warps);
            float2 fa[kWarps], fb[kWarps];
#pragma unroll
            for (int v = 0; v < kWarps; ++v)
                if (v < warps) {
                    fa[v] = f.a[turn][v][lane];
                    fb[v] = f.b[turn][v][lane];
                }
#pragma unroll
            for (int v = 0; v < kWarps; ++v)
                if (v < warps) {
                    float h0, h1;
                    un2(h, h0, h1);
                    f.start[turn][v][lane] = make_float2(h0, h1);
                    h = act2<kPacked>(fa[v], fb[v], h);
                }
            bar_arrive(kTotal + turn, 3);
            if (k > 0) sum(k - 1);
        }
        if (k > 0) sum(k - 1);
        return;
    }
    if (warp == warps + 1) return receive<kPacked>(p, s, p.dht, warps);
    if (warp == warps + 2) return scout<kPacked, true>(p, s, p.dht, p.dh0, warps, more);
    char *const own = stages + warp * kIn * kStep;
    const int other = more ? warps * kIn * kStep : 0;  // from a tile to the next one's, of three
    const T *const tx = static_cast<const T *>(p.x), *const ti = static_cast<const T *>(p.i), *const tr = static_cast<const T *>(p.r);
    const T *const tz = static_cast<const T *>(p.z), *const ty = static_cast<const T *>(p.dy);
    const long long y_batch = (long long)p.T * p.D;
    auto stage = [&](int k) {
        const Info<kTok> &at = s.info[k % kInfos];
        __syncwarp();  // the stage has been read
        if (at.tile < p.tiles) {
            const int t0 = (at.chunk * warps + warp) * kRun, rows = p.T - t0, ch = p.D - at.d0;
            char *to = own + k % 3 * other;
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
    struct Set {  // a tile between its two passes: a, m sigmoid(i), sigmoid(r), sigmoid(i) a^2 (-L / m)
        f32x2 a[kRun], mi[kRun], sr[kRun], g[kRun];
    };
    auto get = [&](const Info<kTok> &at, const char *in, int which, int j) {
        const T *from = nullptr;
        if (kAcc == 2) {
            const long long tt = (at.chunk * warps + warp) * kRun + j;
            from = at.d0 + (which == 0 ? tr + at.b * p.r_batch + tt * p.r_row : which == 1 ? ti + at.b * p.i_batch + tt * p.i_row
                          : which == 2 ? tx + at.b * p.x_batch + tt * p.x_row : which == 3 ? ty + at.b * y_batch + tt * p.D
                                       : tz + at.b * p.z_batch + tt * p.z_row);
        }
        return M::get(in + which * kStep + j * M::kRow, from);
    };
    auto din = [&](const Info<kTok> &at, const char *in, int j) {
        const f32x2 y = get(at, in, 3, j);
        if (!kZ) return y;
        const f32x2 z = get(at, in, 4, j);
        return mul2(y, mul2(z, sigmoid2(p, z)));
    };
    // Whether one of the warp's tokens is a border.
    auto border = [&](const int (&mark)[kTok]) { return __any_sync(0xffffffffu, lane < kRun && mark[kPacked ? warp * kRun + lane % kRun : 0] >= 0); };
    auto front = [&](int k, Set &o) {
        const Info<kTok> &at = s.info[k % kInfos];
        if (at.tile >= p.tiles) return;
        const int turn = k & 1, d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), t0 = (at.chunk * warps + warp) * kRun, n = min(kRun, p.T - t0);
        const f32x2 sv = mk2(at.s[lane].x, at.s[lane].y);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        char *in = own + k % 3 * other;
        f32x2 A = p.one, B = dup(0.f);
        bool cut = false;
        auto given = [&](const float *t, int q) { return t ? load_f(t + (long long)q * p.D + d, nch) : dup(0.f); };
        auto tell = [&](float2 *ta, float2 *tb) {
            float a0, a1, b0, b1;
            un2(A, a0, a1);
            un2(B, b0, b1);
            ta[lane] = cut ? make_float2(-1.f, -1.f) : make_float2(a0, a1);
            tb[lane] = make_float2(b0, b1);
            A = p.one;
            B = dup(0.f);
            cut = false;
        };
        auto pass = [&](auto sm, auto borders) {
            constexpr bool C = decltype(borders)::value;
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const f32x2 sr = sigmoid2(p, get(at, in, 0, j)), si = sigmoid2(p, get(at, in, 1, j));
                M::put2(in + kStep + j * M::kRow, in + j * M::kRow, si);  // it waits in the place of both gates
                const f32x2 u = mul2(sr, sv);
                f32x2 a, rest;
                decay2<decltype(sm)::value>(p, u, a, rest);
                rest = add2(rest, dup(1e-36f));  // a gate is not quite closed here, so that m has a reciprocal
                const f32x2 inv = rsqrt_2(rest);
                const f32x2 mi = mul2(mul2(rest, inv), si), b = mul2(mi, get(at, in, 2, j));
                o.a[j] = a;
                o.mi[j] = mi;
                o.sr[j] = sr;
                o.g[j] = mul2(mul2(mul2(a, a), mul2(u, inv)), si);
                const int q = C ? at.first[C ? warp * kRun + j : 0] : -1;
                if (C && q >= 0) {
                    B = fma2(a, given(p.h0, q), b);
                    A = p.one;
                    cut = true;
                } else {
                    B = fma2(a, B, b);
                    A = mul2(A, a);
                }
            }
        };
        // branches inside a run would keep its tokens' latencies from overlapping
        if (kPacked && border(at.first)) pass(std::false_type{}, std::integral_constant<bool, kPacked>{});
        else if (at.small) pass(std::true_type{}, std::false_type{});
        else pass(std::false_type{}, std::false_type{});
        tell(f.a[turn][warp], f.b[turn][warp]);
        auto back = [&](auto whole, auto borders) {
            constexpr bool W = decltype(whole)::value, C = decltype(borders)::value;
#pragma unroll
            for (int j = kRun - 1; j >= 0; --j) {
                if (W || j < n) {
                    const int q = C ? at.last[C ? warp * kRun + j : 0] : -1;
                    if (C && q >= 0) {
                        B = given(p.dht, q);
                        A = p.one;
                        cut = true;
                    }
                    A = mul2(A, o.a[j]);
                    B = mul2(o.a[j], add2(din(at, in, j), B));
                }
            }
        };
        if (kPacked && border(at.last)) back(std::false_type{}, std::integral_constant<bool, kPacked>{});
        else if (n == kRun) back(std::true_type{}, std::false_type{});
        else back(std::false_type{}, std::false_type{});
        tell(s.a[turn][warp], s.b[turn][warp]);
        bar_arrive(kReady + turn, warps + 1);
    };
    auto rear = [&](int k, Set &o) {
        const Info<kTok> &at = s.info[k % kInfos];
        const int turn = k & 1, d = at.d0 + 2 * lane, nch = max(0, min(2, p.D - d)), t0 = (at.chunk * warps + warp) * kRun, n = min(kRun, p.T - t0);
        const f32x2 neg_s = mul2(mk2(at.s[lane].x, at.s[lane].y), p.minus);
        const char *in = own + k % 3 * other;
        auto given = [&](const float *t, int q) { return t ? load_f(t + (long long)q * p.D + d, nch) : dup(0.f); };
        bar_sync(kState + turn, warps + 2);
        f32x2 h = mk2(f.start[turn][warp][lane].x, f.start[turn][warp][lane].y), sum = dup(0.f);
        const float2 c = s.carry[turn][lane];
        f32x2 e = act2<kPacked>(s.a[turn][warp][lane], s.b[turn][warp][lane], mk2(c.x, c.y));
        const long long out = ((long long)at.b * p.T + t0) * p.D + d;
        T *const px = static_cast<T *>(p.dx) + out, *const pi = static_cast<T *>(p.di) + out, *const pr = static_cast<T *>(p.dr) + out;
        T *const pz = kZ ? static_cast<T *>(p.dz) + out : nullptr;
        auto finish = [&](auto whole, auto borders) {
            constexpr bool W = decltype(whole)::value, C = decltype(borders)::value;
            auto starts = [&](int j) { return C ? at.first[C ? warp * kRun + j : 0] : -1; };
            auto ends = [&](int j) { return C ? at.last[C ? warp * kRun + j : 0] : -1; };
#pragma unroll
            for (int j = 0; j < kRun; ++j) {  // g becomes G / e
                const int q = starts(j);
                if (C && q >= 0) h = given(p.h0, q);
                const f32x2 x = get(at, in, 2, j), La = mul2(mul2(o.sr[j], neg_s), o.a[j]);
                o.g[j] = fma2(La, h, mul2(o.g[j], x));
                h = fma2(o.a[j], h, mul2(o.mi[j], x));
                if (kZ && (W || j < n)) {
                    const f32x2 z = get(at, in, 4, j), on = sigmoid2(p, z);
                    const f32x2 slope = mul2(on, fma2(z, fma2(on, p.minus, p.one), p.one));
                    M::store(pz + (long long)j * p.D, mul2(mul2(get(at, in, 3, j), h), slope), W ? 2 : nch);
                }
            }
#pragma unroll
            for (int j = kRun - 1; j >= 0; --j) {
                if (W || j < n) {
                    const int q = ends(j);
                    if (C && q >= 0) e = given(p.dht, q);
                    e = add2(e, din(at, in, j));
                    const f32x2 G = mul2(e, o.g[j]), dx = mul2(e, o.mi[j]), si = M::get2(in + kStep + j * M::kRow, in + j * M::kRow);
                    sum = add2(sum, G);
                    const long long to = (long long)j * p.D;
                    M::store(px + to, dx, W ? 2 : nch);
                    M::store(pi + to, mul2(mul2(dx, get(at, in, 2, j)), fma2(si, p.minus, p.one)), W ? 2 : nch);
                    M::store(pr + to, mul2(G, fma2(o.sr[j], p.minus, p.one)), W ? 2 : nch);
                    e = mul2(e, o.a[j]);
                    if (kPacked ? C : j == 0) {
                        const int first = kPacked ? starts(j) : t0 == 0 ? at.b : -1;
                        if (first >= 0 && p.dh0) store_f(p.dh0 + (long long)first * p.D + d, e, nch);
                    }
                }
            }
        };
        if (kPacked && (border(at.first) || border(at.last))) finish(std::false_type{}, std::integral_constant<bool, kPacked>{});
        else if (n == kRun && p.D - at.d0 >= kTile) finish(std::true_type{}, std::false_type{});
        else finish(std::false_type{}, std::false_type{});
        float g0, g1;
        un2(sum, g0, g1);
        f.sums[turn][warp][lane] = make_float2(g0, g1);
        bar_arrive(kSums + turn, warps + 1);
    };
    Set even, odd;  // as in the forward
    stage(0);
    stage(1);
    front(0, even);
    for (int k = 0; s.info[k % kInfos].tile < p.tiles; k += 2) {
        stage(k + 2);
        front(k + 1, odd);
        rear(k, even);
        if (s.info[(k + 1) % kInfos].tile >= p.tiles) break;
        stage(k + 3);
        front(k + 2, even);
        rear(k + 1, odd);
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
        f32x2 a, rest;
        decay2<false>(p.c, mul2(sigmoid2(p.c, r), s), a, rest);
        y = fma2(a, before, mul2(sqrt_2(rest), mul2(sigmoid2(p.c, i), x)));
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
    const float poly[4] = {-4.99999642e-1f, 1.66652888e-1f, -4.15001325e-2f, 7.53017422e-3f};
    for (int i = 0; i < 4; ++i) p.poly[i] = pair_of(poly[i]);
    return p;
}

struct LinPlan {
    int warps;  // with tokens, of a CTA
    long long chunks;
};
LinPlan linear_plan(long long T, bool bwd) {
    const int run = bwd ? kBwdRun : kFwdRun, warps = (int)std::max(1LL, std::min<long long>(kWarps, (T + run - 1) / run));
    return LinPlan{warps, std::max(1LL, (T + warps * run - 1) / (warps * run))};
}

// The workspace: the counter and the records (where there is more than one
// chunk), the backward's sums.
struct LinSpace {
    size_t rec, part, total, zeroed;
};
LinSpace linear_space(long long B, long long T, long long D, bool bwd) {
    const LinPlan pl = linear_plan(T, bwd);
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

// As many CTAs as run at once, with `stages` tiles in shared memory (one where
// every CTA has but one).  `each`: a warp's part of a tile.
template <typename K>
int linear_launch(K *kernel, const LinP &p, const LinPlan &pl, int stages, size_t each, cudaStream_t st) {
    const int threads = 32 * (pl.warps + kHelpers);
    const long long grid = std::min<long long>(p.tiles, (long long)layer_sms() * (65536 / (threads * kRegs)));
    const size_t smem = each * pl.warps * (grid < p.tiles ? stages : 1);
    // the kernel's limit, not this call's need: another thread may set it between this line and the launch
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(each * kWarps * stages));
    if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "linear scan: %s", cudaGetErrorString(e));
    kernel<<<(unsigned)grid, threads, smem, st>>>(p);
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
    LinP p;
    LinPlan pl;
    if ((rc = linear_fill(a, s, false, sp, &p, &pl, st))) return rc;
    const int access = linear_access(a->dtype, {a->x, a->input_gate, a->decay_gate, a->z, a->y},
                                     {a->x_row, a->x_batch, a->i_row, a->i_batch, a->r_row, a->r_batch, a->z ? a->z_row : 0, a->z ? a->z_batch : 0, a->D});
    linear_by_type(a, access, [&](auto t, auto c, auto z, auto k) {
        using E = decltype(t);
        using M = Mem<E, decltype(c)::value>;
        constexpr int kEach = (decltype(z)::value ? 4 : 3) * kFwdRun * M::kRow;
        static_assert(2 * kWarps * kEach + sizeof(Talk<kWarps * kFwdRun>) <= 227 * 1024, "shared memory");
        rc = linear_launch(k_linear_fwd<E, decltype(c)::value, decltype(z)::value, decltype(k)::value>, p, pl, 2, kEach, st);
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
    const LinSpace sp = linear_space(a->B, a->T, a->D, true);
    if ((rc = linear_workspace(a, sp, "linear scan backward"))) return rc;
    LinP p;
    LinPlan pl;
    if ((rc = linear_fill(a, s, true, sp, &p, &pl, st))) return rc;
    const int access = linear_access(a->dtype, {a->x, a->input_gate, a->decay_gate, a->z, a->dy, a->dx, a->di, a->dr, a->dz},
                                     {a->x_row, a->x_batch, a->i_row, a->i_batch, a->r_row, a->r_batch, a->z ? a->z_row : 0, a->z ? a->z_batch : 0, a->D});
    linear_by_type(a, access, [&](auto t, auto c, auto z, auto k) {
        using E = decltype(t);
        using M = Mem<E, decltype(c)::value>;
        constexpr int kEach = (decltype(z)::value ? 5 : 4) * kBwdRun * M::kRow;
        static_assert(3 * kWarps * kEach + sizeof(Talk<kWarps * kBwdRun>) + sizeof(BackTalk) <= 227 * 1024, "shared memory");
        rc = linear_launch(k_linear_bwd<E, decltype(c)::value, decltype(z)::value, decltype(k)::value>, p, pl, 3, kEach, st);
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
