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
// Bound by memory: a row is read once, reduced in the registers of its threads,
// and written once.  Short rows (the heads of a mixer's output) share a warp: 16 or
// 32 lanes a row and shuffles alone; longer ones have a CTA.  The backward's CTAs
// stay, for the weights' gradients, and take rows in turn: each thread copies its
// pieces of the rows to come to shared memory of its own, asynchronously, so that
// reads are on their way while a row is reduced, and no thread waits for
// another's copies.
//
// bf16: 16384 x 4096 with stream and next norm 89 us (6.0 TB/s); 8192 x 4096 with
// all parts 62 us (5.4 TB/s) and 121 backward (4.4 TB/s); 262144 heads of 128 with
// their gate 37 us (5.5 TB/s) and 88 (3.8 TB/s).  The backward is bound by
// instructions, 63 an element of a head (issue slots 62 % used, 24 warps an SM; at
// 4096 channels 47 %, 16 warps), and by one reduction after another.
// Plans that these figures do not speak for, 33.5 million elements with all parts,
// backward, bf16 | fp32: 512 channels 147 | 252 us and 1024 channels 178 | 333 (one
// or four small CTAs an SM), above 8192 channels 391 | 596 (threads at 64
// registers, which spill), rows that are not whole vectors on 16-byte
// boundaries 683 to 752 | 617 to 677 (element by element, no rows ahead, spills).
#include <string.h>

#include "gdr_layer.h"

namespace {

constexpr int kMaxD = 16384, kWide = 1024, kNarrow = 512, kShort = 256;  // greatest row; threads of a CTA
constexpr int kStreams = 5;  // most tensors that a row is read from

struct BlockP {
    const void *x, *gate, *residual, *dr, *dy;
    const float *weight, *next;
    void *r, *y, *dx, *dgate, *dres;
    float *stats, *part;  // part: [CTAs, 2, D], the sums of dw and dw'
    long long M, x_row, x_outer, gate_row, gate_outer, res_row, res_outer;
    int D, lanes, inner, depth;  // lanes: threads of a row; depth: rows in shared memory (0: none)
    float scale, eps;
    // Pairs of constants, read from the parameters: packed instructions take no
    // immediate operand, and the compiler would make a pair of one at each use.
    f32x2 neg_log2e, one, minus, scale2;
};

// Where a row of x, gate and residual begins: `inner` heads of a token have a stride of their own.
struct Row {
    long long outer, head;
    __device__ __forceinline__ Row(long long row, int inner) : outer(row), head(0) {
        if (inner > 1) {
            const unsigned r = (unsigned)row, n = (unsigned)inner, o = r / n;  // fewer than 2^31 rows
            outer = o;
            head = r - o * n;
        }
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
    static constexpr int kSlot = kN * (int)sizeof(T), kPer = (int)sizeof(T) / 2;  // bytes of a thread's part, pieces of a vector
    // Copies a thread's part to its place in shared memory, asynchronously (kV = 8): pieces of 16 bytes, a CTA's threads apart.
    static __device__ __forceinline__ void fetch(const T *row, int D, int tid, int lanes, uint32_t place) {
#pragma unroll
        for (int i = 0; i < kSlot / 16; ++i) {
            const int c = Part::at(i / kPer * 8, tid, lanes) + i % kPer * (16 / (int)sizeof(T));
            if (c < D) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place + i * blockDim.x * 16), "l"(row + c) : "memory");
        }
    }
    static __device__ __forceinline__ void fetched(uint32_t place, int D, int tid, int lanes, Raw &raw) {
#pragma unroll
        for (int i = 0; i < kSlot / 16; ++i) {
            uint4 &v = raw.v[i / kPer].w[i % kPer];
            v = make_uint4(0, 0, 0, 0);
            if (Part::at(i / kPer * 8, tid, lanes) < D)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(place + i * blockDim.x * 16) : "memory");
        }
    }
    // Elements in pairs, for packed fp32 instructions.
    static constexpr int kH = kN / 2;
    static __device__ __forceinline__ void get(const Raw &raw, f32x2 (&f)[kH]) {
#pragma unroll
        for (int i = 0; i < kN; i += kV == 8 ? 8 : 2) {
            if (kV == 8) {
                float e[8];
                unpack8(raw.v[i / 8], e);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[i / 2 + k < kH ? i / 2 + k : 0] = mk2(e[2 * k], e[2 * k + 1]);
            } else {
                f[i / 2] = mk2(to_f(raw.s[kV == 8 ? 0 : i]), to_f(raw.s[kV == 8 ? 0 : i + 1]));
            }
        }
    }
    static __device__ __forceinline__ void store(T *row, int D, int tid, int lanes, const f32x2 (&f)[kH]) {
        float e[kN];
#pragma unroll
        for (int i = 0; i < kH; ++i) un2(f[i], e[2 * i], e[2 * i + 1]);
        if (kV == 8) {
#pragma unroll
            for (int i = 0; i < kN / 8; ++i) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = e[8 * i + k];
                store8<T, true>(row + at(8 * i, tid, lanes), v, D - at(8 * i, tid, lanes));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int c = at(i, tid, lanes);
                if (c < D) from_f(row[c], e[i]);
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

__device__ __forceinline__ f32x2 dup(float v) { return mk2(v, v); }
__device__ __forceinline__ float both(f32x2 v) {
    float a, b;
    un2(v, a, b);
    return a + b;
}
__device__ __forceinline__ f32x2 sigmoid2(const BlockP &p, f32x2 v) {
    float a, b;
    un2(mul2(v, p.neg_log2e), a, b);
    un2(add2(mk2(ex2f(a), ex2f(b)), p.one), a, b);
    return mk2(rcpf(a), rcpf(b));
}
__device__ __forceinline__ f32x2 silu2(const BlockP &p, f32x2 v) { return mul2(v, sigmoid2(p, v)); }

// The rows of a CTA, `group` at a time, from kMost tensors, of which those that
// are there have a place in each stage.  What a row costs beside its elements
// counts: addresses go from row to row by additions.
template <typename P, typename T, int kMost, int kMask>
struct Rows {
    // Whether tensor k is there: bit k of kMask, or as the call says (kMask < 0).
    __device__ __forceinline__ bool has(int k) const { return kMask >= 0 ? kMask >> k & 1 : from[k] != nullptr; }
    const T *from[kMost];
    long long row_stride[kMost], outer_stride[kMost];
    long long M, first, step, row;  // row: this thread's of the current group
    int D, tid, lanes, inner, depth, len;
    uint32_t stages, stage, get, put;   // the thread's places: of the first stage, from stage to stage, of the current row's, of the next to be filled
    const T *next_row[kMost];           // of the next group to be fetched

    __device__ __forceinline__ Rows(const BlockP &p, int group, char *smem) {
        M = p.M;
        first = (long long)blockIdx.x * group;
        step = (long long)gridDim.x * group;
        D = p.D;
        lanes = p.lanes;
        tid = lanes == (int)blockDim.x ? threadIdx.x : threadIdx.x % lanes;
        inner = p.inner;
        stages = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    }
    __device__ __forceinline__ void tensor(int k, const void *t, long long row, long long outer) {
        from[k] = static_cast<const T *>(t);
        row_stride[k] = row;
        outer_stride[k] = outer;
    }
    // the place of tensor k among those that are there
    __device__ __forceinline__ uint32_t place(int k) const {
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kMost; ++i) n += i < k && has(i);
        return n * blockDim.x * P::kSlot;
    }
    __device__ __forceinline__ const T *at(int k, const Row &q) const { return from[k] + q.at(row_stride[k], outer_stride[k]); }
    __device__ __forceinline__ long long mine(long long group) const { return group + (lanes == (int)blockDim.x ? 0 : (int)threadIdx.x / lanes); }
    __device__ __forceinline__ uint32_t after(uint32_t at) const { return at + stage < stages + depth * stage ? at + stage : stages; }
    __device__ __forceinline__ void fetch(long long group) {
        const long long r = mine(group);
        if (r < M) {
            if (inner > 1) {
                const Row q(r, inner);
#pragma unroll
                for (int k = 0; k < kMost; ++k) next_row[k] = has(k) ? at(k, q) : nullptr;
            }
            uint32_t to = put;
#pragma unroll
            for (int k = 0; k < kMost; ++k)
                if (has(k)) {
                    P::fetch(next_row[k], D, tid, lanes, to);
                    to += blockDim.x * P::kSlot;
                    next_row[k] += step * outer_stride[k];
                }
        }
        put = after(put);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void begin(int depth_) {
        depth = depth_;
        stage = place(kMost);
        get = put = stages;
#pragma unroll
        for (int k = 0; k < kMost; ++k) next_row[k] = has(k) ? from[k] + mine(first) * outer_stride[k] : nullptr;
        for (int i = 0; i + 1 < depth; ++i) fetch(first + i * step);
    }
    // Whether there is a group; its rows may be read then.
    __device__ __forceinline__ bool there() {
        if (first >= M) return false;
        row = mine(first);
        len = row < M ? D : 0;
        if (depth) {
            fetch(first + (depth - 1) * step);  // in the place of the group before, which has been read
            if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
            else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
            else asm volatile("cp.async.wait_group 1;" ::: "memory");
        }
        return true;
    }
    __device__ __forceinline__ void read(int k, typename P::Raw &raw) const {
        if (depth) P::fetched(get + place(k), len, tid, lanes, raw);
        else P::load(at(k, Row(row, inner)), len, tid, lanes, raw);
    }
    __device__ __forceinline__ void next() {
        first += step;
        if (depth) get = after(get);
    }
};

// What a call has beside x: bits of kHas (or, kHas < 0, as the pointers say: rows
// of other widths and alignments).
constexpr int kGate = 1, kStream = 2, kNext = 4;

// Forward: one row a CTA (kCta) or `lanes` lanes of a warp.
template <typename T, int kV, int kN, int kThreads, bool kCta, int kHas>
__global__ void __launch_bounds__(kThreads) k_block_fwd(const __grid_constant__ BlockP p) {
    using P = Part<T, kV, kN>;
    __shared__ float buf[2][1][32];
    const int tid = kCta ? threadIdx.x : threadIdx.x % p.lanes, D = p.D;
    const long long row = kCta ? blockIdx.x : (long long)blockIdx.x * (blockDim.x / p.lanes) + threadIdx.x / p.lanes;
    const bool on = row < p.M;  // lanes of rows past the last only join the shuffles
    typename P::Raw rx, rg, rr;
    const int len = on ? D : 0;
    const bool gate = kHas < 0 ? p.gate != nullptr : kHas & kGate, stream = kHas < 0 ? p.residual != nullptr : kHas & kStream,
               next = kHas < 0 ? p.next != nullptr : kHas & kNext;
    const Row from(row, p.inner);
    P::load(static_cast<const T *>(p.x) + from.at(p.x_row, p.x_outer), len, tid, p.lanes, rx);
    if (gate) P::load(static_cast<const T *>(p.gate) + from.at(p.gate_row, p.gate_outer), len, tid, p.lanes, rg);
    if (stream) P::load(static_cast<const T *>(p.residual) + from.at(p.res_row, p.res_outer), len, tid, p.lanes, rr);
    f32x2 v[P::kH], acc = dup(0.f);
    P::get(rx, v);
#pragma unroll
    for (int i = 0; i < P::kH; ++i) acc = fma2(v[i], v[i], acc);
    float sum[1] = {both(acc)};
    f32x2 g[P::kH], w[P::kH];
    typename Part<float, kV, kN>::Raw rw;
    Part<float, kV, kN>::load(p.weight, D, tid, p.lanes, rw);
    Part<float, kV, kN>::get(rw, w);
#pragma unroll
    for (int i = 0; i < P::kH; ++i) v[i] = mul2(v[i], w[i]);
    if (gate) {
        P::get(rg, g);
#pragma unroll
        for (int i = 0; i < P::kH; ++i) v[i] = mul2(v[i], silu2(p, g[i]));
    }
    row_sum<1, kCta>(sum, p.lanes, buf[0]);
    const float inv_x = 1.f / sqrtf(sum[0] / (float)D + p.eps);
    const f32x2 k = dup(p.scale * inv_x);
    if (stream) P::get(rr, g);
#pragma unroll
    for (int i = 0; i < P::kH; ++i) v[i] = stream ? fma2(v[i], k, g[i]) : mul2(v[i], k);
    P::store(static_cast<T *>(p.r) + row * D, len, tid, p.lanes, v);
    float inv_r = 0.f;
    if (next) {
        // places behind a row's end hold zeros
        acc = dup(0.f);
#pragma unroll
        for (int i = 0; i < P::kH; ++i) acc = fma2(v[i], v[i], acc);
        sum[0] = both(acc);
        row_sum<1, kCta>(sum, p.lanes, buf[1]);
        inv_r = 1.f / sqrtf(sum[0] / (float)D + p.eps);
        Part<float, kV, kN>::load(p.next, D, tid, p.lanes, rw);
        Part<float, kV, kN>::get(rw, w);
#pragma unroll
        for (int i = 0; i < P::kH; ++i) v[i] = mul2(mul2(v[i], dup(inv_r)), w[i]);
        P::store(static_cast<T *>(p.y) + row * D, len, tid, p.lanes, v);
    }
    if (p.stats && on && tid == 0) *reinterpret_cast<float2 *>(p.stats + 2 * row) = make_float2(inv_x, inv_r);
}

// A CTA keeps its part of the weights' gradients in registers.
template <typename T, int kV, int kN, int kThreads, bool kCta, int kHas>
__global__ void __launch_bounds__(kThreads, kThreads == kShort && kN == 8 ? 3 : 1) k_block_bwd(const __grid_constant__ BlockP p) {
    using P = Part<T, kV, kN>;
    using W = Part<float, kV, kN>;
    extern __shared__ __align__(16) char stages[];
    __shared__ float buf[2][3][32];
    const int tid = kCta ? threadIdx.x : threadIdx.x % p.lanes, D = p.D, group = kCta ? 1 : blockDim.x / p.lanes;
    constexpr int kH = P::kH;
    f32x2 gw[kH], gn[kH];
#pragma unroll
    for (int i = 0; i < kH; ++i) gw[i] = gn[i] = dup(0.f);
    // kHas: the gradients of all outputs are there
    constexpr int kMask = kHas < 0 ? -1 : 1 | (kHas & kGate ? 2 : 0) | ((kHas & kStream) && (kHas & kNext) ? 4 : 0) | 8 | (kHas & kNext ? 16 : 0);
    const bool gate = kHas < 0 ? p.gate != nullptr : kHas & kGate, stream = kHas < 0 ? p.residual != nullptr : kHas & kStream,
               next = kHas < 0 ? p.next != nullptr : kHas & kNext;
    const bool has_dr = kHas >= 0 || p.dr, has_dy = kHas >= 0 || p.dy;
    Rows<P, T, kStreams, kMask> rows(p, group, stages);
    rows.tensor(0, p.x, p.x_row, p.x_outer);
    rows.tensor(1, p.gate, p.gate_row, p.gate_outer);
    rows.tensor(2, next ? p.residual : nullptr, p.res_row, p.res_outer);  // read only for the norm of the stream
    rows.tensor(3, p.dr, D, (long long)p.inner * D);
    rows.tensor(4, next ? p.dy : nullptr, D, (long long)p.inner * D);
    rows.begin(kV == 8 ? p.depth : 0);
    auto stats = [&](long long first) {  // a row's reciprocal roots, read a turn ahead
        const long long r = rows.mine(first);
        return first < p.M && r < p.M ? *reinterpret_cast<const float2 *>(p.stats + 2 * r) : make_float2(0.f, 0.f);
    };
    float2 inv_next = stats(rows.first);
    int turn = 0;
    for (; rows.there(); rows.next(), turn ^= 1) {
        const float2 inv = inv_next;
        const f32x2 inv_x = dup(inv.x), inv_y = dup(inv.y);
        inv_next = stats(rows.first + rows.step);
        typename P::Raw raw;
        typename W::Raw rw;
        f32x2 n[kH], c[kH], u[kH], r[kH];  // c: n w silu(gate)
        rows.read(0, raw);
        P::get(raw, n);
        W::load(p.weight, D, tid, p.lanes, rw);
        W::get(rw, c);
        if (gate) {
            rows.read(1, raw);
            P::get(raw, r);
#pragma unroll
            for (int i = 0; i < kH; ++i) c[i] = mul2(c[i], silu2(p, r[i]));
        }
#pragma unroll
        for (int i = 0; i < kH; ++i) {
            n[i] = mul2(n[i], inv_x);
            c[i] = mul2(c[i], n[i]);
            u[i] = dup(0.f);
        }
        if (has_dr) {
            rows.read(3, raw);
            P::get(raw, u);
        }
        f32x2 s0 = dup(0.f), s1 = s0, s2 = s0;
        if (next) {
#pragma unroll
            for (int i = 0; i < kH; ++i) r[i] = dup(0.f);
            if (stream) {
                rows.read(2, raw);
                P::get(raw, r);
            }
            f32x2 f[kH], w2[kH];
#pragma unroll
            for (int i = 0; i < kH; ++i) f[i] = dup(0.f);
            if (has_dy) {
                rows.read(4, raw);
                P::get(raw, f);
            }
            W::load(p.next, D, tid, p.lanes, rw);
            W::get(rw, w2);
#pragma unroll
            for (int i = 0; i < kH; ++i) {
                r[i] = fma2(p.scale2, c[i], r[i]);
                gn[i] = fma2(f[i], mul2(r[i], inv_y), gn[i]);
                f[i] = mul2(f[i], w2[i]);
                s0 = fma2(f[i], r[i], s0);
                u[i] = fma2(inv_y, f[i], u[i]);
                s2 = fma2(r[i], c[i], s2);
            }
        }
#pragma unroll
        for (int i = 0; i < kH; ++i) s1 = fma2(u[i], c[i], s1);
        float s[3] = {both(s0), both(s1), both(s2)};
        row_sum<3, kCta>(s, p.lanes, buf[turn]);
        const float k = next ? inv.y * inv.y * inv.y * s[0] / (float)D : 0.f;
        const float mean = p.scale * (s[1] - k * s[2]) / (float)D;  // of b n
        const f32x2 minus_k = dup(-k);
        if (next) {
#pragma unroll
            for (int i = 0; i < kH; ++i) u[i] = fma2(minus_k, r[i], u[i]);
            if (stream) P::store(static_cast<T *>(p.dres) + rows.row * D, rows.len, tid, p.lanes, u);
        }
        W::load(p.weight, D, tid, p.lanes, rw);
        f32x2 w[kH];
        W::get(rw, w);
        const f32x2 drop = dup(-mean * inv.x);
#pragma unroll
        for (int i = 0; i < kH; ++i) u[i] = mul2(u[i], p.scale2);
        if (gate) {
            f32x2 g[kH];
            rows.read(1, raw);
            P::get(raw, g);
#pragma unroll
            for (int i = 0; i < kH; ++i) {
                const f32x2 on = sigmoid2(p, g[i]), sl = mul2(g[i], on), ds = fma2(sl, fma2(on, p.minus, p.one), on), un = mul2(u[i], n[i]);
                gw[i] = fma2(un, sl, gw[i]);
                g[i] = mul2(mul2(un, w[i]), ds);
                u[i] = fma2(n[i], drop, mul2(mul2(mul2(u[i], w[i]), sl), inv_x));
            }
            P::store(static_cast<T *>(p.dgate) + rows.row * D, rows.len, tid, p.lanes, g);
        } else {
#pragma unroll
            for (int i = 0; i < kH; ++i) {
                gw[i] = fma2(u[i], n[i], gw[i]);
                u[i] = fma2(n[i], drop, mul2(mul2(u[i], w[i]), inv_x));
            }
        }
        P::store(static_cast<T *>(p.dx) + rows.row * D, rows.len, tid, p.lanes, u);
    }
    float ew[kN], en[kN];
#pragma unroll
    for (int i = 0; i < kH; ++i) {
        un2(gw[i], ew[2 * i], ew[2 * i + 1]);
        un2(gn[i], en[2 * i], en[2 * i + 1]);
    }
    float *to = p.part + (long long)blockIdx.x * 2 * D;
    if (kCta) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int c = P::at(i, tid, p.lanes);
            if (c < D) {
                to[c] = ew[i];
                to[D + c] = en[i];
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
                    sums[0][c] = v ? sums[0][c] + ew[i] : ew[i];
                    sums[1][c] = v ? sums[1][c] + en[i] : en[i];
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
BlockPlan block_plan(long long D) {
    if (D <= 128) return {8, 16, kShort, false};
    if (D <= 256) return {8, 32, kShort, false};
    if (D <= 512) return {16, 32, kShort, false};
    // two CTAs of 256 threads an SM for 4096 channels (the gradient of 8192 x 4096 120 us; one of 512, eight elements a thread, 146)
    const int t = (int)((D + 511) / 512 * 32);
    return {16, t, t, true};
}

// Rows that a thread keeps on their way (none where two have no room), and CTAs: as
// many as run at once.
struct BlockGrid {
    int depth, ctas;
    size_t smem;
};
constexpr size_t block_room(int per_sm) { return (size_t)(224 * 1024) / per_sm - 2048; }  // shared memory of a CTA for rows
static_assert(block_room(1) + 2 * 32 * 16 * 4 + 2 * 3 * 32 * 4 <= 227 * 1024, "rows, the groups' sums and the rows' sums");
BlockGrid block_grid(long long M, const BlockPlan &pl, bool vec, int dtype, int streams, int per_sm) {
    const size_t stage = (size_t)streams * pl.threads * pl.n * (dtype == GDR_BF16 ? 2 : 4);
    const int depth = vec ? (int)std::min<size_t>(4, block_room(per_sm) / stage) : 0;
    const long long need = (M + pl.rows() - 1) / pl.rows();
    BlockGrid g{};
    g.depth = depth >= 2 ? depth : 0;
    g.smem = g.depth * stage;
    g.ctas = (int)std::max(1LL, std::min(need, (long long)per_sm * layer_sms()));
    return g;
}
// CTAs of an SM of the backward: as many as registers allow of the threads that a
// kernel may have at most (512; 64-thread CTAs of 513 to 1024 channels would fit
// eight times, and take four).
int block_per_sm(const BlockPlan &pl) {
    if (!pl.cta) return pl.n == 8 ? 3 : 1;
    return std::max(1, std::min(4, 512 / pl.threads));
}
int block_ctas(long long M, long long D) { return block_grid(M, block_plan(D), false, GDR_BF16, 0, block_per_sm(block_plan(D))).ctas; }

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
    p.D = (int)a->D; p.lanes = pl.lanes; p.inner = (int)a->inner; p.depth = 0;
    p.scale = a->scale; p.eps = a->eps;
    auto pair = [](float v) {
        uint32_t bits;
        memcpy(&bits, &v, sizeof bits);
        return (f32x2)bits << 32 | bits;
    };
    p.neg_log2e = pair(-kLog2e); p.one = pair(1.f); p.minus = pair(-1.f); p.scale2 = pair(a->scale);
    return p;
}

// f(type, vector, elements, most threads, a CTA a row, what the call has): kernels
// for what a call has where rows are vectors; with the pointers looked at for each
// row the gradient of 8192 x 4096 took 169 us, without 147.  Rows of 257 to 512
// channels and of more than 8192 have only the kernel that looks: each plan's own
// set is sixteen more kernels to build, whose gain there was not measured.
template <typename F>
void block_by_type(int dtype, bool vec, int has, const BlockPlan &pl, F f) {
    using std::integral_constant;
    auto w = [&](auto t, auto v, auto h) {
        if (!pl.cta && pl.n == 8) f(t, v, integral_constant<int, 8>{}, integral_constant<int, kShort>{}, std::false_type{}, h);
        else if (pl.cta && pl.threads <= kNarrow) f(t, v, integral_constant<int, 16>{}, integral_constant<int, kNarrow>{}, std::true_type{}, h);
        else if constexpr (!(decltype(h)::value >= 0)) {
            if (!pl.cta) f(t, v, integral_constant<int, 16>{}, integral_constant<int, kShort>{}, std::false_type{}, h);
            else f(t, v, integral_constant<int, 16>{}, integral_constant<int, kWide>{}, std::true_type{}, h);
        }
    };
    auto k = [&](auto t) {
        const integral_constant<int, 8> eight{};
        if (!vec) w(t, integral_constant<int, 1>{}, integral_constant<int, -1>{});
        else if (!(pl.n == 8 || (pl.cta && pl.threads <= kNarrow)) || has < 0) w(t, eight, integral_constant<int, -1>{});
        else if (has == 0) w(t, eight, integral_constant<int, 0>{});
        else if (has == 1) w(t, eight, integral_constant<int, 1>{});
        else if (has == 2) w(t, eight, integral_constant<int, 2>{});
        else if (has == 3) w(t, eight, integral_constant<int, 3>{});
        else if (has == 4) w(t, eight, integral_constant<int, 4>{});
        else if (has == 5) w(t, eight, integral_constant<int, 5>{});
        else if (has == 6) w(t, eight, integral_constant<int, 6>{});
        else w(t, eight, integral_constant<int, 7>{});
    };
    if (dtype == GDR_BF16) k(bf16_t{}); else k(float{});
}
int block_has(const gdr_block_norm_args *a) { return (a->gate ? kGate : 0) | (a->residual ? kStream : 0) | (a->next_weight ? kNext : 0); }
template <typename K>
int block_launch(K *kernel, const BlockP &p, const BlockGrid &g, int threads, cudaStream_t st) {
    // the most that any call takes, not this call's need: another thread may set it between this line and the launch
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)block_room(1));
    if (e != cudaSuccess) return layer_fail(GDR_ERR_CUDA, "block norm: %s", cudaGetErrorString(e));
    kernel<<<g.ctas, threads, g.smem, st>>>(p);
    return GDR_OK;
}

}  // namespace

extern "C" {

int gdr_block_norm_fwd(const gdr_block_norm_args *a, void *stream) {
    const int rc = block_common(a, false);
    if (rc || a->M == 0) return rc;
    const BlockPlan pl = block_plan(a->D);
    const BlockP p = block_fill(a, pl);
    const bool vec = block_vec(a);
    const unsigned ctas = (unsigned)((a->M + pl.rows() - 1) / pl.rows());
    block_by_type(a->dtype, vec, block_has(a), pl, [&](auto t, auto v, auto n, auto th, auto cta, auto has) {
        k_block_fwd<decltype(t), decltype(v)::value, decltype(n)::value, decltype(th)::value, decltype(cta)::value, decltype(has)::value>
            <<<ctas, pl.threads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    });
    return layer_launched("block norm forward");
}

size_t gdr_block_norm_bwd_workspace_size(long long M, long long D) {
    if (M < 0 || D < 1 || D > kMaxD || M >= (1LL << 31)) return 0;
    return ((size_t)block_ctas(M, D) * 2 * D * 4 + 15) & ~size_t(15);
}

int gdr_block_norm_bwd(const gdr_block_norm_args *a, void *stream) {
    int rc = block_common(a, true);
    if (rc) return rc;
    if (!a->workspace) return layer_fail(GDR_ERR_WORKSPACE, "block norm backward: workspace is null");
    if (!multiple16(a->workspace)) return layer_fail(GDR_ERR_ALIGN, "block norm backward: workspace must be 16-byte aligned");
    if (a->workspace_bytes < gdr_block_norm_bwd_workspace_size(a->M, a->D))
        return layer_fail(GDR_ERR_WORKSPACE, "block norm backward: workspace too small");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const BlockPlan pl = block_plan(a->D);
    BlockP p = block_fill(a, pl);
    const bool vec = block_vec(a), next = a->next_weight != nullptr;
    const int streams = 1 + (a->gate != nullptr) + (a->residual && next) + (a->dr != nullptr) + (a->dy && next);
    const BlockGrid g = block_grid(a->M, pl, vec, a->dtype, streams, block_per_sm(pl));
    const int ctas = g.ctas;
    p.depth = g.depth;
    const int has = a->dr && (a->dy || !next) ? block_has(a) : -1;
    block_by_type(a->dtype, vec, has, pl, [&](auto t, auto v, auto n, auto th, auto cta, auto h) {
        rc = block_launch(k_block_bwd<decltype(t), decltype(v)::value, decltype(n)::value, decltype(th)::value, decltype(cta)::value, decltype(h)::value>, p, g,
                          pl.threads, st);
    });
    if (rc) return rc;
    k_block_sum<<<dim3((unsigned)((a->D + 31) / 32), a->next_weight ? 2 : 1), dim3(32, 32), 0, st>>>(p.part, ctas, p.D, a->dweight, a->dnext_weight);
    return layer_launched("block norm backward");
}

}  // extern "C"
