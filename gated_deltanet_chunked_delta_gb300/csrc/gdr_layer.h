// gdr_layer.h -- shared by the layer operators around a recurrent mixer
// (gdr_conv.cu, gdr_ssm.cu, gdr_norm.cu, gdr_fp8.cu): element access, the
// scalar functions, sequence lookup and argument checks.  Not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <type_traits>

#include "gdr.h"
#include "gdr_once.h"

namespace gdr {
int set_last_error(int code, const char *msg);  // gdr_api.cu
// Each translation unit's device status word, read and cleared (gdr_check_status).
unsigned conv_take_status(cudaStream_t st);
unsigned ssm_take_status(cudaStream_t st);
unsigned fp8_take_status(cudaStream_t st);
}  // namespace gdr

namespace {

constexpr unsigned kStatusTimeout = 1u, kStatusIndex = 2u;  // bits of a status word
constexpr float kLog2e = 1.4426950408889634f;

// ---- host ------------------------------------------------------------------

inline int layer_fail(int code, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return gdr::set_last_error(code, msg);
}

// A required or optional pointer whose address is a multiple of `align` bytes.
inline int layer_ptr(const char *name, const void *p, bool required, unsigned align) {
    if (!p) return required ? layer_fail(GDR_ERR_ARG, "%s is null", name) : GDR_OK;
    if (reinterpret_cast<uintptr_t>(p) & (align - 1))
        return layer_fail(GDR_ERR_ALIGN, "%s is not %u-byte aligned", name, align);
    return GDR_OK;
}

inline int layer_launched(const char *what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GDR_OK : layer_fail(GDR_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
}

inline bool multiple16(const void *p) { return !(reinterpret_cast<uintptr_t>(p) & 15u); }

// The current device, -1 when there is none.
inline int layer_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) return dev;
    cudaGetLastError();
    return -1;
}

// SM count of the current device, asked once a device (152 when none answers).
inline int layer_sms() {
    static gdr::OncePerDevice known;
    const int dev = layer_device();
    return known.get(dev, 152, [&] {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) return sms;
        cudaGetLastError();
        return 0;
    });
}

// ---- device ----------------------------------------------------------------

struct bf16_t {
    uint16_t bits;
};

__device__ __forceinline__ float to_f(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {  // round to nearest even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void from_f(bf16_t &d, float v) { d.bits = (uint16_t)pack2(v, 0.f); }
__device__ __forceinline__ void from_f(float &d, float v) { d = v; }

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};
__device__ __forceinline__ void unpack8(const Raw8<bf16_t> &r, float (&f)[8]) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(r.w[i].x);
        f[4 * i + 1] = __uint_as_float(r.w[i].y);
        f[4 * i + 2] = __uint_as_float(r.w[i].z);
        f[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
}
__device__ __forceinline__ void pack8(const float (&f)[8], Raw8<bf16_t> &r) {
    r.w[0] = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void pack8(const float (&f)[8], Raw8<float> &r) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r.w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                            __float_as_uint(f[4 * i + 3]));
}
// Loads eight elements from p (16-byte aligned), zeros if n is not positive.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T *p, int n) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
        r.w[i] = n > 0 ? reinterpret_cast<const uint4 *>(p)[i] : make_uint4(0, 0, 0, 0);
    return r;
}
// Stores the first n of eight elements (kVec: p is 16-byte aligned and n is 8 or not positive).
template <typename T, bool kVec>
__device__ __forceinline__ void store8(T *p, const float (&f)[8], int n) {
    if (kVec) {
        if (n <= 0) return;
        Raw8<T> r;
        pack8(f, r);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) from_f(p[i], f[i]);
    }
}

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpf(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-v)
__device__ __forceinline__ float sigmoidf(float v) { return rcpf(1.f + ex2f(-kLog2e * v)); }
// log(1 + e^v) = max(v, 0) + log1p(u), u = e^-|v| in (0, 1].  log1p(u) is
// 2 atanh(s) with s = u / (2 + u) <= 1/3; its series to s^13 leaves a relative
// remainder below 2^-26.  A plain log(1 + u) would round 1 + u and lose the
// small steps (u near 1e-3) to 2^-14 relative.
__device__ __forceinline__ float softplusf(float v) {
    const float u = ex2f(-kLog2e * fabsf(v));
    const float s = u * rcpf(2.f + u), s2 = s * s;
    float p = fmaf(s2, 1.f / 13, 1.f / 11);
    p = fmaf(s2, p, 1.f / 9);
    p = fmaf(s2, p, 1.f / 7);
    p = fmaf(s2, p, 1.f / 5);
    p = fmaf(s2, p, 1.f / 3);
    p = fmaf(s2, p, 1.f);
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

// Packed pairs of fp32 (one instruction for two elements).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 mk2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void un2(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The sequences of a call: `n` packed ones with bounds cu[0..n], or (cu null)
// one per batch row covering its T tokens.  Bounds are clamped into [0, T], so
// that whatever cu holds no index leaves the tensors.
struct Seqs {
    const int32_t *cu;
    int n, T;
    __device__ __forceinline__ int bound(int i) const {
        const int v = cu ? cu[i] : (i ? T : 0);
        return min(max(v, 0), T);
    }
    __device__ __forceinline__ int count() const { return cu ? n : 1; }
    // The last sequence that starts at or before token t: the one that holds
    // t (the empty ones before it start at the same place).
    __device__ __forceinline__ int find(int t) const {
        int lo = 0, hi = count() - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (bound(mid) <= t) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
};
// The bounds are meant to rise from 0 to T: one block looks them over.
__device__ __forceinline__ void check_bounds(const Seqs &s, unsigned *status) {
    if (!s.cu) return;
    for (int i = threadIdx.x; i <= s.n; i += blockDim.x) {
        const int v = s.cu[i];
        if ((i == 0 && v != 0) || (i == s.n && v != s.T) || (i > 0 && v < s.cu[i - 1])) atomicOr(status, kStatusIndex);
    }
}

}  // namespace
