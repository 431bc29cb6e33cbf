// gdr_delta.cu -- one token of every sequence through the gated delta rule.
//
//   h <- e^g h,  w = beta (v - h^T k),  h <- h + k w^T,  o = scale h^T q
//
// A column of the state (a channel of v) needs only itself, k and q.  With
// p = h^T k and s = h^T q of the old state
//   w = beta (v - e^g p),   o = scale (e^g s + (k . q) w),
// so that both sums are taken while the state is read, and it is read and
// written once: 8 K V bytes a head against 7 K V flops, bound by memory.  A CTA
// holds kCols columns in registers, so that one row of 16 heads has 64 CTAs; 8
// lanes share a row of 32 columns, a line of 128 bytes.  64 rows x 32 heads of 128
// x 128: 42.7 us, 6.3 TB/s; one row of 16 heads 3.3 us, 13 rows x 8 heads of 64 x 192
// 4.9 us (a CTA's one chain of slot, state, sums and store).
#include "gdr_layer.h"

namespace {

__device__ unsigned g_delta_status;

constexpr int kThreads = 128, kCols = 32;
constexpr int kRows = kThreads / 8;  // rows of the state read at a time

struct DeltaP {
    const void *q, *k, *v;
    const float *g, *beta;
    float *state;
    const int32_t *slots;
    void *o;
    long long q_row, k_row, v_row, n_slots;
    int Hv, V, per;  // per: v-heads a qk-head
    float scale;
};

template <typename T, int kK>
__global__ void __launch_bounds__(kThreads) k_delta_step(const DeltaP p) {
    constexpr int kN = kK / kRows;
    __shared__ float4 part[kThreads / 32][2][8];
    __shared__ float dots[kThreads / 32];
    const int head = blockIdx.y, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const long long row = blockIdx.z;
    const int col = blockIdx.x * kCols + lane % 8 * 4, r0 = threadIdx.x / 8;
    const long long slot = p.slots ? p.slots[row] : row;
    T *o = static_cast<T *>(p.o) + (row * p.Hv + head) * p.V + col;
    if (slot < 0 || slot >= p.n_slots) {
        if (slot >= p.n_slots && threadIdx.x == 0) atomicOr(&g_delta_status, kStatusIndex);
        if (r0 == 0)
#pragma unroll
            for (int e = 0; e < 4; ++e) from_f(o[e], 0.f);
        return;
    }
    float *st = p.state + (slot * p.Hv + head) * kK * p.V + (long long)r0 * p.V + col;
    const T *kp = static_cast<const T *>(p.k) + row * p.k_row + (head / p.per) * kK + r0;
    const T *qp = static_cast<const T *>(p.q) + row * p.q_row + (head / p.per) * kK + r0;
    float4 h[kN];
    float k[kN], q[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) h[i] = *reinterpret_cast<const float4 *>(st + (long long)i * kRows * p.V);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        k[i] = to_f(kp[i * kRows]);
        q[i] = to_f(qp[i * kRows]);
    }
    const float alpha = expf(p.g[row * p.Hv + head]), beta = p.beta[row * p.Hv + head];
    float v[4];
    {
        const T *vp = static_cast<const T *>(p.v) + row * p.v_row + (long long)head * p.V + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = to_f(vp[e]);
    }
    float sums[9] = {};  // h^T k and h^T q of the four columns, k . q
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const float f[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sums[e] = fmaf(f[e], k[i], sums[e]);
            sums[4 + e] = fmaf(f[e], q[i], sums[4 + e]);
        }
        sums[8] = fmaf(k[i], q[i], sums[8]);
    }
#pragma unroll
    for (int e = 0; e < 9; ++e) {
        sums[e] += __shfl_xor_sync(0xffffffffu, sums[e], 8);
        sums[e] += __shfl_xor_sync(0xffffffffu, sums[e], 16);
    }
    if (lane < 8) {
        part[warp][0][lane] = make_float4(sums[0], sums[1], sums[2], sums[3]);
        part[warp][1][lane] = make_float4(sums[4], sums[5], sums[6], sums[7]);
        if (lane == 0) dots[warp] = sums[8];
    }
    __syncthreads();
    float hk[4] = {}, hq[4] = {}, kq = 0.f;
#pragma unroll
    for (int u = 0; u < kThreads / 32; ++u) {
        const float4 a = part[u][0][lane % 8], b = part[u][1][lane % 8];
        hk[0] += a.x; hk[1] += a.y; hk[2] += a.z; hk[3] += a.w;
        hq[0] += b.x; hq[1] += b.y; hq[2] += b.z; hq[3] += b.w;
        kq += dots[u];
    }
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = beta * fmaf(-alpha, hk[e], v[e]);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        float4 n;
        n.x = fmaf(k[i], w[0], alpha * h[i].x);
        n.y = fmaf(k[i], w[1], alpha * h[i].y);
        n.z = fmaf(k[i], w[2], alpha * h[i].z);
        n.w = fmaf(k[i], w[3], alpha * h[i].w);
        *reinterpret_cast<float4 *>(st + (long long)i * kRows * p.V) = n;
    }
    if (r0 == 0)
#pragma unroll
        for (int e = 0; e < 4; ++e) from_f(o[e], p.scale * fmaf(kq, w[e], alpha * hq[e]));
}

}  // namespace

namespace gdr {
unsigned delta_take_status(cudaStream_t st) {
    unsigned v = 0, z = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_delta_status, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return 0x80000000u;
    cudaMemcpyToSymbolAsync(g_delta_status, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    if (cudaStreamSynchronize(st) != cudaSuccess) return 0x80000000u;
    return v;
}
}  // namespace gdr

extern "C" {

int gdr_delta_step(const gdr_delta_step_args *a, void *stream) {
    if (!a) return layer_fail(GDR_ERR_ARG, "args is null");
    int rc;
    if (a->rows < 0 || a->rows > 65535) return layer_fail(GDR_ERR_SHAPE, "delta step: 0 to 65535 rows (got %lld)", a->rows);
    if (a->Hq < 1 || a->Hv < 1 || a->Hv % a->Hq || a->Hv > 65535)
        return layer_fail(GDR_ERR_SHAPE, "delta step: Hq must be >= 1 and Hv a multiple of it, at most 65535 (got %lld, %lld)", a->Hq, a->Hv);
    if (a->K != 64 && a->K != 128 && a->K != 192) return layer_fail(GDR_ERR_SHAPE, "delta step: K must be 64, 128 or 192 (got %d)", a->K);
    if (a->V != 64 && a->V != 128 && a->V != 192 && a->V != 256)
        return layer_fail(GDR_ERR_SHAPE, "delta step: V must be 64, 128, 192 or 256 (got %d)", a->V);
    if (a->dtype != GDR_BF16 && a->dtype != GDR_F32) return layer_fail(GDR_ERR_DTYPE, "delta step: unknown dtype %d", a->dtype);
    if (a->n_slots < 0 || (!a->slots && a->n_slots < a->rows))
        return layer_fail(GDR_ERR_SHAPE, "delta step: %lld state slots for %lld rows", a->n_slots, a->rows);
    const unsigned e = a->dtype == GDR_BF16 ? 2 : 4;
    const bool any = a->rows > 0;
    if ((rc = layer_ptr("q", a->q, any, e)) || (rc = layer_ptr("k", a->k, any, e)) || (rc = layer_ptr("v", a->v, any, e)) ||
        (rc = layer_ptr("g", a->g, any, 4)) || (rc = layer_ptr("beta", a->beta, any, 4)) ||
        (rc = layer_ptr("state", a->state, any && a->n_slots > 0, 16)) || (rc = layer_ptr("slots", a->slots, false, 4)) ||
        (rc = layer_ptr("o", a->o, any, e)))
        return rc;
    if (!any) return GDR_OK;
    const DeltaP p{a->q, a->k, a->v, a->g, a->beta, a->state, a->slots, a->o, a->q_row, a->k_row, a->v_row, a->n_slots,
                   (int)a->Hv, a->V, (int)(a->Hv / a->Hq), a->scale};
    const dim3 grid((unsigned)(a->V / kCols), (unsigned)a->Hv, (unsigned)a->rows);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto run = [&](auto t) {
        using T = decltype(t);
        if (a->K == 64) k_delta_step<T, 64><<<grid, kThreads, 0, st>>>(p);
        else if (a->K == 128) k_delta_step<T, 128><<<grid, kThreads, 0, st>>>(p);
        else k_delta_step<T, 192><<<grid, kThreads, 0, st>>>(p);
    };
    if (a->dtype == GDR_BF16) run(bf16_t{}); else run(float{});
    return layer_launched("delta step");
}

}  // extern "C"
