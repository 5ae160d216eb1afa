// gdn_decay_decode.cu -- one token per sequence of the decayed linear
// attention, the state updated in place:
//     s_i <- a s_i + v_i k^T,   o_i = s_i . q        (rows s_i of S)
// One read and one write of S, which is all the work there is: at 256
// sequences x 32 heads x 128 x 128 the states are 1.07 GB of traffic beside
// 10 MB of everything else, so the bound is memory bandwidth.  A group of
// lanes holds a row as 16-byte pieces (32 lanes for d_k up to 128, 16 up to
// 64, 8 up to 32; two pieces a lane up to 256) and keeps eight rows' loads in
// flight; a row's dot product takes one shuffle tree, interleaved over the
// rows.  d_k not a multiple of 4 takes a scalar form of the same walk.  256
// sequences x 32 heads x 128 x 128: 168 us, 0.98 of the copy bandwidth; one
// sequence is the host's time for a call (11 us).
#include <algorithm>

#include "gdn_decay.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 8;  // rows in flight per lane group

__device__ __forceinline__ void vec4(const float *p, float (&o)[4]) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
}
__device__ __forceinline__ void vec4(const __nv_bfloat16 *p, float (&o)[4]) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    o[0] = __uint_as_float(x.x << 16); o[1] = __uint_as_float(x.x & 0xffff0000u);
    o[2] = __uint_as_float(x.y << 16); o[3] = __uint_as_float(x.y & 0xffff0000u);
}

// kLanes lanes a row, kV 16-byte pieces a lane.  Block (x: sequence and head,
// y: a share of the rows).
template <typename T, int kLanes, int kV>
__global__ void __launch_bounds__(kWarps * 32)
decay_decode_kernel(int hk, int hv, int dk, int dv, int rows_per_block, const T *__restrict__ q,
                    const T *__restrict__ k, const T *__restrict__ v, const float *__restrict__ g, int g_const,
                    float *__restrict__ state, T *__restrict__ o) {
    const int unit = blockIdx.x, n = unit / hv, h = unit % hv;
    const size_t hq = size_t(n) * hk + h / (hv / hk);
    const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    constexpr int kGroups = kWarps * 32 / kLanes;
    const int row0 = blockIdx.y * rows_per_block, row1 = min(dv, row0 + rows_per_block);
    float *S = state + size_t(unit) * dv * dk;
    const T *vr = v + size_t(unit) * dv;
    T *orow = o + size_t(unit) * dv;
    float kf[kV][4], qf[kV][4];
    bool in[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        const int c = 4 * (lane + e * kLanes);
        in[e] = c < dk;
        if (in[e]) {
            vec4(k + hq * dk + c, kf[e]);
            vec4(q + hq * dk + c, qf[e]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) kf[e][j] = qf[e][j] = 0.f;
        }
    }
    const float alpha = expf(floored(g[g_const ? h : unit]));
    for (int i0 = row0 + grp * kRows; i0 - grp * kRows < row1; i0 += kGroups * kRows) {
        float4 s[kRows][kV];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (i0 + r < row1 && in[e])
                    s[r][e] = __ldcs(reinterpret_cast<const float4 *>(S + size_t(i0 + r) * dk + 4 * (lane + e * kLanes)));
        float p[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            p[r] = 0.f;
            if (i0 + r >= row1) continue;
            const float vv = to_f32(vr[i0 + r]);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                if (!in[e]) continue;
                float4 x = s[r][e];
                x.x = fmaf(alpha, x.x, vv * kf[e][0]);
                x.y = fmaf(alpha, x.y, vv * kf[e][1]);
                x.z = fmaf(alpha, x.z, vv * kf[e][2]);
                x.w = fmaf(alpha, x.w, vv * kf[e][3]);
                __stcs(reinterpret_cast<float4 *>(S + size_t(i0 + r) * dk + 4 * (lane + e * kLanes)), x);
                p[r] += fmaf(x.x, qf[e][0], fmaf(x.y, qf[e][1], fmaf(x.z, qf[e][2], x.w * qf[e][3])));
            }
        }
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1)
#pragma unroll
            for (int r = 0; r < kRows; ++r) p[r] += __shfl_xor_sync(0xffffffffu, p[r], m);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (lane == r && i0 + r < row1) orow[i0 + r] = from_f32<T>(p[r]);
    }
}

// Any d_k up to 256, a warp per row, element by element.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
decay_decode_any_kernel(int hk, int hv, int dk, int dv, int rows_per_block, const T *__restrict__ q,
                        const T *__restrict__ k, const T *__restrict__ v, const float *__restrict__ g, int g_const,
                        float *__restrict__ state, T *__restrict__ o) {
    const int unit = blockIdx.x, n = unit / hv, h = unit % hv;
    const size_t hq = size_t(n) * hk + h / (hv / hk);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = blockIdx.y * rows_per_block, row1 = min(dv, row0 + rows_per_block);
    float kf[8], qf[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = lane + 32 * e;
        kf[e] = c < dk ? to_f32(k[hq * dk + c]) : 0.f;
        qf[e] = c < dk ? to_f32(q[hq * dk + c]) : 0.f;
    }
    const float alpha = expf(floored(g[g_const ? h : unit]));
    for (int i = row0 + warp; i < row1; i += kWarps) {
        float *S = state + (size_t(unit) * dv + i) * dk;
        const float vv = to_f32(v[size_t(unit) * dv + i]);
        float p = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = lane + 32 * e;
            if (c >= dk) continue;
            const float x = fmaf(alpha, S[c], vv * kf[e]);
            S[c] = x;
            p = fmaf(x, qf[e], p);
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) p += __shfl_xor_sync(0xffffffffu, p, m);
        if (lane == 0) o[size_t(unit) * dv + i] = from_f32<T>(p);
    }
}

template <typename T>
void launch_as(dim3 grid, int hk, int hv, int dk, int dv, int rows, const void *q_, const void *k_, const void *v_,
               const float *g, int g_const, float *state, void *o_, cudaStream_t stream) {
    const T *q = static_cast<const T *>(q_), *k = static_cast<const T *>(k_), *v = static_cast<const T *>(v_);
    T *o = static_cast<T *>(o_);
    const dim3 block(kWarps * 32);
    if (dk % 4 != 0)
        decay_decode_any_kernel<T><<<grid, block, 0, stream>>>(hk, hv, dk, dv, rows, q, k, v, g, g_const, state, o);
    else if (dk > 128)
        decay_decode_kernel<T, 32, 2><<<grid, block, 0, stream>>>(hk, hv, dk, dv, rows, q, k, v, g, g_const, state, o);
    else if (dk > 64)
        decay_decode_kernel<T, 32, 1><<<grid, block, 0, stream>>>(hk, hv, dk, dv, rows, q, k, v, g, g_const, state, o);
    else if (dk > 32)
        decay_decode_kernel<T, 16, 1><<<grid, block, 0, stream>>>(hk, hv, dk, dv, rows, q, k, v, g, g_const, state, o);
    else
        decay_decode_kernel<T, 8, 1><<<grid, block, 0, stream>>>(hk, hv, dk, dv, rows, q, k, v, g, g_const, state, o);
}

}  // namespace

cudaError_t launch_decay_decode(int32_t n, int32_t hk, int32_t hv, int32_t dk, int32_t dv, int32_t dtype,
                                const void *q, const void *k, const void *v, const float *g, bool g_const,
                                float *state, void *o, cudaStream_t stream) {
    const int64_t units = int64_t(n) * hv;
    if (units > INT32_MAX) return cudaErrorInvalidValue;
    // few (sequence, head) pairs: their rows go to several blocks, 32 rows each
    const bool few = units < 4 * kDecayPlanSms;
    const int rows = few ? 32 : dv;
    const dim3 grid(static_cast<unsigned>(units), unsigned((dv + rows - 1) / rows));
    if (dtype == GDN_DTYPE_BF16)
        launch_as<__nv_bfloat16>(grid, hk, hv, dk, dv, rows, q, k, v, g, g_const, state, o, stream);
    else
        launch_as<float>(grid, hk, hv, dk, dv, rows, q, k, v, g, g_const, state, o, stream);
    count_launch();
    return cudaGetLastError();
}

}  // namespace gdn
