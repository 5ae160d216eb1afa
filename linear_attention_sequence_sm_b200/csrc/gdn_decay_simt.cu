// gdn_decay_simt.cu -- the decayed linear attention's pass on CUDA cores:
// fp32 or bf16 storage, any head sizes up to 128, all arithmetic in fp32
// (differences of prefix sums in 64 bits).
//
// One block of 256 threads walks a segment for one value head, 64 tokens at a
// time, with the state (dz x dy) in shared memory.  Per chunk: P = decay mask
// . (x y^T) as 4 x 4 register tiles, out = P z + decay . (x Sigma^T) as 4 x 8
// tiles, Sigma = e^G Sigma + z^T (w y) as 8 x 8 tiles.  Shared-memory reads
// are 16 bytes; rows are padded by 4 floats so that a quarter-warp's rows fall
// into different banks.
//
// What bounds it is the chain of phases inside a chunk (loads, P, out, Sigma,
// with barriers between them), which two blocks an SM overlap only in part:
// 5003 ragged tokens of 8 heads, 64 x 96, take 154 us -- 95 for the pass, 36
// for the sweep at the cuts, the rest for the join, the schedule and the
// launches -- where the multiply-adds (1.4 M a chunk, 11,300 cycles of an SM's
// fp32 lanes) would take 35.  Tiles sized by the heads instead of 128 wide, two
// blocks an SM: 336 -> 246 us; paired arithmetic and loads in batches: 246 ->
// 158 us.
#include <algorithm>

#include "gdn_decay.cuh"
#include "gdn_f32x2.cuh"

namespace gdn {

namespace {

constexpr int C = kDecayChunk;
constexpr int kThreads = 256;
constexpr int LP = 68;    // row pitch of the 64 x 64 mask tile (floats)

__host__ __device__ constexpr int padded(int d) { return (d + 7) & ~7; }
__host__ __device__ constexpr int pitch(int d) { return padded(d) + 4; }  // of a tile of d columns

// Token vectors, then the tiles x, y, z (64 rows), S (dz x dy) and P, sized by
// the head sizes: up to 64 x 96 two blocks fit on an SM.
struct SimtVec {
    double G[C];
    float w_in[C], w_st[C];
    float red[kThreads / 32];
    float gamma;
    float pad[3];
};
static_assert(sizeof(SimtVec) % 16 == 0, "tiles are 16-byte aligned");
constexpr size_t simt_smem(int dy, int dz, bool state_only) {
    const size_t tiles = size_t(state_only ? 1 : 2) * C * pitch(dy) + size_t(C) * pitch(dz) + size_t(padded(dz)) * pitch(dy);
    return sizeof(SimtVec) + 4 * (tiles + (state_only ? 0 : C * LP));
}
// The most that any call asks for.  A kernel's limit is one value for all host
// threads: set to a call's own size, another thread could lower it before this
// call's launch, which would then be refused.
constexpr size_t kSimtMaxSmem = simt_smem(128, 128, false);
static_assert(kSimtMaxSmem <= 232448, "shared memory over the sm_100 per-block limit");

// rows [0, L) of a [tokens, heads, d] tensor's head into a tile, the rest of
// the 64 rows and of the columns up to a multiple of 8 zero
// (read four at a time before any is stored: one trip's latency, not four)
template <typename T>
__device__ __forceinline__ void load_tile(float *__restrict__ dst, int ld, const T *__restrict__ src, size_t stride,
                                          int d, int L, int dpad) {
    constexpr int kBatch = 4;
    if (d % 4 == 0) {
        const int n4 = dpad / 4, total = C * n4;
        for (int e0 = threadIdx.x; e0 < total; e0 += kBatch * kThreads) {
            float4 v[kBatch];
            int at[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int e = e0 + b * kThreads, r = e / n4, c = 4 * (e - r * n4);
                v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                at[b] = e < total ? r * ld + c : -1;
                if (e < total && r < L && c < d) {
                    if constexpr (sizeof(T) == 4) {
                        v[b] = *reinterpret_cast<const float4 *>(src + r * stride + c);
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2 *>(src + r * stride + c);
                        v[b] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (at[b] >= 0) *reinterpret_cast<float4 *>(dst + at[b]) = v[b];
        }
    } else {
        const int total = C * dpad;
        for (int e0 = threadIdx.x; e0 < total; e0 += kBatch * kThreads) {
            float v[kBatch];
            int at[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int e = e0 + b * kThreads, r = e / dpad, c = e - r * dpad;
                at[b] = e < total ? r * ld + c : -1;
                v[b] = (e < total && r < L && c < d) ? to_f32(src[r * stride + c]) : 0.f;
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (at[b] >= 0) dst[at[b]] = v[b];
        }
    }
}

// Prefix sums of a chunk's floored log-decays (warp 0), and the weights.
__device__ void load_gates(SimtVec &sm, const float *g, size_t g_stride, int L, bool reverse) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const float g0 = 2 * lane < L ? floored(g[(2 * lane) * g_stride]) : 0.f;
        const float g1 = 2 * lane + 1 < L ? floored(g[(2 * lane + 1) * g_stride]) : 0.f;
        double s = double(g0) + double(g1);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const double a = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += a;
        }
        const double last = __shfl_sync(0xffffffffu, s, 31);
        const double G0 = s - double(g1), G1 = s;
        sm.G[2 * lane] = G0;
        sm.G[2 * lane + 1] = G1;
        const float a0 = expf(float(G0)), a1 = expf(float(G1));
        const float b0 = expf(float(last - G0)), b1 = expf(float(last - G1));
        sm.w_in[2 * lane] = reverse ? b0 : a0;
        sm.w_in[2 * lane + 1] = reverse ? b1 : a1;
        sm.w_st[2 * lane] = reverse ? a0 : b0;
        sm.w_st[2 * lane + 1] = reverse ? a1 : b1;
        if (lane == 0) sm.gamma = expf(float(last));
    }
}

// Four floats as two pairs, and their product sums kept as a pair (even and
// odd terms), added at the end.
__device__ __forceinline__ ulonglong2 ld4(const float *p) { return *reinterpret_cast<const ulonglong2 *>(p); }
__device__ __forceinline__ f32x2 dot4(const ulonglong2 &a, const ulonglong2 &b, f32x2 c) {
    return fma2(a.x, b.x, fma2(a.y, b.y, c));
}
__device__ __forceinline__ float sum_of(f32x2 x) { return lo_of(x) + hi_of(x); }

// 4 x 4 tile of a 64 x 64 product of rows: acc[i][j] = a[r0 + 16 i] . b[c0 + 16 j]
__device__ __forceinline__ void gram(float (&out)[4][4], const float *a, const float *b, int ld, int r0, int c0, int d) {
    f32x2 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = both(0.f);
    for (int k = 0; k < d; k += 4) {
        ulonglong2 u[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = ld4(a + (r0 + 16 * i) * ld + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = ld4(b + (c0 + 16 * j) * ld + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = dot4(u[i], v[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) out[i][j] = sum_of(acc[i][j]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
decay_pass_simt_kernel(const __grid_constant__ DecayPass a0, const __grid_constant__ DecayPass a1) {
    const DecayPass &a = blockIdx.y ? a1 : a0;  // two passes that do not wait for one another share a launch
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SimtVec &sm = *reinterpret_cast<SimtVec *>(smem_raw);
    const DecayHeader *hdr = a.sched.hdr;
    if (hdr->status != GDN_OK) return;
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
    const int dy = a.dy, dz = a.dz, hv = a.hv;
    const int dyp = padded(dy), dzp = padded(dz), ly = pitch(dy), lz = pitch(dz);
    float *ty = reinterpret_cast<float *>(smem_raw + sizeof(SimtVec)), *tz = ty + C * ly, *tS = tz + C * lz;
    float *tx = tS + dzp * ly, *tp = tx + C * ly;
    const int64_t units = int64_t(hdr->num_segs) * hv;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const DecaySeg seg = a.sched.segs[u / hv];
        const int h = int(u % hv);
        const bool first = a.reverse ? seg.pos + seg.len == seg.seq_len : seg.pos == 0;
        const bool last = a.reverse ? seg.pos == 0 : seg.pos + seg.len == seg.seq_len;
        if (a.state_only && (seg.slot < 0 || last)) continue;
        const T *x = static_cast<const T *>(a.x) + (size_t(seg.start) * a.hx + h / (hv / a.hx)) * dy;
        const T *y = static_cast<const T *>(a.y) + (size_t(seg.start) * a.hy + h / (hv / a.hy)) * dy;
        const T *z = static_cast<const T *>(a.z) + (size_t(seg.start) * a.hz + h / (hv / a.hz)) * dz;
        const T *aux = a.aux ? static_cast<const T *>(a.aux) + (size_t(seg.start) * a.haux + h / (hv / a.haux)) * dz
                             : nullptr;
        const float *g = a.g_const ? a.g + h : a.g + size_t(seg.start) * hv + h;
        const size_t gs = a.g_const ? 0 : hv;
        // start state
        const bool own = seg.slot >= 0 && !a.state_only;
        const float *src = own ? a.seg_state + (size_t(seg.slot) * hv + h) * 16384
                               : (a.s_in && first && !a.state_only) ? a.s_in + (size_t(seg.seq) * hv + h) * dz * dy : nullptr;
        __syncthreads();
        for (int e0 = tid; e0 < dzp * dyp; e0 += 8 * kThreads) {
            float v[8];
            int at[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const int e = e0 + b * kThreads, r = e / dyp, c = e - r * dyp;
                at[b] = e < dzp * dyp ? r * ly + c : -1;
                v[b] = 0.f;
                if (src && at[b] >= 0 && r < dz && c < dy)
                    v[b] = own ? src[a.seg_trans ? c * 128 + r : r * 128 + c] : src[a.s_trans ? c * dz + r : r * dy + c];
            }
#pragma unroll
            for (int b = 0; b < 8; ++b)
                if (at[b] >= 0) tS[at[b]] = v[b];
        }
        const int nch = (seg.len + C - 1) / C;
        float seg_sum = 0.f;
        for (int i = 0; i < nch; ++i) {
            const int n = a.reverse ? nch - 1 - i : i;
            const int t0 = n * C, L = min(C, seg.len - t0);
            __syncthreads();
            load_tile(ty, ly, y + size_t(t0) * a.hy * dy, size_t(a.hy) * dy, dy, L, dyp);
            load_tile(tz, lz, z + size_t(t0) * a.hz * dz, size_t(a.hz) * dz, dz, L, dzp);
            if (!a.state_only) load_tile(tx, ly, x + size_t(t0) * a.hx * dy, size_t(a.hx) * dy, dy, L, dyp);
            load_gates(sm, g + size_t(t0) * gs, gs, L, a.reverse);
            __syncthreads();
            seg_sum += float(sm.G[C - 1]);
            if (a.starts) {
                const bool start = seg.pos + t0 == 0;
                float *at = a.starts + (size_t((seg.start + t0) / C) * hv + h) * dz * dy;
                if (!a.span) {
                    if (!start)
                        for (int q = tid; q < dz * dy; q += kThreads) at[q] = tS[(q / dy) * ly + q % dy];
                } else {
                    // <Sigma at the chunk's end, the state at its start>
                    const float *cp = !start ? at : a.s_first ? a.s_first + (size_t(seg.seq) * hv + h) * dz * dy : nullptr;
                    float s = 0.f;
                    if (cp) {
                        const bool tr = start && a.s_trans;
                        for (int q0 = tid; q0 < dz * dy; q0 += 8 * kThreads) {
                            float v[8];
#pragma unroll
                            for (int b = 0; b < 8; ++b) v[b] = q0 + b * kThreads < dz * dy ? cp[q0 + b * kThreads] : 0.f;
#pragma unroll
                            for (int b = 0; b < 8; ++b) {
                                const int q = q0 + b * kThreads;
                                if (q < dz * dy) s = fmaf(v[b], tS[(tr ? q % dz : q / dy) * ly + (tr ? q / dz : q % dy)], s);
                            }
                        }
                    }
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                    if ((tid & 31) == 0) sm.red[tid >> 5] = s;
                }
            }
            if (!a.state_only) {
                {
                    float acc[4][4];
                    gram(acc, tx, ty, ly, rg, cg, dyp);
#pragma unroll
                    for (int p = 0; p < 4; ++p)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int r = rg + 16 * p, c = cg + 16 * q;
                            const bool in = a.reverse ? c >= r : c <= r;
                            const double d = a.reverse ? sm.G[c] - sm.G[r] : sm.G[r] - sm.G[c];
                            tp[r * LP + c] = in ? acc[p][q] * expf(float(d)) : 0.f;
                        }
                }
                __syncthreads();
                if (a.span && tid < 8)
                    a.span[(size_t(seg.chunk + (seg.pos + t0) / C) * hv + h) * 8 + tid] = sm.gamma * sm.red[tid];
                // out rows 4 rg .. 4 rg + 3, columns cg + 16 q (the rows of Sigma a quarter-warp reads are then
                // next to one another and fall into different banks)
                float in[4][8], ex[4][8];
                {
                    f32x2 acc[4][8];
#pragma unroll
                    for (int p = 0; p < 4; ++p)
#pragma unroll
                        for (int q = 0; q < 8; ++q) acc[p][q] = both(0.f);
                    // Only pairs inside the mask are multiplied: a zero of P times an infinity or a NaN further on (back in
                    // time, backward) would be NaN.  Tokens 4 rg .. are this thread's rows: whole groups of four before
                    // (behind) them, and a triangle of their own.
                    for (int c = a.reverse ? 4 * rg + 4 : 0; c < (a.reverse ? C : 4 * rg); c += 4) {
                        ulonglong2 pr[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) pr[p] = ld4(tp + (4 * rg + p) * LP + c);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (16 * q >= dzp) break;
                            const float *zc = tz + c * lz + cg + 16 * q;  // (past dz: the row's padding, not used)
                            const ulonglong2 zv = make_ulonglong2(pair(zc[0], zc[lz]), pair(zc[2 * lz], zc[3 * lz]));
#pragma unroll
                            for (int p = 0; p < 4; ++p) acc[p][q] = dot4(pr[p], zv, acc[p][q]);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        if (16 * q >= dzp) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float zj = tz[(4 * rg + j) * lz + cg + 16 * q];
#pragma unroll
                            for (int p = 0; p < 4; ++p)
                                if (a.reverse ? j >= p : j <= p)
                                    acc[p][q] = fma2(pair(tp[(4 * rg + p) * LP + 4 * rg + j], 0.f), pair(zj, 0.f), acc[p][q]);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p)
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            in[p][q] = sum_of(acc[p][q]);
                            acc[p][q] = both(0.f);
                        }
                    for (int k = 0; k < dyp; k += 4) {
                        ulonglong2 xr[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) xr[p] = ld4(tx + (4 * rg + p) * ly + k);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (16 * q >= dzp) break;
                            const ulonglong2 s = ld4(tS + min(cg + 16 * q, dzp - 1) * ly + k);
#pragma unroll
                            for (int p = 0; p < 4; ++p) acc[p][q] = dot4(xr[p], s, acc[p][q]);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p)
#pragma unroll
                        for (int q = 0; q < 8; ++q) ex[p][q] = sum_of(acc[p][q]);
                }
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int r = 4 * rg + p;
                    const float w = sm.w_in[r];
                    const size_t row = size_t(seg.start + t0 + r);
                    float dot = 0.f, av[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int c = cg + 16 * q;
                        av[q] = aux && r < L && c < dz ? to_f32(aux[(size_t(t0) + r) * a.haux * dz + c]) : 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int c = cg + 16 * q;
                        const float e = w * ex[p][q];
                        if (r < L && c < dz) {
                            const size_t at = (row * hv + h) * dz + c;
                            if (a.out_f32) static_cast<float *>(a.out)[at] = in[p][q] + e;
                            else static_cast<T *>(a.out)[at] = from_f32<T>(in[p][q] + e);
                            dot = fmaf(av[q], e, dot);
                        }
                    }
                    if (aux) {
#pragma unroll
                        for (int m = 8; m > 0; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
                        if (cg == 0 && r < L) a.dot[size_t(h) * a.tokens + row] = dot;
                    }
                }
                __syncthreads();
            }
            // Sigma = gamma Sigma + z^T (w y): z rows 4 rg (and 64 +), y columns 4 cg (and 64 +)
            for (int zb = 4 * rg; zb < dzp; zb += 64)
                for (int yb = 4 * cg; yb < dyp; yb += 64) {
                    f32x2 acc[4][2];
                    const f32x2 gamma = both(sm.gamma);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const ulonglong2 s = ld4(tS + (zb + p) * ly + yb);
                        acc[p][0] = mul2(gamma, s.x);
                        acc[p][1] = mul2(gamma, s.y);
                    }
#pragma unroll 2
                    for (int c = 0; c < L; ++c) {
                        const f32x2 w = both(sm.w_st[c]);
                        const ulonglong2 zv = ld4(tz + c * lz + zb), yv = ld4(ty + c * ly + yb);
                        const f32x2 z01 = mul2(w, zv.x), z23 = mul2(w, zv.y);
                        const f32x2 zw[4] = {both(lo_of(z01)), both(hi_of(z01)), both(lo_of(z23)), both(hi_of(z23))};
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            acc[p][0] = fma2(zw[p], yv.x, acc[p][0]);
                            acc[p][1] = fma2(zw[p], yv.y, acc[p][1]);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        *reinterpret_cast<ulonglong2 *>(tS + (zb + p) * ly + yb) = make_ulonglong2(acc[p][0], acc[p][1]);
                }
        }
        __syncthreads();
        if (a.state_only) {
            float *dst = a.seg_local + (size_t(seg.slot) * hv + h) * 16384;
            for (int e = tid; e < dz * dy; e += kThreads) dst[(e / dy) * 128 + e % dy] = tS[(e / dy) * ly + e % dy];
            if (tid == 0) a.seg_dec[size_t(seg.slot) * hv + h] = expf(seg_sum);
            continue;
        }
        if (last && a.s_out) {
            float *dst = a.s_out + (size_t(seg.seq) * hv + h) * dz * dy;
            for (int e = tid; e < dz * dy; e += kThreads) {
                const int r = a.s_trans ? e % dz : e / dy, c = a.s_trans ? e / dz : e % dy;
                dst[e] = tS[r * ly + c];
            }
        }
    }
}

// The pairs inside one chunk: intra_t = sum of W_ij over j < t <= i,
// W_ij = e^{G_i - G_j} (q_i . k_j) (do_i . v_j).  Row i's running sums over j
// give X_i,t = sum_{j < t} W_ij; column t then sums X_i,t over i >= t.
constexpr int LD = 132;  // row pitch of 128-wide tiles
struct IntraSmem {
    float q[C * LD], k[C * LD], v[C * LD], o[C * LD];
    float w[C * LP];
    float part[4 * C];
    double G[C];
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
decay_intra_simt_kernel(const DecaySched sc, int num_seqs, int hk, int hv, int dk, int dv, int tokens, int batched_len,
                        const int32_t *__restrict__ cu, const T *__restrict__ q, const T *__restrict__ k,
                        const T *__restrict__ v, const T *__restrict__ d_o, const float *__restrict__ g, int g_const,
                        float *__restrict__ intra) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    IntraSmem &sm = *reinterpret_cast<IntraSmem *>(smem_raw);
    if (sc.hdr->status != GDN_OK) return;
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
    const int dkp = (dk + 7) & ~7, dvp = (dv + 7) & ~7;
    const int64_t units = int64_t(sc.hdr->total_chunks) * hv;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int gc = int(u / hv), h = int(u % hv), hq = h / (hv / hk);
        const int n = chunk_sequence(sc.chunk_base, num_seqs, gc);
        const int start = cu ? cu[n] : n * batched_len, len = cu ? cu[n + 1] - cu[n] : batched_len;
        const int t0 = (gc - sc.chunk_base[n]) * C, L = min(C, len - t0);
        const size_t tok = size_t(start) + t0;
        __syncthreads();
        load_tile(sm.q, LD, q + (tok * hk + hq) * dk, size_t(hk) * dk, dk, L, dkp);
        load_tile(sm.k, LD, k + (tok * hk + hq) * dk, size_t(hk) * dk, dk, L, dkp);
        load_tile(sm.v, LD, v + (tok * hv + h) * dv, size_t(hv) * dv, dv, L, dvp);
        load_tile(sm.o, LD, d_o + (tok * hv + h) * dv, size_t(hv) * dv, dv, L, dvp);
        if (tid < 32) {
            const float *gp = g_const ? g + h : g + tok * hv + h;
            const size_t gs = g_const ? 0 : hv;
            const float g0 = 2 * tid < L ? floored(gp[(2 * tid) * gs]) : 0.f;
            const float g1 = 2 * tid + 1 < L ? floored(gp[(2 * tid + 1) * gs]) : 0.f;
            double s = double(g0) + double(g1);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double e = __shfl_up_sync(0xffffffffu, s, d);
                if (tid >= d) s += e;
            }
            sm.G[2 * tid] = s - double(g1);
            sm.G[2 * tid + 1] = s;
        }
        __syncthreads();
        {
            float A[4][4], B[4][4];
            gram(A, sm.q, sm.k, LD, rg, cg, dkp);
            gram(B, sm.o, sm.v, LD, rg, cg, dvp);
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = rg + 16 * p, c = cg + 16 * e;
                    sm.w[r * LP + c] = c < r ? A[p][e] * B[p][e] * expf(float(sm.G[r] - sm.G[c])) : 0.f;
                }
        }
        __syncthreads();
        {
            // thread: row tid / 4, columns 16 (tid % 4) ..; exclusive running sums of the row
            const int r = tid >> 2, c0 = 16 * (tid & 3);
            float x[16], run = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[e] = run;
                run += sm.w[r * LP + c0 + e];
            }
            float before = 0.f;
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                const float o = __shfl_sync(0xffffffffu, run, (tid & 28) + m);
                if ((tid & 3) > m) before += o;
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; ++e) sm.w[r * LP + c0 + e] = x[e] + before;
        }
        __syncthreads();
        {
            const int t = tid & 63, quarter = tid >> 6;
            float s = 0.f;
            for (int r = max(16 * quarter, t); r < 16 * quarter + 16; ++r) s += sm.w[r * LP + t];
            sm.part[quarter * C + t] = s;
        }
        __syncthreads();
        if (tid < L)
            intra[size_t(h) * tokens + tok + tid] =
                (sm.part[tid] + sm.part[C + tid]) + (sm.part[2 * C + tid] + sm.part[3 * C + tid]);
    }
}

}  // namespace

cudaError_t launch_decay_pass_simt(const DecayPass &p, const DecayPass *also, int32_t dtype, int64_t max_units,
                                   cudaStream_t stream) {
    if (max_units <= 0) return cudaSuccess;
    const void *kern = dtype == GDN_DTYPE_BF16 ? reinterpret_cast<const void *>(decay_pass_simt_kernel<__nv_bfloat16>)
                                               : reinterpret_cast<const void *>(decay_pass_simt_kernel<float>);
    const size_t bytes = std::max(simt_smem(p.dy, p.dz, p.state_only),
                                  also ? simt_smem(also->dy, also->dz, also->state_only) : 0);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSimtMaxSmem));
    if (e != cudaSuccess) return e;
    const dim3 grid(unsigned(std::min<int64_t>(max_units, kDecayPlanSms * 8)), also ? 2 : 1);
    if (dtype == GDN_DTYPE_BF16) decay_pass_simt_kernel<__nv_bfloat16><<<grid, kThreads, bytes, stream>>>(p, also ? *also : p);
    else decay_pass_simt_kernel<float><<<grid, kThreads, bytes, stream>>>(p, also ? *also : p);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_decay_intra_simt(const gdn_shape_t &s, const int32_t *cu, const DecayLayout &L, const DecaySched &sc,
                                    const void *q, const void *k, const void *v, const void *d_o, const float *g,
                                    bool g_const, float *intra, cudaStream_t stream) {
    const int64_t units = L.max_chunks * s.num_v_heads;
    if (units <= 0) return cudaSuccess;
    const int tokens = s.batch * s.seq_len;
    const unsigned grid = unsigned(std::min<int64_t>(units, kDecayPlanSms * 8));
    cudaError_t e;
    if (s.dtype == GDN_DTYPE_BF16) {
        using bf = __nv_bfloat16;
        e = cudaFuncSetAttribute(decay_intra_simt_kernel<bf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(sizeof(IntraSmem)));
        if (e != cudaSuccess) return e;
        decay_intra_simt_kernel<bf><<<grid, kThreads, sizeof(IntraSmem), stream>>>(
            sc, s.num_seqs, s.num_qk_heads, s.num_v_heads, s.head_dim_k, s.head_dim_v, tokens, s.seq_len, cu,
            static_cast<const bf *>(q), static_cast<const bf *>(k), static_cast<const bf *>(v),
            static_cast<const bf *>(d_o), g, g_const, intra);
    } else {
        e = cudaFuncSetAttribute(decay_intra_simt_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(sizeof(IntraSmem)));
        if (e != cudaSuccess) return e;
        decay_intra_simt_kernel<float><<<grid, kThreads, sizeof(IntraSmem), stream>>>(
            sc, s.num_seqs, s.num_qk_heads, s.num_v_heads, s.head_dim_k, s.head_dim_v, tokens, s.seq_len, cu,
            static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(v),
            static_cast<const float *>(d_o), g, g_const, intra);
    }
    count_launch();
    return cudaGetLastError();
}

}  // namespace gdn
