// gdn_decay_intra.cu -- the decays' gradient from the pairs inside a chunk,
// bf16 inputs with head sizes a multiple of 8 (gdn_decay_simt.cu has the form
// for every other shape):
//     intra_t = sum over j < t <= i of W_ij,
//     W_ij = e^{G_i - G_j} (q_i . k_j) (do_i . v_j).
// Every term is added, none taken off, so a gradient that is small because
// its decay is strong keeps its digits.
//
// A block of four warps takes (chunk of 64 tokens, q/k head): the 64 x 64
// products q k^T once, then do v^T for each value head of the group; warp w
// has rows i of 16 w .. 16 w + 15 and skips the tiles above the diagonal.  W
// is formed in the accumulators' registers; running sums along a row (two
// shuffles in a quad, then tile by tile) give X_it = sum_{j < t} W_ij, and the
// sum of X_it over rows i >= t is a halving exchange over the eight lanes of a
// column pair and a sum over warps.
//
// What bounds it is reading q, k, v and do once: two warp-level products
// (mma.sync) of 2 x 64 x 64 x 128 per value head are a tenth of the time that
// takes, so their accumulators may as well be where the scan wants them, in
// registers; the tensor-memory path would only add a round trip.  4 x 4096
// tokens, 16 q/k and 32 value heads, d = 128: 127 us for 405 MB, 0.49 of the
// copy bandwidth (a block for each value head, reading q and k again: 178 us;
// on CUDA cores 941 us); three blocks an SM wait for their tiles in turn.
#include <algorithm>

#include "gdn_decay.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
using namespace sm100;

namespace {

constexpr int C = kDecayChunk;
constexpr int kThreads = 128;
constexpr uint32_t kTile = C * 256;  // 64 rows of up to 128 bf16, 16-byte pieces swizzled by the row

struct IntraVec {
    float hi[2][C], lo[2][C];  // prefix sums of the log-decays in log2 units, as a sum of two floats (two heads)
    float part[4][C];
};
constexpr uint32_t kSmem = 4 * kTile + sizeof(IntraVec);

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {  // within 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Rows [0, L) of a head into a swizzled tile by 16-byte asynchronous copies;
// the other rows, and columns past d up to dpad, zero.
__device__ __forceinline__ void tile_in(uint32_t dst, const __nv_bfloat16 *src, size_t stride, int d, int dpad, int L) {
    const int pieces = dpad / 8, c = threadIdx.x & 15;
    if (c >= pieces) return;
#pragma unroll
    for (int r = threadIdx.x >> 4; r < C; r += kThreads / 16) {
        const bool in = r < L && 8 * c < d;
        const uint32_t at = dst + uint32_t(r) * 256 + (uint32_t(c ^ (r & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(src + (in ? r * stride + 8 * c : 0)),
                     "r"(in ? 16 : 0)
                     : "memory");
    }
}

// acc[n] = rows 16 warp .. + 15 of a times rows 8 n .. 8 n + 7 of b, n < tiles (even)
__device__ __forceinline__ void gram(float (&acc)[8][4], uint32_t a, uint32_t b, int dpad, int warp, int lane, int tiles) {
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    const uint32_t ra = uint32_t(16 * warp + (lane & 15));
    const uint32_t rb = uint32_t((lane & 7) + ((lane >> 4) << 3));
    for (int k = 0; k < dpad / 16; ++k) {
        uint32_t av[4];
        ldsm4(a + ra * 256 + ((uint32_t(2 * k + (lane >> 4)) ^ (ra & 7)) << 4), av);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            if (n >= tiles) break;
            uint32_t bv[4];
            ldsm4(b + (8 * n + rb) * 256 + ((uint32_t(2 * k + ((lane >> 3) & 1)) ^ (rb & 7)) << 4), bv);
            mma16816(acc[n], av, bv[0], bv[1]);
            mma16816(acc[n + 1], av, bv[2], bv[3]);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 3)
decay_intra_kernel(const DecaySched sc, int num_seqs, int hk, int hv, int dk, int dv, int tokens, int batched_len,
                   const int32_t *__restrict__ cu, const __nv_bfloat16 *__restrict__ q,
                   const __nv_bfloat16 *__restrict__ k, const __nv_bfloat16 *__restrict__ v,
                   const __nv_bfloat16 *__restrict__ d_o, const float *__restrict__ g, int g_const,
                   float *__restrict__ intra) {
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sb = smem_u32(smem);
    IntraVec &sm = *reinterpret_cast<IntraVec *>(smem + 4 * kTile);
    if (sc.hdr->status != GDN_OK) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = hv / hk, dkp = (dk + 15) & ~15, dvp = (dv + 15) & ~15;
    const int tiles = 2 * warp + 2;  // column tiles of 8 up to the diagonal
    const int64_t units = int64_t(sc.hdr->total_chunks) * hk;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int gc = int(u / hk), hq = int(u % hk);
        const int n = chunk_sequence(sc.chunk_base, num_seqs, gc);
        const int start = cu ? cu[n] : n * batched_len, len = cu ? cu[n + 1] - cu[n] : batched_len;
        const int t0 = (gc - sc.chunk_base[n]) * C, L = min(C, len - t0);
        const size_t tok = size_t(start) + t0;
        __syncthreads();  // the previous unit's tiles have been read
        // v and do of the j-th head of the group: tiles 2 and 3, then (q and k have been used) 0 and 1, in turn
        auto head_in = [&](int j) {
            const int h = hq * group + j;
            const uint32_t at = sb + ((j & 1) ? 0u : 2 * kTile);
            tile_in(at, v + (tok * hv + h) * dv, size_t(hv) * dv, dv, dvp, L);
            tile_in(at + kTile, d_o + (tok * hv + h) * dv, size_t(hv) * dv, dv, dvp, L);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (warp == 0) {
                const float *gp = g_const ? g + h : g + tok * hv + h;
                const size_t gs = g_const ? 0 : hv;
                const float g0 = 2 * lane < L ? floored(gp[(2 * lane) * gs]) : 0.f;
                const float g1 = 2 * lane + 1 < L ? floored(gp[(2 * lane + 1) * gs]) : 0.f;
                double s = double(g0) + double(g1);
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const double e = __shfl_up_sync(0xffffffffu, s, d);
                    if (lane >= d) s += e;
                }
                constexpr double kLog2e = 1.4426950408889634;
                const double G0 = (s - double(g1)) * kLog2e, G1 = s * kLog2e;
                const float h0 = float(G0), h1 = float(G1);
                *reinterpret_cast<float2 *>(sm.hi[j & 1] + 2 * lane) = make_float2(h0, h1);
                *reinterpret_cast<float2 *>(sm.lo[j & 1] + 2 * lane) = make_float2(float(G0 - h0), float(G1 - h1));
            }
        };
        tile_in(sb, q + (tok * hk + hq) * dk, size_t(hk) * dk, dk, dkp, L);
        tile_in(sb + kTile, k + (tok * hk + hq) * dk, size_t(hk) * dk, dk, dkp, L);
        head_in(0);
        float A[8][4];
        for (int j = 0; j < group; ++j) {
            const int h = hq * group + j;
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();  // this head's tiles are here, and the one before has been read
            if (j == 0) {
                gram(A, sb, sb + kTile, dkp, warp, lane, tiles);
                if (group > 1) __syncthreads();  // q and k have been read
            }
            if (j + 1 < group) head_in(j + 1);
            float W[8][4];
            const uint32_t at = sb + ((j & 1) ? 0u : 2 * kTile);
            gram(W, at + kTile, at, dvp, warp, lane, tiles);
            // rows of this thread: i = 16 warp + lane / 4 (and + 8); columns 8 n + 2 (lane % 4) (and the next)
            const int i0 = 16 * warp + (lane >> 2), c0 = 2 * (lane & 3);
            float X[16];  // column sums of this thread's rows
#pragma unroll
            for (int e = 0; e < 16; ++e) X[e] = 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = i0 + 8 * r;
                const float Ghi = sm.hi[j & 1][i], Glo = sm.lo[j & 1][i];
                float base = 0.f;
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    if (m >= tiles) break;
                    const float2 hi = *reinterpret_cast<const float2 *>(sm.hi[j & 1] + 8 * m + c0);
                    const float2 lo = *reinterpret_cast<const float2 *>(sm.lo[j & 1] + 8 * m + c0);
                    const int c = 8 * m + c0;
                    const float w0 = c < i ? W[m][2 * r] * A[m][2 * r] * ex2((Ghi - hi.x) + (Glo - lo.x)) : 0.f;
                    const float w1 = c + 1 < i ? W[m][2 * r + 1] * A[m][2 * r + 1] * ex2((Ghi - hi.y) + (Glo - lo.y)) : 0.f;
                    float s = w0 + w1;
                    const float a = __shfl_up_sync(0xffffffffu, s, 1, 4);
                    if ((lane & 3) >= 1) s += a;
                    const float b = __shfl_up_sync(0xffffffffu, s, 2, 4);
                    if ((lane & 3) >= 2) s += b;
                    float before = __shfl_up_sync(0xffffffffu, s, 1, 4);
                    if ((lane & 3) == 0) before = 0.f;
                    before += base;
                    if (c <= i) X[2 * m] += before;
                    if (c + 1 <= i) X[2 * m + 1] += before + w0;
                    base += __shfl_sync(0xffffffffu, s, 3, 4);
                }
            }
            // over the eight lanes of a column pair: halving exchanges leave two of the 16 columns
#pragma unroll
            for (int s = 8, bit = 16; s >= 2; s >>= 1, bit >>= 1) {
                const bool up = (lane & bit) != 0;
#pragma unroll
                for (int e = 0; e < s; ++e) {
                    const float send = up ? X[e] : X[e + s], keep = up ? X[e + s] : X[e];
                    X[e] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
                }
            }
            const int tile = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
            *reinterpret_cast<float2 *>(&sm.part[warp][8 * tile + c0]) = make_float2(X[0], X[1]);
            __syncthreads();
            if (tid < L)
                intra[size_t(h) * tokens + tok + tid] =
                    (sm.part[0][tid] + sm.part[1][tid]) + (sm.part[2][tid] + sm.part[3][tid]);
        }
    }
}

}  // namespace

cudaError_t launch_decay_intra(const gdn_shape_t &s, const int32_t *cu, const DecayLayout &L, const DecaySched &sc,
                               const void *q, const void *k, const void *v, const void *d_o, const float *g,
                               bool g_const, float *intra, cudaStream_t stream) {
    const int64_t units = L.max_chunks * s.num_qk_heads;
    if (units <= 0) return cudaSuccess;
    using bf = __nv_bfloat16;
    const cudaError_t e = cudaFuncSetAttribute(decay_intra_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
    if (e != cudaSuccess) return e;
    const unsigned grid = unsigned(std::min<int64_t>(units, kDecayPlanSms * 3));
    decay_intra_kernel<<<grid, kThreads, kSmem, stream>>>(
        sc, s.num_seqs, s.num_qk_heads, s.num_v_heads, s.head_dim_k, s.head_dim_v, s.batch * s.seq_len, s.seq_len, cu,
        static_cast<const bf *>(q), static_cast<const bf *>(k), static_cast<const bf *>(v), static_cast<const bf *>(d_o), g,
        g_const, intra);
    count_launch();
    return cudaGetLastError();
}

}  // namespace gdn
