// gdn_block_norm.cu -- the norms around a block, fused with its gate and the
// residual connection (gdn_block_norm_forward, gdn_block_norm_backward).
//
// Per row of `width` values, with mean-square norms (fp32 throughout):
//     n1 = x / sqrt(mean(x^2) + eps)                (x itself without POST_NORM)
//     b  = n1 * w1 * act(z)
//     h  = rho r + c s * b
//     n2 = h / sqrt(mean(h^2) + eps),   y = n2 * w2
// and, for upstream gradients dh and dy, with dn2 = dy * w2,
//     e   = dh + (dn2 - n2 mean(dn2 . n2)) / rms(h)         (h's whole gradient)
//     dr  = rho e,     db = c s e,     du = db act(z),   dz = db n1 w1 act'(z),
//     dn1 = du w1,     dx = (dn1 - n1 mean(dn1 . n1)) / rms(x),
//     dw2 = sum dy n2, ds = sum c e b, dw1 = sum du n1      (sums over rows)
//
// Each input row is read once; h and the norms are recomputed in the backward
// instead of kept.  The forward is bound by memory: 16,384 x 4096 rows in bf16
// with a gate and a residual take 116 us, 0.88 of the copy bandwidth.  The
// gradients of the same take 246 us, 0.67: a row is a chain of sums over the
// block and of what follows from them, and one block of 16 warps an SM leaves
// about half of the issue slots empty while it waits for them.
#include <algorithm>

#include "gdn_block_norm.cuh"
#include "gdn_f32x2.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
using namespace sm100;

namespace {

constexpr int kMaxThreads = 512;  // per block

__device__ __forceinline__ void load8w(const float *p, float (&v)[8]) {  // weights: cached
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// A thread's values of a row.  Aligned rows (16-byte multiples) are staged in
// shared memory, and group i holds columns 8 (i n + t) .. + 7 (n threads a
// row); other rows are read directly, columns (8 i + e) n + t.
template <typename T>
__device__ __forceinline__ void row_load(const T *row, int i, int t, int n, int width, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = (8 * i + e) * n + t;
        v[e] = c < width ? to_f32(row[c]) : 0.f;
    }
}
// Weights of the same columns; `none` where the pointer is NULL.
template <bool kVec>
__device__ __forceinline__ void weight_load(const float *w, float none, float add, int i, int t, int n, int width,
                                            float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = none;
    } else if constexpr (kVec) {
        const int c = 8 * (i * n + t);
        if (c < width) {
            load8w(w + c, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = (8 * i + e) * n + t;
            v[e] = c < width ? __ldg(w + c) : 0.f;
        }
    }
    if (add != 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += add;
    }
}
template <typename T>
__device__ __forceinline__ void row_store(T *row, int i, int t, int n, int width, const float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = (8 * i + e) * n + t;
        if (c < width) row[c] = from_f32<T>(v[e]);
    }
}

// Eight values of a staged row as four pairs.
template <typename T>
__device__ __forceinline__ void staged8(const unsigned char *at, f32x2 (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(at);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(at + 16);
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(at);
        v[0] = from_bf16x2(a.x); v[1] = from_bf16x2(a.y); v[2] = from_bf16x2(a.z); v[3] = from_bf16x2(a.w);
    }
}
// The same, zeros past the row's end.
template <typename T>
__device__ __forceinline__ void staged(const unsigned char *row, int c, int width, f32x2 (&v)[4]) {
    if (c >= width) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = both(0.f);
    } else {
        staged8<T>(row + sizeof(T) * c, v);
    }
}
template <typename T> __device__ __forceinline__ void store_pairs(T *p, const f32x2 (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(lo_of(v[0]), hi_of(v[0]), lo_of(v[1]), hi_of(v[1])));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(lo_of(v[2]), hi_of(v[2]), lo_of(v[3]), hi_of(v[3])));
    } else {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(to_bf16x2(v[0]), to_bf16x2(v[1]), to_bf16x2(v[2]), to_bf16x2(v[3])));
    }
}

// The staged rows: a block takes the same number of consecutive rows at a time,
// and kStages groups of them are in flight.  A thread copies the bytes that it
// will read itself (a warp, where 32 bytes a thread are copied as two runs of
// 16 bytes a lane), so it waits for its own copies only: no barrier of the block
// stands between a copy, its readers and the next copy, and there is no wait
// that could run out.  (Bulk copies by one thread, counted on mbarriers, were 2
// to 10 % slower forward, 2 % faster for the gradients of 4096 bf16 columns and
// 3 to 9 % for fp32 ones up to 2048, and a copy that did not arrive in time
// left its rows out without a word.)
constexpr int kMaxTensors = 5;  // x, gate, residual, d_y, d_h
struct Stages {
    const unsigned char *src[kMaxTensors];  // NULL: not wanted
    uint32_t row_bytes[kMaxTensors], off[kMaxTensors];  // a row's bytes; where its group starts in a stage
    uint32_t stage_bytes;
};
__device__ __forceinline__ void copy16(uint32_t dst, const unsigned char *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// kRows consecutive rows a thread.
template <typename T, typename R, int kStages, int kGroups, int kRows> struct Pipe {
    static constexpr bool kShared = sizeof(T) == 4 || sizeof(R) == 4;  // lanes copy for one another
    uint32_t buf, stage;
    int rows, stride, next;  // this thread's first row of the next group to fetch
    __device__ Pipe(const unsigned char *smem, int rows_)
        : buf(smem_u32(smem)), stage(0), rows(rows_), stride(int(gridDim.x * blockDim.y) * kRows),
          next((int(blockIdx.x * blockDim.y) + int(threadIdx.y)) * kRows) {}
    // the copies of this thread's next rows, into stage `st` (a group of copies, possibly of none)
    __device__ __forceinline__ void fetch(const Stages &s, uint32_t st, int width) {
        const uint32_t dst = buf + st * s.stage_bytes;
        if constexpr (kShared) __syncwarp();
#pragma unroll
        for (int i = 0; i < kMaxTensors; ++i) {
            if (!s.src[i]) continue;
            constexpr int kT = sizeof(T), kR = sizeof(R);
            const int size = i == 2 || i == 4 ? kR : kT;
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (next + k >= rows) continue;
                const unsigned char *row = s.src[i] + int64_t(next + k) * s.row_bytes[i];
                const uint32_t to = dst + s.off[i] + (threadIdx.y * kRows + k) * s.row_bytes[i];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int mine = 8 * (g * int(blockDim.x) + int(threadIdx.x));
                    if (size == 2) {
                        if (mine < width) copy16(to + 2 * mine, row + 2 * mine);
                    } else {
                        const int c = mine - 4 * int(threadIdx.x & 31);
                        if (c < width) copy16(to + 4 * c, row + 4 * c);
                        if (c + 128 < width) copy16(to + 4 * c + 512, row + 4 * c + 512);
                    }
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next = next > rows - stride ? rows : next + stride;
    }
    __device__ __forceinline__ void start(const Stages &s, int width) {
#pragma unroll
        for (uint32_t i = 0; i < kStages; ++i) fetch(s, i, width);
    }
    // all copies are here but those of the last kLeft fetches
    template <int kLeft> __device__ __forceinline__ void wait() const {
        asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
        if constexpr (kShared) __syncwarp();
    }
    __device__ __forceinline__ void advance() { stage = stage + 1 == kStages ? 0 : stage + 1; }
};

// Sums of kN values over the n threads of a row (n a multiple of 32, at most
// 32 kWarps; the block's rows reduce together).  `red` has kN * kWarps floats
// per row, aligned to 16 bytes and zero where a row has no warp (clear_red).
// Every thread adds the warps' sums itself: the reads are broadcasts, and the
// chain is shorter than a second tree of shuffles.
template <int kN, int kWarps>
__device__ __forceinline__ void row_sum(float (&v)[kN], float *red, int t, int n) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], m);
    if (n == 32) return;
    __syncthreads();  // the previous use of `red` has been read
    if ((t & 31) == 0)
#pragma unroll
        for (int j = 0; j < kN; ++j) red[kWarps * j + (t >> 5)] = v[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        f32x2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < kWarps; i += 4) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(red + kWarps * j + i);
            s = i == 0 ? add2(x.x, x.y) : add2(s, add2(x.x, x.y));
        }
        v[j] = lo_of(s) + hi_of(s);
    }
}
template <int kFloats>
__device__ __forceinline__ void clear_red(float (&red)[kFloats]) {
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < kFloats; i += blockDim.x * blockDim.y) red[i] = 0.f;
    __syncthreads();
}

// Sigmoid: the exact exponential for fp32 rows; for bf16 rows the fast one,
// about 1e-6 off relative to the result, far below their rounding.
template <typename T> __device__ __forceinline__ float gate_sigmoid(float z) {
    if constexpr (sizeof(T) == 4) return sigmoid(z);
    return sigmoid_fast(z);
}

// A thread's weights of eight columns of an aligned row: w1 and w2 as the norms
// use them, and branch_scale s (zeros past the row's end).
struct Weights {
    f32x2 w1[4], s[4], w2[4];
    __device__ __forceinline__ void load(const BlockNormArgs &a, int i, int t, int n, int width) {
        const bool post = a.flags & GDN_BLOCK_POST_NORM;
        const float zc = (a.flags & GDN_BLOCK_ZERO_CENTRED) ? 1.f : 0.f, none = 1.f - zc;
        float u[8], v[8], x[8];
        weight_load(post ? a.post_weight : nullptr, post ? none : 1.f, post ? zc : 0.f, i, t, n, width, u);
        weight_load(a.scale, 1.f, 0.f, i, t, n, width, v);
        weight_load(a.pre_weight, none, zc, i, t, n, width, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w1[e] = pair(u[2 * e], u[2 * e + 1]);
            s[e] = mul2(pair(v[2 * e], v[2 * e + 1]), both(a.branch_scale));
            w2[e] = pair(x[2 * e], x[2 * e + 1]);
        }
    }
    // the same for aligned columns 8 (i n + t) .. + 7
    static __device__ __forceinline__ void weight_load(const float *w, float none, float add, int i, int t, int n,
                                                       int width, float (&v)[8]) {
        gdn::weight_load<true>(w, none, add, i, t, n, width, v);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {  // (of infinity: 0)
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The gate of four pairs of pre-activations, and its derivative:
// act' = g + act (1 - g) for SiLU, g (1 - g) for the sigmoid (g the sigmoid).
template <typename T, bool kGrad>
__device__ __forceinline__ void gate(bool silu, f32x2 (&z)[4], f32x2 (&slope)[4]) {
    f32x2 g[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
            g[e] = pair(sigmoid(lo_of(z[e])), sigmoid(hi_of(z[e])));
        } else {
            // 1 / (1 + 2^(-z log2 e)) by the hardware's exponential and reciprocal
            const f32x2 x = mul2(z[e], both(-1.4426950408889634f));
            f32x2 d = add2(pair(ex2(lo_of(x)), ex2(hi_of(x))), both(1.f));
            g[e] = pair(rcp(lo_of(d)), rcp(hi_of(d)));
        }
    }
    if (silu) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            z[e] = mul2(z[e], g[e]);
            if (kGrad) slope[e] = fma2(z[e], fma2(g[e], both(-1.f), both(1.f)), g[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            z[e] = g[e];
            if (kGrad) slope[e] = mul2(g[e], fma2(g[e], both(-1.f), both(1.f)));
        }
    }
}

// Aligned rows.  A block walks the rows with a stride and keeps kFwdStages
// groups of them coming; a thread's weights stay in registers (up to 8192
// columns).  About 20 instructions a column against 10 bytes of memory
// traffic at bf16: both take about as long, so the fixed work of a row (two
// sums over the block) is spread over 16 columns a thread.
constexpr int kFwdStages = 3;
template <typename T, typename R, int kGroups, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 1)
block_norm_forward_kernel(const BlockNormArgs a, const Stages sg) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int kWarps = kThreads / 32;
    __shared__ __align__(16) float red_all[kWarps * 8];
    clear_red(red_all);
    constexpr bool kKeep = kGroups <= 2;
    const int n = blockDim.x, t = threadIdx.x, width = a.width;
    float *red = red_all + kWarps * threadIdx.y;
    Pipe<T, R, kFwdStages, kGroups, 1> pipe(smem, int(a.rows));
    const bool post = a.flags & GDN_BLOCK_POST_NORM, pre = a.flags & GDN_BLOCK_PRE_NORM;
    const bool silu = a.flags & GDN_BLOCK_GATE_SILU, gated = sg.src[1] != nullptr, res = sg.src[2] != nullptr;
    const float inv_width = 1.f / float(width);
    const int rows = int(a.rows), stride = int(gridDim.x * blockDim.y);
    pipe.start(sg, width);
    f32x2 w1s[kKeep ? kGroups : 1][4], w2[kKeep ? kGroups : 1][4];  // w1 branch_scale s, w2
    auto weights = [&](int i, f32x2 (&u)[4], f32x2 (&v)[4]) {
        Weights w;
        w.load(a, i, t, n, width);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[e] = mul2(w.w1[e], w.s[e]);
            v[e] = w.w2[e];
        }
    };
    if constexpr (kKeep)
#pragma unroll
        for (int i = 0; i < kGroups; ++i) weights(i, w1s[i], w2[i]);
    for (int first = int(blockIdx.x * blockDim.y), left = 1; left > 0; first += stride) {
        left = rows - first - stride;  // (rows < 2^31, and so is first: `left` > 0 while another group follows)
        const int row = first + int(threadIdx.y);
        const bool live = row < rows;
        pipe.template wait<kFwdStages - 1>();
        const unsigned char *st = smem + pipe.stage * sg.stage_bytes;
        auto at = [&](int i) { return st + sg.off[i] + threadIdx.y * sg.row_bytes[i]; };
        const int64_t base = int64_t(row) * width + 8 * t;
        const int lw = live ? width : 0;
        f32x2 xv[kGroups][4];
        float scale1 = 1.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) staged<T>(at(0), 8 * (i * n + t), lw, xv[i]);
        if (post) {
            f32x2 ss = both(0.f);
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) ss = fma2(xv[i][e], xv[i][e], ss);
            float s1[1] = {lo_of(ss) + hi_of(ss)};
            row_sum<1, kWarps>(s1, red, t, n);
            scale1 = rsqrtf(fmaf(s1[0], inv_width, a.eps));
        }
        f32x2 ss = both(0.f);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = 8 * (i * n + t);
            if constexpr (!kKeep) weights(i, w1s[0], w2[0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) xv[i][e] = mul2(mul2(xv[i][e], both(scale1)), w1s[kKeep ? i : 0][e]);
            if (gated) {
                f32x2 zv[4], none[4];
                staged<T>(at(1), c, lw, zv);
                gate<T, false>(silu, zv, none);
#pragma unroll
                for (int e = 0; e < 4; ++e) xv[i][e] = mul2(xv[i][e], zv[e]);
            }
            if (res) {
                f32x2 rv[4];
                staged<R>(at(2), c, lw, rv);
#pragma unroll
                for (int e = 0; e < 4; ++e) xv[i][e] = fma2(both(a.residual_scale), rv[e], xv[i][e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = fma2(xv[i][e], xv[i][e], ss);  // h
        }
        pipe.fetch(sg, pipe.stage, width);  // (the stage has been read)
        pipe.advance();
        if (live && a.h)
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (8 * (i * n + t) < width) store_pairs(static_cast<R *>(a.h) + base + 8 * i * n, xv[i]);
        if (!pre) continue;
        float s2[1] = {lo_of(ss) + hi_of(ss)};
        row_sum<1, kWarps>(s2, red, t, n);
        const float scale2 = rsqrtf(fmaf(s2[0], inv_width, a.eps));
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            if constexpr (!kKeep) weights(i, w1s[0], w2[0]);
            f32x2 yv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) yv[e] = mul2(mul2(xv[i][e], both(scale2)), w2[kKeep ? i : 0][e]);
            if (8 * (i * n + t) < width) store_pairs(static_cast<T *>(a.y) + base + 8 * i * n, yv);
        }
    }
}

// Rows of any alignment, read directly.
template <typename T, typename R, int kGroups>
__global__ void __launch_bounds__(kMaxThreads)
block_norm_forward_any_kernel(const BlockNormArgs a) {
    __shared__ __align__(16) float red_all[16 * 8];
    clear_red(red_all);
    const int n = blockDim.x, t = threadIdx.x, width = a.width;
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    float *red = red_all + 16 * threadIdx.y;
    const int64_t at = (live ? row : 0) * width;
    const T *x = static_cast<const T *>(a.x) + at, *z = a.gate ? static_cast<const T *>(a.gate) + at : nullptr;
    const R *r = a.residual ? static_cast<const R *>(a.residual) + at : nullptr;
    const float zc = (a.flags & GDN_BLOCK_ZERO_CENTRED) ? 1.f : 0.f;
    const float none = zc != 0.f ? 0.f : 1.f;
    float xv[kGroups][8], hv[kGroups][8];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) row_load(x, i, t, n, width, xv[i]);
    float scale1 = 1.f;
    const bool post = a.flags & GDN_BLOCK_POST_NORM;
    if (post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss[0] = fmaf(xv[i][e], xv[i][e], ss[0]);
        row_sum<1, 16>(ss, red, t, n);
        scale1 = 1.f / sqrtf(ss[0] / float(width) + a.eps);
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        float w1[8], s[8], zv[8], rv[8];
        weight_load<false>(post ? a.post_weight : nullptr, post ? none : 1.f, post ? zc : 0.f, i, t, n, width, w1);
        weight_load<false>(a.scale, 1.f, 0.f, i, t, n, width, s);
        if (z) row_load(z, i, t, n, width, zv);
        if (r) row_load(r, i, t, n, width, rv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float b = xv[i][e] * scale1 * w1[e];
            if (z) {
                const float sg = gate_sigmoid<T>(zv[e]);
                b *= (a.flags & GDN_BLOCK_GATE_SILU) ? zv[e] * sg : sg;
            }
            b *= a.branch_scale * s[e];
            hv[i][e] = r ? fmaf(a.residual_scale, rv[e], b) : b;
            ss[0] = fmaf(hv[i][e], hv[i][e], ss[0]);
        }
    }
    if (live && a.h)
#pragma unroll
        for (int i = 0; i < kGroups; ++i) row_store(static_cast<R *>(a.h) + at, i, t, n, width, hv[i]);
    if (!(a.flags & GDN_BLOCK_PRE_NORM)) return;
    row_sum<1, 16>(ss, red, t, n);
    const float scale2 = 1.f / sqrtf(ss[0] / float(width) + a.eps);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        float w2[8];
        weight_load<false>(a.pre_weight, none, zc, i, t, n, width, w2);
#pragma unroll
        for (int e = 0; e < 8; ++e) w2[e] *= hv[i][e] * scale2;
        row_store(static_cast<T *>(a.y) + at, i, t, n, width, w2);
    }
}

// Aligned rows: as the forward, with a thread's sums over rows in registers
// beside its weights (the sums go to the row group's own line of the workspace
// at the end).  Three sums a row: x^2; h^2 and dy w2 h together; dn1 . n1.
// 512 threads of 128 registers fill an SM at 4096 columns.
constexpr int kBwdStages = 2;
template <typename T, typename R, int kGroups>
__global__ void __launch_bounds__(512, 1)
block_norm_backward_kernel(const BlockNormArgs a, const Stages sg) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float red_all[32 * 8];
    clear_red(red_all);
    constexpr bool kKeep = kGroups == 1;
    const int n = blockDim.x, t = threadIdx.x, width = a.width;
    float *red = red_all + 32 * threadIdx.y;
    Pipe<T, R, kBwdStages, kGroups, 1> pipe(smem, int(a.rows));
    const bool post = a.flags & GDN_BLOCK_POST_NORM, pre = sg.src[3] != nullptr;
    const bool silu = a.flags & GDN_BLOCK_GATE_SILU, gated = sg.src[1] != nullptr, res = sg.src[2] != nullptr;
    const bool has_dh = sg.src[4] != nullptr;
    const float inv_width = 1.f / float(width);
    const int rows = int(a.rows), stride = int(gridDim.x * blockDim.y);
    pipe.start(sg, width);
    Weights w;
    if constexpr (kKeep) w.load(a, 0, t, n, width);
    f32x2 sw1[kGroups][4], sw2[kGroups][4], ssc[kGroups][4];
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sw1[i][e] = sw2[i][e] = ssc[i][e] = both(0.f);
    for (int first = int(blockIdx.x * blockDim.y), left = 1; left > 0; first += stride) {
        left = rows - first - stride;  // (rows < 2^31, and so is first: `left` > 0 while another group follows)
        const int row = first + int(threadIdx.y);
        const bool live = row < rows;
        pipe.template wait<kBwdStages - 1>();
        const unsigned char *st = smem + pipe.stage * sg.stage_bytes;
        auto at = [&](int i) { return st + sg.off[i] + threadIdx.y * sg.row_bytes[i]; };
        const int64_t base = int64_t(row) * width + 8 * t;
        const int lw = live ? width : 0;  // rows past the end read as zeros and add zeros
        f32x2 nv[kGroups][4];
        float scale1 = 1.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) staged<T>(at(0), 8 * (i * n + t), lw, nv[i]);
        if (post) {
            f32x2 ss = both(0.f);
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) ss = fma2(nv[i][e], nv[i][e], ss);
            float s1[1] = {lo_of(ss) + hi_of(ss)};
            row_sum<1, 16>(s1, red, t, n);
            scale1 = rsqrtf(fmaf(s1[0], inv_width, a.eps));
        }
        // n1, the gate and its derivative, h, and the sums of h^2 and dy w2 h
        f32x2 hv[kGroups][4], gv[kGroups][4], dv[kGroups][4], sh = both(0.f), sy = both(0.f);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = 8 * (i * n + t);
            if constexpr (!kKeep) w.load(a, i, t, n, width);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                nv[i][e] = mul2(nv[i][e], both(scale1));
                hv[i][e] = mul2(mul2(nv[i][e], w.w1[e]), w.s[e]);
            }
            if (gated) {
                staged<T>(at(1), c, lw, gv[i]);
                gate<T, true>(silu, gv[i], dv[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[i][e] = mul2(hv[i][e], gv[i][e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    gv[i][e] = both(1.f);
                    dv[i][e] = both(0.f);
                }
            }
            if (res) {
                f32x2 rv[4];
                staged<R>(at(2), c, lw, rv);
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[i][e] = fma2(both(a.residual_scale), rv[e], hv[i][e]);
            }
            if (pre) {
                f32x2 yv[4];
                staged<T>(at(3), c, lw, yv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sh = fma2(hv[i][e], hv[i][e], sh);
                    sy = fma2(mul2(yv[e], w.w2[e]), hv[i][e], sy);
                }
            }
        }
        float scale2 = 0.f, mean2 = 0.f;
        if (pre) {
            float s2[2] = {lo_of(sh) + hi_of(sh), lo_of(sy) + hi_of(sy)};
            row_sum<2, 16>(s2, red, t, n);
            scale2 = rsqrtf(fmaf(s2[0], inv_width, a.eps));
            mean2 = scale2 * s2[1] * inv_width;  // mean(dn2 . n2)
        }
        f32x2 sd = both(0.f);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = 8 * (i * n + t);
            const bool in = live && c < width;
            if constexpr (!kKeep) w.load(a, i, t, n, width);
            f32x2 ev[4];  // h's whole gradient
            if (has_dh) {
                staged<R>(at(4), c, lw, ev);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) ev[e] = both(0.f);
            }
            if (pre) {
                f32x2 yv[4];
                staged<T>(at(3), c, lw, yv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 n2 = mul2(hv[i][e], both(scale2));
                    sw2[i][e] = fma2(yv[e], n2, sw2[i][e]);
                    ev[e] = fma2(both(scale2), fma2(n2, both(-mean2), mul2(yv[e], w.w2[e])), ev[e]);
                }
            }
            if (in && a.d_residual) {
                f32x2 dr[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) dr[e] = mul2(both(a.residual_scale), ev[e]);
                store_pairs(static_cast<R *>(a.d_residual) + base + 8 * i * n, dr);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 n1 = nv[i][e], u = mul2(n1, w.w1[e]), db = mul2(ev[e], w.s[e]), du = mul2(db, gv[i][e]);
                ssc[i][e] = fma2(ev[e], mul2(u, gv[i][e]), ssc[i][e]);  // (branch_scale at the end)
                dv[i][e] = mul2(dv[i][e], mul2(db, u));                  // dz
                sw1[i][e] = fma2(du, n1, sw1[i][e]);
                hv[i][e] = mul2(du, w.w1[e]);                            // dn1 (dx without the norm)
                sd = fma2(hv[i][e], n1, sd);
            }
            if (in && a.d_gate) store_pairs(static_cast<T *>(a.d_gate) + base + 8 * i * n, dv[i]);
        }
        if (post) {
            float s3[1] = {lo_of(sd) + hi_of(sd)};
            row_sum<1, 16>(s3, red, t, n);
            const float mean1 = s3[0] * inv_width;
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    hv[i][e] = mul2(both(scale1), fma2(nv[i][e], both(-mean1), hv[i][e]));
        }
        if (live && a.dx)
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (8 * (i * n + t) < width) store_pairs(static_cast<T *>(a.dx) + base + 8 * i * n, hv[i]);
        pipe.fetch(sg, pipe.stage, width);  // (the stage has been read; here fewer values are held than where it was)
        pipe.advance();
    }
    float *out = a.partial + (int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * 3 * width + 8 * t;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        if (8 * (i * n + t) >= width) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) ssc[i][e] = mul2(ssc[i][e], both(a.branch_scale));
        if (a.d_post_weight) store_pairs(out + 8 * i * n, sw1[i]);
        if (a.d_scale) store_pairs(out + width + 8 * i * n, ssc[i]);
        if (a.d_pre_weight) store_pairs(out + 2 * width + 8 * i * n, sw2[i]);
    }
}

// The same for rows up to 4096 columns, two rows a thread at a time: what the
// form above waits for is a row's chain of three sums over the block, so here
// a sum carries both rows' terms, and x^2 of the next two rows is summed with
// dn1 . n1 of these (two sums for two rows, not six).  A row keeps its h and
// the gate's sigmoid in registers; x, z and dy are read again from the stage.
// kParts says at compile time which parts there are (with a residual and both
// upstream gradients; kAnyParts: looked up), which takes instructions off the
// chain.  16,384 x 4096 in bf16, each with bulk copies: 318 us in the form
// above, 345 us with two rows and parts looked up at every use, 297 us with
// one row and parts known, 242 us with both.
enum { kPartPost = 1, kPartGate = 2, kPartSilu = 4, kAnyParts = 8 };
template <typename T, typename R, int kParts>
__global__ void __launch_bounds__(512, 1)
block_norm_backward_pair_kernel(const BlockNormArgs a, const Stages sg) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float red_all[64 * 8], zeros[8];
    if (threadIdx.y == 0 && threadIdx.x < 8) zeros[threadIdx.x] = 0.f;
    clear_red(red_all);
    const int n = blockDim.x, t = threadIdx.x, width = a.width, c = 8 * t;
    float *red = red_all + 64 * threadIdx.y;
    Pipe<T, R, kBwdStages, 1, 2> pipe(smem, int(a.rows));
    const int per = 2 * blockDim.y;
    constexpr bool kAny = kParts == kAnyParts;
    const bool post = kAny ? bool(a.flags & GDN_BLOCK_POST_NORM) : bool(kParts & kPartPost);
    const bool gated = kAny ? sg.src[1] != nullptr : bool(kParts & kPartGate);
    const bool silu = kAny ? bool(a.flags & GDN_BLOCK_GATE_SILU) : bool(kParts & kPartSilu);
    const bool pre = !kAny || sg.src[3] != nullptr, res = !kAny || sg.src[2] != nullptr, has_dh = !kAny || sg.src[4] != nullptr;
    const float inv_width = 1.f / float(width);
    const int rows = int(a.rows), stride = int(gridDim.x) * per;
    pipe.start(sg, width);
    Weights w;
    w.load(a, 0, t, n, width);
    f32x2 sw1[4], sw2[4], ssc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sw1[e] = sw2[e] = ssc[e] = both(0.f);
    // of the group being read: whether its rows are there (past the end: read as zeros, add zeros)
    const int mine = 2 * int(threadIdx.y);
    // this thread's values of a row in a stage (of zeros, where it has none)
    auto at = [&](int i, int k, uint32_t stage, bool in) -> const unsigned char * {
        return in ? smem + stage * sg.stage_bytes + sg.off[i] + (mine + k) * sg.row_bytes[i] +
                        t * 8 * (i == 2 || i == 4 ? int(sizeof(R)) : int(sizeof(T)))
                  : reinterpret_cast<const unsigned char *>(zeros);
    };
    auto squares = [&](int k, bool in) {  // this thread's part of a row's x^2
        f32x2 x[4], ss = both(0.f);
        staged8<T>(at(0, k, pipe.stage, in), x);
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fma2(x[e], x[e], ss);
        return lo_of(ss) + hi_of(ss);
    };
    int first = int(blockIdx.x) * per;
    bool live[2];
    auto arrive = [&](bool more) {  // the group at `first`, if there is one
        live[0] = more && first + mine < rows && c < width;
        live[1] = live[0] && first + mine + 1 < rows;
    };
    pipe.template wait<kBwdStages - 1>();
    arrive(first < rows);
    float s3[4] = {0.f, 0.f, 0.f, 0.f};  // dn1 . n1 of two rows, x^2 of the next two
    if (post) {
        float s[2] = {squares(0, live[0]), squares(1, live[1])};
        row_sum<2, 16>(s, red, t, n);
        s3[2] = s[0];
        s3[3] = s[1];
    }
    for (bool more = first < rows; more;) {
        float scale1[2];
        f32x2 hv[2][4], gv[2][4];  // h (then dn1), the gate's sigmoid
        float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            scale1[k] = post ? rsqrtf(fmaf(s3[2 + k], inv_width, a.eps)) : 1.f;
            staged8<T>(at(0, k, pipe.stage, live[k]), hv[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[k][e] = mul2(mul2(mul2(hv[k][e], both(scale1[k])), w.w1[e]), w.s[e]);
            if (gated) {
                f32x2 zv[4];
                staged8<T>(at(1, k, pipe.stage, live[k]), zv);
#pragma unroll
                for (int e = 0; e < 4; ++e) gv[k][e] = zv[e];
                f32x2 none[4];
                gate<T, false>(false, gv[k], none);
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[k][e] = mul2(hv[k][e], silu ? mul2(zv[e], gv[k][e]) : gv[k][e]);
            }
            if (res) {
                f32x2 rv[4];
                staged8<R>(at(2, k, pipe.stage, live[k]), rv);
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[k][e] = fma2(both(a.residual_scale), rv[e], hv[k][e]);
            }
            if (pre) {
                f32x2 yv[4], sh = both(0.f), sy = both(0.f);
                staged8<T>(at(3, k, pipe.stage, live[k]), yv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sh = fma2(hv[k][e], hv[k][e], sh);
                    sy = fma2(mul2(yv[e], w.w2[e]), hv[k][e], sy);
                }
                s2[2 * k] = lo_of(sh) + hi_of(sh);
                s2[2 * k + 1] = lo_of(sy) + hi_of(sy);
            }
        }
        if (pre) row_sum<4, 16>(s2, red, t, n);
        const int64_t base = int64_t(first + mine) * width + c;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool in = live[k];
            f32x2 ev[4], sd = both(0.f);  // h's whole gradient
            if (has_dh) {
                staged8<R>(at(4, k, pipe.stage, live[k]), ev);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) ev[e] = both(0.f);
            }
            if (pre) {
                const float scale2 = rsqrtf(fmaf(s2[2 * k], inv_width, a.eps));
                const float mean2 = scale2 * s2[2 * k + 1] * inv_width;  // mean(dn2 . n2)
                f32x2 yv[4];
                staged8<T>(at(3, k, pipe.stage, live[k]), yv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 n2 = mul2(hv[k][e], both(scale2));
                    sw2[e] = fma2(yv[e], n2, sw2[e]);
                    ev[e] = fma2(both(scale2), fma2(n2, both(-mean2), mul2(yv[e], w.w2[e])), ev[e]);
                }
            }
            if (in && a.d_residual) {
                f32x2 dr[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) dr[e] = mul2(both(a.residual_scale), ev[e]);
                store_pairs(static_cast<R *>(a.d_residual) + base + int64_t(k) * width, dr);
            }
            f32x2 xv[4], zv[4];
            staged8<T>(at(0, k, pipe.stage, live[k]), xv);
            if (gated) staged8<T>(at(1, k, pipe.stage, live[k]), zv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 n1 = mul2(xv[e], both(scale1[k])), u = mul2(n1, w.w1[e]), db = mul2(ev[e], w.s[e]);
                f32x2 act = both(1.f), du = db;
                if (gated) {
                    // act' = g + act (1 - g) for SiLU, g (1 - g) for the sigmoid
                    const f32x2 g = gv[k][e], not_g = fma2(g, both(-1.f), both(1.f));
                    act = silu ? mul2(zv[e], g) : g;
                    du = mul2(db, act);
                    zv[e] = mul2(silu ? fma2(act, not_g, g) : mul2(g, not_g), mul2(db, u));  // dz
                }
                ssc[e] = fma2(ev[e], mul2(u, act), ssc[e]);  // (branch_scale at the end)
                sw1[e] = fma2(du, n1, sw1[e]);
                hv[k][e] = mul2(du, w.w1[e]);  // dn1 (dx without the norm)
                sd = fma2(hv[k][e], n1, sd);
            }
            s3[k] = lo_of(sd) + hi_of(sd);
            if (in && a.d_gate) store_pairs(static_cast<T *>(a.d_gate) + base + int64_t(k) * width, zv);
        }
        // the next two rows' x^2, with the sums of these
        const uint32_t stage = pipe.stage;
        const bool in0 = live[0], in1 = live[1];
        more = first < rows - stride;
        if (more) first += stride;
        pipe.advance();
        pipe.template wait<kBwdStages - 2>();  // (this stage's next copies are not on their way yet)
        arrive(more);
        if (post) {
            s3[2] = squares(0, live[0]);
            s3[3] = squares(1, live[1]);
            row_sum<4, 16>(s3, red, t, n);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool in = k ? in1 : in0;
            if (post) {
                f32x2 xv[4];
                const float mean1 = s3[k] * inv_width;
                staged8<T>(at(0, k, stage, in), xv);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    hv[k][e] = mul2(both(scale1[k]), fma2(mul2(xv[e], both(scale1[k])), both(-mean1), hv[k][e]));
            }
            if (in && a.dx) store_pairs(static_cast<T *>(a.dx) + base + int64_t(k) * width, hv[k]);
        }
        pipe.fetch(sg, stage, width);  // (the stage has been read)
    }
    float *out = a.partial + (int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * 3 * width + c;
    if (c >= width) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) ssc[e] = mul2(ssc[e], both(a.branch_scale));
    if (a.d_post_weight) store_pairs(out, sw1);
    if (a.d_scale) store_pairs(out + width, ssc);
    if (a.d_pre_weight) store_pairs(out + 2 * width, sw2);
}

// A block row-group (threadIdx.y) walks rows with a stride; its columns' sums
// stay in registers and go to its own line of the workspace.
template <typename T, typename R, int kGroups>
__global__ void __launch_bounds__(512)
block_norm_backward_any_kernel(const BlockNormArgs a) {
    __shared__ __align__(16) float red_all[32 * 8];
    clear_red(red_all);
    const int n = blockDim.x, t = threadIdx.x, width = a.width;
    float *red = red_all + 32 * threadIdx.y;
    const int64_t lines = int64_t(gridDim.x) * blockDim.y, line = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const float zc = (a.flags & GDN_BLOCK_ZERO_CENTRED) ? 1.f : 0.f;
    const float none = zc != 0.f ? 0.f : 1.f;
    const bool post = a.flags & GDN_BLOCK_POST_NORM, pre = (a.flags & GDN_BLOCK_PRE_NORM) && a.d_y;
    const bool silu = a.flags & GDN_BLOCK_GATE_SILU;
    float sw1[kGroups][8], sw2[kGroups][8], ssc[kGroups][8];
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sw1[i][e] = sw2[i][e] = ssc[i][e] = 0.f;
    const int64_t turns = (a.rows + lines - 1) / lines;
    for (int64_t turn = 0; turn < turns; ++turn) {
        const int64_t row = turn * lines + line;
        const bool live = row < a.rows;
        const int64_t at = (live ? row : 0) * width;
        const T *x = static_cast<const T *>(a.x) + at, *z = a.gate ? static_cast<const T *>(a.gate) + at : nullptr;
        const R *r = a.residual ? static_cast<const R *>(a.residual) + at : nullptr;
        float xv[kGroups][8], zv[kGroups][8], hv[kGroups][8], yv[kGroups][8], ev[kGroups][8];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            row_load(x, i, t, n, width, xv[i]);
            if (z) row_load(z, i, t, n, width, zv[i]);
            if (r) {
                row_load(r, i, t, n, width, hv[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) hv[i][e] = 0.f;
            }
            if (pre) row_load(static_cast<const T *>(a.d_y) + at, i, t, n, width, yv[i]);
            if (a.d_h) {
                row_load(static_cast<const R *>(a.d_h) + at, i, t, n, width, ev[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) ev[i][e] = 0.f;
            }
        }
        float scale1 = 1.f;
        if (post) {
            float ss[1] = {0.f};
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) ss[0] = fmaf(xv[i][e], xv[i][e], ss[0]);
            row_sum<1, 16>(ss, red, t, n);
            scale1 = 1.f / sqrtf(ss[0] / float(width) + a.eps);
        }
        // h, and the sums of h^2 and dy w2 h
        float s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            float w1[8], s[8], w2[8];
            weight_load<false>(post ? a.post_weight : nullptr, post ? none : 1.f, post ? zc : 0.f, i, t, n, width, w1);
            weight_load<false>(a.scale, 1.f, 0.f, i, t, n, width, s);
            if (pre) weight_load<false>(a.pre_weight, none, zc, i, t, n, width, w2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xv[i][e] *= scale1;  // n1
                float b = xv[i][e] * w1[e];
                if (z) {
                    const float sg = gate_sigmoid<T>(zv[i][e]);
                    b *= silu ? zv[i][e] * sg : sg;
                }
                hv[i][e] = fmaf(a.residual_scale, hv[i][e], a.branch_scale * s[e] * b);
                if (pre) {
                    s2[0] = fmaf(hv[i][e], hv[i][e], s2[0]);
                    s2[1] = fmaf(yv[i][e] * w2[e], hv[i][e], s2[1]);
                }
            }
        }
        float scale2 = 0.f, mean2 = 0.f;
        if (pre) {
            row_sum<2, 16>(s2, red, t, n);
            scale2 = 1.f / sqrtf(s2[0] / float(width) + a.eps);
            mean2 = scale2 * s2[1] / float(width);  // mean(dn2 . n2)
        }
        float s3[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            float w1[8], s[8], w2[8], dr[8], dzv[8];
            weight_load<false>(post ? a.post_weight : nullptr, post ? none : 1.f, post ? zc : 0.f, i, t, n, width, w1);
            weight_load<false>(a.scale, 1.f, 0.f, i, t, n, width, s);
            if (pre) weight_load<false>(a.pre_weight, none, zc, i, t, n, width, w2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float g = ev[i][e];
                if (pre) {
                    const float n2 = hv[i][e] * scale2;
                    g = fmaf(scale2, fmaf(-n2, mean2, yv[i][e] * w2[e]), g);
                    if (live) sw2[i][e] = fmaf(yv[i][e], n2, sw2[i][e]);
                }
                dr[e] = a.residual_scale * g;
                const float n1 = xv[i][e], u = n1 * w1[e], cg = a.branch_scale * g;
                const float db = cg * s[e];
                float act = 1.f, du = db;
                dzv[e] = 0.f;
                if (z) {
                    const float zz = zv[i][e], sg = gate_sigmoid<T>(zz);
                    act = silu ? zz * sg : sg;
                    du = db * act;
                    dzv[e] = db * u * (silu ? sg * fmaf(zz, 1.f - sg, 1.f) : sg * (1.f - sg));
                }
                if (live) {
                    ssc[i][e] = fmaf(cg, u * act, ssc[i][e]);
                    sw1[i][e] = fmaf(du, n1, sw1[i][e]);
                }
                ev[i][e] = du * w1[e];  // dn1 (dx without the norm)
                s3[0] = fmaf(ev[i][e], n1, s3[0]);
            }
            if (live && a.d_residual) row_store(static_cast<R *>(a.d_residual) + at, i, t, n, width, dr);
            if (live && a.d_gate) row_store(static_cast<T *>(a.d_gate) + at, i, t, n, width, dzv);
        }
        if (post) {
            row_sum<1, 16>(s3, red, t, n);
            const float mean1 = s3[0] / float(width);
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) ev[i][e] = scale1 * fmaf(-xv[i][e], mean1, ev[i][e]);
        }
        if (live && a.dx)
#pragma unroll
            for (int i = 0; i < kGroups; ++i) row_store(static_cast<T *>(a.dx) + at, i, t, n, width, ev[i]);
    }
    float *out = a.partial + line * 3 * width;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        if (a.d_post_weight) row_store(out, i, t, n, width, sw1[i]);
        if (a.d_scale) row_store(out + width, i, t, n, width, ssc[i]);
        if (a.d_pre_weight) row_store(out + 2 * width, i, t, n, width, sw2[i]);
    }
}

// Column sums of the lines, 16 partial sums per column joined in a fixed order.
__global__ void __launch_bounds__(512)
block_norm_columns_kernel(const float *__restrict__ part, int lines, int width, float *dw1, float *ds, float *dw2) {
    __shared__ float sum[16][33];
    float *dst = blockIdx.y == 0 ? dw1 : blockIdx.y == 1 ? ds : dw2;
    if (!dst) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < width) {
        const float *p = part + size_t(blockIdx.y) * width + c;
#pragma unroll 8
        for (int i = threadIdx.y; i < lines; i += 16) s += p[size_t(i) * 3 * width];
    }
    sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < width) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += sum[i][threadIdx.x];
        dst[c] = s;
    }
}

// Threads a row takes (a multiple of 32) with `groups` 8-value groups each.
int row_threads(int width, int groups) { return ((width + 8 * groups - 1) / (8 * groups) + 31) / 32 * 32; }

// Launch shape: threads per row and rows per block (as many whole rows as 256
// threads take, eight at most, or one row), 8 columns a thread up to 4096
// columns.
struct Shape {
    int groups, n, per;
};
Shape shape_of(int width) {
    Shape s;
    s.groups = width <= 4096 ? 1 : width <= 8192 ? 2 : 4;
    s.n = row_threads(width, s.groups);
    s.per = std::max(1, std::min(8, 256 / s.n));
    return s;
}

Shape forward_shape_of(int width) {  // 16 columns a thread above 2048
    Shape s;
    s.groups = width <= 2048 ? 1 : width <= 8192 ? 2 : 4;
    s.n = row_threads(width, s.groups);
    s.per = std::max(1, std::min(8, 256 / s.n));
    return s;
}

Stages stages_of(const void *const *src, const int *size, int count, int width, int per) {
    Stages s = {};
    for (int i = 0; i < count; ++i) {
        s.src[i] = static_cast<const unsigned char *>(src[i]);
        s.row_bytes[i] = uint32_t(width) * uint32_t(size[i]);
        s.off[i] = s.stage_bytes;
        if (src[i]) s.stage_bytes += s.row_bytes[i] * uint32_t(per);
    }
    return s;
}

// Rows whose bytes are multiples of 16 (8 columns), and kFwdStages or
// kBwdStages stages of which fit in shared memory, are staged.
constexpr size_t kStageRoom = 220 * 1024;

template <typename K>
cudaError_t staged_launch(K kern, int stages, const BlockNormArgs &a, const Stages &sg, int grid, dim3 block,
                          cudaStream_t stream) {
    const size_t bytes = size_t(stages) * sg.stage_bytes;
    if (bytes > 40 * 1024) {  // (a kernel may have 48 KB in all without asking)
        // The limit is one value for all host threads: the most that any call asks for, never this call's own size,
        // which another thread could lower before the launch.
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kStageRoom));
        if (e != cudaSuccess) return e;
    }
    kern<<<unsigned(grid), block, bytes, stream>>>(a, sg);
    count_launch();
    return cudaGetLastError();
}

bool aligned_rows(const BlockNormArgs &a) { return a.width % 8 == 0; }

template <typename T, typename R>
cudaError_t forward_as(const BlockNormArgs &a, cudaStream_t stream) {
    const Shape s = forward_shape_of(a.width);
    const dim3 block(s.n, s.per);
    const int64_t groups = (a.rows + s.per - 1) / s.per;
    const void *src[] = {a.x, a.gate, a.residual};
    const int size[] = {sizeof(T), sizeof(T), sizeof(R)};
    const Stages sg = stages_of(src, size, 3, a.width, s.per);
    if (aligned_rows(a) && kFwdStages * size_t(sg.stage_bytes) <= kStageRoom) {
        const int fit = int(std::max<size_t>(1, kStageRoom / (kFwdStages * size_t(sg.stage_bytes) + 1024)));
        const bool small = s.n * s.per <= 256;
        const int grid = int(std::min<int64_t>(groups, int64_t(148) * (small ? std::min(fit, 3) : 1)));
        if (s.groups == 1) return staged_launch(block_norm_forward_kernel<T, R, 1, 256>, kFwdStages, a, sg, grid, block, stream);
        if (s.groups == 2 && small)
            return staged_launch(block_norm_forward_kernel<T, R, 2, 256>, kFwdStages, a, sg, grid, block, stream);
        if (s.groups == 2) return staged_launch(block_norm_forward_kernel<T, R, 2, 512>, kFwdStages, a, sg, grid, block, stream);
        return staged_launch(block_norm_forward_kernel<T, R, 4, 512>, kFwdStages, a, sg, grid, block, stream);
    }
    if (groups > INT32_MAX) return cudaErrorInvalidValue;
    if (s.groups == 1) block_norm_forward_any_kernel<T, R, 1><<<unsigned(groups), block, 0, stream>>>(a);
    else if (s.groups == 2) block_norm_forward_any_kernel<T, R, 2><<<unsigned(groups), block, 0, stream>>>(a);
    else block_norm_forward_any_kernel<T, R, 4><<<unsigned(groups), block, 0, stream>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t backward_as(const BlockNormArgs &a, cudaStream_t stream) {
    const Shape s = shape_of(a.width);
    const dim3 block(s.n, s.per);
    const int lines = block_norm_lines(a.rows, a.width), grid = lines / s.per;
    const void *src[] = {a.x, a.gate, a.residual, a.d_y, a.d_h};
    const int size[] = {sizeof(T), sizeof(T), sizeof(R), sizeof(T), sizeof(R)};
    const Stages sg = stages_of(src, size, 5, a.width, s.per);
    cudaError_t e;
    const Stages pair = stages_of(src, size, 5, a.width, 2 * s.per);
    // two rows at a time where a block then still has two groups of them or more, and as many blocks fit an SM
    if (aligned_rows(a) && s.groups == 1 && a.rows >= 4 * int64_t(lines) &&
        kBwdStages * size_t(pair.stage_bytes) * (lines > 148 * s.per ? 2 : 1) <= kStageRoom) {
        const bool known = (a.flags & GDN_BLOCK_PRE_NORM) && a.residual && a.d_y && a.d_h;
        const int parts = !known ? kAnyParts
                                 : ((a.flags & GDN_BLOCK_POST_NORM) ? kPartPost : 0) | (a.gate ? kPartGate : 0) |
                                       (a.gate && (a.flags & GDN_BLOCK_GATE_SILU) ? kPartSilu : 0);
        auto go = [&](auto kern) { return staged_launch(kern, kBwdStages, a, pair, grid, block, stream); };
        e = parts == 0   ? go(block_norm_backward_pair_kernel<T, R, 0>)
            : parts == 1 ? go(block_norm_backward_pair_kernel<T, R, 1>)
            : parts == 2 ? go(block_norm_backward_pair_kernel<T, R, 2>)
            : parts == 3 ? go(block_norm_backward_pair_kernel<T, R, 3>)
            : parts == 6 ? go(block_norm_backward_pair_kernel<T, R, 6>)
            : parts == 7 ? go(block_norm_backward_pair_kernel<T, R, 7>)
                         : go(block_norm_backward_pair_kernel<T, R, kAnyParts>);
    } else if (aligned_rows(a) && kBwdStages * size_t(sg.stage_bytes) <= kStageRoom) {
        e = s.groups == 1   ? staged_launch(block_norm_backward_kernel<T, R, 1>, kBwdStages, a, sg, grid, block, stream)
            : s.groups == 2 ? staged_launch(block_norm_backward_kernel<T, R, 2>, kBwdStages, a, sg, grid, block, stream)
                            : staged_launch(block_norm_backward_kernel<T, R, 4>, kBwdStages, a, sg, grid, block, stream);
    } else {
        if (s.groups == 1) block_norm_backward_any_kernel<T, R, 1><<<unsigned(grid), block, 0, stream>>>(a);
        else if (s.groups == 2) block_norm_backward_any_kernel<T, R, 2><<<unsigned(grid), block, 0, stream>>>(a);
        else block_norm_backward_any_kernel<T, R, 4><<<unsigned(grid), block, 0, stream>>>(a);
        count_launch();
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    if (a.d_post_weight || a.d_scale || a.d_pre_weight) {
        block_norm_columns_kernel<<<dim3(unsigned((a.width + 31) / 32), 3), dim3(32, 16), 0, stream>>>(
            a.partial, lines, a.width, a.d_post_weight, a.d_scale, a.d_pre_weight);
        count_launch();
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

// Row groups of the backward, each with a line of column sums in the workspace.
int block_norm_lines(int64_t rows, int32_t width) {
    const Shape s = shape_of(width);
    const int resident = std::max(1, 512 / (s.n * s.per));  // blocks an SM holds at the kernel's registers
    const int64_t blocks = std::min<int64_t>((rows + s.per - 1) / s.per, int64_t(148) * resident);
    return int(std::max<int64_t>(blocks, 1)) * s.per;
}

cudaError_t launch_block_norm_forward(const BlockNormArgs &a, int32_t dtype, int32_t rdtype, cudaStream_t stream) {
    using bf = __nv_bfloat16;
    if (dtype == GDN_DTYPE_F32) return forward_as<float, float>(a, stream);
    return rdtype == GDN_DTYPE_F32 ? forward_as<bf, float>(a, stream) : forward_as<bf, bf>(a, stream);
}
cudaError_t launch_block_norm_backward(const BlockNormArgs &a, int32_t dtype, int32_t rdtype, cudaStream_t stream) {
    using bf = __nv_bfloat16;
    if (dtype == GDN_DTYPE_F32) return backward_as<float, float>(a, stream);
    return rdtype == GDN_DTYPE_F32 ? backward_as<bf, float>(a, stream) : backward_as<bf, bf>(a, stream);
}

}  // namespace gdn
