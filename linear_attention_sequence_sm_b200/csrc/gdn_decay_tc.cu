// gdn_decay_tc.cu -- the decayed linear attention's pass on the tensor cores
// (bf16, head sizes a multiple of 8 up to 128), see gdn_decay.cuh for the
// pass and its operands x, y, z, out.
//
// Chunk of 64 tokens, state Sigma (z x y, fp32, tensor memory), every product
// one tcgen05.mma stream with fp32 accumulators:
//   (QK) x y^T                     64 x 64 x dy      -> P = QK . decay mask, bf16
//   (KV) Sigma += z^T (w y)        128 x dy x 64     the state's critical path
//   (X1) X1 = Sigma x^T            128 x 64 x dy     bf16 copies of Sigma (tensor memory) times x
//   (X2) X2 = z^T P^T              128 x 64 x 64
// out^T = X2 + w_in X1.  x, y, z come by TMA as 128-byte-swizzled tiles and
// serve as the K-major and MN-major operands they are; head sizes below 128
// are padded with zeros by TMA.
//
// Precision.  The state is fp32 in and out, so the scaled operand w y is split
// into three bf16 terms (24 bits; one term would leave 2^-9 of the state, two
// terms 2^-17).  For `dot` passes, whose products with the start state feed
// the decays' fp32 gradient, Sigma's copy is split into three terms as well;
// otherwise X1 ends in a bf16 output, and one bf16 copy costs it as much as
// the output's own rounding.  P is one bf16 term for the same reason.
//
// Roles (18 warps):
//   state warps 0-7    two per tensor-memory quarter, 64 state columns each:
//                      before chunk n: copies of Sigma, Sigma <- e^G Sigma
//   out warps 8-11     X1, X2 -> out (and the dot with aux)
//   prep warps 12-15   decays, the split of w y, P from QK
//   warp 16            TMA loads;  warp 17  issues every product, in the order
//                      KV(n), X1(n), X2(n), QK(n + 1): the state warps work on
//                      chunk n + 1's state while X1, X2 and QK run.  (With
//                      three copies of Sigma there is tensor memory for one
//                      set only, so X1(n) goes before KV(n).)
// All hand-overs are mbarriers with bounded waits; a timeout records
// GDN_ERR_DEVICE_CHECK (bad_index -2).  A CTA takes units (segment, head) with
// a stride of the grid; nothing synchronises it between units.
#include <algorithm>

#include "gdn_decay.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
using namespace sm100;

namespace {

constexpr int kThreads = 576;
constexpr int kWarpOut = 8, kWarpPrep = 12, kWarpTma = 16, kWarpMma = 17;
constexpr int kBarPrep = 1, kBarOut = 2;  // named barriers (128 threads each)
constexpr uint32_t kTile = 16384, kAtom = 8192, kPTile = 8192;
constexpr uint32_t kTmemCols = 512;

// token vectors of a chunk (floats): prefix sums in log2 units, the output's
// and the state operand's weights, e^G of the whole chunk
constexpr int kVecG = 0, kVecIn = 64, kVecSt = 128, kVecGamma = 192, kVecFloats = 196;

// kKind: what a pass leaves out or adds
enum { kPlain = 0, kDot = 1, kStateOnly = 2 };

template <int kKind> struct Cfg {
    static constexpr int kCopies = kKind == kDot ? 3 : 1;        // bf16 terms of Sigma's copy
    static constexpr int kQkBufs = kKind == kDot ? 1 : 2;
    static constexpr int kNX = kKind == kDot ? 2 : 3, kNZ = kNX, kNY = 2;
    // shared memory, from a 1024-byte-aligned base
    static constexpr uint32_t kOffX = 0;
    static constexpr uint32_t kOffZ = kOffX + kNX * kTile;
    static constexpr uint32_t kOffY = kOffZ + kNZ * kTile;
    static constexpr uint32_t kOffAux = kOffY + kNY * kTile;                    // [2], kDot only
    static constexpr uint32_t kOffYs = kOffAux + (kKind == kDot ? 2 * kTile : 0);  // three terms of w y
    static constexpr uint32_t kOffP = kOffYs + 3 * kTile;                       // [2]
    static constexpr uint32_t kOffVec = kOffP + 2 * kPTile;                     // [4]
    static constexpr uint32_t kOffRed = kOffVec + 4 * kVecFloats * 4;           // [4 warps][64]
    static constexpr uint32_t kOffBar = kOffRed + 1024;
    static constexpr uint32_t kSmem = kOffBar + 320 + 1024;
    static_assert(kSmem <= 232448, "shared memory over the sm_100 per-block limit");
    // tensor memory columns
    static constexpr uint32_t kColS = 0, kColC = 128;  // Sigma; its copies (64 columns each, two buffers or three terms)
    static constexpr uint32_t kColX1 = kCopies == 1 ? 256 : 320, kColX2 = kColX1 + 64, kColQK = kColX2 + 64;
};

// mbarriers
enum {
    kBX = 0,        // [3] x landed
    kBZ = 3,        // [3] z
    kBY = 6,        // [2] y
    kBA = 8,        // [2] aux
    kBXFree = 10,   // [3] X1 and QK of the slot's chunk done
    kBZFree = 13,   // [3] KV and X2 done
    kBYFree = 16,   // [2] QK done, w y written (4 prep warps)
    kBAFree = 18,   // [2] dot taken (4 out warps)
    kBVec = 20,     // [2] token vectors written
    kBYs = 22,      // w y written (4 prep warps)
    kBSt = 23,      // state pass done (8 state warps)
    kBKV = 24,      // KV done
    kBQK = 25,      // [2] QK done
    kBP = 27,       // [2] P written (4 prep warps)
    kBPFree = 29,   // [2] X2 done
    kBOut = 31,     // X1, X2 done (and an arrival of the issuing thread, which orders the token vectors)
    kBOutFree = 32, // X1, X2 read (4 out warps)
    kBDrain = 33,
    kNumBars = 34
};

struct Maps {
    CUtensorMap x, y, z, aux;
};

// The units of this CTA, one after the other.
struct UnitWalk {
    const DecayPass &a;
    int64_t u, units;
    DecaySeg seg;
    int h, nch;
    bool first, last;
    __device__ UnitWalk(const DecayPass &a_, bool dead) : a(a_), u(int64_t(blockIdx.x) - gridDim.x) {
        units = dead ? 0 : int64_t(a.sched.hdr->num_segs) * a.hv;
    }
    __device__ bool next(bool state_only) {
        for (;;) {
            u += gridDim.x;
            if (u >= units) return false;
            seg = a.sched.segs[u / a.hv];
            h = int(u % a.hv);
            nch = (seg.len + kDecayChunk - 1) / kDecayChunk;
            first = a.reverse ? seg.pos + seg.len == seg.seq_len : seg.pos == 0;
            last = a.reverse ? seg.pos == 0 : seg.pos + seg.len == seg.seq_len;
            if (!(state_only && (seg.slot < 0 || last))) return true;
        }
    }
    // first token of the n-th chunk in pass order, from the segment's start
    __device__ int chunk_at(int n) const { return kDecayChunk * (a.reverse ? nch - 1 - n : n); }
};

// A bounded wait of a whole warp; every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Rows 16 (warp % 4) + lane % 16 of an M = 64 accumulator, columns 0-31 in
// lanes 0-15 and 32-63 in lanes 16-31.
__device__ __forceinline__ void tmem_ld_m64(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32], 32;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 state columns at c: copies of Sigma (kCopies bf16 terms, `step` columns
// apart), Sigma <- gamma Sigma.
template <int kCopies>
__device__ __forceinline__ void state_slice(uint32_t s_addr, uint32_t c_addr, float gamma, float (&v)[32]) {
    uint32_t pk[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    tmem_st16u(c_addr, pk);
    if constexpr (kCopies == 3) {
        float r[32];
#pragma unroll
        for (int t = 1; t < 3; ++t) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                r[2 * j] = (t == 1 ? v[2 * j] : r[2 * j]) - bf_lo(pk[j]);
                r[2 * j + 1] = (t == 1 ? v[2 * j + 1] : r[2 * j + 1]) - bf_hi(pk[j]);
                pk[j] = pack_bf16x2(r[2 * j], r[2 * j + 1]);
            }
            tmem_st16u(c_addr + 64 * t, pk);
        }
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= gamma;
    tmem_st32(s_addr, v);
}

template <int kKind>
__global__ void __launch_bounds__(kThreads, 1)
decay_pass_tc_kernel(const __grid_constant__ Maps tm, const DecayPass a) {
    using K = Cfg<kKind>;
    constexpr bool kDots = kKind == kDot, kSt = kKind == kStateOnly;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + K::kOffBar + 8 * kNumBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) { return sb + K::kOffBar + 8u * uint32_t(i); };
    auto vecs = [&](uint32_t m) { return reinterpret_cast<float *>(smem + K::kOffVec) + (m & 3u) * kVecFloats; };

    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            int n = 1;
            if (i == kBYFree || i == kBYFree + 1) n = kSt ? 4 : 5;
            if (i == kBAFree || i == kBAFree + 1 || i == kBYs || i == kBP || i == kBP + 1 || i == kBOutFree) n = 4;
            if (i == kBSt) n = 8;
            if (i == kBOut) n = 2;
            mbar_init(bar(i), uint32_t(n));
        }
        fence_mbarrier_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tslot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    grid_dep_wait();  // the segment table (and start states) are written
    bool ok = a.sched.hdr->status == GDN_OK;
    const int hv = a.hv, dy = a.dy, dz = a.dz;
    const int ya = dy > 64 ? 2 : 1;  // 64-column halves of y and of the state
    UnitWalk w(a, !ok);
    const bool dead = !ok;
    uint32_t m = 0;  // chunks this CTA has processed

    if (warp < kWarpOut) {
        // ==================== state warps: thread = state row ====================
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t trow = tmem + (uint32_t((warp & 3) * 32) << 16);
        const int c0 = 64 * half;
        const bool mine = half < ya;
        const bool zin = row < dz;
        while (ok && w.next(kSt)) {
            const size_t sbase = (size_t(w.seg.seq) * hv + w.h) * dz * dy;
            const bool own = !kSt && w.seg.slot >= 0;
            if (mine) {  // the start state
                const float *src = nullptr;
                bool tr = false;
                int ld = 0;
                if (own) {
                    src = a.seg_state + (size_t(w.seg.slot) * hv + w.h) * 16384;
                    tr = a.seg_trans;
                    ld = 128;
                } else if (!kSt && a.s_in && w.first) {
                    src = a.s_in + sbase;
                    tr = a.s_trans;
                    ld = tr ? dz : dy;
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float v[32];
                    const int c = c0 + 32 * p;
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                    if (src && zin) {
                        if (tr) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c + j < dy) v[j] = src[size_t(c + j) * ld + row];
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)  // dy and ld are multiples of 8
                                if (c + j < dy) load4(src + size_t(row) * ld + c + j, v + j);
                        }
                    }
                    tmem_st32(trow + K::kColS + uint32_t(c), v);
                }
                tmem_wait_st();
            }
            float dec = 1.f;
            for (int n = 0; n <= w.nch; ++n) {
                // before chunk n, or after the last one
                const bool end = n == w.nch;
                const uint32_t mm = m + uint32_t(n);
                if (!end) ok = warp_wait(bar(kBVec + int(mm & 1u)), (mm >> 1) & 1u);
                if (ok && n > 0) ok = warp_wait(bar(kBKV), (mm - 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                const float gamma = end ? 1.f : vecs(mm)[kVecGamma];
                // where the state is wanted: a checkpoint to write (forward) or to be dotted with (backward)
                float *ck = nullptr;
                const float *cd = nullptr;
                bool cd_first = false;
                float *zs = nullptr;
                if (kDots && a.ckpt) {
                    const int ick = a.sched.hdr->ick;
                    if (!a.zsum) {
                        const int p = w.seg.pos + w.chunk_at(n);
                        if (!end && p > 0 && p % ick == 0) ck = a.ckpt + (size_t(w.seg.ck + p / ick) * hv + w.h) * 16384;
                    } else if (n > 0) {
                        const int p = w.seg.pos + w.chunk_at(n - 1);  // the state is the one at this chunk's start
                        if (p % ick == 0) {
                            const size_t slot = size_t(w.seg.ck + p / ick) * hv + w.h;
                            zs = a.zsum + slot * 8;
                            cd_first = p == 0;
                            cd = cd_first ? (a.s_first ? a.s_first + sbase : nullptr) : a.ckpt + slot * 16384;
                        }
                    }
                }
                float dot = 0.f;
                if (mine) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int c = c0 + 32 * p;
                        float v[32];
                        tmem_ld32(trow + K::kColS + uint32_t(c), v);
                        tmem_wait_ld();
                        if constexpr (kDots) {
                            if (ck) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) ck[(c + j) * 128 + row] = v[j];
                            }
                            if (cd && zin) {
                                if (cd_first) {  // stored [y][z] (s_trans)
#pragma unroll
                                    for (int j = 0; j < 32; ++j)
                                        if (c + j < dy) dot = fmaf(cd[size_t(c + j) * dz + row], v[j], dot);
                                } else {
#pragma unroll
                                    for (int j = 0; j < 32; ++j) dot = fmaf(cd[(c + j) * 128 + row], v[j], dot);
                                }
                            }
                        }
                        if (!end) {
                            if constexpr (kSt) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[j] *= gamma;
                                tmem_st32(trow + K::kColS + uint32_t(c), v);
                            } else {
                                const uint32_t ca = trow + K::kColC + (K::kCopies == 1 ? 64u * (mm & 1u) : 0u) + uint32_t(c / 2);
                                state_slice<K::kCopies>(trow + K::kColS + uint32_t(c), ca, gamma, v);
                            }
                        } else {
                            float *dst = nullptr;
                            bool tr = false;
                            int ld = 128;
                            if constexpr (kSt) {
                                dst = a.seg_local + (size_t(w.seg.slot) * hv + w.h) * 16384;
                            } else if (w.last && a.s_out) {
                                dst = a.s_out + sbase;
                                tr = a.s_trans;
                                ld = tr ? dz : dy;
                            }
                            if (dst && zin) {
                                if (tr) {
#pragma unroll
                                    for (int j = 0; j < 32; ++j)
                                        if (c + j < dy) dst[size_t(c + j) * ld + row] = v[j];
                                } else {
#pragma unroll
                                    for (int j = 0; j < 32; j += 4)
                                        if (c + j < dy)
                                            *reinterpret_cast<float4 *>(dst + size_t(row) * ld + c + j) =
                                                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                                }
                            }
                        }
                    }
                    tmem_wait_st();
                }
                if (kDots && zs) {
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
                    if (lane == 0) zs[warp] = dot;
                }
                dec *= gamma;
                tc_fence_before();
                __syncwarp();
                if (!end && lane == 0) mbar_arrive(bar(kBSt));
            }
            if (kSt && ok && tid == 0) a.seg_dec[size_t(w.seg.slot) * hv + w.h] = dec;
            m += uint32_t(w.nch);
        }
    } else if (warp < kWarpPrep) {
        // ==================== out warps: thread = z row ====================
        if constexpr (!kSt) {
            const int quarter = warp & 3, row = quarter * 32 + lane, ot = tid - 32 * kWarpOut;
            const uint32_t trow = tmem + (uint32_t(quarter * 32) << 16);
            float *red = reinterpret_cast<float *>(smem + K::kOffRed);
            while (ok && w.next(false)) {
                for (int n = 0; n < w.nch; ++n) {
                    const uint32_t mm = m + uint32_t(n);
                    const int t0 = w.chunk_at(n), L = min(kDecayChunk, w.seg.len - t0);
                    ok = warp_wait(bar(kBOut), mm & 1u);
                    if (kDots && a.aux) {
                        if (ok) ok = warp_wait(bar(kBA + int(mm & 1u)), (mm >> 1) & 1u);
                        ok = !named_sync_or(kBarOut, 128, !ok);  // the four warps stay together (and `red` was read)
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const float *win = vecs(mm) + kVecIn;
                    const size_t tok = size_t(w.seg.start) + t0;
                    const size_t step = size_t(hv) * dz;
                    const size_t at = (tok * hv + w.h) * dz + row;
                    const uint32_t aux = sb + K::kOffAux + (mm & 1u) * kTile + uint32_t(row >> 6) * kAtom;
                    float x[64];  // out, all 64 tokens of this row
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        float x1[32], x2[32];
                        tmem_ld32(trow + K::kColX1 + 32 * p, x1);
                        tmem_ld32(trow + K::kColX2 + 32 * p, x2);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            float wi[4];
                            load4(win + 32 * p + 4 * q, wi);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                x1[4 * q + e] *= wi[e];
                                x[32 * p + 4 * q + e] = x2[4 * q + e] + x1[4 * q + e];
                            }
                        }
                        if constexpr (kDots) {
                            if (a.aux) {
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    float d[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const int r = 32 * p + 16 * q + e;
                                        unsigned short b;
                                        const uint32_t ad = aux + uint32_t(r) * 128 +
                                                            ((uint32_t((row & 63) >> 3) ^ uint32_t(r & 7)) << 4) + 2 * (row & 7);
                                        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(b) : "r"(ad) : "memory");
                                        d[e] = row < dz ? __uint_as_float(uint32_t(b) << 16) * x1[16 * q + e] : 0.f;
                                    }
                                    const float s = warp_colsum16(d, lane);
                                    if ((lane & 1) == 0) red[quarter * 64 + 32 * p + 16 * q + (lane >> 1)] = s;
                                }
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(kBOutFree));
                        if (kDots && a.aux) mbar_arrive(bar(kBAFree + int(mm & 1u)));
                    }
                    if (row < dz) {
                        if (a.out_f32) {
                            float *o = static_cast<float *>(a.out) + at;
                            if (L == 64) {
#pragma unroll
                                for (int r = 0; r < 64; ++r) __stcs(o + r * step, x[r]);
                            } else {
#pragma unroll
                                for (int r = 0; r < 64; ++r)
                                    if (r < L) o[r * step] = x[r];
                            }
                        } else {
                            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + at;
                            if (L == 64) {
#pragma unroll
                                for (int r = 0; r < 64; ++r) o[r * step] = __float2bfloat16_rn(x[r]);
                            } else {
#pragma unroll
                                for (int r = 0; r < 64; ++r)
                                    if (r < L) o[r * step] = __float2bfloat16_rn(x[r]);
                            }
                        }
                    }
                    if (kDots && a.aux) {
                        named_sync(kBarOut, 128);
                        if (ot < L)
                            a.dot[size_t(w.h) * a.tokens + tok + ot] =
                                (red[ot] + red[64 + ot]) + (red[128 + ot] + red[192 + ot]);
                    }
                }
                m += uint32_t(w.nch);
            }
        }
    } else if (warp < kWarpTma) {
        // ============ prep warps: decays, w y in three terms, P ============
        const int pt = tid - 32 * kWarpPrep, quarter = warp & 3;
        while (w.next(kSt)) {
            const float *g = a.g_const ? a.g + w.h : a.g + size_t(w.seg.start) * hv + w.h;
            const size_t gs = a.g_const ? 0 : hv;
            float g0 = 0.f, g1 = 0.f;
            auto load_g = [&](int n) {  // this lane's two tokens of the n-th chunk
                const int t = w.chunk_at(n) + 2 * lane;
                g0 = t < w.seg.len ? fmaxf(g[size_t(t) * gs], kGFloor) : 0.f;
                g1 = t + 1 < w.seg.len ? fmaxf(g[size_t(t + 1) * gs], kGFloor) : 0.f;
            };
            if (quarter == 0 && w.nch > 0) load_g(0);
            for (int n = 0; n < w.nch; ++n) {
                const uint32_t mm = m + uint32_t(n);
                const int t0 = w.chunk_at(n), L = min(kDecayChunk, w.seg.len - t0);
                float *vec = vecs(mm);
                if (quarter == 0) {
                    // prefix sums and suffix sums (each without a subtraction)
                    float pre = g0 + g1, suf = g0 + g1;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const float u = __shfl_up_sync(0xffffffffu, pre, d), v = __shfl_down_sync(0xffffffffu, suf, d);
                        if (lane >= d) pre += u;
                        if (lane + d < 32) suf += v;
                    }
                    float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
                    if (lane == 0) before = 0.f;
                    if (lane == 31) after = 0.f;
                    const float G0 = before + g0, G1 = pre, R0 = g1 + after, R1 = after;
                    const float total = __shfl_sync(0xffffffffu, pre, 31);
                    const float e0 = expf(G0), e1 = expf(G1), f0 = expf(R0), f1 = expf(R1);
                    constexpr float kLog2e = 1.4426950408889634f;
                    *reinterpret_cast<float2 *>(vec + kVecG + 2 * lane) = make_float2(G0 * kLog2e, G1 * kLog2e);
                    *reinterpret_cast<float2 *>(vec + kVecIn + 2 * lane) = a.reverse ? make_float2(f0, f1) : make_float2(e0, e1);
                    *reinterpret_cast<float2 *>(vec + kVecSt + 2 * lane) = a.reverse ? make_float2(e0, e1) : make_float2(f0, f1);
                    if (lane == 0) vec[kVecGamma] = expf(total);
                    if (n + 1 < w.nch) load_g(n + 1);
                }
                // the four warps go on, or stop, together
                if (named_sync_or(kBarPrep, 128, !ok)) {
                    ok = false;
                    goto prep_done;
                }
                if (pt == 0) mbar_arrive(bar(kBVec + int(mm & 1u)));
                // w y in three bf16 terms, over the previous chunk's
                ok = warp_wait(bar(kBY + int(mm % K::kNY)), (mm / K::kNY) & 1u);
                if (ok && mm > 0) ok = warp_wait(bar(kBKV), (mm - 1) & 1u);
                if (!ok) continue;
                {
                    const uint32_t ys = sb + K::kOffYs, yt = sb + K::kOffY + (mm % K::kNY) * kTile;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // 16 bytes of row r: eight rows and their swizzle stay within a warp's reach
                        const int e = pt + 128 * i, r = (e >> 3) & 63;
                        const uint32_t off = uint32_t(e) * 16;
                        if (e >= 512 * ya) break;
                        const uint4 q = ld_shared_v4(yt + off);
                        const uint32_t ws[4] = {q.x, q.y, q.z, q.w};
                        const float wt = vec[kVecSt + r];
                        uint32_t t0w[4], t1w[4], t2w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float lo = r < L ? bf_lo(ws[j]) * wt : 0.f, hi = r < L ? bf_hi(ws[j]) * wt : 0.f;
                            t0w[j] = pack_bf16x2(lo, hi);
                            lo -= bf_lo(t0w[j]);
                            hi -= bf_hi(t0w[j]);
                            t1w[j] = pack_bf16x2(lo, hi);
                            lo -= bf_lo(t1w[j]);
                            hi -= bf_hi(t1w[j]);
                            t2w[j] = pack_bf16x2(lo, hi);
                        }
                        st_shared_v4(ys + off, make_uint4(t0w[0], t0w[1], t0w[2], t0w[3]));
                        st_shared_v4(ys + kTile + off, make_uint4(t1w[0], t1w[1], t1w[2], t1w[3]));
                        st_shared_v4(ys + 2 * kTile + off, make_uint4(t2w[0], t2w[1], t2w[2], t2w[3]));
                    }
                }
                if (L < kDecayChunk) {
                    // tokens past the end are another sequence's: their z, whatever it holds, must not meet a zero weight
                    const uint32_t zs = mm % K::kNZ, zt = sb + K::kOffZ + zs * kTile;
                    ok = warp_wait(bar(kBZ + int(zs)), (mm / K::kNZ) & 1u);
                    if (!ok) continue;
                    for (int e = pt; e < 1024; e += 128)
                        if (((e >> 3) & 63) >= L) st_shared_v4(zt + uint32_t(e) * 16, make_uint4(0u, 0u, 0u, 0u));
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(kBYs));
                    mbar_arrive(bar(kBYFree + int(mm % K::kNY)));
                }
                if constexpr (!kSt) {
                    const uint32_t qb = K::kQkBufs == 2 ? (mm & 1u) : 0u;
                    ok = K::kQkBufs == 2 ? warp_wait(bar(kBQK + int(qb)), (mm >> 1) & 1u) : warp_wait(bar(kBQK), mm & 1u);
                    if (ok && mm >= 2) ok = warp_wait(bar(kBPFree + int(mm & 1u)), ((mm >> 1) - 1) & 1u);
                    if (!ok) continue;
                    tc_fence_after();
                    float v[32];
                    tmem_ld_m64(tmem + (uint32_t(quarter * 32) << 16) + K::kColQK + 64 * qb, v);
                    tmem_wait_ld();
                    const int r = 16 * quarter + (lane & 15), cb = lane < 16 ? 0 : 32;
                    const float Gr = vec[kVecG + r];
                    const uint32_t base = sb + K::kOffP + (mm & 1u) * kPTile + uint32_t(r) * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float gc[8], x[8];
                        load4(vec + kVecG + cb + 8 * q, gc);
                        load4(vec + kVecG + cb + 8 * q + 4, gc + 4);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int c = cb + 8 * q + j;
                            const bool in = a.reverse ? (c >= r && c < L) : c <= r;
                            const float d = a.reverse ? gc[j] - Gr : Gr - gc[j];
                            float e;
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d));
                            x[j] = in ? v[8 * q + j] * e : 0.f;
                        }
                        st_shared_v4(base + ((uint32_t(cb / 8 + q) ^ uint32_t(r & 7)) << 4), pack_bf16x8(x));
                    }
                    fence_proxy_async_shared();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBP + int(mm & 1u)));
                }
            }
            m += uint32_t(w.nch);
        }
    prep_done:;
    } else if (warp == kWarpTma) {
        if (lane == 0) {
            const uint32_t bytes_y = kAtom * uint32_t(ya);
            while (ok && w.next(kSt)) {
                const int hx = w.h / (hv / a.hx), hy = w.h / (hv / a.hy), hz = w.h / (hv / a.hz);
                const int ha = kDots && a.aux ? w.h / (hv / a.haux) : 0;
                for (int n = 0; n < w.nch; ++n) {
                    const uint32_t mm = m + uint32_t(n);
                    const int tok = w.seg.start + w.chunk_at(n);
                    if constexpr (!kSt) {
                        const uint32_t s = mm % K::kNX, dst = sb + K::kOffX + s * kTile;
                        if (mm >= uint32_t(K::kNX)) ok = mbar_wait(bar(kBXFree + int(s)), (mm / K::kNX - 1) & 1u);
                        if (!ok) break;
                        mbar_arrive_expect_tx(bar(kBX + int(s)), bytes_y);
                        tma_load_3d(dst, &tm.x, 0, hx, tok, bar(kBX + int(s)));
                        if (ya == 2) tma_load_3d(dst + kAtom, &tm.x, 64, hx, tok, bar(kBX + int(s)));
                    }
                    {
                        const uint32_t s = mm % K::kNY, dst = sb + K::kOffY + s * kTile;
                        if (mm >= uint32_t(K::kNY)) ok = mbar_wait(bar(kBYFree + int(s)), (mm / K::kNY - 1) & 1u);
                        if (!ok) break;
                        mbar_arrive_expect_tx(bar(kBY + int(s)), bytes_y);
                        tma_load_3d(dst, &tm.y, 0, hy, tok, bar(kBY + int(s)));
                        if (ya == 2) tma_load_3d(dst + kAtom, &tm.y, 64, hy, tok, bar(kBY + int(s)));
                    }
                    {
                        const uint32_t s = mm % K::kNZ, dst = sb + K::kOffZ + s * kTile;
                        if (mm >= uint32_t(K::kNZ)) ok = mbar_wait(bar(kBZFree + int(s)), (mm / K::kNZ - 1) & 1u);
                        if (!ok) break;
                        mbar_arrive_expect_tx(bar(kBZ + int(s)), kTile);
                        tma_load_3d(dst, &tm.z, 0, hz, tok, bar(kBZ + int(s)));
                        tma_load_3d(dst + kAtom, &tm.z, 64, hz, tok, bar(kBZ + int(s)));
                    }
                    if (kDots && a.aux) {
                        const uint32_t s = mm & 1u, dst = sb + K::kOffAux + s * kTile;
                        if (mm >= 2) ok = mbar_wait(bar(kBAFree + int(s)), ((mm >> 1) - 1) & 1u);
                        if (!ok) break;
                        mbar_arrive_expect_tx(bar(kBA + int(s)), kTile);
                        tma_load_3d(dst, &tm.aux, 0, ha, tok, bar(kBA + int(s)));
                        tma_load_3d(dst + kAtom, &tm.aux, 64, ha, tok, bar(kBA + int(s)));
                    }
                }
                m += uint32_t(w.nch);
            }
        }
    } else if (lane == 0) {
        // ==================== the issuing thread ====================
        uint32_t total = 0;
        while (w.next(kSt)) total += uint32_t(w.nch);
        const uint32_t id_qk = idesc_bf16(64, 64, false, false), id_kv = idesc_bf16(128, 64 * ya, true, true);
        const uint32_t id_x1 = idesc_bf16(128, 64, false, false), id_x2 = idesc_bf16(128, 64, true, false);
        const int ksteps = 4 * ya;
        auto koff = [](int s) { return uint64_t(((s >> 2) * kAtom + (s & 3) * 32) >> 4); };  // K-major steps
        auto issue_qk = [&](uint32_t c) {
            const uint32_t s = c % K::kNX, t = c % K::kNY;
            bool good = mbar_wait(bar(kBX + int(s)), (c / K::kNX) & 1u) && mbar_wait(bar(kBY + int(t)), (c / K::kNY) & 1u);
            if (!good) return false;
            tc_fence_after();
            const uint64_t dx = smem_desc(sb + K::kOffX + s * kTile, 16, 1024), dyd = smem_desc(sb + K::kOffY + t * kTile, 16, 1024);
            const uint32_t qb = K::kQkBufs == 2 ? (c & 1u) : 0u;
            for (int i = 0; i < ksteps; ++i) mma_bf16(tmem + K::kColQK + 64 * qb, dx + koff(i), dyd + koff(i), id_qk, i > 0);
            mma_commit(bar(kBQK + int(qb)));
            mma_commit(bar(kBYFree + int(t)));
            return true;
        };
        auto issue_kv = [&](uint32_t c) {
            const uint32_t s = c % K::kNZ;
            bool good = mbar_wait(bar(kBSt), c & 1u) && mbar_wait(bar(kBYs), c & 1u) &&
                        mbar_wait(bar(kBZ + int(s)), (c / K::kNZ) & 1u);
            if (!good) return false;
            tc_fence_after();
            const uint64_t da = smem_desc(sb + K::kOffZ + s * kTile, 8192, 1024);
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                const uint64_t db = smem_desc(sb + K::kOffYs + uint32_t(t) * kTile, 8192, 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_bf16(tmem + K::kColS, da + uint64_t((i * 2048) >> 4), db + uint64_t((i * 2048) >> 4), id_kv, 1);
            }
            mma_commit(bar(kBKV));
            if (kSt) mma_commit(bar(kBZFree + int(s)));
            return true;
        };
        auto issue_x1 = [&](uint32_t c) {
            const uint32_t s = c % K::kNX;
            bool good = mbar_wait(bar(kBSt), c & 1u);
            if (good && c > 0) good = mbar_wait(bar(kBOutFree), (c - 1) & 1u);
            if (!good) return false;
            tc_fence_after();
            const uint64_t dx = smem_desc(sb + K::kOffX + s * kTile, 16, 1024);
            const uint32_t cb = tmem + K::kColC + (K::kCopies == 1 ? 64u * (c & 1u) : 0u);
#pragma unroll
            for (int t = 0; t < K::kCopies; ++t)
                for (int i = 0; i < ksteps; ++i)
                    mma_bf16_ts(tmem + K::kColX1, cb + 64 * t + 8 * i, dx + koff(i), id_x1, t > 0 || i > 0);
            return true;
        };
        if (!kSt && ok && total > 0) ok = issue_qk(0);
        for (uint32_t c = 0; ok && c < total; ++c) {
            if constexpr (kSt) {
                ok = issue_kv(c);
            } else {
                if (K::kCopies == 1) ok = issue_kv(c) && issue_x1(c);
                else ok = issue_x1(c) && issue_kv(c);
                if (!ok) break;
                const uint32_t s = c % K::kNZ;
                ok = mbar_wait(bar(kBP + int(c & 1u)), (c >> 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                const uint64_t da = smem_desc(sb + K::kOffZ + s * kTile, 8192, 1024);
                const uint64_t db = smem_desc(sb + K::kOffP + (c & 1u) * kPTile, 16, 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_bf16(tmem + K::kColX2, da + uint64_t((i * 2048) >> 4), db + uint64_t((i * 32) >> 4), id_x2, i > 0);
                mma_commit(bar(kBOut));
                mbar_arrive(bar(kBOut));
                mma_commit(bar(kBXFree + int(c % K::kNX)));
                mma_commit(bar(kBZFree + int(s)));
                mma_commit(bar(kBPFree + int(c & 1u)));
                if (c + 1 < total) ok = issue_qk(c + 1);
            }
        }
        // every product done before the tensor memory goes
        mma_commit(bar(kBDrain));
        if (!mbar_wait(bar(kBDrain), 0u)) ok = false;
    }
    if (!ok && !dead) {
        a.sched.hdr->bad_index = -2;
        atomicExch(&a.sched.hdr->status, int(GDN_ERR_DEVICE_CHECK));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int kKind>
cudaError_t launch_as(const Maps &tm, const DecayPass &p, int64_t max_units, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(decay_pass_tc_kernel<kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(Cfg<kKind>::kSmem));
    if (e != cudaSuccess) return e;
    int dev = 0, sms = kDecayPlanSms;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(max_units, sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<kKind>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, decay_pass_tc_kernel<kKind>, tm, p);
    count_launch();
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

bool decay_tc_supported(const gdn_shape_t &s) {
    return s.dtype == GDN_DTYPE_BF16 && s.head_dim_k % 8 == 0 && s.head_dim_v % 8 == 0 &&
           !(s.flags & GDN_FLAG_FORCE_SIMT);
}

cudaError_t launch_decay_pass_tc(const DecayPass &p, int64_t max_units, cudaStream_t stream) {
    if (max_units <= 0) return cudaSuccess;
    Maps tm = {};
    // without tokens no tile is loaded, and there is nothing to map
    if (p.tokens > 0 &&
        ((!p.state_only && !make_head_map(&tm.x, p.x, p.hx, p.dy, p.tokens)) ||
         !make_head_map(&tm.y, p.y, p.hy, p.dy, p.tokens) || !make_head_map(&tm.z, p.z, p.hz, p.dz, p.tokens) ||
         (p.aux && !make_head_map(&tm.aux, p.aux, p.haux, p.dz, p.tokens))))
        return cudaErrorInvalidValue;
    if (p.state_only) return launch_as<kStateOnly>(tm, p, max_units, stream);
    if (p.dot) return launch_as<kDot>(tm, p, max_units, stream);
    return launch_as<kPlain>(tm, p, max_units, stream);
}

}  // namespace gdn
