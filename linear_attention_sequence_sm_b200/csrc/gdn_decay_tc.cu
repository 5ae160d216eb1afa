// gdn_decay_tc.cu -- the decayed linear attention's pass on the tensor cores
// (bf16, head sizes a multiple of 8 up to 128), see gdn_decay.cuh for the
// pass and its operands x, y, z, out.
//
// Chunk of 64 tokens; every product is one tcgen05.mma stream with fp32
// accumulators in tensor memory:
//   (QK) x y^T               64 x 64 x dy    -> P = QK . decay mask, bf16
//   (KV) L = (w z)^T y       128 x dy x 64   -> Sigma <- e^G Sigma + L
//   (X1) X1 = Sigma x^T      128 x 64 x dy   bf16 copies of Sigma times x
//   (X2) X2 = z^T P^T        128 x 64 x 64
// out^T = X2 + w_in X1.  x, y, z come by TMA as 128-byte-swizzled tiles and
// serve as the K-major and MN-major operands they are; head sizes below 128
// are padded with zeros by TMA.  (w z)^T and the copies of Sigma are A
// operands in tensor memory: operands read from shared memory are what the
// products wait for (12 products of 128 x 128 x 16 take 1450 cycles with both
// operands there, 1040 with one), and what shared memory holds goes to a
// third tile of x, y and z, loaded two chunks ahead -- or, in the dot pass
// backward in time, to the chunk's start state (64 KB), which its state warps
// multiply with dS while X1 runs (read from global memory by these warps: 358
// us; by the out warps, with Sigma from its copies: 500; from shared memory:
// 276).
//
// Sigma itself lives in the state warps' registers, so that L's products need
// nothing from the chunk before: the chain from chunk to chunk is one
// multiply-add per element, its rounded copy, and X1.
//
// Precision.  The state is fp32 in and out, so w z is split into three bf16
// terms (24 bits; one term would leave 2^-9 of the state, two 2^-17).  For
// `dot` passes, whose products with the start state feed the decays' fp32
// gradient, Sigma's copy is split into three terms as well; otherwise X1 ends
// in a bf16 output, and one bf16 copy costs it as much as the output's own
// rounding.  P is one bf16 term for the same reason.  An infinity in z leaves
// NaN in the state (its terms are inf and inf - inf).
//
// Roles (8 warpgroups; a role's warps are latency-bound, so the work is spread
// until the products set the pace):
//   0-7     state      two warps per tensor-memory quarter, 64 columns each
//   8-15    out        X1, X2 -> out (and the dot with aux), 32 tokens a warpgroup
//   16-23   split      w z in three terms, 16 tokens at a time, the warpgroups in turn (8-23 where there is no out)
//   24-27   mask       P from QK
//   28 TMA loads, 29 issues X1, X2 and QK, 30 decays, 31 issues KV
// The registers go where the state is (setmaxnreg).  A chunk's products are 32
// instructions with a dozen waits and commits between them; issued by one
// thread these took 3300 cycles a chunk, more than the products themselves.
//
// Chains run side by side, each bound by its own hand-overs: KV(n) -> L read by
// the state warps -> KV(n + 1); QK(n) -> P(n) -> X2(n); X1(n), X2(n) -> out.
// What tensor memory has room for is buffered: X2 twice in plain passes (QK
// takes the columns of its chunk's X2 and runs a chunk ahead), L twice in
// passes for the state alone, w z in quarters of a chunk, four or (with three
// copies of Sigma) two.
//
// Measured on a B200, 4 x 4096 tokens, 32 heads, d = 128 (128 units, 64 chunks
// each): 127 us plain, 231 us with dots and fp32 out (dq) and 284 us backward
// in time (dk); 65,536 x 48 heads: 335 us for the states at the cuts and 635 us
// for the outputs.  A plain chunk
// takes about 3900 cycles, its products 2060 of them (tensor pipe 33 % busy
// over all SMs, 40 % where 148 are used); DRAM traffic is what the operands
// are.  So the bound is latency: hand-overs between roles, and issue slots
// (some 8000 warp instructions a chunk).  With dots, X1 is three times as
// long, tensor memory has no room to double X2 or X1, and a chunk takes 7300.
// One kernel is compiled for each kind, direction and output type: a choice
// made at run time in these loops cost 5 % of a dot pass.  Registers moved
// from the state to the out warps of dot passes (88 and 80) or the other way
// (104 and 64) took the whole backward from 896 to 946 and 915 us; out warps
// that read all of X1 and X2 before using them, 992 us (spills).
// All hand-overs are mbarriers with bounded waits; a timeout records
// GDN_ERR_DEVICE_CHECK (bad_index -2).  A CTA takes units (segment, head) with
// a stride of the grid; nothing synchronises it between units.
#include <algorithm>

#include "gdn_decay.cuh"
#include "gdn_f32x2.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
using namespace sm100;

namespace {

constexpr int kThreads = 1024;
constexpr int kWarpOut = 8, kWarpSplit = 16, kWarpMask = 24, kWarpTma = 28, kWarpMma = 29, kWarpGate = 30, kWarpKv = 31;
constexpr int kBarOut = 1, kBarSplit = 3;  // named barriers (128 threads each; one for each out and split warpgroup)
// Registers a thread: 64 at launch, then by role; the sum over the eight
// warpgroups is what the block was launched with.
constexpr int kRegsLaunch = 64, kRegsState = 96, kRegsOut = 72, kRegsWork = 48, kRegsCtl = 32;
static_assert(128 * (2 * kRegsState + 2 * kRegsOut + 3 * kRegsWork + kRegsCtl) <= kThreads * kRegsLaunch, "registers");
constexpr uint32_t kTile = 16384, kAtom = 8192, kPTile = 8192;
constexpr uint32_t kTmemCols = 512;

// token vectors of a chunk (floats): prefix sums in log2 units, the output's
// and the state operand's weights, e^G of the whole chunk
constexpr int kVecG = 0, kVecIn = 64, kVecSt = 128, kVecGamma = 192, kVecFloats = 196;

// kKind: what a pass leaves out or adds
enum { kPlain = 0, kDot = 1, kStateOnly = 2 };
constexpr uint32_t kStage = 2304;  // an out warp's staging: 32 rows of 64 bytes, or 16 rows of 36 floats

template <int kKind, bool kRev> struct Cfg {
    // Dot passes also keep the start state of every chunk (forward in time) or multiply with it (backward, from a
    // buffer that takes a tile of each ring; a dot pass's chunks are long enough for two).
    static constexpr bool kKeepStarts = kKind == kDot && !kRev, kSpans = kKind == kDot && kRev;
    static constexpr uint32_t kRing = kSpans ? 2 : 3;            // tiles of x, y and z
    static constexpr uint32_t kAuxRing = kSpans ? 1 : 2;         // of aux
    static constexpr int kCopies = kKind == kDot ? 3 : 1;        // bf16 terms of Sigma's copy
    static constexpr int kBufs = kKind == kDot ? 1 : 2;          // of X2 and QK
    static constexpr int kQuarters = kKind == kDot ? 2 : 4;      // of w z
    // shared memory, from a 1024-byte-aligned base
    static constexpr uint32_t kOffX = 0;
    static constexpr uint32_t kOffZ = kOffX + kRing * kTile;
    static constexpr uint32_t kOffY = kOffZ + kRing * kTile;
    static constexpr uint32_t kOffAux = kOffY + kRing * kTile;                     // kDot only
    static constexpr uint32_t kOffStart = kOffAux + (kKind == kDot ? kAuxRing * kTile : 0);  // kSpans only
    static constexpr uint32_t kOffP = kOffStart + (kSpans ? 4 * kTile : 0);        // [2]
    static constexpr uint32_t kOffOut = kOffP + 2 * kPTile;                        // kStage bytes an out warp
    static constexpr uint32_t kOffVec = kOffOut + 8 * kStage;                           // [4]
    static constexpr uint32_t kOffRed = kOffVec + 4 * kVecFloats * 4;              // [4 warps][64]
    static constexpr uint32_t kOffBar = kOffRed + 1024;
    static constexpr uint32_t kSmem = kOffBar + 464 + 1024;
    static_assert(kSmem <= 232448, "shared memory over the sm_100 per-block limit");
    // tensor memory columns
    // L (two for the state alone); quarters of w z (8 columns a term); the copies of Sigma (64 columns a term);
    // X1; X2 or QK (64 each)
    static constexpr uint32_t kColL = 0, kColW = kKind == kStateOnly ? 256 : 128, kColC = kColW + 24 * kQuarters;
    static constexpr uint32_t kColX1 = kColC + 64 * kCopies, kColX2 = kColX1 + 64;
    static_assert(kKind == kStateOnly || kColX2 + 64 * kBufs <= kTmemCols, "tensor memory");
    // columns and barrier phases of chunk m
    static __device__ __forceinline__ uint32_t buf(uint32_t m) { return kBufs == 2 ? (m & 1u) : 0u; }
    static __device__ __forceinline__ uint32_t phase(uint32_t m) { return (kBufs == 2 ? m >> 1 : m) & 1u; }
    static __device__ __forceinline__ uint32_t col_x2(uint32_t m) { return kColX2 + 64u * buf(m); }
    static __device__ __forceinline__ uint32_t aux(uint32_t m) { return m % kAuxRing; }
    static __device__ __forceinline__ uint32_t aux_turn(uint32_t m) { return m / kAuxRing; }
    // quarter q of chunk m: its buffer, and which use of it this is
    static __device__ __forceinline__ uint32_t qbuf(uint32_t q) { return kQuarters == 4 ? q : q & 1u; }
    static __device__ __forceinline__ uint32_t qturn(uint32_t m, uint32_t q) { return kQuarters == 4 ? m : 2 * m + (q >> 1); }
    static __device__ __forceinline__ uint32_t lbuf(uint32_t m) { return kKind == kStateOnly ? (m & 1u) : 0u; }
    static __device__ __forceinline__ uint32_t lphase(uint32_t m) { return (kKind == kStateOnly ? m >> 1 : m) & 1u; }
    static __device__ __forceinline__ uint32_t col_l(uint32_t m) { return kColL + 128u * lbuf(m); }
};

// mbarriers
enum {
    kBX = 0,        // [3] x landed (one barrier a tile of the ring)
    kBZ = 3,        // [3] z
    kBY = 6,        // [3] y
    kBA = 9,        // [2] aux
    kBXFree = 11,   // [3] X1 (and QK) of the slot's chunk done
    kBZFree = 14,   // [3] X2 done, w z taken (every split warp)
    kBYFree = 17,   // [3] KV done, QK done
    kBAFree = 20,   // [2] dot taken (8 out warps)
    kBW = 22,       // [4] a quarter of w z written (4 split warps)
    kBKq = 26,      // [4] its KV done
    kBKV = 30,      // [2] KV done (and an arrival of the issuing thread, which orders the token vectors)
    kBLFree = 32,   // [2] L read (8 state warps)
    kBSt = 34,      // copies of Sigma written (8 state warps)
    kBX1 = 35,      // X1 done
    kBQK = 36,      // [2] QK done
    kBP = 38,       // [2] P written (4 mask warps)
    kBPFree = 40,   // [2] X2 done
    kBOut = 42,     // X1, X2 done (and an arrival of the issuing thread)
    kBOutFree = 43, // X1, X2 read (8 out warps)
    kBVec = 44,     // [4] token vectors written
    kBVecFree = 48, // [4] token vectors read (8 state warps, 8 out warps)
    kBX2Free = 52,  // X2 read (8 out warps; where QK needs its columns)
    kBDrain = 53,
    kBStart = 54,     // the chunk's start state landed
    kBStartFree = 55, // and multiplied (8 state warps)
    kNumBars = 56
};

struct Maps {
    CUtensorMap x, y, z, aux;
};

// The units of this CTA, one after the other.
template <bool kRev> struct UnitWalk {
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
            first = kRev ? seg.pos + seg.len == seg.seq_len : seg.pos == 0;
            last = kRev ? seg.pos == 0 : seg.pos + seg.len == seg.seq_len;
            if (!(state_only && (seg.slot < 0 || last))) return true;
        }
    }
    // first token of the n-th chunk in pass order, from the segment's start
    __device__ int chunk_at(int n) const { return kDecayChunk * (kRev ? nch - 1 - n : n); }
};

// The start state of the chunk that begins at token t, as the state warps hold
// it: 64 columns a thread as 16 pieces of 16 bytes, the threads' first pieces
// one after the other, then their second, and so on.
__device__ __forceinline__ float *start_slot(const DecayPass &a, int t, int h, int ya) {
    return a.starts + (size_t(t / kDecayChunk) * a.hv + h) * size_t(8192 * ya);
}

// A bounded wait that leaves the issue slots to the others: the thread is
// suspended until the phase completes or kIdleNs pass.
constexpr uint32_t kIdleNs = 1000000;
__device__ __forceinline__ bool idle_wait(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < 2000; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(kIdleNs)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// A bounded wait of a whole warp; every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, idle_wait(bar, parity));
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Rows 16 (warp % 4) + lane % 16 of an M = 64 accumulator: 16 columns from
// `taddr` in lanes 0-15, the 16 columns 32 further on in lanes 16-31.
__device__ __forceinline__ void tmem_ld_m64(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16], 32;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 columns of 16 lanes in fragments: registers 4 j .. 4 j + 3 hold columns
// 8 j + 2 (lane % 4) and the next, of lane / 4 and of lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// 8 columns of 16 lanes: column lane % 4 of lane / 4 (a) and of lane / 4 + 8
// (b), and four columns further (c, d).
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// x minus the two bf16 values of w (exact where w is x rounded).
__device__ __forceinline__ f32x2 sub_bf16x2(f32x2 x, uint32_t w) { return fma2(from_bf16x2(w), both(-1.f), x); }
// Consecutive 32-bit columns of this thread's lane, written (raw bits).
__device__ __forceinline__ void tmem_st_words(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_words(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Four 8 x 8 tiles of 16-bit values, transposed on the way: lane l gives the
// address of row l % 8 of tile l / 8, and holds elements (row 2 (l % 4) and
// the next, column l / 4) of each tile.
__device__ __forceinline__ void ldmatrix_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <int kRegs> __device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs> __device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
__device__ __forceinline__ void stmatrix_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ float tmem_ld_1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    tmem_wait_ld();
    return __uint_as_float(r);
}

// An out warp's 32 tokens (from 32 part) x 32 z columns (from z0) once more,
// where X2 is not finite: a zero of P times an infinity or a NaN of z is NaN,
// so z at one token reaches tokens before it (behind it, backward in time) that
// it has nothing to do with.  Those are summed here over the pairs inside the
// mask alone, x, y and z read from global memory, X1 from tensor memory (column
// x1).  The other tokens keep what the products gave, which is not finite.
// Kept short (nothing unrolled) and out of the way: it stands in the out warps'
// loop, and unrolled it cost dq's pass 30 us without ever running.
template <bool kRev, bool kF32>
__device__ __forceinline__ void redo_tile(const DecayPass &a, const UnitWalk<kRev> &w, int t0, int L, int part, int z0, int lane,
                                          uint32_t x1, const float *vec, uint32_t stage) {
    const int hv = a.hv, zc = z0 + lane;
    const size_t tok = size_t(w.seg.start) + t0;
    auto rows = [&](const void *p, int heads, int d) {
        return static_cast<const __nv_bfloat16 *>(p) + (tok * heads + w.h / (hv / heads)) * size_t(d);
    };
    const __nv_bfloat16 *x = rows(a.x, a.hx, a.dy), *y = rows(a.y, a.hy, a.dy), *z = rows(a.z, a.hz, a.dz) + zc;
    const size_t xs = size_t(a.hx) * a.dy, ys = size_t(a.hy) * a.dy, zs = size_t(a.hz) * a.dz;
    int edge = kRev ? -1 : kDecayChunk;  // the first (backward: last) token whose z is not finite
    if (zc < a.dz)
#pragma unroll 1
        for (int c = 0; c < L; ++c)
            if (!isfinite(to_f32(z[c * zs]))) edge = kRev ? c : min(edge, c);
    const bool none = edge < 0 || edge == kDecayChunk;
#pragma unroll 1
    for (int r = 32 * part; r < min(L, 32 * part + 32); ++r) {
        const bool mine = zc < a.dz && !none && (kRev ? r > edge : r < edge);
        if (!__any_sync(0xffffffffu, mine)) continue;
        float o = vec[kVecIn + r] * tmem_ld_1(x1 + uint32_t(r));
#pragma unroll 1
        for (int c = kRev ? r : 0; c < (kRev ? L : r + 1); ++c) {
            float p = 0.f;
#pragma unroll 1
            for (int e = lane; e < a.dy; e += 32) p = fmaf(to_f32(x[r * xs + e]), to_f32(y[c * ys + e]), p);
#pragma unroll 1
            for (int m = 16; m > 0; m >>= 1) p += __shfl_xor_sync(0xffffffffu, p, m);
            p *= exp2f(kRev ? vec[kVecG + c] - vec[kVecG + r] : vec[kVecG + r] - vec[kVecG + c]);
            if (mine) o = fmaf(to_f32(__float2bfloat16_rn(p)), to_f32(z[c * zs]), o);  // (P as the products have it)
        }
        if (mine && kF32) static_cast<float *>(a.out)[((tok + r) * hv + w.h) * a.dz + zc] = o;
        const uint32_t rr = uint32_t(r - 32 * part);
        if (mine && !kF32) st_shared_b16(stage + rr * 64 + (((uint32_t(lane) >> 3) ^ ((rr >> 1) & 3)) << 4) + 2 * (lane & 7), o);
    }
}

template <int kKind, bool kRev, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
decay_pass_tc_kernel(const __grid_constant__ Maps tm, const DecayPass a) {
    using K = Cfg<kKind, kRev>;
    constexpr uint32_t kRing = K::kRing;
    constexpr bool kDots = kKind == kDot, kSt = kKind == kStateOnly;
    constexpr bool kKeepStarts = K::kKeepStarts, kSpans = K::kSpans;
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
            if ((i >= kBW && i < kBW + 4) || i == kBP || i == kBP + 1) n = 4;
            if (i == kBSt || i == kBLFree || i == kBLFree + 1 || i == kBOutFree || i == kBX2Free || i == kBAFree ||
                i == kBAFree + 1 || i == kBStartFree)
                n = 8;
            if (i == kBOut || i == kBKV || i == kBKV + 1) n = 2;
            if (i >= kBZFree && i < kBZFree + int(kRing)) n = kSt ? 16 : 9;  // (each split warp once a chunk)
            if (i >= kBYFree && i < kBYFree + int(kRing)) n = kSt ? 1 : 2;
            if (i == kBDrain) n = 2;
            if (i >= kBVecFree && i < kBVecFree + 4) n = kSt ? 8 : 16;
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
    UnitWalk<kRev> w(a, !ok);
    const bool dead = !ok;
    uint32_t m = 0;  // chunks this CTA has processed

    if (warp < kWarpOut) {
        // ==================== state warps: thread = state row, 64 columns in registers ====================
        regs_up<kRegsState>();
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t trow = tmem + (uint32_t((warp & 3) * 32) << 16);
        const int c0 = 64 * half;
        const bool mine = half < ya;
        const bool zin = row < dz;
        float S[64];
        while (ok && w.next(kSt)) {
            const size_t sbase = (size_t(w.seg.seq) * hv + w.h) * dz * dy;
#pragma unroll
            for (int j = 0; j < 64; ++j) S[j] = 0.f;
            if (mine && zin && !kSt) {  // the start state
                const float *src = nullptr;
                bool tr = false;
                int ld = 0;
                if (w.seg.slot >= 0) {
                    src = a.seg_state + (size_t(w.seg.slot) * hv + w.h) * 16384;
                    tr = a.seg_trans;
                    ld = 128;
                } else if (a.s_in && w.first) {
                    src = a.s_in + sbase;
                    tr = a.s_trans;
                    ld = tr ? dz : dy;
                }
                if (src && tr) {
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (c0 + j < dy) S[j] = src[size_t(c0 + j) * ld + row];
                } else if (src) {
#pragma unroll
                    for (int j = 0; j < 64; j += 4)  // dy and ld are multiples of 8
                        if (c0 + j < dy) load4(src + size_t(row) * ld + c0 + j, S + j);
                }
            }
            float dec = 1.f;
            for (int n = 0; n < w.nch; ++n) {
                const uint32_t mm = m + uint32_t(n);
                if constexpr (!kSt) {
                    // the copies of Sigma, once the previous X1 has read its own
                    if (mm > 0) ok = warp_wait(bar(kBX1), (mm - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    if (mine) {
                        const uint32_t ca = trow + K::kColC + uint32_t(c0 / 2);
constexpr int kW = K::kCopies == 1 ? 8 : 4;  // words of a slice (fewer where its terms take registers too)
#pragma unroll
                        for (int q = 0; q < 32 / kW; ++q) {
                            uint32_t pk[kW];
                            f32x2 r[kW];
#pragma unroll
                            for (int j = 0; j < kW; ++j) {
                                r[j] = pair(S[2 * (kW * q + j)], S[2 * (kW * q + j) + 1]);
                                pk[j] = to_bf16x2(r[j]);
                            }
                            tmem_st_words(ca + kW * q, pk);
#pragma unroll
                            for (int t = 1; t < K::kCopies; ++t) {
#pragma unroll
                                for (int j = 0; j < kW; ++j) {
                                    r[j] = sub_bf16x2(r[j], pk[j]);
                                    pk[j] = to_bf16x2(r[j]);
                                }
                                tmem_st_words(ca + 64 * t + kW * q, pk);
                            }
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBSt));
                }
                if (kKeepStarts && mine && w.seg.pos + w.chunk_at(n) > 0) {
                    float4 *st = reinterpret_cast<float4 *>(start_slot(a, w.seg.start + w.chunk_at(n), w.h, ya)) + tid;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        st[j * 128 * ya] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
                }
                float span = 0.f;  // <Sigma at the chunk's end, the state at its start>, while X1 runs
                if constexpr (kSpans) {
                    ok = warp_wait(bar(kBStart), mm & 1u);
                    if (!ok) break;
                    if (mine && w.seg.pos + w.chunk_at(n) > 0) {
                        const float4 *st = reinterpret_cast<const float4 *>(smem + K::kOffStart) + tid;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float4 x = st[j * 128 * ya];
                            span = fmaf(x.x, S[4 * j], fmaf(x.y, S[4 * j + 1], fmaf(x.z, S[4 * j + 2], fmaf(x.w, S[4 * j + 3], span))));
                        }
                    } else if (mine && a.s_first && zin) {  // the initial state, stored [y][z] (s_trans)
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (c0 + j < dy) span = fmaf(a.s_first[sbase + size_t(c0 + j) * dz + row], S[j], span);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBStartFree));
                }
                ok = warp_wait(bar(kBKV + int(K::lbuf(mm))), K::lphase(mm));
                if (!ok) break;
                tc_fence_after();
                const float gamma = vecs(mm)[kVecGamma];
                if (mine) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float v[16];
                        tmem_ld16(trow + K::col_l(mm) + uint32_t(c0 + 16 * q), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const f32x2 r = fma2(both(gamma), pair(S[16 * q + j], S[16 * q + j + 1]), pair(v[j], v[j + 1]));
                            S[16 * q + j] = lo_of(r);
                            S[16 * q + j + 1] = hi_of(r);
                        }
                    }
                }
                dec *= gamma;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(kBLFree + int(K::lbuf(mm))));
                    mbar_arrive(bar(kBVecFree + int(mm & 3u)));
                }
                if (kSpans) {
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1) span += __shfl_xor_sync(0xffffffffu, span, s);
                    if (lane == 0)
                        a.span[(size_t(w.seg.chunk + (w.seg.pos + w.chunk_at(n)) / kDecayChunk) * hv + w.h) * 8 + warp] = gamma * span;
                }
            }
            if (!ok) break;
            {
                float *dst = nullptr;
                bool tr = false;
                int ld = 128;
                if constexpr (kSt) {
                    dst = a.seg_local + (size_t(w.seg.slot) * hv + w.h) * 16384;
                    if (tid == 0) a.seg_dec[size_t(w.seg.slot) * hv + w.h] = dec;
                } else if (w.last && a.s_out) {
                    dst = a.s_out + sbase;
                    tr = a.s_trans;
                    ld = tr ? dz : dy;
                }
                if (dst && mine && zin) {
                    if (tr) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (c0 + j < dy) dst[size_t(c0 + j) * ld + row] = S[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 64; j += 4)
                            if (c0 + j < dy)
                                *reinterpret_cast<float4 *>(dst + size_t(row) * ld + c0 + j) =
                                    make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
                    }
                }
            }
            m += uint32_t(w.nch);
        }
    } else if (!kSt && warp < kWarpSplit) {
        // ==================== out warps: 32 z rows each, read in fragments ====================
        regs_up<kRegsOut>();
        if constexpr (!kSt) {
            const int quarter = warp & 3, part = (warp - kWarpOut) >> 2, ot = tid - 32 * kWarpOut - 128 * part;
            const uint32_t tq = tmem + (uint32_t(quarter * 32) << 16);
            const int tp = 2 * (lane & 3);                 // first of this thread's two tokens in a group of 8
            float *red = reinterpret_cast<float *>(smem + K::kOffRed);
            float *stage = reinterpret_cast<float *>(smem + K::kOffOut + (warp - kWarpOut) * kStage);
            const uint32_t stage_u = sb + K::kOffOut + uint32_t(warp - kWarpOut) * kStage;
            while (ok && w.next(false)) {
                for (int n = 0; n < w.nch; ++n) {
                    const uint32_t mm = m + uint32_t(n);
                    const int t0 = w.chunk_at(n), L = min(kDecayChunk, w.seg.len - t0);
                    ok = warp_wait(bar(kBOut), mm & 1u);
                    if (kDots && a.aux) {
                        if (ok) ok = warp_wait(bar(kBA + int(K::aux(mm))), K::aux_turn(mm) & 1u);
                        ok = !named_sync_or(kBarOut + part, 128, !ok);  // the four warps stay together (and `red` was read)
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const float *win = vecs(mm) + kVecIn;
                    const size_t tok = size_t(w.seg.start) + t0;
                    const size_t step = size_t(hv) * dz;
                    const size_t at = (tok * hv + w.h) * dz + 32 * quarter;
                    float y2[kDots ? 2 : 1][2][8];
                    f32x2 all = both(0.f);  // the sum of X2's values: whether all of them are finite
                    bool odd = false;
                    if constexpr (kDots) {
                        // X2 first: QK waits for its columns
#pragma unroll
                        for (int pp = 0; pp < 2; ++pp)
#pragma unroll
                            for (int l = 0; l < 2; ++l)
                                tmem_ld_frag(tq + (uint32_t(16 * l) << 16) + K::col_x2(mm) + 16 * (2 * part + pp), y2[pp][l]);
                        tmem_wait_ld();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kBX2Free));
#pragma unroll
                        for (int pp = 0; pp < 2; ++pp)
#pragma unroll
                            for (int l = 0; l < 2; ++l)
#pragma unroll
                                for (int e = 0; e < 8; e += 2) all = add2(all, pair(y2[pp][l][e], y2[pp][l][e + 1]));
                        odd = __any_sync(0xffffffffu, !isfinite(lo_of(all) + hi_of(all)));
                    }
#pragma unroll(kDots ? 2 : 1)
                    for (int pp = 0; pp < 2; ++pp) {  // 16 tokens (rolled: the roles share the instruction caches)
                        const int p = 2 * part + pp;
                        float x1[2][8], x2[2][8];
#pragma unroll
                        for (int l = 0; l < 2; ++l) {
                            tmem_ld_frag(tq + (uint32_t(16 * l) << 16) + K::kColX1 + 16 * p, x1[l]);
                            if constexpr (kDots) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) x2[l][e] = y2[pp][l][e];
                            } else {
                                tmem_ld_frag(tq + (uint32_t(16 * l) << 16) + K::col_x2(mm) + 16 * p, x2[l]);
                            }
                        }
                        tmem_wait_ld();
                        if constexpr (!kDots) {
#pragma unroll
                            for (int l = 0; l < 2; ++l)
#pragma unroll
                                for (int e = 0; e < 8; e += 2) all = add2(all, pair(x2[l][e], x2[l][e + 1]));
                        }
                        if (pp == 1) {
                            if (!kDots) odd = __any_sync(0xffffffffu, !isfinite(lo_of(all) + hi_of(all)));
                            if (__builtin_expect(!odd, 1)) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(bar(kBOutFree));
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const f32x2 wi = *reinterpret_cast<const f32x2 *>(win + 16 * p + 8 * j + tp);
#pragma unroll
                            for (int l = 0; l < 2; ++l)
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    float *u = &x1[l][4 * j + e], *v = &x2[l][4 * j + e];
                                    const f32x2 a1 = pair(u[0], u[1]), a2 = pair(v[0], v[1]);
                                    f32x2 o2;
                                    if constexpr (kDots) {
                                        const f32x2 w1 = mul2(a1, wi);
                                        u[0] = lo_of(w1);
                                        u[1] = hi_of(w1);
                                        o2 = add2(a2, w1);
                                    } else {
                                        o2 = fma2(a1, wi, a2);
                                    }
                                    v[0] = lo_of(o2);
                                    v[1] = hi_of(o2);
                                }
                        }
                        if constexpr (kDots) {
                            if (a.aux) {
                                float d[4];  // dots of this thread's 4 tokens over its 4 rows
                                const uint32_t aux = sb + K::kOffAux + K::aux(mm) * kTile + uint32_t(quarter >> 1) * kAtom;
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    // tiles: tokens 8 j .. 8 j + 7, z 8 i .. 8 i + 7 of this quarter, i = lane / 8
                                    const uint32_t r = uint32_t(16 * p + 8 * j + (lane & 7));
                                    const uint32_t ch = uint32_t(4 * (quarter & 1) + (lane >> 3));
                                    uint32_t q[4];
                                    ldmatrix_t(aux + r * 128 + ((ch ^ (r & 7)) << 4), q);
                                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        s0 = fmaf(bf_lo(q[i]), x1[i >> 1][4 * j + 2 * (i & 1)], s0);
                                        s1 = fmaf(bf_hi(q[i]), x1[i >> 1][4 * j + 2 * (i & 1) + 1], s1);
                                    }
                                    d[2 * j] = s0;
                                    d[2 * j + 1] = s1;
                                }
                                // sums over the 8 lanes of a token pair: two halving exchanges and a plain one
#pragma unroll
                                for (int c = 2, bit = 16; c >= 1; c >>= 1, bit >>= 1) {
                                    const bool up = (lane & bit) != 0;
#pragma unroll
                                    for (int e = 0; e < c; ++e) {
                                        const float send = up ? d[e] : d[e + c], keep = up ? d[e + c] : d[e];
                                        d[e] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
                                    }
                                }
                                d[0] += __shfl_xor_sync(0xffffffffu, d[0], 4);
                                // lane bit 16 chose the group of 8 tokens, bit 8 the token of the pair
                                if ((lane & 4) == 0)
                                    red[quarter * 64 + 16 * p + 8 * (lane >> 4) + tp + ((lane >> 3) & 1)] = d[0];
                            }
                        }
                        if (!kF32) {
                            // bf16 token pairs, transposed into rows of 64 bytes (four 16-byte pieces, swizzled) per token
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t r = uint32_t(16 * pp + 8 * j + (lane & 7));
                                const uint32_t ch = uint32_t(lane >> 3);
                                stmatrix_t(stage_u + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4),
                                           pack_bf16x2(x2[0][4 * j], x2[0][4 * j + 1]),
                                           pack_bf16x2(x2[0][4 * j + 2], x2[0][4 * j + 3]),
                                           pack_bf16x2(x2[1][4 * j], x2[1][4 * j + 1]),
                                           pack_bf16x2(x2[1][4 * j + 2], x2[1][4 * j + 3]));
                            }
                        } else {
                            // fp32 rows of 36 floats (a token pair's lanes fall into other banks)
                            __syncwarp();
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int l = 0; l < 2; ++l)
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        stage[(8 * j + tp + (e & 1)) * 36 + 16 * l + 8 * (e >> 1) + (lane >> 2)] =
                                            x2[l][4 * j + e];
                            __syncwarp();
                            float *o = static_cast<float *>(a.out) + at;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int r = 4 * i + (lane >> 3), c = 4 * (lane & 7), tk = 16 * p + r;
                                if (tk < L && 32 * quarter + c < dz)
                                    *reinterpret_cast<float4 *>(o + tk * step + c) =
                                        *reinterpret_cast<const float4 *>(stage + r * 36 + c);
                            }
                        }
                    }
                    __syncwarp();
                    if (__builtin_expect(odd, 0)) {
                        redo_tile<kRev, kF32>(a, w, t0, L, part, 32 * quarter, lane, tq + K::kColX1, vecs(mm), stage_u);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kBOutFree));
                    }
                    if (lane == 0) mbar_arrive(bar(kBVecFree + int(mm & 3u)));
                    if (!kF32) {
                        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + at;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t r = uint32_t(8 * i + (lane >> 2)), ch = uint32_t(lane & 3);
                            const uint4 q = ld_shared_v4(stage_u + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
                            const int tk = 32 * part + int(r);
                            if (tk < L && 32 * quarter + 8 * int(ch) < dz)
                                *reinterpret_cast<uint4 *>(o + tk * step + 8 * ch) = q;
                        }
                        __syncwarp();
                    }
                    if (kDots && a.aux) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kBAFree + int(K::aux(mm))));
                        named_sync(kBarOut + part, 128);
                        const int tk = 32 * part + ot;
                        if (ot < 32 && tk < L)
                            a.dot[size_t(w.h) * a.tokens + tok + tk] =
                                (red[tk] + red[64 + tk]) + (red[128 + tk] + red[192 + tk]);
                    }
                }
                m += uint32_t(w.nch);
            }
        }
    } else if (warp < kWarpMask) {
        // ============ split warps: w z of 16 tokens, in three terms ============
        regs_down<kRegsWork>();
        constexpr int kGroups = kSt ? 4 : 2;  // warpgroups at it; quarter q of a chunk is the (q % kGroups)-th's
        const int quarter = warp & 3, grp = ((warp - kWarpSplit) >> 2) & (kGroups - 1), st = tid & 127;
        const uint32_t tw = tmem + (uint32_t(quarter * 32) << 16) + K::kColW;
        const uint32_t ch = uint32_t(4 * (quarter & 1) + (lane >> 3)), r7 = uint32_t(lane & 7);
        const uint32_t src = uint32_t(quarter >> 1) * kAtom + r7 * 128 + ((ch ^ r7) << 4);
        while (w.next(kSt)) {
            for (int n = 0; n < w.nch; ++n) {
                const uint32_t mm = m + uint32_t(n);
                const int L = min(kDecayChunk, w.seg.len - w.chunk_at(n));
                const uint32_t s = mm % kRing, ring_phase = (mm / kRing) & 1u;
                if (ok) ok = warp_wait(bar(kBZ + int(s)), ring_phase) && warp_wait(bar(kBVec + int(mm & 3u)), (mm >> 2) & 1u);
                if (L < kDecayChunk) {
                    // tokens past the end are another sequence's: their y, whatever it holds, must not meet a zero
                    // weight (their z is left out below)
                    if (ok) ok = warp_wait(bar(kBY + int(s)), ring_phase);
                    const uint32_t yt = sb + K::kOffY + s * kTile;
                    for (int e = st; e < 256 * ya && ok; e += 128) {
                        // pieces of 16 bytes: 8 a row, 32 rows (two quarters, of which this group may have one), column
                        // halves
                        const int q = (e >> 7) & 1, r = 16 * (grp % 2 + 2 * q) + ((e >> 3) & 15);
                        if (r >= L && (kGroups == 2 || q == grp / 2))
                            st_shared_v4(yt + uint32_t(e >> 8) * kAtom + uint32_t(r) * 128 + uint32_t(e & 7) * 16,
                                         make_uint4(0u, 0u, 0u, 0u));
                    }
                    fence_proxy_async_shared();
                    // all four warps' rows are written before any of them arrives; they go on, or stop, together
                    if (named_sync_or(kBarSplit + grp, 128, !ok)) {
                        ok = false;
                        goto split_done;
                    }
                }
                if (!ok) continue;  // (on to the next meeting of the four, or out)
                const float *wst = vecs(mm) + kVecSt + 2 * (lane & 3);
                const uint32_t zt = sb + K::kOffZ + s * kTile + src;
#pragma unroll 1
                for (int hf = 0; hf < 4 / kGroups; ++hf) {
                    const uint32_t qq = uint32_t(grp + kGroups * hf), turn = K::qturn(mm, qq);
                    const int t16 = 16 * int(qq);  // the quarter's first token
                    uint32_t w0[2][4], w1[2][4], w2[2][4];  // two groups of 8 tokens; 8-row blocks of z
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // transposed reads give token pairs of a z row, the layout of a tensor-memory A operand
                        uint32_t q[4];
                        ldmatrix_t(zt + 128u * uint32_t(t16 + 8 * j), q);
                        if (L < kDecayChunk) {
                            const int tk = t16 + 8 * j + 2 * (lane & 3);
                            const uint32_t keep = (tk < L ? 0xffffu : 0u) | (tk + 1 < L ? 0xffff0000u : 0u);
#pragma unroll
                            for (int i = 0; i < 4; ++i) q[i] &= keep;
                        }
                        const f32x2 wt = *reinterpret_cast<const f32x2 *>(wst + t16 + 8 * j);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f32x2 x = mul2(from_bf16x2(q[i]), wt);
                            w0[j][i] = to_bf16x2(x);
                            x = sub_bf16x2(x, w0[j][i]);
                            w1[j][i] = to_bf16x2(x);
                            x = sub_bf16x2(x, w1[j][i]);
                            w2[j][i] = to_bf16x2(x);
                        }
                    }
                    if (hf == 4 / kGroups - 1 && lane == 0) mbar_arrive(bar(kBZFree + int(s)));  // (its last read of z)
                    // KV has read these columns' previous quarter
                    if (turn > 0) ok = warp_wait(bar(kBKq + int(K::qbuf(qq))), (turn - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int l = 0; l < 2; ++l) {  // 16 z rows: two columns groups of 8 tokens, two 8-row blocks
                        const uint32_t at = tw + 24u * K::qbuf(qq) + (uint32_t(16 * l) << 16);
                        tmem_st_frag(at, w0[0][2 * l], w0[0][2 * l + 1], w0[1][2 * l], w0[1][2 * l + 1]);
                        tmem_st_frag(at + 8, w1[0][2 * l], w1[0][2 * l + 1], w1[1][2 * l], w1[1][2 * l + 1]);
                        tmem_st_frag(at + 16, w2[0][2 * l], w2[0][2 * l + 1], w2[1][2 * l], w2[1][2 * l + 1]);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBW + int(K::qbuf(qq))));
                }
            }
            m += uint32_t(w.nch);
        }
    split_done:;
    } else if (warp < kWarpTma) {
        // ============ mask warps: P = QK . decay mask ============
        regs_down<kRegsWork>();
        if constexpr (!kSt) {
            const int quarter = warp & 3;
            const uint32_t tq = tmem + (uint32_t(quarter * 32) << 16);
            const int r = 16 * quarter + (lane & 15), cb = lane < 16 ? 0 : 32;
            while (ok && w.next(false)) {
                for (int n = 0; n < w.nch; ++n) {
                    const uint32_t mm = m + uint32_t(n);
                    const int L = min(kDecayChunk, w.seg.len - w.chunk_at(n));
                    const float *G = vecs(mm) + kVecG;
                    ok = warp_wait(bar(kBVec + int(mm & 3u)), (mm >> 2) & 1u);
                    if (ok && mm >= 2) ok = warp_wait(bar(kBPFree + int(mm & 1u)), ((mm >> 1) - 1) & 1u);
                    if (ok) ok = warp_wait(bar(kBQK + int(K::buf(mm))), K::phase(mm));
                    const uint32_t s = mm % kRing;
                    if (ok && L < kDecayChunk) ok = warp_wait(bar(kBZ + int(s)), (mm / kRing) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    if (L < kDecayChunk) {
                        // tokens past the end are another sequence's: their z must not meet P's zeros
                        const uint32_t zt = sb + K::kOffZ + s * kTile;
                        for (int e = 32 * quarter + lane; e < 1024; e += 128)
                            if (((e >> 3) & 63) >= L) st_shared_v4(zt + uint32_t(e) * 16, make_uint4(0u, 0u, 0u, 0u));
                    }
                    const float Gr = G[r];
                    const uint32_t base = sb + K::kOffP + (mm & 1u) * kPTile + uint32_t(r) * 128;
#pragma unroll 1
                    for (int p = 0; p < 2; ++p) {
                        float v[16];
                        tmem_ld_m64(tq + K::col_x2(mm) + 16 * p, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float gc[8], x[8];
                            const int c0 = cb + 16 * p + 8 * q;
                            load4(G + c0, gc);
                            load4(G + c0 + 4, gc + 4);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int c = c0 + j;
                                const bool in = kRev ? (c >= r && c < L) : c <= r;
                                const float d = kRev ? gc[j] - Gr : Gr - gc[j];
                                float e;
                                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d));
                                x[j] = in ? v[8 * q + j] * e : 0.f;
                            }
                            st_shared_v4(base + ((uint32_t(c0 / 8) ^ uint32_t(r & 7)) << 4), pack_bf16x8(x));
                        }
                    }
                    fence_proxy_async_shared();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBP + int(mm & 1u)));
                }
                m += uint32_t(w.nch);
            }
        }
    } else {
        regs_down<kRegsCtl>();
        if (warp == kWarpGate) {
            // ============ decays: prefix and suffix sums (each without a subtraction), their exponentials ============
            while (ok && w.next(kSt)) {
                const float *g = a.g_const ? a.g + w.h : a.g + size_t(w.seg.start) * hv + w.h;
                const size_t gs = a.g_const ? 0 : hv;
                float g0 = 0.f, g1 = 0.f;
                auto load_g = [&](int n) {  // this lane's two tokens of the n-th chunk (floored where they are used)
                    const int t = w.chunk_at(n) + 2 * lane;
                    g0 = t < w.seg.len ? g[size_t(t) * gs] : 0.f;
                    g1 = t + 1 < w.seg.len ? g[size_t(t + 1) * gs] : 0.f;
                };
                if (w.nch > 0) load_g(0);
                for (int n = 0; n < w.nch; ++n) {
                    const uint32_t mm = m + uint32_t(n);
                    float *vec = vecs(mm);
                    const float a0 = floored(g0), a1 = floored(g1);
                    if (n + 1 < w.nch) load_g(n + 1);
                    float pre = a0 + a1, suf = a0 + a1;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const float u = __shfl_up_sync(0xffffffffu, pre, d), v = __shfl_down_sync(0xffffffffu, suf, d);
                        if (lane >= d) pre += u;
                        if (lane + d < 32) suf += v;
                    }
                    float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
                    if (lane == 0) before = 0.f;
                    if (lane == 31) after = 0.f;
                    const float G0 = before + a0, G1 = pre, R0 = a1 + after, R1 = after;
                    const float total = __shfl_sync(0xffffffffu, pre, 31);
                    const float e0 = expf(G0), e1 = expf(G1), f0 = expf(R0), f1 = expf(R1), et = expf(total);
                    constexpr float kLog2e = 1.4426950408889634f;
                    if (mm >= 4) ok = warp_wait(bar(kBVecFree + int(mm & 3u)), ((mm >> 2) - 1) & 1u);
                    if (!ok) break;
                    *reinterpret_cast<float2 *>(vec + kVecG + 2 * lane) = make_float2(G0 * kLog2e, G1 * kLog2e);
                    *reinterpret_cast<float2 *>(vec + kVecIn + 2 * lane) = kRev ? make_float2(f0, f1) : make_float2(e0, e1);
                    *reinterpret_cast<float2 *>(vec + kVecSt + 2 * lane) = kRev ? make_float2(e0, e1) : make_float2(f0, f1);
                    if (lane == 0) vec[kVecGamma] = et;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBVec + int(mm & 3u)));
                }
                m += uint32_t(w.nch);
            }
        } else if (warp == kWarpTma && elect_one()) {
            const uint32_t bytes_y = kAtom * uint32_t(ya);
            while (ok && w.next(kSt)) {
                const int hx = kSt ? 0 : w.h / (hv / a.hx), hy = w.h / (hv / a.hy), hz = w.h / (hv / a.hz);
                const int ha = kDots && a.aux ? w.h / (hv / a.haux) : 0;
                for (int n = 0; n < w.nch; ++n) {
                    const uint32_t mm = m + uint32_t(n);
                    const int tok = w.seg.start + w.chunk_at(n);
                    const uint32_t s = mm % kRing, freed = (mm / kRing - 1) & 1u;
                    const bool wait = mm >= kRing;
                    {
                        const uint32_t dst = sb + K::kOffY + s * kTile, b = bar(kBY + int(s));
                        if (wait) ok = mbar_wait(bar(kBYFree + int(s)), freed);
                        if (!ok) break;
                        mbar_arrive_expect_tx(b, bytes_y);
                        tma_load_3d(dst, &tm.y, 0, hy, tok, b);
                        if (ya == 2) tma_load_3d(dst + kAtom, &tm.y, 64, hy, tok, b);
                    }
                    if constexpr (!kSt) {
                        const uint32_t dst = sb + K::kOffX + s * kTile, b = bar(kBX + int(s));
                        if (wait) ok = mbar_wait(bar(kBXFree + int(s)), freed);
                        if (!ok) break;
                        mbar_arrive_expect_tx(b, bytes_y);
                        tma_load_3d(dst, &tm.x, 0, hx, tok, b);
                        if (ya == 2) tma_load_3d(dst + kAtom, &tm.x, 64, hx, tok, b);
                    }
                    {
                        const uint32_t dst = sb + K::kOffZ + s * kTile, b = bar(kBZ + int(s));
                        if (wait) ok = mbar_wait(bar(kBZFree + int(s)), freed);
                        if (!ok) break;
                        mbar_arrive_expect_tx(b, kTile);
                        tma_load_3d(dst, &tm.z, 0, hz, tok, b);
                        tma_load_3d(dst + kAtom, &tm.z, 64, hz, tok, b);
                    }
                    if constexpr (kSpans) {
                        if (mm > 0) ok = mbar_wait(bar(kBStartFree), (mm - 1) & 1u);
                        if (!ok) break;
                        if (w.seg.pos + w.chunk_at(n) > 0) {
                            mbar_arrive_expect_tx(bar(kBStart), 32768u * uint32_t(ya));
                            bulk_load(sb + K::kOffStart, start_slot(a, tok, w.h, ya), 32768u * uint32_t(ya), bar(kBStart));
                        } else {
                            mbar_arrive(bar(kBStart));  // (the initial state is read where it is)
                        }
                    }
                    if (kDots && a.aux) {
                        const uint32_t i = K::aux(mm), dst = sb + K::kOffAux + i * kTile, b = bar(kBA + int(i));
                        if (mm >= K::kAuxRing) ok = mbar_wait(bar(kBAFree + int(i)), (K::aux_turn(mm) - 1) & 1u);
                        if (!ok) break;
                        mbar_arrive_expect_tx(b, kTile);
                        tma_load_3d(dst, &tm.aux, 0, ha, tok, b);
                        tma_load_3d(dst + kAtom, &tm.aux, 64, ha, tok, b);
                    }
                }
                m += uint32_t(w.nch);
            }
        } else if ((warp == kWarpMma || warp == kWarpKv) && elect_one()) {
        // ==================== the issuing threads ====================
        uint32_t total = 0;
        while (w.next(kSt)) total += uint32_t(w.nch);
        const uint32_t id_qk = idesc_bf16(64, 64, false, false), id_kv = idesc_bf16(128, 64 * ya, false, true);
        const uint32_t id_x1 = idesc_bf16(128, 64, false, false), id_x2 = idesc_bf16(128, 64, true, false);
        auto koff = [](int s) { return uint64_t(((s >> 2) * kAtom + (s & 3) * 32) >> 4); };  // K-major steps
        // the out warps have read chunk c's X1 and X2
        auto out_read = [&](uint32_t c) { return mbar_wait(bar(kBOutFree), c & 1u); };
        auto issue_qk = [&](uint32_t c) {
            const uint32_t s = c % kRing, ph = (c / kRing) & 1u;
            if (!mbar_wait(bar(kBX + int(s)), ph) || !mbar_wait(bar(kBY + int(s)), ph)) return false;
            // (its columns were the X2 of kBufs chunks ago)
            if (kDots ? c > 0 && !mbar_wait(bar(kBX2Free), (c - 1) & 1u) : c > 1 && !out_read(c - 2)) return false;
            tc_fence_after();
            const uint64_t dx = smem_desc(sb + K::kOffX + s * kTile, 16, 1024), dyd = smem_desc(sb + K::kOffY + s * kTile, 16, 1024);
#pragma unroll 1
            for (int j = 0; j < ya; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_bf16(tmem + K::col_x2(c), dx + koff(4 * j) + koff(i), dyd + koff(4 * j) + koff(i), id_qk, i > 0 || j > 0);
            mma_commit(bar(kBQK + int(K::buf(c))));
            mma_commit(bar(kBYFree + int(s)));
            return true;
        };
        auto issue_kv = [&](uint32_t c) {
            const uint32_t s = c % kRing;
            if (!mbar_wait(bar(kBY + int(s)), (c / kRing) & 1u)) return false;
            const uint32_t back = kSt ? 2u : 1u;  // the chunk whose L these columns held
            if (c >= back && !mbar_wait(bar(kBLFree + int(K::lbuf(c))), K::lphase(c - back))) return false;
            const uint64_t db = smem_desc(sb + K::kOffY + s * kTile, 8192, 1024);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                const uint32_t b = K::qbuf(uint32_t(q));
                if (!mbar_wait(bar(kBW + int(b)), K::qturn(c, uint32_t(q)) & 1u)) return false;
                tc_fence_after();
                const uint32_t col = tmem + K::kColW + 24u * b;
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    mma_bf16_ts(tmem + K::col_l(c), col + 8 * t, db + uint64_t((q * 2048) >> 4), id_kv, q > 0 || t > 0);
                mma_commit(bar(kBKq + int(b)));
            }
            mma_commit(bar(kBKV + int(K::lbuf(c))));
            mbar_arrive(bar(kBKV + int(K::lbuf(c))));
            mma_commit(bar(kBYFree + int(s)));
            return true;
        };
        auto issue_x1 = [&](uint32_t c) {
            const uint32_t s = c % kRing;
            if (!mbar_wait(bar(kBSt), c & 1u)) return false;
            if (c > 0 && !out_read(c - 1)) return false;
            tc_fence_after();
            const uint64_t dx = smem_desc(sb + K::kOffX + s * kTile, 16, 1024);
#pragma unroll 1
            for (int j = 0; j < 2 * K::kCopies; ++j) {
                if ((j & 1) >= ya) continue;  // (j & 1: 64 columns of y; j / 2: term)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_bf16_ts(tmem + K::kColX1, tmem + K::kColC + 32 * j + 8 * i, dx + koff(4 * (j & 1)) + koff(i), id_x1,
                                j > 0 || i > 0);
            }
            mma_commit(bar(kBX1));
            mma_commit(bar(kBXFree + int(s)));
            return true;
        };
        auto issue_x2 = [&](uint32_t c) {
            const uint32_t s = c % kRing;
            if (!mbar_wait(bar(kBP + int(c & 1u)), (c >> 1) & 1u)) return false;
            if (!mbar_wait(bar(kBZ + int(s)), (c / kRing) & 1u)) return false;
            tc_fence_after();
            const uint64_t da = smem_desc(sb + K::kOffZ + s * kTile, 8192, 1024);
            const uint64_t db = smem_desc(sb + K::kOffP + (c & 1u) * kPTile, 16, 1024);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_bf16(tmem + K::col_x2(c), da + uint64_t((i * 2048) >> 4), db + uint64_t((i * 32) >> 4), id_x2, i > 0);
            mma_commit(bar(kBOut));
            mbar_arrive(bar(kBOut));
            mma_commit(bar(kBZFree + int(s)));
            mma_commit(bar(kBPFree + int(c & 1u)));
            return true;
        };
        if (warp == kWarpKv) {
            for (uint32_t c = 0; ok && c < total; ++c) ok = issue_kv(c);
        } else if constexpr (kKind == kPlain) {
            // QK a chunk ahead
            if (total > 0) ok = ok && issue_qk(0);
            for (uint32_t c = 0; ok && c < total; ++c)
                ok = (c + 1 == total || issue_qk(c + 1)) && issue_x1(c) && issue_x2(c);
        } else if constexpr (kDots) {
            if (total > 0) ok = ok && issue_qk(0);
            for (uint32_t c = 0; ok && c < total; ++c)
                ok = issue_x1(c) && issue_x2(c) && (c + 1 == total || issue_qk(c + 1));
        }
        // every product done before the tensor memory goes
        mma_commit(bar(kBDrain));
        if (!mbar_wait(bar(kBDrain), 0u)) ok = false;
        }
    }
    if (!ok && !dead) {
        a.sched.hdr->bad_index = -2;
        atomicExch(&a.sched.hdr->status, int(GDN_ERR_DEVICE_CHECK));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int kKind, bool kRev, bool kF32>
cudaError_t launch_as(const Maps &tm, const DecayPass &p, int64_t max_units, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(decay_pass_tc_kernel<kKind, kRev, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(Cfg<kKind, kRev>::kSmem));
    if (e != cudaSuccess) return e;
    static const int regs = [] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, decay_pass_tc_kernel<kKind, kRev, kF32>) == cudaSuccess ? fa.numRegs : -1;
    }();
    if (regs != kRegsLaunch) return cudaErrorInvalidKernelImage;  // the roles' registers are dealt out of these
    const int sms = device_sm_count(nullptr);
    if (sms <= 0) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(max_units, sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<kKind, kRev>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, decay_pass_tc_kernel<kKind, kRev, kF32>, tm, p);
    count_launch();
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <int kKind>
cudaError_t launch_out(const Maps &tm, const DecayPass &p, int64_t max_units, cudaStream_t stream) {
    if (p.reverse)
        return p.out_f32 ? launch_as<kKind, true, true>(tm, p, max_units, stream)
                         : launch_as<kKind, true, false>(tm, p, max_units, stream);
    return p.out_f32 ? launch_as<kKind, false, true>(tm, p, max_units, stream)
                     : launch_as<kKind, false, false>(tm, p, max_units, stream);
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
    if (p.state_only)
        return p.reverse ? launch_as<kStateOnly, true, false>(tm, p, max_units, stream)
                         : launch_as<kStateOnly, false, false>(tm, p, max_units, stream);
    return p.dot ? launch_out<kDot>(tm, p, max_units, stream) : launch_out<kPlain>(tm, p, max_units, stream);
}

}  // namespace gdn
