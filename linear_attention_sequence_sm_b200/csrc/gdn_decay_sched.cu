// gdn_decay_sched.cu -- the decayed linear attention's plan and its small
// kernels: the segment table, the start states of cut sequences, the decays'
// gradient from its parts, and sums over grouped heads.
#include <algorithm>

#include "gdn_decay.cuh"

namespace gdn {

namespace {

constexpr int kSchedThreads = 1024;
// Above this many sequences the longest-first ranking (quadratic in N) is
// skipped and sequences keep their given order.
constexpr int kMaxRankedSeqs = 8192;

// Tokens times heads each of `ways` CTAs takes when the work is spread evenly.
__host__ __device__ inline int64_t balanced_tokens(int64_t tokens, int hv, int ways) {
    return (tokens * hv + ways - 1) / ways;
}

// How finely a pass is cut: a tensor-core CTA has an SM to itself, of the
// CUDA-core pass's blocks two share one.
struct DecayPlan {
    int ways, min_seg;
};
inline DecayPlan plan_of(const gdn_shape_t &s) {
    return decay_tc_supported(s) ? DecayPlan{kDecayPlanSms, kDecayMinSeg} : DecayPlan{2 * kDecayPlanSms, kDecayMinSeg / 2};
}

// Whether any sequence may be cut: the longest has at most seq_len tokens (all
// of them, with cu_seqlens).
inline bool may_split(const gdn_shape_t &s) {
    const DecayPlan p = plan_of(s);
    return s.seq_len > p.min_seg &&
           s.seq_len >= 2 * balanced_tokens(int64_t(s.batch) * s.seq_len, s.num_v_heads, p.ways);
}

// Exclusive prefix sums over the block of kN values per thread; totals gets the sums.
template <int kN>
__device__ void block_scan(int (&v)[kN], int (&totals)[kN], int *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int mine[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        mine[j] = v[j];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, mine[j], d);
            if (lane >= d) mine[j] += u;
        }
        if (lane == 31) part[32 * j + warp] = mine[j];
    }
    __syncthreads();
    if (warp < kN) {
        int x = part[32 * warp + lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += u;
        }
        part[32 * warp + lane] = x;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        totals[j] = part[32 * j + 31];
        v[j] = mine[j] - v[j] + (warp ? part[32 * j + warp - 1] : 0);
    }
    __syncthreads();
}

// Checks cu_seqlens and writes the segment table, longest sequences first.
// A sequence is a chain of dependent chunks, so a call with few sequences and
// heads would leave SMs idle: with B = tokens * Hv / ways (a perfect spread) and
// the longest sequence at least 2 B, sequences are cut into segments of
// ceil(longest / floor(longest / B)) tokens, rounded up, whose start states come from a
// first sweep over all segments but one end's (k and v are then read twice, a
// third of the prefill's traffic; the uncut chain would take at least twice as
// long).  At 1 x 65,536 tokens and 48 heads: 3 segments of 21,888 tokens.
// Below 2 B nothing is cut, and units go to CTAs with a fixed stride: 160 equal
// units on 148 SMs take two chains' time, 96 leave 52 SMs idle.
__global__ void __launch_bounds__(kSchedThreads)
decay_schedule_kernel(int32_t num_seqs, int32_t tokens, int32_t batched_len, int32_t hv, DecayPlan plan,
                      const int32_t *__restrict__ cu, DecaySched sc, int32_t *order) {
    __shared__ int bad, longest;
    __shared__ int part[96];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    DecayHeader *hdr = sc.hdr;
    if (threadIdx.x == 0) {
        bad = -1;
        longest = 0;
        hdr->status = GDN_OK;
        hdr->bad_index = -1;
        hdr->num_segs = hdr->num_split = hdr->total_chunks = 0;
        hdr->seg_len = 0;
    }
    __syncthreads();
    auto start_of = [&](int n) { return cu ? cu[n] : n * batched_len; };
    auto len_of = [&](int n) { return cu ? cu[n + 1] - cu[n] : batched_len; };
    int most = 0;
    for (int n = threadIdx.x; n < num_seqs; n += blockDim.x) {
        if (cu) {
            const int s0 = cu[n], s1 = cu[n + 1];
            const bool ok = s1 >= s0 && s0 >= 0 && s1 <= tokens && (n != 0 || s0 == 0) &&
                            (n != num_seqs - 1 || s1 == tokens);
            if (!ok) atomicMax(&bad, n);
        }
        most = max(most, len_of(n));
    }
    atomicMax(&longest, most);
    __syncthreads();
    if (bad >= 0) {
        if (threadIdx.x == 0) {
            hdr->status = GDN_ERR_DEVICE_CHECK;
            hdr->bad_index = bad;
        }
        return;
    }
    // segment length: whole chunks
    int seg_len = INT32_MAX;
    {
        const int64_t balanced = balanced_tokens(tokens, hv, plan.ways);
        const int64_t k = balanced > 0 ? longest / balanced : 1;
        if (k >= 2 && longest > plan.min_seg) {
            int64_t L = (longest + k - 1) / k;
            L = max(int64_t(plan.min_seg), (L + kDecayChunk - 1) / kDecayChunk * kDecayChunk);
            seg_len = int(L);
        }
    }
    // longest first, ties by index
    const bool rank_it = cu != nullptr && num_seqs <= kMaxRankedSeqs;
    for (int n = threadIdx.x; n < num_seqs; n += blockDim.x) {
        int r = n;
        if (rank_it) {
            const int ln = len_of(n);
            r = 0;
            for (int m = 0; m < num_seqs; ++m) {
                const int lm = len_of(m);
                r += (lm > ln) || (lm == ln && m < n);
            }
        }
        order[r] = n;
    }
    // chunks before each sequence: each thread takes a run of sequences
    const int per = (num_seqs + kSchedThreads - 1) / kSchedThreads;
    const int n0 = min(num_seqs, int(threadIdx.x) * per), n1 = min(num_seqs, n0 + per);
    int one[1] = {0}, total1[1];
    for (int n = n0; n < n1; ++n) one[0] += (len_of(n) + kDecayChunk - 1) / kDecayChunk;
    block_scan(one, total1, part);
    int chunks = one[0];
    for (int n = n0; n < n1; ++n) {
        sc.chunk_base[n] = chunks;
        chunks += (len_of(n) + kDecayChunk - 1) / kDecayChunk;
    }
    __syncthreads();  // order, chunk_base
    // segments, sequences by rank
    auto segs_of = [&](int n) { return len_of(n) <= seg_len ? 1 : (len_of(n) + seg_len - 1) / seg_len; };
    int three[3] = {0, 0, 0}, total3[3];
    for (int r = n0; r < n1; ++r) {
        const int c = segs_of(order[r]);
        three[0] += c;
        three[1] += c > 1;
        three[2] += c > 1 ? c : 0;
    }
    block_scan(three, total3, part);
    int segs = three[0], cut = three[1], slots = three[2];
    for (int r = n0; r < n1; ++r) {
        const int n = order[r], c = segs_of(n), len = len_of(n);
        if (c > 1) sc.split[cut++] = segs;
        for (int i = 0; i < c; ++i) {
            DecaySeg g;
            g.pos = i * seg_len * (c > 1);
            g.len = c > 1 ? min(seg_len, len - g.pos) : len;
            g.start = start_of(n) + g.pos;
            g.seq_len = len;
            g.seq = n;
            g.slot = c > 1 ? slots++ : -1;
            g.chunk = sc.chunk_base[n];
            g.pad = 0;
            sc.segs[segs++] = g;
        }
    }
    if (threadIdx.x == 0) {
        sc.chunk_base[num_seqs] = total1[0];
        hdr->num_segs = total3[0];
        hdr->num_split = total3[1];
        hdr->seg_len = seg_len;
        hdr->total_chunks = total1[0];
    }
}

// Start states of cut sequences: thread = four elements of a (cut sequence,
// head) state, walking its segments in pass order; each slot's local state
// becomes the state its segment starts from.  Four segments' local states are
// read ahead of the chain.
__global__ void __launch_bounds__(256)
decay_combine_kernel(DecaySched sc, float *__restrict__ states, const float *__restrict__ seg_dec,
                     const float *__restrict__ s_in, int s_trans, int hv, int dz, int dy, int reverse) {
    if (sc.hdr->status != GDN_OK) return;
    const int h = blockIdx.y;
    const int el = 4 * (blockIdx.x * 256 + threadIdx.x);  // of the 128 x 128 padded state
    const int r = el >> 7, c = el & 127;                  // z row, y columns c .. c + 3
    for (int j = blockIdx.z; j < sc.hdr->num_split; j += gridDim.z) {
        const DecaySeg first = sc.segs[sc.split[j]];
        const int n = (first.seq_len + sc.hdr->seg_len - 1) / sc.hdr->seg_len;
        float run[4] = {0.f, 0.f, 0.f, 0.f};
        if (s_in && r < dz) {
            const float *src = s_in + (size_t(first.seq) * hv + h) * dz * dy;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < dy) run[e] = src[s_trans ? size_t(c + e) * dz + r : size_t(r) * dy + c + e];
        }
        auto slot = [&](int i) { return size_t(first.slot + (reverse ? n - 1 - i : i)) * hv + h; };
        for (int i0 = 0; i0 < n; i0 += 4) {
            float4 local[4];
            float dec[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                local[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                dec[i] = 0.f;
                if (i0 + i + 1 < n) {  // the last segment's local state is not needed
                    local[i] = *reinterpret_cast<const float4 *>(states + slot(i0 + i) * 16384 + el);
                    dec[i] = seg_dec[slot(i0 + i)];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i0 + i >= n) break;
                *reinterpret_cast<float4 *>(states + slot(i0 + i) * 16384 + el) = make_float4(run[0], run[1], run[2], run[3]);
                run[0] = fmaf(dec[i], run[0], local[i].x);
                run[1] = fmaf(dec[i], run[1], local[i].y);
                run[2] = fmaf(dec[i], run[2], local[i].z);
                run[3] = fmaf(dec[i], run[3], local[i].w);
            }
        }
    }
}

// The decays' gradient: one warp per (chunk, head), two tokens a lane.  For
// token t of the chunk
//   dg_t = intra_t + sum_{i >= t} dot_q_i + sum_{j < t} dot_k_j + span.
__global__ void __launch_bounds__(128)
decay_dg_kernel(int num_seqs, int hv, int tokens, const int32_t *__restrict__ cu, int batched_len, DecaySched sc,
                const float *__restrict__ dot_q, const float *__restrict__ dot_k, const float *__restrict__ intra,
                const float *__restrict__ span, const float *__restrict__ g, int g_const, float *__restrict__ dg_tok,
                float *__restrict__ dg) {
    if (sc.hdr->status != GDN_OK) return;
    const int lane = threadIdx.x & 31;
    const int64_t units = int64_t(sc.hdr->total_chunks) * hv;
    for (int64_t u = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5); u < units; u += int64_t(gridDim.x) * 4) {
        const int gc = int(u / hv), h = int(u % hv);
        const int n = chunk_sequence(sc.chunk_base, num_seqs, gc);
        const int start = cu ? cu[n] : n * batched_len, len = cu ? cu[n + 1] - cu[n] : batched_len;
        const int t0 = (gc - sc.chunk_base[n]) * kDecayChunk + 2 * lane;
        const size_t at = size_t(start) + t0, of = size_t(h) * tokens + at;
        const bool v0 = t0 < len, v1 = t0 + 1 < len;
        const float q0 = v0 ? dot_q[of] : 0.f, q1 = v1 ? dot_q[of + 1] : 0.f;
        const float k0 = v0 ? dot_k[of] : 0.f, k1 = v1 ? dot_k[of + 1] : 0.f;
        const float i0 = v0 ? intra[of] : 0.f, i1 = v1 ? intra[of + 1] : 0.f;
        const float *sp = span + (size_t(gc) * hv + h) * 8;
        const float outside = ((sp[0] + sp[1]) + (sp[2] + sp[3])) + ((sp[4] + sp[5]) + (sp[6] + sp[7]));
        float qs = q0 + q1, ks = k0 + k1;  // inclusive: qs from the end, ks from the start
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, qs, d), e = __shfl_up_sync(0xffffffffu, ks, d);
            if (lane + d < 32) qs += a;
            if (lane >= d) ks += e;
        }
        float q_after = __shfl_down_sync(0xffffffffu, qs, 1), k_before = __shfl_up_sync(0xffffffffu, ks, 1);
        if (lane == 31) q_after = 0.f;  // sums of the lanes after and before this one
        if (lane == 0) k_before = 0.f;
        float val[2] = {i0 + qs + k_before + outside, i1 + (q1 + q_after) + (k_before + k0) + outside};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!(e ? v1 : v0)) continue;
            const size_t to = (at + e) * hv + h;
            if ((g_const ? g[h] : g[to]) < kGFloor) val[e] = 0.f;
            if (g_const) dg_tok[of + e] = val[e];
            else dg[to] = val[e];
        }
    }
}

// One value per head: the sum of its tokens' gradients, in 64 bits and a fixed order.
__global__ void __launch_bounds__(512)
decay_dg_head_kernel(const DecayHeader *hdr, const float *__restrict__ dg_tok, int tokens, float *__restrict__ dg) {
    __shared__ double part[512];
    if (hdr->status != GDN_OK) return;
    double s = 0.0;
    for (int t = threadIdx.x; t < tokens; t += 512) s += double(dg_tok[size_t(blockIdx.x) * tokens + t]);
    part[threadIdx.x] = s;
    __syncthreads();
    for (int d = 256; d > 0; d >>= 1) {
        if (int(threadIdx.x) < d) part[threadIdx.x] += part[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[blockIdx.x] = float(part[0]);
}

// out[t, hq, :] = the sum over the group's value heads of part[t, h, :], in head order.
// Bound by reading the parts: 268 MB (4 x 4096 tokens, 32 heads, d = 128) in 53 us, 0.77 of the copy bandwidth
// without the writes (0.96 with those that reach memory later).
template <typename T>
__global__ void __launch_bounds__(256)
decay_group_sum_kernel(const DecayHeader *hdr, const float *__restrict__ part, T *__restrict__ out, int64_t n4,
                       int group, int d4) {
    if (hdr->status != GDN_OK) return;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n4; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / d4;  // (token, q/k head)
        const int c = int(i % d4);
        const float4 *src = reinterpret_cast<const float4 *>(part) + row * group * d4 + c;
        float4 s = __ldcs(src);
        for (int j = 1; j < group; ++j) {
            const float4 x = __ldcs(src + int64_t(j) * d4);
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(out)[i] = s;
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(s.x, s.y), b = __floats2bfloat162_rn(s.z, s.w);
            reinterpret_cast<uint2 *>(out)[i] = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                                           *reinterpret_cast<const uint32_t *>(&b));
        }
    }
}
template <typename T>
__global__ void __launch_bounds__(256)
decay_group_sum_any_kernel(const DecayHeader *hdr, const float *__restrict__ part, T *__restrict__ out, int64_t n,
                           int group, int d) {
    if (hdr->status != GDN_OK) return;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / d;
        const float *src = part + row * group * d + i % d;
        float s = src[0];
        for (int j = 1; j < group; ++j) s += src[int64_t(j) * d];
        out[i] = from_f32<T>(s);
    }
}

}  // namespace

DecayLayout decay_layout(const gdn_shape_t &s, bool backward) {
    const int64_t tokens = int64_t(s.batch) * s.seq_len, N = s.num_seqs, hv = s.num_v_heads;
    // segments are at least max(min_seg, tokens * hv / ways) tokens long, and a
    // cut sequence is longer than one: it has at most 2 len / L of them
    const DecayPlan plan = plan_of(s);
    const int64_t balanced = balanced_tokens(tokens, s.num_v_heads, plan.ways);
    const int64_t shortest = std::max<int64_t>(plan.min_seg, balanced);
    DecayLayout L = {};
    L.max_slots = may_split(s) ? 2 * tokens / shortest + 1 : 0;
    L.max_split = may_split(s) ? tokens / shortest + 1 : 0;
    L.max_segs = N + L.max_slots;
    L.max_chunks = (tokens + 63 * N) / kDecayChunk;
    L.max_starts = tokens / kDecayChunk + 1;  // (a sequence's first needs no room: it is the initial state)
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    L.segs_off = take(size_t(L.max_segs) * sizeof(DecaySeg));
    L.split_off = take(size_t(L.max_split) * 4);
    L.order_off = take(size_t(N) * 4);
    L.cbase_off = take(size_t(N + 1) * 4);
    L.segdec_off[0] = take(size_t(L.max_slots) * hv * 4);
    L.state_off[0] = take(size_t(L.max_slots) * hv * 65536);
    if (backward) {
        L.segdec_off[1] = take(size_t(L.max_slots) * hv * 4);
        L.state_off[1] = take(size_t(L.max_slots) * hv * 65536);
        // (the tensor-core pass keeps 128 rows and 64 or 128 columns whatever the head sizes)
        const size_t state = decay_tc_supported(s) ? (s.head_dim_v > 64 ? 16384 : 8192)
                                                   : size_t(s.head_dim_k) * s.head_dim_v;
        L.start_off = take(size_t(L.max_starts) * hv * state * 4);
        L.span_off = take(size_t(L.max_chunks) * hv * 32);
        for (int i = 0; i < 2; ++i) L.dot_off[i] = take(size_t(tokens) * hv * 4);
        L.intra_off = take(size_t(tokens) * hv * 4);
        L.dgtok_off = take(size_t(tokens) * hv * 4);
        if (s.num_v_heads != s.num_qk_heads)
            for (int i = 0; i < 2; ++i) L.part_off[i] = take(size_t(tokens) * hv * s.head_dim_k * 4);
    }
    L.total = off;
    return L;
}

DecaySched decay_sched(char *ws, const DecayLayout &L) {
    DecaySched sc;
    sc.hdr = reinterpret_cast<DecayHeader *>(ws);
    sc.segs = reinterpret_cast<DecaySeg *>(ws + L.segs_off);
    sc.split = reinterpret_cast<int32_t *>(ws + L.split_off);
    sc.chunk_base = reinterpret_cast<int32_t *>(ws + L.cbase_off);
    return sc;
}

cudaError_t launch_decay_schedule(const gdn_shape_t &s, const int32_t *cu, char *ws, const DecayLayout &L,
                                  cudaStream_t stream) {
    decay_schedule_kernel<<<1, kSchedThreads, 0, stream>>>(s.num_seqs, s.batch * s.seq_len, cu ? 0 : s.seq_len,
                                                           s.num_v_heads, plan_of(s), cu, decay_sched(ws, L),
                                                           reinterpret_cast<int32_t *>(ws + L.order_off));
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_decay_combine(const gdn_shape_t &s, const DecayLayout &L, const DecaySched &sc, float *states,
                                 const float *seg_dec, const float *s_in, bool s_trans, int dz, int dy, bool reverse,
                                 cudaStream_t stream) {
    if (L.max_split == 0) return cudaSuccess;
    const int hv = s.num_v_heads;
    const int deep = int(std::min<int64_t>(L.max_split, std::max(1, 64 / hv)));
    decay_combine_kernel<<<dim3(16, unsigned(hv), unsigned(deep)), 256, 0, stream>>>(sc, states, seg_dec, s_in,
                                                                                     s_trans, hv, dz, dy, reverse);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_decay_dg(const gdn_shape_t &s, const int32_t *cu, const DecayLayout &L, const DecaySched &sc,
                            const float *dot_q, const float *dot_k, const float *intra, const float *span,
                            const float *g, bool g_const, float *dg_tok, float *dg, cudaStream_t stream) {
    const int64_t tokens = int64_t(s.batch) * s.seq_len, units = L.max_chunks * s.num_v_heads;
    const unsigned grid = unsigned(std::min<int64_t>((units + 3) / 4, 148 * 16));
    if (grid > 0) {
        decay_dg_kernel<<<grid, 128, 0, stream>>>(s.num_seqs, s.num_v_heads, int(tokens), cu, s.seq_len, sc, dot_q,
                                                  dot_k, intra, span, g, g_const, dg_tok, dg);
        count_launch();
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (g_const) {
        decay_dg_head_kernel<<<unsigned(s.num_v_heads), 512, 0, stream>>>(sc.hdr, dg_tok, int(tokens), dg);
        count_launch();
    }
    return cudaGetLastError();
}

cudaError_t launch_decay_group_sum(const DecayHeader *hdr, const float *part, void *out, int64_t tokens, int32_t hk,
                                   int32_t hv, int32_t d, int32_t dtype, cudaStream_t stream) {
    const int64_t n = tokens * hk * d;
    if (n == 0) return cudaSuccess;
    const int group = hv / hk;
    const bool by4 = d % 4 == 0;
    const int64_t items = by4 ? n / 4 : n;
    const unsigned grid = unsigned(std::min<int64_t>((items + 255) / 256, 148 * 8));
    using bf = __nv_bfloat16;
    if (by4 && dtype == GDN_DTYPE_BF16)
        decay_group_sum_kernel<bf><<<grid, 256, 0, stream>>>(hdr, part, static_cast<bf *>(out), items, group, d / 4);
    else if (by4)
        decay_group_sum_kernel<float><<<grid, 256, 0, stream>>>(hdr, part, static_cast<float *>(out), items, group,
                                                                  d / 4);
    else if (dtype == GDN_DTYPE_BF16)
        decay_group_sum_any_kernel<bf><<<grid, 256, 0, stream>>>(hdr, part, static_cast<bf *>(out), items, group, d);
    else
        decay_group_sum_any_kernel<float><<<grid, 256, 0, stream>>>(hdr, part, static_cast<float *>(out), items, group, d);
    count_launch();
    return cudaGetLastError();
}

}  // namespace gdn
