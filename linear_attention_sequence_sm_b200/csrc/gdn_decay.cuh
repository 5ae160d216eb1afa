// gdn_decay.cuh -- declarations shared by the decayed linear attention's
// translation units (not part of the public ABI).
//
// The operation, per sequence and value head (S is d_v x d_k, fp32):
//     S_t = a_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t,   a_t = e^{max(g_t, -20)}
// and its reverse mode (dS_t: the gradient of S_t, later tokens included)
//     dS_t = do_t q_t^T + a_{t+1} dS_{t+1},
//     dq_t = S_t^T do_t,  dk_t = dS_t^T v_t,  dv_t = dS_t k_t,
//     dg_t = a_t <dS_t, S_{t-1}>.
// All four token outputs are one "pass" over the tokens with other operands:
//     out_t = Sigma_t x_t,  Sigma = decayed sums of z y^T,
//         o:  x = q,  y = k,  z = v,  forward in time
//         dq: x = do, y = v,  z = k,  forward  (Sigma = S^T)
//         dv: x = k,  y = q,  z = do, backward (Sigma = dS)
//         dk: x = v,  y = do, z = q,  backward (Sigma = dS^T)
// Over a chunk of 64 tokens with prefix sums G of g (inclusive) and start
// state Sigma, a forward pass is
//     out_r = sum_{c <= r} e^{G_r - G_c} (x_r . y_c) z_c + e^{G_r} Sigma x_r,
//     Sigma <- e^{G_last} Sigma + sum_c e^{G_last - G_c} z_c y_c^T,
// and a backward pass, whose chunks run last to first,
//     out_r = sum_{c >= r} e^{G_c - G_r} (x_r . y_c) z_c + e^{G_last - G_r} Sigma x_r,
//     Sigma <- e^{G_last} Sigma + sum_c e^{G_c} z_c y_c^T.
// No exponent is positive, so nothing overflows whatever the decays.
//
// The decays' gradient sums the weights W_ij = e^{G_i - G_j} (q_i . k_j)
// (do_i . v_j) of all pairs j < t <= i.  Inside t's chunk they are summed
// directly; pairs with one end in the chunk are q_i . dq_i's and k_j . dk_j's
// parts that come from the chunk's start and end states (`dot` below), and
// the pairs that span the chunk are e^{G_last} <dS at its end, S at its start>:
// the pass forward in time keeps each chunk's start state, the one backward in
// time multiplies it with dS.  Every part is a sum of decayed terms and none is
// taken off, so a token whose decay is far stronger than its neighbours' keeps
// the digits of its small gradient.  (dg_t = dg_{t+1} + q_t . dq_t - k_t . dk_t
// over the sequence cancels there, and so does carrying the pairs across a
// chunk's start from one chunk to the next: with g = -15 among -0.01, dg = 2.5e-5
// is what remains of some 80 in fp32.  The states cost 64 KB a chunk and head,
// written once and read once.)
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

constexpr int kDecayChunk = 64;      // tokens of a chunk
constexpr int kDecayMinSeg = 256;    // shortest segment a split sequence is cut into
constexpr int kDecayMaxTokens = INT32_MAX - 2048;  // (positions past a sequence's end stay in 32 bits)
constexpr int kDecayPlanSms = 148;   // SMs the split aims to fill (B200)

// A log-decay as the recurrence uses it.  A NaN stays one (fmaxf would make it
// the floor, and the call would answer as if nothing were wrong).
__device__ __forceinline__ float floored(float g) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(g), "f"(kGFloor));
    return r;
}

// A segment: the tokens one CTA walks for one value head.  Sequences are cut
// only where whole sequences would leave SMs idle (see decay_schedule_kernel).
struct DecaySeg {
    int32_t start, len;     // first token (of all tokens) and token count
    int32_t pos, seq_len;   // offset in the sequence, the sequence's length
    int32_t seq, slot;      // sequence; slot of its start state, -1 for an uncut sequence
    int32_t chunk;          // chunks before the sequence
    int32_t pad;
};

// Header of the workspace (shares its status word with the other operators').
struct DecayHeader {
    int32_t status, bad_index;
    int32_t num_segs, num_split, seg_len, total_chunks;
    int32_t pad[58];
};
static_assert(sizeof(DecayHeader) == 256, "header must be 256 bytes");

struct DecaySched {
    DecayHeader *hdr;
    DecaySeg *segs;         // [max_segs], longest sequences first
    int32_t *split;         // [max_split] first segment of each cut sequence
    int32_t *chunk_base;    // [N + 1] chunks before each sequence
};

// Workspace (offsets 256-byte aligned).  Every bound is a function of the
// shape alone; see decay_layout for the arithmetic.
struct DecayLayout {
    size_t segs_off, split_off, cbase_off, order_off;
    size_t state_off[2];    // start states of cut sequences, [slots][Hv][128][128] fp32 (backward: two directions)
    size_t segdec_off[2];   // [slots][Hv] decay across each segment (each direction writes its own)
    size_t start_off, span_off, dot_off[2], intra_off, part_off[2], dgtok_off;
    size_t total;
    int64_t max_segs, max_split, max_slots, max_starts, max_chunks;
};
DecayLayout decay_layout(const gdn_shape_t &s, bool backward);

// One pass (see above).  Heads: value head h reads head h / (hv / hx) of x.
struct DecayPass {
    const void *x, *y, *z, *aux;  // aux: rows dotted with the start state's part of out (NULL: none)
    int32_t hx, hy, hz, haux, hv;
    int32_t dy, dz;               // x, y: dy wide; z, out, aux: dz wide
    int32_t tokens;
    const float *g;               // [tokens, hv], or [hv] with g_const
    int32_t g_const, reverse;
    const float *s_in;            // state before the first chunk of a sequence, [N, hv, ...] or NULL
    float *s_out;                 // state after its last chunk, or NULL
    int32_t s_trans;              // s_in and s_out are stored [dy][dz] (0: [dz][dy])
    const float *seg_state;       // start states of cut sequences
    int32_t seg_trans;            // they are stored [dy][dz]
    float *seg_local, *seg_dec;   // state_only: where local states and decays go
    int32_t state_only;
    void *out;                    // [tokens, hv, dz]
    int32_t out_f32;              // 32-bit out whatever the inputs' type
    float *dot;                   // [hv][tokens], or NULL
    // Start states of the chunks behind a sequence's first, or NULL: [tokens / 64 + 1][hv][a state], at slot
    // (first token / 64), in an order of the pass's own.  Two of them are at least 64 tokens apart, whatever the sequences, so no slot is used twice;
    // a sequence's first is s_first.
    float *starts;
    float *span;                  // backward in time: e^G <Sigma, start state>, [chunks][hv][8 parts]; NULL: write starts
    const float *s_first;         // a sequence's first start state, stored as s_in, or NULL for zeros
    DecaySched sched;
};

cudaError_t launch_decay_schedule(const gdn_shape_t &s, const int32_t *cu, char *ws, const DecayLayout &L,
                                  cudaStream_t stream);
DecaySched decay_sched(char *ws, const DecayLayout &L);

// Start states of cut sequences from the segments' local states, in place.
cudaError_t launch_decay_combine(const gdn_shape_t &s, const DecayLayout &L, const DecaySched &sc, float *states,
                                 const float *seg_dec, const float *s_in, bool s_trans, int dz, int dy, bool reverse,
                                 cudaStream_t stream);

// The pass on CUDA cores (fp32 or bf16 storage, any d <= 128; with `also`, two
// independent passes in one launch), and on the tensor cores (bf16, d a
// multiple of 8).
cudaError_t launch_decay_pass_simt(const DecayPass &p, const DecayPass *also, int32_t dtype, int64_t max_units,
                                   cudaStream_t stream);
bool decay_tc_supported(const gdn_shape_t &s);
cudaError_t launch_decay_pass_tc(const DecayPass &p, int64_t max_units, cudaStream_t stream);

// Pairs inside a chunk for the decays' gradient: intra [hv][tokens]; the first
// for every shape, the second for bf16 with head sizes a multiple of 8.
cudaError_t launch_decay_intra_simt(const gdn_shape_t &s, const int32_t *cu, const DecayLayout &L,
                                    const DecaySched &sc, const void *q, const void *k, const void *v,
                                    const void *d_o, const float *g, bool g_const, float *intra, cudaStream_t stream);
cudaError_t launch_decay_intra(const gdn_shape_t &s, const int32_t *cu, const DecayLayout &L, const DecaySched &sc,
                               const void *q, const void *k, const void *v, const void *d_o, const float *g,
                               bool g_const, float *intra, cudaStream_t stream);

// dg from its parts, and the sums over grouped value heads.
cudaError_t launch_decay_dg(const gdn_shape_t &s, const int32_t *cu, const DecayLayout &L, const DecaySched &sc, const float *dot_q,
                            const float *dot_k, const float *intra, const float *span, const float *g, bool g_const,
                            float *dg_tok, float *dg, cudaStream_t stream);
cudaError_t launch_decay_group_sum(const DecayHeader *hdr, const float *part, void *out, int64_t tokens, int32_t hk,
                                   int32_t hv, int32_t d, int32_t dtype, cudaStream_t stream);

cudaError_t launch_decay_decode(int32_t n, int32_t hk, int32_t hv, int32_t dk, int32_t dv, int32_t dtype,
                                const void *q, const void *k, const void *v, const float *g, bool g_const,
                                float *state, void *o, cudaStream_t stream);

}  // namespace gdn
