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
// pairs that span the chunk follow from <dS, S> at its start, known exactly
// at checkpoints every `ick` tokens and carried from chunk to chunk by taking
// off and adding the one-ended sums.  (The shorter dg_t = dg_{t+1} + q_t .
// dq_t - k_t . dk_t over the whole sequence loses digits where decays are
// strong: its terms hold the undecayed q_t . k_t, and cancel.  So would
// <dS, S> at a chunk's end: at the last one it holds the undecayed pairs of
// the last token and the final state's gradient.)
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

constexpr int kDecayChunk = 64;      // tokens of a chunk
constexpr int kDecayMinSeg = 256;    // shortest segment a split sequence is cut into
constexpr int kDecayMaxIck = 1024;   // checkpoint spacing of the decays' gradient (tokens)
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
    int32_t ck;             // first checkpoint slot of the sequence
    int32_t pad;
};

// Header of the workspace (shares its status word with the other operators').
struct DecayHeader {
    int32_t status, bad_index;
    int32_t num_segs, num_split, ick, seg_len, num_cks, total_chunks;
    int32_t pad[56];
};
static_assert(sizeof(DecayHeader) == 256, "header must be 256 bytes");

struct DecaySched {
    DecayHeader *hdr;
    DecaySeg *segs;         // [max_segs], longest sequences first
    int32_t *split;         // [max_split] first segment of each cut sequence
    int32_t *chunk_base;    // [N + 1] chunks before each sequence
    int32_t *ck_base;       // [N + 1] checkpoint slots before each sequence
};

// Workspace (offsets 256-byte aligned).  Every bound is a function of the
// shape alone; see decay_layout for the arithmetic.
struct DecayLayout {
    size_t segs_off, split_off, cbase_off, ckbase_off, order_off;
    size_t state_off[2];    // start states of cut sequences, [slots][Hv][128][128] fp32 (backward: two directions)
    size_t segdec_off[2];   // [slots][Hv] decay across each segment (each direction writes its own)
    size_t ckpt_off, zsum_off, dot_off[2], intra_off, part_off[2], dgtok_off;
    size_t total;
    int64_t max_segs, max_split, max_slots, max_cks, max_ckpt, max_chunks;
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
    // States at positions p > 0 that are multiples of `ick`, or NULL: [tokens / ick + 1][hv][128 * 128], at slot
    // (token / ick).  Two of them are at least ick tokens apart, whatever the sequences, so no slot is used twice;
    // the state at p = 0 is s_first.
    float *ckpt;
    float *zsum;                  // backward in time: <Sigma, checkpoint>, [cks][hv][8 parts]; NULL: write checkpoints
    const float *s_first;         // the checkpoint at a sequence's start, stored as s_in, or NULL for zeros
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
                            const float *dot_k, const float *intra, const float *zsum, const float *g, bool g_const,
                            float *dg_tok, float *dg, cudaStream_t stream);
cudaError_t launch_decay_group_sum(const DecayHeader *hdr, const float *part, void *out, int64_t tokens, int32_t hk,
                                   int32_t hv, int32_t d, int32_t dtype, cudaStream_t stream);

cudaError_t launch_decay_decode(int32_t n, int32_t hk, int32_t hv, int32_t dk, int32_t dv, int32_t dtype,
                                const void *q, const void *k, const void *v, const float *g, bool g_const,
                                float *state, void *o, cudaStream_t stream);

}  // namespace gdn
