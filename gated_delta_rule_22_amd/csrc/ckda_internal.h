// Internal declarations shared by the host entry points and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <stddef.h>
#include <stdint.h>

#include "ckda.h"

namespace ckda {

constexpr int kChunk = 64;          // tokens per chunk of the chunkwise forward

// ---------------------------------------------------------------- input loads
// q, k, v arrive as bf16 or fp32; both widen exactly to fp32 (and fp64).
__device__ __forceinline__ float to_f32(__hip_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
// Four consecutive elements (8-byte aligned for bf16, 16-byte for fp32) as fp32.
__device__ __forceinline__ float4 load4_f32(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4_f32(const __hip_bfloat16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}

// ---------------------------------------------------------------- schedule
// Per-call sequence table, computed on the device from cu_seqlens (or the
// uniform B x T layout) into the workspace:
//   seq_start[n], seq_len[n]  token offset and length of sequence n
//   chunk_off[n]              first flat chunk index of sequence n (N+1 entries)
//   order[r]                  sequence index of rank r, longest first
struct SeqTable {
    int32_t *seq_start;
    int32_t *seq_len;
    int32_t *chunk_off;
    int32_t *order;
};
// Sequences are ordered by length up to this many (the ranking is quadratic).
constexpr int kRankedSeqs = 1024;

// The sequences of a call: the table, or for uniform rows of T tokens (T >= 0)
// plain arithmetic, which spares the table's launch.
struct Seqs {
    SeqTable tab;
    int T;                               // -1: packed
    __device__ int start(int n) const { return T >= 0 ? n * T : tab.seq_start[n]; }
    __device__ int len(int n) const { return T >= 0 ? T : tab.seq_len[n]; }
    __device__ int first_chunk(int n) const {      // n = N: the number of chunks
        return T >= 0 ? n * ((T + kChunk - 1) / kChunk) : tab.chunk_off[n];
    }
    __device__ int order(int r) const { return T >= 0 ? r : tab.order[r]; }
    // Sequence of a flat chunk index below first_chunk(N).
    __device__ int of_chunk(int chunk, int N) const {
        if (T >= 0) return chunk / ((T + kChunk - 1) / kChunk);
        int lo = 0, hi = N;              // first_chunk(lo) <= chunk < first_chunk(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tab.chunk_off[mid] <= chunk) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

// Workspace layout for a forward call (host-side arithmetic only).
struct FwdLayout {
    size_t table_bytes;      // the SeqTable arrays, 256-byte aligned
    size_t rec_bytes;        // fp64 path: bytes of one (chunk, head) record
    size_t n_chunks_ub;      // upper bound of chunks over all sequences
    size_t total;            // total workspace bytes
};
FwdLayout fwd_layout(int B, int T, int H, int dk, int dv, int N, int in_dtype);
SeqTable seq_table(void *workspace, int N);

hipError_t launch_seq_table(const int32_t *cu_seqlens, int B, int T, int N, SeqTable tab,
                            hipStream_t stream);
// Fills `bytes` (a multiple of 4; 4-byte aligned) with a NaN bit pattern.
hipError_t launch_poison(void *buf, size_t bytes, hipStream_t stream);

hipError_t launch_decode(const void *q, const void *k, const void *v, const float *g,
                         const float *beta, float *S, float *o, int N, int H, int dk, int dv,
                         int in_dtype, hipStream_t stream);

// fp64 chunkwise forward (fp32 inputs).
hipError_t launch_fwd_f64(const void *q, const void *k, const void *v, const float *g,
                          const float *beta, const float *S0, int T_rows, int H, int dk, int dv,
                          int N, int in_dtype, SeqTable tab, size_t n_chunks_ub, void *records,
                          size_t rec_bytes, void *o, float *S_T, int signed_gates, int l2norm,
                          int o_bf16, hipStream_t stream);

// Fused bf16 chunkwise forward on matrix cores (bf16 inputs).
// signed_gates = 0 is KDA mode: the gates' signs are ignored (|g| is used).
// l2norm: q and k are L2-normalised per (token, head) inside the kernel.
// o_bf16: o is bfloat16 (else fp32).
hipError_t launch_fwd_bf16(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, const float *S0, void *o, float *S_T, int T, int H,
                           int dk, int dv, int N, SeqTable tab, int packed, int signed_gates,
                           int l2norm, int o_bf16, hipStream_t stream);

// The same forward as two kernels (uniform rows, no fused options): a
// preparation kernel writes every prepared 16-token block's slot image to
// `img` (fwd_bf16_split_bytes bytes), then a state kernel loads them.  Kept to
// measure the hand-off the fused kernel replaced; results are bit-identical.
size_t fwd_bf16_split_bytes(int T, int H, int dk, int N);
hipError_t launch_fwd_bf16_split(const void *q, const void *k, const void *v, const float *g,
                                 const float *beta, const float *S0, void *o, float *S_T, int T,
                                 int H, int dk, int dv, int N, SeqTable tab, int signed_gates,
                                 void *img, hipStream_t stream);

// fp64 chunkwise backward (both input dtypes).  Runs the records and the
// forward's serial pass (keeping per-chunk states and U), the reverse pass of
// the state gradient, then the per-chunk gradients.  signed_gates = 0 is KDA
// mode (|g| is used; the gradient with respect to g is then dlog|g| / g, the
// same formula).  l2norm: q and k are L2-normalised per (token, head) before
// use, and their gradients pass back through that normalisation.
size_t f64_bwd_scratch_bytes(int dk, int dv);
hipError_t launch_bwd_f64(const void *q, const void *k, const void *v, const float *g,
                          const float *beta, const float *S0, const float *dO, const float *dS_T,
                          int H, int dk, int dv, int N, int in_dtype, SeqTable tab,
                          size_t n_chunks_ub, void *records, size_t rec_bytes, double *S_chunks,
                          double *U_chunks, double *dU_chunks, double *dSe_chunks,
                          double *scratch, float *dq, float *dk_out, float *dv_out, float *dg,
                          float *dbeta, float *dS0, int signed_gates, int l2norm,
                          hipStream_t stream);

// ---------------------------------------------------------------- gated delta rule
// One log-gate per (token, head); Hv value heads share Hk query/key heads in
// groups of Hv / Hk.
struct GdrArgs {
    const void *q, *k, *v;
    const float *g, *beta, *S0;
    Seqs seqs;
    size_t n_chunks_ub;
    int N, Hk, Hv, dk, dv;
    void *o;
    float *S_T;
};
hipError_t launch_gdr_step(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, float *S, const int32_t *slots, int pool, void *o,
                           int N, int Hk, int Hv, int dk, int dv, int in_dtype,
                           hipStream_t stream);
// Token by token, fp32 arithmetic, any input type.
hipError_t launch_gdr_token(const GdrArgs &a, hipStream_t stream);
// Chunkwise on bf16 matrix cores (bf16 inputs): `rec` holds
// gdr_forward_rec_bytes() for every chunk and value head.
size_t gdr_forward_rec_bytes();
hipError_t launch_gdr_forward(const GdrArgs &a, void *rec, hipStream_t stream);
// The backward's records, which hold P's second term too.
hipError_t launch_gdr_prepare_backward(const GdrArgs &a, void *rec, hipStream_t stream);
struct GdrBwdArgs {
    GdrArgs fwd;                         // fwd.S_T is NULL
    const void *d_o;
    const float *dS_T;
    void *rec, *S, *U, *dS, *F;          // per (chunk, value head): see GdrBwdBytes
    void *dq, *dk, *dv;
    float *dg, *dbeta, *dS0;
};
struct GdrBwdBytes { size_t rec, state, rows; };   // rec; S and dS; U and F
GdrBwdBytes gdr_backward_bytes(int dk, int dv);
hipError_t launch_gdr_backward(const GdrBwdArgs &a, hipStream_t stream);
// Layouts to and from the per-channel fp64 backward: everything in fp32 and per
// value head and channel.  vx, dox and dvx are NULL where v, d_o and dv are
// fp32 themselves.
struct GdrF64Args {
    const void *q, *k, *v, *d_o;
    const float *g;
    Seqs seqs;
    size_t rows;
    int N, Hk, Hv, dk, dv;
    float *qx, *kx, *gx, *vx, *dox, *dqx, *dkx, *dgx, *dvx;
    void *dq, *dk_out, *dv_out;
    float *dg;
    bool zero_start;                     // sequences start from zero states
};
hipError_t launch_gdr_expand(const GdrF64Args &a, int in_dtype, hipStream_t stream);
hipError_t launch_gdr_collect(const GdrF64Args &a, int in_dtype, hipStream_t stream);

// ---------------------------------------------------------------- norm and rotation
struct RotaryArgs {
    const void *q, *k, *dq, *dk;         // rows; upstream gradients (backward)
    void *qo, *ko;                       // results (backward: gradients of q, k)
    size_t ldq, ldk, lddq, lddk, ldqo, ldko;   // elements from token to token
    const int32_t *pos;
    const double *freqs;                 // radians per position, rd / 2 of them
    const float *wq, *wk;
    float *dwq, *dwk, *partial;
    int tokens, Hq, Hk, d, rd, lanes;
    int norm, half, inverse;             // norm: 0 none, else rows are normalised
    float norm_scale, eps, q_scale, rotary_scale;   // norm_scale: 1/d (rms) or 1 (l2)
};
int rotary_bwd_groups(int tokens);       // workspace rows of 2 d floats
hipError_t launch_rotary(const RotaryArgs &a, int in_dtype, bool backward, hipStream_t stream);

}  // namespace ckda
