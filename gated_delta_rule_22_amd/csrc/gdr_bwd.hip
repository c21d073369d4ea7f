// Backward of the chunkwise gated delta rule for bf16 inputs.
//
// With dS' the gradient of the state behind the chunk and the forward's
// symbols (gdr_chunk.hip):
//
//   dU = P^T dO + (gam_n / gam) K dS'        F = T^T dU   ( = dV )
//   dS = gam_n dS' + Q^T (gam dO) - K^T (gam F)
//   dP_ij = r_ij dO_i.U_j                    dA_ij = -r_ij F_i.U_j
//   dQ = gam dO S^T + dP K
//   dK = [-gam F S^T + dA K] + [dP^T Q + dA^T K + (gam_n / gam) U dS'^T]
//   dbeta = F.U / beta^2
//   dG_i = q_i.dQ_i + k_i.dK_i[first bracket] - k_i.dK_i[second bracket]
//   dg_t = sum_{i >= t} dG_i + sum_j w_j + gam_n <S, dS'>
//
// where w_j is the last term's part of k_j.dK_j.  (F and U carry a factor beta
// each, and beta is kept off zero by kBetaFloor, so F.U / beta^2 holds at
// beta = 0 too.)
//
// Three passes: the forward's chain kept per chunk (S, U), the chain of dS
// backwards (dS', F), each serial in the chunks of a (sequence, head), and the
// gradients, parallel over chunks.  Everything that feeds an fp32 gradient
// (dg, dbeta, dS0) runs in two bf16 terms, as in the forward.
#include "gdr_chunk.h"

namespace ckda {
using namespace gdr;
namespace {

__device__ __forceinline__ bool chain_block(int nblk, int pairs, int &pair, int &blk) {
  const int b = blockIdx.x;              // as in the forward: a head's blocks share an XCD
  blk = (b / 8) % nblk;
  pair = (b / 8 / nblk) * 8 + b % 8;
  return pair < pairs;
}

// The chain of dS, last chunk first.  As in the forward's chain four waves own
// 16 of the DV columns each, so dS -> dU -> F -> dS stays in their registers,
// and four helper waves run beside them: they load, and one chunk ahead they
// compute the chain's inputs that do not depend on dS, P^T dO and
// Q^T (gam dO), which the chain takes from LDS as result tiles.
// Barrier A: the chunk's operands and those tiles are in LDS; barrier B: the
// chain has read all of them but K.
template <int DK> struct ReverseLds {
  static constexpr int kBufK = kTile<DK>, kWave = (4 + DK / 16) * 1024;   // a wave's tiles
  static constexpr int kK = 0, kT = 2 * kBufK, kQ = kT + 2 * kTri, kD = kQ + kTile<DK>;
  static constexpr int kP = kD + kTile<64>, kGam = kP + 2 * kTri;
  static constexpr int kTiles = kGam + C * 4, kBytes = kTiles + 4 * kWave;
};

template <int DK, int DV>
__global__ __launch_bounds__(2 * kThreads, 2) void reverse_kernel(
    const __hip_bfloat16 *__restrict__ q, const __hip_bfloat16 *__restrict__ k,
    const __hip_bfloat16 *__restrict__ d_o, const float *__restrict__ dS_T, SeqTable tab, int N,
    int Hk, int Hv, const char *__restrict__ rec_base, char *__restrict__ dS_keep,
    char *__restrict__ F_keep, float *__restrict__ dS0) {
  using L = ReverseLds<DK>;
  constexpr int KS = DK / 32, MT = DK / 16, BV = 64;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int pair, blk;
  if (!chain_block(DV / BV, N * Hv, pair, blk)) return;
  const int seq = tab.order[pair / Hv], hv = pair % Hv, hk = hv / (Hv / Hk);
  const int wave = (threadIdx.x >> 6) & 3, lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
  const int len = tab.seq_len[seq], chunks = (len + C - 1) / C;
  const size_t row0 = tab.seq_start[seq];
  const size_t c0 = tab.chunk_off[seq];
  const int col = blk * BV + 16 * wave;
  char *tiles = lds + L::kTiles + wave * L::kWave + lane * 16;

  if (threadIdx.x >= kThreads) {         // helper waves
    const int t = threadIdx.x - kThreads;
    const char *Q = lds + L::kQ, *D = lds + L::kD, *P = lds + L::kP;
    const float *s_gam = reinterpret_cast<const float *>(lds + L::kGam);
    Stage<DK> gk, gq;
    Stage<BV> gd;
    Linear<2 * kTri> gt, gp;
    float gam = 0.f;
    // The chain's operands of chunk c, and the helpers' own of the chunk before.
    auto fetch_chain = [&](int c) {
      const size_t row = row0 + (size_t)c * C;
      const char *rec = rec_base + ((c0 + c) * Hv + hv) * kRecBwd;
      gk.load(k + (row * Hk + hk) * DK, (size_t)Hk * DK, min(C, len - c * C), t);
      gt.load(rec + kRecTh, t);
    };
    auto put_chain = [&](int c, int buf) {
      gk.store(lds + L::kK + (buf & 1) * L::kBufK, min(C, len - c * C), t);
      gt.store(lds + L::kT, t);
    };
    auto fetch_own = [&](int c) {
      const int valid = min(C, len - c * C);
      const size_t row = row0 + (size_t)c * C;
      const char *rec = rec_base + ((c0 + c) * Hv + hv) * kRecBwd;
      gq.load(q + (row * Hk + hk) * DK, (size_t)Hk * DK, valid, t);
      gd.load(d_o + (row * Hv + hv) * DV + blk * BV, (size_t)Hv * DV, valid, t);
      // P hi and P lo: two matrices, not next to each other in the record
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int at = (t + i * kThreads) * 16;
        gp.r[i] = load16(rec + (at < kTri ? kRecPh + at : kRecPl + at - kTri), true);
      }
      gam = reinterpret_cast<const float *>(rec + kRecGate)[kGam * C + t % C];
    };
    auto put_own = [&](int c) {
      const int valid = min(C, len - c * C);
      gq.store(lds + L::kQ, valid, t);
      gd.store(lds + L::kD, valid, t);
      gp.store(lds + L::kP, t);
      if (t < C) reinterpret_cast<float *>(lds + L::kGam)[t] = gam;
    };
    f4 pd[4], qd[MT];
    auto ahead = [&]() {
      f4 d[4];                           // dO: lane = column, 4 tokens a tile
      bf4 r[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) r[it] = cols_quad<BV>(D, 16 * it, 16 * wave, lane);
      const bf8 d0 = join(r[0], r[1]), d1 = join(r[2], r[3]);
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        pd[jt] = 0.f;
#pragma unroll
        for (int ks = jt / 2; ks < 2; ++ks) {
          const Split p = {tri_frag_t(P, jt, ks, lane), tri_frag_t(P + kTri, jt, ks, lane)};
          pd[jt] = dot2(p, ks ? d1 : d0, pd[jt]);
        }
        d[jt] = widen4(r[jt]) * *reinterpret_cast<const f4 *>(s_gam + 16 * jt + 4 * h);
      }
      const Split e0 = split8(d[0], d[1]), e1 = split8(d[2], d[3]);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        qd[i] = dot2(cols_frag<DK>(Q, 32, 16 * i, lane), e1,
                     dot2(cols_frag<DK>(Q, 0, 16 * i, lane), e0, f4(0.f)));
    };
    auto put_tiles = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<f4 *>(tiles + i * 1024) = pd[i];
#pragma unroll
      for (int i = 0; i < MT; ++i) *reinterpret_cast<f4 *>(tiles + (4 + i) * 1024) = qd[i];
    };
    // Behind the first chunk the first one is staged again, read by nobody.
    const int last = chunks - 1;
    if (chunks > 0) {
      fetch_own(last);
      fetch_chain(last);
      put_own(last);
      put_chain(last, last);
    }
    lds_barrier();                       // the helpers' operands of the last chunk
    if (chunks > 0) {
      fetch_own(max(last - 1, 0));
      ahead();
      put_tiles();
    }
    lds_barrier();                       // all helpers have read them
    if (chunks > 0) put_own(max(last - 1, 0));
    for (int c = last; c >= 0; --c) {
      lds_barrier();                     // A
      const int c1 = max(c - 1, 0), c2 = max(c - 2, 0);
      fetch_chain(c1);
      fetch_own(c2);
      ahead();
      lds_barrier();                     // B
      put_tiles();
      put_chain(c1, c - 1);
      put_own(c2);
    }
    return;
  }

  f4 S[MT];                              // dS
  const size_t sbase = ((size_t)seq * Hv + hv) * DK * DV + col + m;
#pragma unroll
  for (int i = 0; i < MT; ++i) S[i] = 0.f;
  if (dS_T)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = dS_T[sbase + (size_t)(16 * i + 4 * h + r) * DV];
  // The gate factors of a lane's tokens, from memory a chunk ahead.
  f4 gam[4], last[4];
  float gn = 0.f;
  auto fetch_gates = [&](int c) {
    const float *g = reinterpret_cast<const float *>(rec_base + ((c0 + c) * Hv + hv) * kRecBwd +
                                                     kRecGate);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      gam[jt] = *reinterpret_cast<const f4 *>(g + kGam * C + 16 * jt + 4 * h);
      last[jt] = *reinterpret_cast<const f4 *>(g + kLast * C + 16 * jt + 4 * h);
    }
    gn = g[kGam * C + C - 1];
  };
  if (chunks > 0) fetch_gates(chunks - 1);
  lds_barrier();                         // the helpers' two, before the loop
  lds_barrier();
  for (int c = chunks - 1; c >= 0; --c) {
    const char *K = lds + L::kK + (c & 1) * L::kBufK, *T = lds + L::kT;
    Split sf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) sf[ks] = split8(S[2 * ks], S[2 * ks + 1]);
    lds_barrier();                       // A
    char *p = dS_keep + (((c0 + c) * Hv + hv) * (2 * KS * (DV / 16)) + col / 16) * kFrag + lane * 16;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      *reinterpret_cast<bf8 *>(p + ks * (DV / 16) * kFrag) = sf[ks].hi;
      *reinterpret_cast<bf8 *>(p + (KS + ks) * (DV / 16) * kFrag) = sf[ks].lo;
    }
    bf8 kf[KS][4];
    f4 X[4];                             // dU
    auto read_k = [&](int ks) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) kf[ks][jt] = rows_frag<DK>(K, 16 * jt, 32 * ks, lane);
    };
    auto times_s = [&](int ks) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) X[jt] = mfma(kf[ks][jt], sf[ks].hi, ks ? X[jt] : f4(0.f));
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) X[jt] = mfma(kf[ks][jt], sf[ks].lo, X[jt]);
    };
    read_k(0);
    read_k(1);
    fence_schedule();
    if (KS > 2) {
      read_k(KS - 2);
      read_k(KS - 1);
    }
    times_s(0);
    fence_schedule();
    f4 pd[4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) pd[jt] = *reinterpret_cast<const f4 *>(tiles + jt * 1024);
    Split t[4][2];                       // T^T: tiles jt, rows of ks >= jt / 2
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
#pragma unroll
      for (int ks = jt / 2; ks < 2; ++ks)
        t[jt][ks] = {tri_frag_t(T, jt, ks, lane), tri_frag_t(T + kTri, jt, ks, lane)};
#pragma unroll
    for (int ks = 1; ks < KS; ++ks) times_s(ks);
    fence_schedule();
    bf8 kt[2][MT];                       // K^T for the update, read meanwhile
    f4 qd[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) kt[0][i] = cols_frag<DK>(K, 0, 16 * i, lane);
#pragma unroll
    for (int i = 0; i < MT; ++i) qd[i] = *reinterpret_cast<const f4 *>(tiles + (4 + i) * 1024);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) X[jt] = X[jt] * last[jt] + pd[jt];
    const Split x0 = split8(X[0], X[1]), x1 = split8(X[2], X[3]);
    fence_schedule();
    f4 F[4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) F[jt] = 0.f;
#pragma unroll
    for (int term = 0; term < 3; ++term)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int jt = 0; jt < 2 * ks + 2; ++jt) {
          const Split &x = ks ? x1 : x0;
          F[jt] = mfma(term == 2 ? t[jt][ks].lo : t[jt][ks].hi, term == 1 ? x.lo : x.hi, F[jt]);
        }
#pragma unroll
    for (int i = 0; i < MT; ++i) S[i] = S[i] * gn + qd[i];
#pragma unroll
    for (int i = 0; i < MT; ++i) kt[1][i] = cols_frag<DK>(K, 32, 16 * i, lane);
    lds_barrier();                       // B
    p = F_keep + (((c0 + c) * Hv + hv) * (4 * (DV / 16)) + col / 16) * kFrag + lane * 16;
    const Split f0 = split8(F[0], F[1]), f1 = split8(F[2], F[3]);
    *reinterpret_cast<bf8 *>(p) = f0.hi;
    *reinterpret_cast<bf8 *>(p + (DV / 16) * kFrag) = f1.hi;
    *reinterpret_cast<bf8 *>(p + 2 * (DV / 16) * kFrag) = f0.lo;
    *reinterpret_cast<bf8 *>(p + 3 * (DV / 16) * kFrag) = f1.lo;
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) F[jt] *= -gam[jt];
    fetch_gates(max(c - 1, 0));
    const Split w0 = split8(F[0], F[1]), w1 = split8(F[2], F[3]);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int term = 0; term < 2; ++term)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const Split &w = ks ? w1 : w0;
          S[i] = mfma(kt[ks][i], term ? w.lo : w.hi, S[i]);
        }
  }
  if (dS0)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        dS0[sbase + (size_t)(16 * i + 4 * h + r) * DV] = S[i][r];
}

// ---------------------------------------------------------------- gradients
// One workgroup per (chunk, query/key head); it goes over the group's value
// heads one after another, so dQ and dK of a shared head are summed in
// registers, in a fixed order.  Wave w owns tokens 16 w .. 16 w + 15: as rows
// i it needs the tiles j <= w of the triangular products, as columns j the
// tiles i >= w, five tiles for every wave.  Results have lane = token and 4
// key channels a lane, so stores are 8 bytes and q.dq needs two exchanges.
template <int DK, int DV> struct GradLds {
  static constexpr int kK = 0, kQ = kK + kTile<DK>, kGate = kQ + kTile<DK>;
  static constexpr int kSum = kGate + kGateBytes, kX = kSum + 512;
  static constexpr int kD = kX, kU = kD + kTile<DV>, kF = kU + 4 * C * DV;
  static constexpr int kEnd1 = kF + 4 * C * DV, kEnd2 = kX + 4 * DK * DV;
  static constexpr int kBytes = kEnd1 > kEnd2 ? kEnd1 : kEnd2;
};

__device__ __forceinline__ float sum4(f4 a) { return (a[0] + a[1]) + (a[2] + a[3]); }
__device__ __forceinline__ float over_quarters(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

template <int DK, int DV>
__global__ __launch_bounds__(kThreads, 1) void grad_kernel(
    const __hip_bfloat16 *__restrict__ q, const __hip_bfloat16 *__restrict__ k,
    const float *__restrict__ g, const float *__restrict__ beta,
    const __hip_bfloat16 *__restrict__ d_o, SeqTable tab, int N, int Hk, int Hv,
    const char *__restrict__ rec_base, const char *__restrict__ S_keep,
    const char *__restrict__ U_keep, const char *__restrict__ dS_keep,
    const char *__restrict__ F_keep, __hip_bfloat16 *__restrict__ dq,
    __hip_bfloat16 *__restrict__ dk_out, __hip_bfloat16 *__restrict__ dv_out,
    float *__restrict__ dg, float *__restrict__ dbeta) {
  using L = GradLds<DK, DV>;
  constexpr int MT = DK / 16, NT = DV / 16, KV = DV / 32;
  constexpr int kPlane = DK * DV * 2;    // bytes of one term of a state
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int chunk = blockIdx.x / Hk, hk = blockIdx.x % Hk, rep = Hv / Hk;
  if (chunk >= tab.chunk_off[N]) return;
  const int seq = find_seq(tab, N, chunk);
  const int at = (chunk - tab.chunk_off[seq]) * C;
  const int valid = min(C, tab.seq_len[seq] - at);
  const size_t row0 = (size_t)tab.seq_start[seq] + at;
  const int t = threadIdx.x, w = t >> 6, lane = t & 63, m = lane & 15, h = lane >> 4;
  const int tok = 16 * w + m;            // this lane's token
  const char *K = lds + L::kK, *Q = lds + L::kQ;
  float *gate = reinterpret_cast<float *>(lds + L::kGate);
  float *s_dG = reinterpret_cast<float *>(lds + L::kSum), *s_n = s_dG + C;

  {
    Stage<DK> a, b;
    a.load(k + (row0 * Hk + hk) * DK, (size_t)Hk * DK, valid, t);
    b.load(q + (row0 * Hk + hk) * DK, (size_t)Hk * DK, valid, t);
    a.store(lds + L::kK, valid, t);
    b.store(lds + L::kQ, valid, t);
  }
  f4 dQ[MT], dK[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) dQ[i] = dK[i] = 0.f;

  for (int u = 0; u < rep; ++u) {
    const int hv = hk * rep + u;
    const size_t ch = (size_t)chunk * Hv + hv;
    {
      Stage<DV> a;
      Linear<4 * C * DV> e, f;
      a.load(d_o + (row0 * Hv + hv) * DV, (size_t)Hv * DV, valid, t);
      e.load(U_keep + ch * (4 * C * DV), t);
      f.load(F_keep + ch * (4 * C * DV), t);
      const float *rg = reinterpret_cast<const float *>(rec_base + ch * kRecBwd + kRecGate);
      float ga = rg[t], gb = t < C ? rg[kThreads + t] : 0.f;
      a.store(lds + L::kD, valid, t);
      e.store(lds + L::kU, t);
      f.store(lds + L::kF, t);
      gate[t] = ga;
      if (t < C) gate[kThreads + t] = gb;
    }
    __syncthreads();
    const char *D = lds + L::kD;
    auto tile_split = [&](const char *base, int row, int rows, int ks) {
      const char *a = base + ((row >> 1) * NT + 2 * ks) * kFrag;
      const char *b = a + (rows / 2) * NT * kFrag;
      const int half = row & 1;
      return Split{join(pair_quad_t(a, half, lane), pair_quad_t(a + kFrag, half, lane)),
                   join(pair_quad_t(b, half, lane), pair_quad_t(b + kFrag, half, lane))};
    };
    auto Uf = [&](int tile, int ks) { return tile_split(lds + L::kU, tile, 4, ks); };
    auto Ff = [&](int tile, int ks) { return tile_split(lds + L::kF, tile, 4, ks); };
    bf8 d[KV];
    Split u_[KV], f[KV];
#pragma unroll
    for (int ks = 0; ks < KV; ++ks) {
      d[ks] = rows_frag<DV>(D, 16 * w, 32 * ks, lane);
      u_[ks] = Uf(w, ks);
      f[ks] = Ff(w, ks);
    }
    const float ghi = gate[kGhi * C + tok], glo = gate[kGlo * C + tok];
    const float bet = gate[kBeta * C + tok], gam = gate[kGam * C + tok];

    // The triangular products, as operands: [lane i, over j] and [lane j, over i].
    Split pt[2], at_[2], pn[2], an[2];
    {
      f4 p[4], a[4];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        p[jt] = a[jt] = 0.f;
        if (jt <= w) {
#pragma unroll
          for (int ks = 0; ks < KV; ++ks) {
            const Split x = Uf(jt, ks);
            p[jt] = dot2(x, d[ks], p[jt]);
            a[jt] = dot3(x, f[ks], a[jt]);
          }
          const f4 hj = *reinterpret_cast<const f4 *>(gate + kGhi * C + 16 * jt + 4 * h);
          const f4 lj = *reinterpret_cast<const f4 *>(gate + kGlo * C + 16 * jt + 4 * h);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * jt + 4 * h + r;
            const float x = exp2f((ghi - hj[r]) + (glo - lj[r]));
            p[jt][r] = tok >= j ? p[jt][r] * x : 0.f;
            a[jt][r] = tok > j ? -a[jt][r] * x : 0.f;
          }
        }
      }
      pt[0] = split8(p[0], p[1]); pt[1] = split8(p[2], p[3]);
      at_[0] = split8(a[0], a[1]); at_[1] = split8(a[2], a[3]);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        p[it] = a[it] = 0.f;
        if (it >= w) {
#pragma unroll
          for (int ks = 0; ks < KV; ++ks) {
            p[it] = dot2(rows_frag<DV>(D, 16 * it, 32 * ks, lane), u_[ks], p[it]);
            a[it] = dot3(Ff(it, ks), u_[ks], a[it]);
          }
          const f4 hi = *reinterpret_cast<const f4 *>(gate + kGhi * C + 16 * it + 4 * h);
          const f4 li = *reinterpret_cast<const f4 *>(gate + kGlo * C + 16 * it + 4 * h);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * it + 4 * h + r;
            const float x = exp2f((hi[r] - ghi) + (li[r] - glo));
            p[it][r] = i >= tok ? p[it][r] * x : 0.f;
            a[it][r] = i > tok ? -a[it][r] * x : 0.f;
          }
        }
      }
      pn[0] = split8(p[0], p[1]); pn[1] = split8(p[2], p[3]);
      an[0] = split8(a[0], a[1]); an[1] = split8(a[2], a[3]);
    }
    // dV and dbeta from the wave's own rows.
    {
      float s = 0.f;
      const float own = tok < valid ? beta[(row0 + tok) * Hv + hv] : 0.f;
      const float back = own / bet;      // 1, or below 1 where beta was raised
      __hip_bfloat16 *o = dv_out + ((row0 + tok) * Hv + hv) * DV;
#pragma unroll
      for (int ks = 0; ks < KV; ++ks)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          auto part = [&](const Split &x) {
            const bf4 a = half ? __builtin_shufflevector(x.hi, x.hi, 4, 5, 6, 7)
                               : __builtin_shufflevector(x.hi, x.hi, 0, 1, 2, 3);
            const bf4 b = half ? __builtin_shufflevector(x.lo, x.lo, 4, 5, 6, 7)
                               : __builtin_shufflevector(x.lo, x.lo, 0, 1, 2, 3);
            return widen4(a) + widen4(b);
          };
          const f4 x = part(f[ks]);
          s += sum4(x * part(u_[ks]));
          if (tok < valid)
            *reinterpret_cast<bf4 *>(o + 32 * ks + 16 * half + 4 * h) = round4(x * back);
        }
      s = over_quarters(s);
      if (h == 0 && tok < valid) dbeta[(row0 + tok) * Hv + hv] = s / (bet * bet);
    }
    __syncthreads();
    {
      Linear<2 * kPlane> s;
      s.load(S_keep + ch * (2 * kPlane), t);
      s.store(lds + L::kX, t);
    }
    __syncthreads();
    auto Sf = [&](int mt, int ks) { return tile_split(lds + L::kX, mt, MT, ks); };
    float dG = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      f4 a = 0.f, b = 0.f;
#pragma unroll
      for (int ks = 0; ks < KV; ++ks) {
        const Split s = Sf(mt, ks);
        a = dot2(s, d[ks], a);
        b = dot3(s, f[ks], b);
      }
      a *= gam;
      b *= -gam;
      const bf8 k0 = cols_frag<DK>(K, 0, 16 * mt, lane), k1 = cols_frag<DK>(K, 32, 16 * mt, lane);
      const bf8 q0 = cols_frag<DK>(Q, 0, 16 * mt, lane), q1 = cols_frag<DK>(Q, 32, 16 * mt, lane);
      a = dot2(k0, pt[0], a);
      b = dot2(k0, at_[0], b);
      if (w >= 2) {                      // tiles j >= 32 lie above the diagonal for w < 2
        a = dot2(k1, pt[1], a);
        b = dot2(k1, at_[1], b);
      }
      f4 c = 0.f;
      if (w < 2) {
        c = dot2(q0, pn[0], c);
        c = dot2(k0, an[0], c);
      }
      c = dot2(q1, pn[1], c);
      c = dot2(k1, an[1], c);
      const int off = place_of<DK>(tok, 16 * mt + 4 * h);
      const f4 qv = widen4(*reinterpret_cast<const bf4 *>(Q + off));
      const f4 kv = widen4(*reinterpret_cast<const bf4 *>(K + off));
      dG += sum4(qv * a) + sum4(kv * (b - c));
      dQ[mt] += a;
      dK[mt] += b + c;
    }
    // <S, dS'>, then dS' in place of S.
    float dot = 0.f;
    {
      Linear<2 * kPlane> s;
      s.load(dS_keep + ch * (2 * kPlane), t);
      constexpr int kHalf = kPlane / (kThreads * 16);
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        const char *p = lds + L::kX + (t + i * kThreads) * 16;
        const u4 x = *reinterpret_cast<const u4 *>(p);
        const u4 y = *reinterpret_cast<const u4 *>(p + kPlane);
        const u4 z = s.r[i], v = s.r[i + kHalf];
        auto low = [](uint32_t a) { return __uint_as_float(a << 16); };
        auto high = [](uint32_t a) { return __uint_as_float(a & 0xFFFF0000u); };
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dot += (low(x[j]) + low(y[j])) * (low(z[j]) + low(v[j])) +
                 (high(x[j]) + high(y[j])) * (high(z[j]) + high(v[j]));
      }
      __syncthreads();
      s.store(lds + L::kX, t);
    }
    __syncthreads();
    const float last = gate[kLast * C + tok];
    float ws = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      f4 c = 0.f;
#pragma unroll
      for (int ks = 0; ks < KV; ++ks) c = dot3(Sf(mt, ks), u_[ks], c);
      c *= last;
      const f4 kv = widen4(*reinterpret_cast<const bf4 *>(K + place_of<DK>(tok, 16 * mt + 4 * h)));
      ws += sum4(kv * c);
      dK[mt] += c;
    }
    dG = over_quarters(dG - ws);
    if (h == 0) s_dG[tok] = dG;
    // sum_j w_j + gam_n <S, dS'> over the workgroup
    float n = ws + gate[kGam * C + C - 1] * dot;
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
    if (lane == 0) s_n[w] = n;
    __syncthreads();
    if (w == 0) {
      float x = s_dG[lane];
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float y = __shfl_down(x, o);
        if (lane + o < 64) x += y;
      }
      x += (s_n[0] + s_n[1]) + (s_n[2] + s_n[3]);
      if (lane < valid) {
        const size_t gi = (row0 + lane) * Hv + hv;
        dg[gi] = g[gi] < (float)kGateFloor ? 0.f : x;   // a floored gate is constant
      }
    }
    __syncthreads();
  }
  if (tok < valid) {
    const size_t o = ((row0 + tok) * Hk + hk) * DK + 4 * h;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      *reinterpret_cast<bf4 *>(dq + o + 16 * mt) = round4(dQ[mt]);
      *reinterpret_cast<bf4 *>(dk_out + o + 16 * mt) = round4(dK[mt]);
    }
  }
}

template <int DK, int DV> hipError_t backward_typed(const GdrBwdArgs &a, hipStream_t st) {
  const GdrArgs &f = a.fwd;
  const auto *q = static_cast<const __hip_bfloat16 *>(f.q);
  const auto *k = static_cast<const __hip_bfloat16 *>(f.k);
  const auto *d_o = static_cast<const __hip_bfloat16 *>(a.d_o);
  char *rec = static_cast<char *>(a.rec), *S = static_cast<char *>(a.S);
  char *U = static_cast<char *>(a.U), *dS = static_cast<char *>(a.dS);
  char *F = static_cast<char *>(a.F);
  if (hipError_t e = launch_gdr_keep(f, rec, S, U, st); e != hipSuccess) return e;
  constexpr int lds = ReverseLds<DK>::kBytes;
  auto *rev = reverse_kernel<DK, DV>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(rev),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  const unsigned pairs = (unsigned)((f.N * f.Hv + 7) / 8 * 8);
  hipLaunchKernelGGL(rev, dim3(pairs * (DV / 64)), dim3(2 * kThreads), lds, st, q, k, d_o, a.dS_T,
                     f.tab, f.N, f.Hk, f.Hv, rec, dS, F, a.dS0);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (f.n_chunks_ub == 0) return hipSuccess;
  auto *gr = grad_kernel<DK, DV>;
  constexpr int gl = GradLds<DK, DV>::kBytes;
  e = hipFuncSetAttribute(reinterpret_cast<const void *>(gr),
                          hipFuncAttributeMaxDynamicSharedMemorySize, gl);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gr, dim3((unsigned)(f.n_chunks_ub * f.Hk)), dim3(kThreads), gl, st, q, k, f.g,
                     f.beta, d_o, f.tab, f.N, f.Hk, f.Hv, rec, S, U, dS, F,
                     static_cast<__hip_bfloat16 *>(a.dq), static_cast<__hip_bfloat16 *>(a.dk),
                     static_cast<__hip_bfloat16 *>(a.dv), a.dg, a.dbeta);
  return hipGetLastError();
}

}  // namespace

GdrBwdBytes gdr_backward_bytes(int dk, int dv) {
  return {(size_t)kRecBwd, (size_t)4 * dk * dv, (size_t)4 * C * dv};
}

hipError_t launch_gdr_backward(const GdrBwdArgs &a, hipStream_t stream) {
  if (a.fwd.dk == 64)
    return a.fwd.dv == 64 ? backward_typed<64, 64>(a, stream) : backward_typed<64, 128>(a, stream);
  return a.fwd.dv == 64 ? backward_typed<128, 64>(a, stream) : backward_typed<128, 128>(a, stream);
}

}  // namespace ckda
