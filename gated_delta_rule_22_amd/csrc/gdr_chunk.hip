// Chunkwise gated delta rule for bf16 inputs.
//
// With a = exp(g), G_i the running sum of g in a 64-token chunk, r_ij =
// e^(G_i - G_j), gam_i = e^(G_i) and S the state that enters the chunk:
//
//   Ah_ij = r_ij k_i.k_j (i > j)          P_ij = r_ij q_i.k_j (i >= j)
//   I + T = (I + Ah diag(beta))^-1        X = V - gam K S
//   U = beta (X + T X)                    O = gam Q S + P U
//   S <- gam_n S + K^T (gam_n / gam U)
//
// The gate is one number per token and head, so decays scale rows and columns
// of products of the bf16 inputs themselves: k and q stay exact bf16 operands
// (per-channel gates would have to be multiplied into them).
//
// prepare_kernel makes T, P and the gate factors of every chunk in parallel;
// chain_kernel runs the chunks of a (sequence, head) in order.
#include "gdr_chunk.h"

namespace ckda {
using namespace gdr;
namespace {

// ------------------------------------------------------------------ prepare
// One wave per (chunk, value head), four to a workgroup, no barriers.  The
// 64 x 64 unit lower triangular inverse is taken in fp32: its 16 x 16 diagonal
// blocks by substitution, what is below them by matrix products (substitution
// over all 64 rows takes 2016 steps a wave and as many LDS broadcasts: 127 us
// where this takes 94).  8 x 4096 tokens, 16 heads, 128 channels: 94 us for 448 MB
// read and written (4.8 TB/s), 108 us for 508 MB with the backward's records, so
// memory bounds it.
constexpr int kMStride = C + 4;          // floats; keeps rows 16-byte aligned

template <int DK, bool BWD>
__global__ __launch_bounds__(kThreads) void prepare_kernel(
    const __hip_bfloat16 *__restrict__ q, const __hip_bfloat16 *__restrict__ k,
    const float *__restrict__ g, const float *__restrict__ beta, Seqs seqs, int N, int Hk,
    int Hv, char *__restrict__ rec_base) {
  constexpr int KS = DK / 32;
  constexpr int kRec = BWD ? kRecBwd : kRecFwd;
  __shared__ float s_M[4][C * kMStride];
  __shared__ float s_g[4][3][C];         // G hi, G lo (log2 units), beta
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int m = lane & 15, h = lane >> 4;
  const int per = (Hv + 3) / 4;
  const int chunk = blockIdx.x / per, hv = (blockIdx.x % per) * 4 + wave;
  if (hv >= Hv || chunk >= seqs.first_chunk(N)) return;   // waves share nothing
  const int seq = seqs.of_chunk(chunk, N);
  const int at = (chunk - seqs.first_chunk(seq)) * C;
  const int valid = min(C, seqs.len(seq) - at);
  const size_t row0 = (size_t)seqs.start(seq) + at;
  const int hk = hv / (Hv / Hk);
  char *rec = rec_base + ((size_t)chunk * Hv + hv) * kRec;
  float *M = s_M[wave], *s_hi = s_g[wave][0], *s_lo = s_g[wave][1], *s_b = s_g[wave][2];

  // Gate factors.  The running sum is fp64: a forgetful token early in the
  // chunk must not cost the later tokens' differences their low bits.
  double G = 0.;
  float b = 0.f;
  if (lane < valid) {
    const float x = g[(row0 + lane) * Hv + hv];
    G = x < (float)kGateFloor ? kGateFloor : (double)x;
    b = beta[(row0 + lane) * Hv + hv];
  }
  if (fabsf(b) < kBetaFloor) b = copysignf(kBetaFloor, b);
  G *= 1.4426950408889634074;            // log2 units
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(G, o);
    if (lane >= o) G += y;
  }
  const double Gn = __shfl(G, 63);
  auto pow2d = [](double x) {             // 2^x; whole and fractional part apart
    const double w = rint(x);
    return ldexpf(exp2f((float)(x - w)), (int)fmin(fmax(w, -3e4), 3e4));
  };
  const float gam = pow2d(G), last = pow2d(Gn - G);
  const float ghi = (float)G, glo = (float)(G - (double)ghi);
  s_hi[lane] = ghi;
  s_lo[lane] = glo;
  s_b[lane] = b;
  float *gate = reinterpret_cast<float *>(rec + kRecGate);
  gate[kGam * C + lane] = gam;
  gate[kLast * C + lane] = last;
  gate[kBeta * C + lane] = b;
  gate[kGhi * C + lane] = ghi;
  gate[kGlo * C + lane] = glo;

  bf8 kf[4][KS];
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int r = 16 * it + m;
      kf[it][ks] = __builtin_bit_cast(
          bf8, load16(k + ((row0 + r) * Hk + hk) * DK + 32 * ks + 8 * h, r < valid));
    }
  wave_sync();

  // Ah diag(beta) to LDS: tile (it, jt), lane = column j, rows i = 4h ..
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const f4 hi_i = *reinterpret_cast<const f4 *>(s_hi + 16 * it + 4 * h);
    const f4 lo_i = *reinterpret_cast<const f4 *>(s_lo + 16 * it + 4 * h);
#pragma unroll
    for (int jt = 0; jt <= it; ++jt) {
      f4 a = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) a = mfma(kf[it][ks], kf[jt][ks], a);
      const int j = 16 * jt + m;
      const float hj = s_hi[j], lj = s_lo[j], bj = s_b[j];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * it + 4 * h + r;
        const float e = (hi_i[r] - hj) + (lo_i[r] - lj);
        M[i * kMStride + j] = i > j ? a[r] * pow2(e) * bj : 0.f;
      }
    }
  }

  // P in operand order: tiles transposed, lane = row i, 4 columns j at a time.
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    bf8 qf[KS];
    const int i = 16 * it + m;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qf[ks] = __builtin_bit_cast(
          bf8, load16(q + ((row0 + i) * Hk + hk) * DK + 32 * ks + 8 * h, i < valid));
    }
    const float hi_i = s_hi[i], lo_i = s_lo[i];
#pragma unroll
    for (int kp = 0; kp <= it / 2; ++kp) {
      auto tile = [&](int jt) {
        f4 p = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) p = mfma(kf[jt][ks], qf[ks], p);
        const f4 hj = *reinterpret_cast<const f4 *>(s_hi + 16 * jt + 4 * h);
        const f4 lj = *reinterpret_cast<const f4 *>(s_lo + 16 * jt + 4 * h);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = (hi_i - hj[r]) + (lo_i - lj[r]);
          const int j = 16 * jt + 4 * h + r;
          if (BWD && i == j) gate[kDiagP * C + i] = p[r];
          p[r] = (BWD ? i > j : i >= j) ? p[r] * pow2(x) : 0.f;
        }
        return p;
      };
      const f4 p0 = tile(2 * kp);
      f4 p1 = 0.f;
      if (2 * kp + 1 <= it) p1 = tile(2 * kp + 1);
      const Split s = split8(p0, p1);
      *reinterpret_cast<bf8 *>(rec + kRecPh + frag_at(it, kp) + lane * 16) = s.hi;
      if (BWD) *reinterpret_cast<bf8 *>(rec + kRecPl + frag_at(it, kp) + lane * 16) = s.lo;
    }
  }
  wave_sync();

  // The inverse, in place.  Diagonal 16 x 16 blocks by forward substitution,
  // one column of one block a lane.
  {
    float x[16];
    float *D = M + (16 * h) * kMStride + 16 * h;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      f4 s = 0.f;
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const f4 a = *reinterpret_cast<const f4 *>(D + i * kMStride + j);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < i) s[e] += a[e] * x[j + e];
      }
      x[i] = (i == m ? 1.f : 0.f) - ((s[0] + s[1]) + (s[2] + s[3]));
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i * kMStride + m] = x[i];
    wave_sync();
  }
  // The blocks below them, T21 = -T22 (A21 T11), on fp32 matrix products.  A
  // product's left operand is read as rows; its right one has the layout of a
  // result (column m, rows 4h ..), so products follow each other in registers.
  auto block = [&](int i, int j) {
    return *reinterpret_cast<const f4 *>(M + (16 * i + m) * kMStride + 16 * j + 4 * h);
  };
  auto times = [](f4 a, f4 b, f4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
  };
  auto keep = [&](int i, int j, f4 x) {
#pragma unroll
    for (int r = 0; r < 4; ++r) M[(16 * i + 4 * h + r) * kMStride + 16 * j + m] = x[r];
  };
  {
    f4 t[4];                             // diagonal blocks as right operands
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) t[d][r] = M[(16 * d + 4 * h + r) * kMStride + 16 * d + m];
    const f4 none = 0.f;
    const f4 t10 = -times(block(1, 1), times(block(1, 0), t[0], none), none);
    const f4 t32 = -times(block(3, 3), times(block(3, 2), t[2], none), none);
    wave_sync();
    keep(1, 0, t10);
    keep(3, 2, t32);
    wave_sync();
    f4 x[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f4 a0 = block(2 + i, 0), a1 = block(2 + i, 1);
      x[i][0] = times(a1, t10, times(a0, t[0], none));
      x[i][1] = times(a1, t[1], none);
    }
    const f4 b22 = block(2, 2), b32 = block(3, 2), b33 = block(3, 3);
    wave_sync();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      keep(2, j, -times(b22, x[0][j], none));
      keep(3, j, -times(b33, x[1][j], times(b32, x[0][j], none)));
    }
  }
  wave_sync();
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int ks = 0; ks <= it / 2; ++ks) {
      const float *p = M + (16 * it + m) * kMStride + 32 * ks + 4 * h;
      // without the unit diagonal, which the chain adds in fp32; the tile right
      // of an even diagonal one lies above the diagonal
      f4 left = *reinterpret_cast<const f4 *>(p), right = 0.f;
      if (2 * ks + 1 <= it) right = *reinterpret_cast<const f4 *>(p + 16);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (2 * ks == it && 4 * h + r == m) left[r] = 0.f;
        if (2 * ks + 1 == it && 4 * h + r == m) right[r] = 0.f;
      }
      const Split s = split8(left, right);
      *reinterpret_cast<bf8 *>(rec + kRecTh + frag_at(it, ks) + lane * 16) = s.hi;
      *reinterpret_cast<bf8 *>(rec + kRecTl + frag_at(it, ks) + lane * 16) = s.lo;
    }
}

// Workgroups of one (sequence, head) -- its column blocks -- share an XCD's
// L2: consecutive workgroups go round the 8 XCDs.
__device__ __forceinline__ bool chain_block(int nblk, int pairs, int &pair, int &blk) {
  const int b = blockIdx.x;
  blk = (b / 8) % nblk;
  pair = (b / 8 / nblk) * 8 + b % 8;
  return pair < pairs;
}

// -------------------------------------------------------------------- chain
// A workgroup runs BV of the state's DV columns of one (sequence, head) over
// its chunks.  Its chain waves own 16 columns each for the whole sequence, so
// the chain S -> K S -> U -> S of a column never leaves its wave: S is 4 DK /
// 16 accumulator registers, and each product's result tiles are the next one's
// operand.  Four helper waves do what the chain does not wait for: they load
// the next chunk and make the output of this one.  Two barriers a chunk:
// A, when the chunk's operands and S's terms are in LDS, and B, when the chain
// has read all of them into registers and has written U; the next chunk's
// operands take their places between B and the next A.
// STORE: for the backward, keeps the state before each chunk and U (two bf16
// terms each) and makes no output.
//
// A chunk takes 2.6 to 3.1 us (5800 cycles) on 64 columns, and 2.26 on 32, where
// two helpers share a chain wave's output: the chain's own latency, K S (1300
// cycles), T X (1000), U's terms and the barrier (700), K^T U (1600) and the
// next state's terms (1000), each of which waits for the one before; 1400 of
// them are matrix instructions.  8 x 4096 tokens of 16 heads of 128 x 128: 203 to
// 212 us for 714 MB (3.5 TB/s); STORE 240 us for 1.24 GB (5.2 TB/s, a copy's
// rate).  Tried and slower: operands a whole chunk ahead (255 us, too many
// registers), half of the products with the state behind barrier B with K and Q
// twice in LDS (217), U's terms and barrier B behind the products of the next
// state (238: the helpers wait), rows padded instead of the swizzle (+15%).
template <int DK, int BV, bool STORE> struct ChainLds {
  static constexpr int kK = 0, kV = gdr::kTile<DK>, kRec = kV + gdr::kTile<BV>;
  static constexpr int kQ = kRec + kRecFwd;                      // the rest: !STORE
  static constexpr int kS = kQ + gdr::kTile<DK>, kSWave = 2 * (DK / 32) * kFrag;
  static constexpr int kU = kS + BV / 16 * kSWave;
  static constexpr int kBytes = STORE ? kQ : kU + BV / 16 * 4 * kFrag;
};

template <int DK, int DV, int BV, bool STORE>
__global__ __launch_bounds__(4 * BV + kThreads, 2) void chain_kernel(
    const __hip_bfloat16 *__restrict__ q, const __hip_bfloat16 *__restrict__ k,
    const __hip_bfloat16 *__restrict__ v, const float *__restrict__ S0, Seqs seqs, int N,
    int Hk, int Hv, const char *__restrict__ rec_base, __hip_bfloat16 *__restrict__ o,
    float *__restrict__ S_T, char *__restrict__ S_keep, char *__restrict__ U_keep,
    bool by_lengths) {
  using L = ChainLds<DK, BV, STORE>;
  constexpr int KS = DK / 32, MT = DK / 16, kWaves = BV / 16;
  constexpr int kRec = STORE ? kRecBwd : kRecFwd;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int pair, blk;
  if (!chain_block(DV / BV, N * Hv, pair, blk)) return;
  if (!STORE && by_lengths) {            // as many pairs as the longest one's time has room for
    const size_t longest = (seqs.len(seqs.order(0)) + C - 1) / C;
    const bool few = (size_t)seqs.first_chunk(N) * Hv * (DV / 64) <= kFewBlocks * longest;
    if (few != (BV == 32)) return;
  }
  const int seq = seqs.order(pair / Hv), hv = pair % Hv, hk = hv / (Hv / Hk);
  const bool helper = threadIdx.x >= 64 * kWaves;
  const int wave = (threadIdx.x >> 6) % kWaves;   // its columns
  const int lane = threadIdx.x & 63, m = lane & 15, h = lane >> 4;
  const int len = seqs.len(seq), chunks = (len + C - 1) / C;
  const size_t row0 = seqs.start(seq);
  const size_t c0 = seqs.first_chunk(seq);
  const int col = blk * BV + 16 * wave;  // of the head's DV
  const char *K = lds + L::kK, *V = lds + L::kV, *R = lds + L::kRec, *Q = lds + L::kQ;
  const float *gate = reinterpret_cast<const float *>(R + kRecGate);
  char *s_S = lds + L::kS + wave * L::kSWave + lane * 16;
  char *s_U = lds + L::kU + wave * 4 * kFrag + lane * 16;

  if (helper) {
    const int t = threadIdx.x - 64 * kWaves;
    // A helper's 16-token tiles of the output: all four, or half where two
    // helpers share 16 columns.
    constexpr int kIt = kWaves;
    const int it0 = kIt == 4 ? 0 : __builtin_amdgcn_readfirstlane(t / 64 / kWaves) * kIt;
    Stage<DK> gk, gq;
    Stage<BV> gv;
    Linear<kRecFwd> gr;
    auto fetch = [&](int c) {
      const int valid = min(C, len - c * C);
      const size_t row = row0 + (size_t)c * C;
      gk.load(k + (row * Hk + hk) * DK, (size_t)Hk * DK, valid, t);
      if (!STORE) gq.load(q + (row * Hk + hk) * DK, (size_t)Hk * DK, valid, t);
      gv.load(v + (row * Hv + hv) * DV + blk * BV, (size_t)Hv * DV, valid, t);
      gr.load(rec_base + ((c0 + c) * Hv + hv) * kRec, t);
    };
    auto put = [&](int c) {
      const int valid = min(C, len - c * C);
      gk.store(lds + L::kK, valid, t);
      if (!STORE) gq.store(lds + L::kQ, valid, t);
      gv.store(lds + L::kV, valid, t);
      gr.store(lds + L::kRec, t);
    };
    if (chunks > 0) {
      fetch(0);
      put(0);
    }
    for (int c = 0; c < chunks; ++c) {
      lds_barrier();                     // A
      const int next = min(c + 1, chunks - 1);   // the last one again: read by nobody
      fetch(next);
      f4 a[kIt];
      bf8 p[kIt][2];
      if (!STORE) {
        // O, transposed: lane = token, 4 columns a lane.
        Split s[KS];
        bf8 qf[KS][kIt];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          s[ks] = {*reinterpret_cast<const bf8 *>(s_S + ks * kFrag),
                   *reinterpret_cast<const bf8 *>(s_S + (KS + ks) * kFrag)};
#pragma unroll
          for (int i = 0; i < kIt; ++i)
            qf[ks][i] = rows_frag<DK>(Q, 16 * (it0 + i), 32 * ks, lane);
        }
        fence_schedule();
#pragma unroll
        for (int i = 0; i < kIt; ++i) a[i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
          for (int i = 0; i < kIt; ++i) a[i] = mfma(s[ks].hi, qf[ks][i], a[i]);
#pragma unroll
          for (int i = 0; i < kIt; ++i) a[i] = mfma(s[ks].lo, qf[ks][i], a[i]);
        }
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          a[i] *= gate[kGam * C + 16 * (it0 + i) + m];
          p[i][0] = tri_frag(R + kRecPh, it0 + i, 0, lane);
          p[i][1] = it0 + i < 2 ? p[i][0] : tri_frag(R + kRecPh, it0 + i, 1, lane);
        }
      }
      lds_barrier();                     // B
      put(next);                         // before the stores, which loads' waits count too
      if (!STORE) {
        // One term of P: it is within 2^-9 of its value, and so is the bf16
        // output itself.
        const Split u0 = {*reinterpret_cast<const bf8 *>(s_U),
                          *reinterpret_cast<const bf8 *>(s_U + 2 * kFrag)};
        const Split u1 = {*reinterpret_cast<const bf8 *>(s_U + kFrag),
                          *reinterpret_cast<const bf8 *>(s_U + 3 * kFrag)};
#pragma unroll
        for (int i = 0; i < kIt; ++i) a[i] = dot2(u0, p[i][0], a[i]);
        if (kIt == 4 || it0 > 0)
#pragma unroll
          for (int i = kIt == 4 ? 2 : 0; i < kIt; ++i) a[i] = dot2(u1, p[i][1], a[i]);
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          const int tok = c * C + 16 * (it0 + i) + m;
          if (tok < len)
            *reinterpret_cast<bf4 *>(o + ((row0 + tok) * Hv + hv) * DV + col + 4 * h) =
                round4(a[i]);
        }
      }
    }
    return;
  }

  f4 S[MT];
  const size_t sbase = ((size_t)seq * Hv + hv) * DK * DV + col + m;
#pragma unroll
  for (int i = 0; i < MT; ++i) S[i] = 0.f;
  if (S0)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = S0[sbase + (size_t)(16 * i + 4 * h + r) * DV];

  // The gate factors of a lane's tokens come from memory a chunk ahead: read
  // from LDS they would be 9 cycles of its time each for 64 bytes.
  f4 gam[4], last[4], bet[4];
  float gn = 0.f;
  auto fetch_gates = [&](int c) {
    const float *g = reinterpret_cast<const float *>(rec_base + ((c0 + c) * Hv + hv) * kRec +
                                                     kRecGate);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      gam[it] = *reinterpret_cast<const f4 *>(g + kGam * C + 16 * it + 4 * h);
      last[it] = *reinterpret_cast<const f4 *>(g + kLast * C + 16 * it + 4 * h);
      bet[it] = *reinterpret_cast<const f4 *>(g + kBeta * C + 16 * it + 4 * h);
    }
    gn = g[kGam * C + C - 1];
  };
  if (chunks > 0) fetch_gates(0);
  __builtin_amdgcn_s_setprio(2);         // the chain before the helper on its SIMD
  for (int c = 0; c < chunks; ++c) {
    Split sf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      sf[ks] = split8(S[2 * ks], S[2 * ks + 1]);
      if (!STORE) {
        *reinterpret_cast<bf8 *>(s_S + ks * kFrag) = sf[ks].hi;
        *reinterpret_cast<bf8 *>(s_S + (KS + ks) * kFrag) = sf[ks].lo;
      }
    }
    lds_barrier();                       // A
    if (STORE) {
      char *p = S_keep + (((c0 + c) * Hv + hv) * (2 * KS * (DV / 16)) + col / 16) * kFrag +
                lane * 16;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        *reinterpret_cast<bf8 *>(p + ks * (DV / 16) * kFrag) = sf[ks].hi;
        *reinterpret_cast<bf8 *>(p + (KS + ks) * (DV / 16) * kFrag) = sf[ks].lo;
      }
    }
    // X = V - gam K S, as the operand of T' X
    bf8 kf[KS][4];
    f4 X[4];
    auto read_k = [&](int ks) {
#pragma unroll
      for (int it = 0; it < 4; ++it) kf[ks][it] = rows_frag<DK>(K, 16 * it, 32 * ks, lane);
    };
    auto times_s = [&](int ks) {
#pragma unroll
      for (int it = 0; it < 4; ++it) X[it] = mfma(kf[ks][it], sf[ks].hi, ks ? X[it] : f4(0.f));
#pragma unroll
      for (int it = 0; it < 4; ++it) X[it] = mfma(kf[ks][it], sf[ks].lo, X[it]);
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
    bf4 vq[4];
    Split T[6];
#pragma unroll
    for (int it = 0; it < 4; ++it) vq[it] = cols_quad<BV>(V, 16 * it, 16 * wave, lane);
#pragma unroll
    for (int f = 0; f < 6; ++f)
      T[f] = {*reinterpret_cast<const bf8 *>(R + kRecTh + f * kFrag + lane * 16),
              *reinterpret_cast<const bf8 *>(R + kRecTl + f * kFrag + lane * 16)};
#pragma unroll
    for (int ks = 1; ks < KS; ++ks) times_s(ks);
    fence_schedule();
    bf8 kt[2][MT];                       // K^T for the update, read meanwhile
#pragma unroll
    for (int i = 0; i < MT; ++i) kt[0][i] = cols_frag<DK>(K, 0, 16 * i, lane);
#pragma unroll
    for (int it = 0; it < 4; ++it) X[it] = widen4(vq[it]) - gam[it] * X[it];
    const Split x0 = split8(X[0], X[1]), x1 = split8(X[2], X[3]);
    fence_schedule();
    f4 U[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) U[it] = X[it];
    // the four tiles' products turn by turn: each waits for its own last one
#pragma unroll
    for (int term = 0; term < 4; ++term)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int it = 2 * ks; it < 4; ++it) {
          const Split &t = T[frag_at(it, ks) / kFrag];
          const Split &x = ks ? x1 : x0;
          U[it] = mfma(term & 2 ? t.lo : t.hi, term & 1 ? x.lo : x.hi, U[it]);
        }
#pragma unroll
    for (int i = 0; i < MT; ++i) S[i] *= gn;
#pragma unroll
    for (int i = 0; i < MT; ++i) kt[1][i] = cols_frag<DK>(K, 32, 16 * i, lane);
#pragma unroll
    for (int it = 0; it < 4; ++it) U[it] *= bet[it];
    {
      const Split u0 = split8(U[0], U[1]), u1 = split8(U[2], U[3]);
      char *p = STORE ? U_keep + (((c0 + c) * Hv + hv) * (4 * (DV / 16)) + col / 16) * kFrag +
                            lane * 16
                      : s_U;
      constexpr int step = STORE ? (DV / 16) * kFrag : kFrag;
      *reinterpret_cast<bf8 *>(p) = u0.hi;
      *reinterpret_cast<bf8 *>(p + step) = u1.hi;
      *reinterpret_cast<bf8 *>(p + 2 * step) = u0.lo;
      *reinterpret_cast<bf8 *>(p + 3 * step) = u1.lo;
    }
    fence_schedule();
    lds_barrier();                       // B
    fence_schedule();
#pragma unroll
    for (int it = 0; it < 4; ++it) U[it] *= last[it];
    fetch_gates(min(c + 1, chunks - 1));
    const Split w0 = split8(U[0], U[1]), w1 = split8(U[2], U[3]);
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
  if (S_T)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S_T[sbase + (size_t)(16 * i + 4 * h + r) * DV] = S[i][r];
}

unsigned chain_grid(int pairs, int nblk) { return (unsigned)((pairs + 7) / 8 * 8) * nblk; }

template <typename F> hipError_t allow_lds(F *f, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void *>(f),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DK, int DV, int BV, bool STORE>
hipError_t launch_chain(const GdrArgs &a, char *rec, char *S, char *U, bool by_lengths,
                        hipStream_t st) {
  constexpr int lds = ChainLds<DK, BV, STORE>::kBytes;
  auto *kernel = chain_kernel<DK, DV, BV, STORE>;
  if (hipError_t e = allow_lds(kernel, lds); e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(chain_grid(a.N * a.Hv, DV / BV)), dim3(4 * BV + kThreads), lds, st,
                     static_cast<const __hip_bfloat16 *>(a.q),
                     static_cast<const __hip_bfloat16 *>(a.k),
                     static_cast<const __hip_bfloat16 *>(a.v), a.S0, a.seqs, a.N, a.Hk, a.Hv, rec,
                     static_cast<__hip_bfloat16 *>(a.o), a.S_T, S, U, by_lengths);
  return hipGetLastError();
}

// prepare, then the chain; with STORE it keeps S and U and makes no output.
template <int DK, int DV, bool STORE>
hipError_t forward_typed(const GdrArgs &a, char *rec, char *S, char *U, hipStream_t st) {
  const auto *q = static_cast<const __hip_bfloat16 *>(a.q);
  const auto *k = static_cast<const __hip_bfloat16 *>(a.k);
  if (a.n_chunks_ub > 0) {
    hipLaunchKernelGGL((prepare_kernel<DK, STORE>),
                       dim3((unsigned)(a.n_chunks_ub * ((a.Hv + 3) / 4))), dim3(kThreads), 0, st,
                       q, k, a.g, a.beta, a.seqs, a.N, a.Hk, a.Hv, rec);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  const bool few = chain_columns(a.N * a.Hv, DV) == 32;
  // Packed sequences that are many, but of which a few may be long: the lengths
  // say on the device which of the two kernels runs, and the other one ends at
  // once (ten sequences, the longest 8192 tokens, of 16 heads of 128 x 128: 289
  // against 336 us).  Both are launched where the order by length is known, and
  // where the longest can have so many chunks that their 0.35 us each pay for the
  // 4 us of the other launch: 64 chunks in all.
  const bool by_lengths = !STORE && !few && a.seqs.T < 0 && a.N <= kRankedSeqs &&
                          a.n_chunks_ub >= 64 + (size_t)a.N;
  if (few || by_lengths) {
    const hipError_t e = launch_chain<DK, DV, 32, STORE>(a, rec, S, U, by_lengths, st);
    if (e != hipSuccess || few) return e;
  }
  return launch_chain<DK, DV, 64, STORE>(a, rec, S, U, by_lengths, st);
}

template <bool STORE>
hipError_t forward_any(const GdrArgs &a, void *rec, void *S, void *E, hipStream_t st) {
  char *r = static_cast<char *>(rec), *s = static_cast<char *>(S), *e = static_cast<char *>(E);
  if (a.dk == 64)
    return a.dv == 64 ? forward_typed<64, 64, STORE>(a, r, s, e, st)
                      : forward_typed<64, 128, STORE>(a, r, s, e, st);
  return a.dv == 64 ? forward_typed<128, 64, STORE>(a, r, s, e, st)
                    : forward_typed<128, 128, STORE>(a, r, s, e, st);
}

}  // namespace

size_t gdr_forward_rec_bytes() { return kRecFwd; }

hipError_t launch_gdr_forward(const GdrArgs &a, void *rec, hipStream_t stream) {
  return forward_any<false>(a, rec, nullptr, nullptr, stream);
}
hipError_t launch_gdr_keep(const GdrArgs &a, void *rec, void *S, void *E, hipStream_t stream) {
  return forward_any<true>(a, rec, S, E, stream);
}

}  // namespace ckda
