// Norm of every query and key head with the position rotation in the same
// pass, its backward, and the rotation alone.
//
// A row is one (token, head) of d channels.  Forward:
//
//   n = x (sum x^2 [/ d] + eps)^(-1/2) [* w]           (or n = x [* w])
//   (y0, y1) = s (n0 cos - n1 sin, n1 cos + n0 sin)     over the pairs of the
//   first rd channels (i, i + rd/2) or (2i, 2i + 1);  y = n behind them
//
// and q rows are multiplied by q_scale.  Backward, with dn the rotation of dy
// by the opposite angle: dw = sum dn n / w over all rows, and
// dx = rs (w dn - xh m), xh = rs x, m = sum (w dn) xh [/ d].
//
// Everything here reads its rows once and writes them once, so HBM traffic is
// the bound.  One thread holds 2V channels that are V whole pairs, so nothing
// but the row's sum crosses lanes: G = d / 2V lanes (rounded up to a power of
// two) share a row.  A workgroup takes the query or the key heads of kTok
// tokens at a time (one weight to keep, not two), loads a row ahead, and
// computes the tokens' cosines and sines once into LDS for all of their heads:
// an angle costs an fp64 product (pos * f in turns, reduced exactly, so that
// positions of a million and more lose nothing) and an fp32 sincospi, about as
// much work as the rest of a pair.
//
// 32768 tokens of 16 query and 16 key heads of 128 channels, bf16, norm and full
// rotation: forward 102 us for 537 MB (5.3 TB/s; a copy reaches 5.16), backward
// 153 + 4.3 us for 805 MB (5.2 TB/s); the rotation alone of 65536 x 16 heads,
// half of their channels, 95 us (5.6 TB/s).  64 tokens: 3.9 us.
#include "ckda_internal.h"

namespace ckda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;          // rd <= 256
constexpr int kRotaryTile = 8;          // tokens of a workgroup's tile where there are many
constexpr int kRotaryManyTokens = 1024;

// V elements of T as they lie in memory.
template <int BYTES> struct RawOf { struct Type { uint4 a[BYTES / 16]; }; };
template <> struct RawOf<8> { using Type = uint2; };
template <> struct RawOf<4> { using Type = uint32_t; };
template <> struct RawOf<2> { using Type = uint16_t; };
template <typename T, int V> struct Raw {
  typename RawOf<V * (int)sizeof(T)>::Type r[2];
};

// 2V channels of a row: V first and V second elements of its pairs.
template <int V> struct Unit { float a[V], b[V]; };

// Offsets within a row of a unit's first and second V channels in memory, and
// whether they are rotated.  In the interleaved layout (and behind the rotated
// part) the 2V channels are contiguous and the pairs are (even, odd).
struct Place { int p0, p1, pair; bool rot, half; };
template <int V> __device__ __forceinline__ Place place(int u, int rd, bool half) {
  Place pl;
  pl.rot = u < rd / (2 * V);
  pl.half = half && pl.rot;
  pl.pair = u * V;
  pl.p0 = pl.half ? u * V : 2 * V * u;
  pl.p1 = pl.half ? rd / 2 + u * V : 2 * V * u + V;
  return pl;
}

template <int V, typename T>
__device__ __forceinline__ Raw<T, V> load_raw(const T *row, const Place &pl) {
  Raw<T, V> x;
  using R = typename RawOf<V * (int)sizeof(T)>::Type;
  x.r[0] = *reinterpret_cast<const R *>(row + pl.p0);
  x.r[1] = *reinterpret_cast<const R *>(row + pl.p1);
  return x;
}
template <int V, typename T>
__device__ __forceinline__ Unit<V> unpack(const Raw<T, V> &raw, const Place &pl) {
  struct Both { T v[2 * V]; };
  const Both b = __builtin_bit_cast(Both, raw);
  float x[2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) x[i] = to_f32(b.v[i]);
  Unit<V> u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    u.a[i] = pl.half ? x[i] : x[2 * i];
    u.b[i] = pl.half ? x[V + i] : x[2 * i + 1];
  }
  return u;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  b2 r = {(__bf16)a, (__bf16)b};         // v_cvt_pk_bf16_f32: nearest even
  return __builtin_bit_cast(uint32_t, r);
}
template <int V> __device__ __forceinline__ void store_vec(__hip_bfloat16 *p, const float *x) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]),
                                               pack2(x[4], x[5]), pack2(x[6], x[7]));
  else if constexpr (V == 4)
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
  else
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = __float2bfloat16(x[i]);
}
template <int V> __device__ __forceinline__ void store_vec(float *p, const float *x) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = x[i];
  }
}
template <int V, typename T>
__device__ __forceinline__ void store_unit(T *row, const Place &pl, const Unit<V> &r) {
  float x[2 * V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[2 * i] = pl.half ? 0.f : r.a[i];
    x[2 * i + 1] = pl.half ? 0.f : r.b[i];
  }
  if (pl.half) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = r.a[i];
      x[V + i] = r.b[i];
    }
  }
  store_vec<V>(row + pl.p0, x);
  store_vec<V>(row + pl.p1, x + V);
}
template <int V>
__device__ __forceinline__ Unit<V> load_weight(const float *w, const Place &pl) {
  Unit<V> u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    u.a[i] = w ? w[pl.half ? pl.p0 + i : pl.p0 + 2 * i] : 1.f;
    u.b[i] = w ? w[pl.half ? pl.p1 + i : pl.p0 + 2 * i + 1] : 1.f;
  }
  return u;
}

template <int V>
__device__ __forceinline__ void rotate(Unit<V> &x, const float2 *cs, const Place &pl,
                                       bool inverse) {
  if (!pl.rot) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float2 t = cs[pl.pair + i];
    const float s = inverse ? -t.y : t.y;
    const float a = x.a[i], b = x.b[i];
    x.a[i] = a * t.x - b * s;
    x.b[i] = b * t.x + a * s;
  }
}

// cos and sin (times `scale`) of nt tokens' angles into LDS.
__device__ __forceinline__ void angles(float2 (*s_cs)[kMaxPairs], const int32_t *pos,
                                       const double *freqs, int t0, int nt, int pairs,
                                       float scale) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    const double turns = (double)pos[t0 + t] * (freqs[p] * kInvTwoPi);
    const float f = (float)(turns - rint(turns));   // in [-1/2, 1/2]
    float s, c;
    sincospif(2.0f * f, &s, &c);
    s_cs[t][p] = make_float2(c * scale, s * scale);
  }
}

// The rows of a workgroup's tile that a lane group goes through: (token, head)
// `groups` apart, without a division a row.
struct Rows {
  int t, h, step_t, step_h, H, nt;
  __device__ Rows(int group, int groups, int H_, int nt_) : H(H_), nt(nt_) {
    step_t = groups / H;
    step_h = groups - step_t * H;
    t = group / H;
    h = group - t * H;
  }
  __device__ bool inside() const { return t < nt; }
  __device__ void next() {
    t += step_t;
    h += step_h;
    if (h >= H) {
      h -= H;
      ++t;
    }
  }
};

// kTok: 8 tokens share a workgroup where there are many (fewer, fuller
// workgroups); 1 where there are few, so that they spread over the chip.
template <typename T, int V, bool kNorm, int kTok>
__global__ __launch_bounds__(kThreads) void rotary_fwd_kernel(RotaryArgs a) {
  constexpr int kU = V == 1 ? 2 : 1;     // units a lane holds (V = 1: up to 128 pairs a row)
  __shared__ float2 s_cs[kTok][kMaxPairs];
  const bool isq = blockIdx.y == 0 && a.Hq > 0;
  const int H = isq ? a.Hq : a.Hk;
  const size_t ldi = isq ? a.ldq : a.ldk, ldo = isq ? a.ldqo : a.ldko;
  const int t0 = blockIdx.x * kTok, nt = min(kTok, a.tokens - t0);
  const T *in = static_cast<const T *>(isq ? a.q : a.k) + (size_t)t0 * ldi;
  T *out = static_cast<T *>(isq ? a.qo : a.ko) + (size_t)t0 * ldo;
  const float scale = isq ? a.q_scale : 1.f;

  const int G = a.lanes, units = a.d / (2 * V);
  const int lane = threadIdx.x % G;
  Place pl[kU];
  bool on[kU];
  Raw<T, V> raw[kU];
  Unit<V> w[kU];
  Rows at(threadIdx.x / G, kThreads / G, H, nt);
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    const int u = lane + j * G;
    on[j] = u < units;
    pl[j] = place<V>(on[j] ? u : 0, a.rd, a.half);
    if (on[j] && at.inside())
      raw[j] = load_raw<V>(in + (size_t)at.t * ldi + (size_t)at.h * a.d, pl[j]);
    w[j] = load_weight<V>(isq ? a.wq : a.wk, pl[j]);
  }
  if (a.rd) angles(s_cs, a.pos, a.freqs, t0, nt, a.rd / 2, a.rotary_scale);
  __syncthreads();
  while (at.inside()) {
    const int t = at.t;
    T *dst = out + (size_t)t * ldo + (size_t)at.h * a.d;
    Unit<V> x[kU];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (on[j]) {
        x[j] = unpack<V, T>(raw[j], pl[j]);
        if (kNorm)
#pragma unroll
          for (int i = 0; i < V; ++i) ss += x[j].a[i] * x[j].a[i] + x[j].b[i] * x[j].b[i];
      }
    at.next();
#pragma unroll
    for (int j = 0; j < kU; ++j)         // the next row, on its way meanwhile
      if (on[j] && at.inside())
        raw[j] = load_raw<V>(in + (size_t)at.t * ldi + (size_t)at.h * a.d, pl[j]);
    float f = scale;
    if (kNorm) {
      for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
      f *= 1.f / sqrtf(ss * a.norm_scale + a.eps);
    }
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (on[j]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[j].a[i] *= f * w[j].a[i];
          x[j].b[i] *= f * w[j].b[i];
        }
        rotate<V>(x[j], s_cs[t], pl[j], a.inverse);
        store_unit<V>(dst, pl[j], x[j]);
      }
  }
}

// Workgroups go over tiles of 8 tokens, a fixed set each, and keep the weight
// gradient's terms of their rows in registers.
template <typename T, int V, bool kNorm>
__global__ __launch_bounds__(kThreads, 4) void rotary_bwd_kernel(RotaryArgs a) {
  constexpr int kU = V == 1 ? 2 : 1, kTok = kRotaryTile;
  __shared__ float2 s_cs[kTok][kMaxPairs];
  __shared__ float s_red[2 * V * kU * kThreads];   // a row of d (<= 2 V kU G) for every lane group
  const bool isq = blockIdx.y == 0 && a.Hq > 0;
  const int H = isq ? a.Hq : a.Hk;
  const size_t ldi = isq ? a.ldq : a.ldk, ldu = isq ? a.lddq : a.lddk;
  const size_t ldo = isq ? a.ldqo : a.ldko;
  const T *in = static_cast<const T *>(isq ? a.q : a.k);
  const T *up = static_cast<const T *>(isq ? a.dq : a.dk);
  T *out = static_cast<T *>(isq ? a.qo : a.ko);
  const float scale = isq ? a.q_scale : 1.f;
  const bool has_w = (isq ? a.wq : a.wk) != nullptr;

  const int G = a.lanes, units = a.d / (2 * V);
  const int lane = threadIdx.x % G, group = threadIdx.x / G, groups = kThreads / G;
  Place pl[kU];
  bool on[kU];
  Unit<V> w[kU], dw[kU];
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    const int u = lane + j * G;
    on[j] = u < units;
    pl[j] = place<V>(on[j] ? u : 0, a.rd, a.half);
    w[j] = load_weight<V>(isq ? a.wq : a.wk, pl[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j].a[i] = dw[j].b[i] = 0.f;
  }
  const int tiles = (a.tokens + kTok - 1) / kTok;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int t0 = tile * kTok, nt = min(kTok, a.tokens - t0);
    Rows at(group, groups, H, nt);
    Raw<T, V> rx[kU], ry[kU];
    auto fetch = [&]() {
      if (!at.inside()) return;
      const size_t t = (size_t)(t0 + at.t), hh = (size_t)at.h * a.d;
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (on[j]) {
          rx[j] = load_raw<V>(in + t * ldi + hh, pl[j]);
          ry[j] = load_raw<V>(up + t * ldu + hh, pl[j]);
        }
    };
    fetch();
    if (a.rd) angles(s_cs, a.pos, a.freqs, t0, nt, a.rd / 2, a.rotary_scale);
    __syncthreads();
    while (at.inside()) {
      const int t = at.t;
      T *dst = out + (size_t)(t0 + t) * ldo + (size_t)at.h * a.d;
      Unit<V> x[kU], y[kU];
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (on[j]) {
          x[j] = unpack<V, T>(rx[j], pl[j]);
          y[j] = unpack<V, T>(ry[j], pl[j]);
          if (kNorm)
#pragma unroll
            for (int i = 0; i < V; ++i) ss += x[j].a[i] * x[j].a[i] + x[j].b[i] * x[j].b[i];
        }
      at.next();
      fetch();                           // the next row, on its way meanwhile
      float rs = 1.f;
      if (kNorm) {
        for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
        rs = 1.f / sqrtf(ss * a.norm_scale + a.eps);
      }
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (on[j]) {
          rotate<V>(y[j], s_cs[t], pl[j], true);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            x[j].a[i] *= rs;
            x[j].b[i] *= rs;
            y[j].a[i] *= scale;
            y[j].b[i] *= scale;
            dw[j].a[i] += y[j].a[i] * x[j].a[i];
            dw[j].b[i] += y[j].b[i] * x[j].b[i];
            y[j].a[i] *= w[j].a[i];
            y[j].b[i] *= w[j].b[i];
            if (kNorm) m += y[j].a[i] * x[j].a[i] + y[j].b[i] * x[j].b[i];
          }
        }
      if (kNorm) {
        for (int o = G >> 1; o > 0; o >>= 1) m += __shfl_xor(m, o);
        m *= a.norm_scale;
      }
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (on[j]) {
          if (kNorm)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              y[j].a[i] = rs * (y[j].a[i] - x[j].a[i] * m);
              y[j].b[i] = rs * (y[j].b[i] - x[j].b[i] * m);
            }
          store_unit<V>(dst, pl[j], y[j]);
        }
    }
    __syncthreads();                     // s_cs is rewritten for the next tile
  }
  if (!has_w) return;
  // The groups' rows of terms, then their sum in a fixed order.
  float *mine = s_red + group * a.d;
#pragma unroll
  for (int j = 0; j < kU; ++j)
    if (on[j])
#pragma unroll
      for (int i = 0; i < V; ++i) {
        mine[pl[j].half ? pl[j].p0 + i : pl[j].p0 + 2 * i] = dw[j].a[i];
        mine[pl[j].half ? pl[j].p1 + i : pl[j].p0 + 2 * i + 1] = dw[j].b[i];
      }
  __syncthreads();
  float *part = a.partial + ((size_t)blockIdx.x * 2 + (isq ? 0 : 1)) * a.d;
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    float s = 0.f;
    for (int g = 0; g < groups; ++g) s += s_red[g * a.d + c];
    part[c] = s;
  }
}

// dw[c] = the sum of the workgroups' rows, always in the same order: 64
// threads a column, each over every 64th row, then their sums.
__global__ __launch_bounds__(kThreads) void weight_sum_kernel(const float *part, int rows, int d,
                                                              float *dwq, float *dwk, int Hq,
                                                              int Hk) {
  __shared__ float s[64][5];
  const int cx = threadIdx.x % 4, ry = threadIdx.x / 4;
  const int c = blockIdx.x * 4 + cx;     // column of the pair of rows [dwq | dwk]
  const bool isq = c < d;
  const bool want = c < 2 * d && (isq ? dwq : dwk) != nullptr;
  float sum = 0.f;
  if (want && (isq ? Hq : Hk) > 0) {     // without heads there are no rows
#pragma unroll 8
    for (int r = ry; r < rows; r += 64) sum += part[(size_t)r * 2 * d + c];
  }
  s[ry][cx] = sum;
  __syncthreads();
  if (ry == 0 && want) {
    float t = 0.f;
#pragma unroll 8
    for (int i = 0; i < 64; ++i) t += s[i][cx];
    (isq ? dwq : dwk)[isq ? c : c - d] = t;
  }
}

// Channels per thread: the widest V such that every vector of V channels that
// a thread touches is whole pairs of the row and aligned.  Rows that allow 4
// only, or single pairs, take 103 and 217 us where 8 take 100 (32768 tokens of
// 32 heads), the backward 173 and 470 against 157.
template <typename T> int unit_width(const RotaryArgs &a) {
  for (int V = 8; V > 1; V >>= 1) {
    if (V == 2) continue;                // V = 4 or 8 vectors, else single pairs
    bool ok = a.d % (2 * V) == 0 && (a.rd / 2) % V == 0;
    const size_t ld[] = {a.ldq, a.ldk, a.ldqo, a.ldko, a.lddq, a.lddk};
    for (size_t l : ld) ok = ok && l % V == 0;
    const void *ps[] = {a.q, a.k, a.qo, a.ko, a.dq, a.dk};
    const size_t bytes = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
    for (const void *p : ps) ok = ok && reinterpret_cast<uintptr_t>(p) % bytes == 0;
    if (ok) return V;
  }
  return 1;
}

template <typename T, int V> hipError_t launch_v(RotaryArgs a, bool backward, hipStream_t st) {
  const int units = a.d / (2 * V);
  int G = 1;
  while (G < units && G < 64) G *= 2;
  a.lanes = G;
  const unsigned both = a.Hq > 0 && a.Hk > 0 ? 2 : 1;   // query heads, key heads
  if (backward) {
    const dim3 grid(rotary_bwd_groups(a.tokens), both);
    if (a.norm) hipLaunchKernelGGL((rotary_bwd_kernel<T, V, true>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((rotary_bwd_kernel<T, V, false>), grid, dim3(kThreads), 0, st, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (a.dwq || a.dwk)
      hipLaunchKernelGGL(weight_sum_kernel, dim3((2 * a.d + 3) / 4), dim3(kThreads), 0, st,
                         a.partial, (int)grid.x, a.d, a.dwq, a.dwk, a.Hq, a.Hk);
    return hipGetLastError();
  }
  // Tiles of 8 tokens pay their angles once for all heads and fill the chip from
  // 1024 tokens on: with 16 query and 16 key heads of 128 channels 10.3 us
  // against 11.8 (a token a workgroup) at 1024 tokens, 10.7 against 19.7 at 2048,
  // 100 against 248 at 32768; at 512 both take the launch's own time.
  if (a.tokens >= kRotaryManyTokens) {
    const dim3 grid((a.tokens + kRotaryTile - 1) / kRotaryTile, both);
    if (a.norm)
      hipLaunchKernelGGL((rotary_fwd_kernel<T, V, true, kRotaryTile>), grid, dim3(kThreads), 0, st, a);
    else
      hipLaunchKernelGGL((rotary_fwd_kernel<T, V, false, kRotaryTile>), grid, dim3(kThreads), 0, st, a);
  } else {
    const dim3 grid(a.tokens, both);
    if (a.norm) hipLaunchKernelGGL((rotary_fwd_kernel<T, V, true, 1>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((rotary_fwd_kernel<T, V, false, 1>), grid, dim3(kThreads), 0, st, a);
  }
  return hipGetLastError();
}

template <typename T> hipError_t launch_t(const RotaryArgs &a, bool backward, hipStream_t st) {
  switch (unit_width<T>(a)) {
    case 8: return launch_v<T, 8>(a, backward, st);
    case 4: return launch_v<T, 4>(a, backward, st);
    default: return launch_v<T, 1>(a, backward, st);
  }
}

}  // namespace

// Workgroups of the backward for query and for key heads: each keeps its
// weight-gradient sums over many tiles, so their number is bounded (a row of
// the workspace each) and fixed by the number of tokens alone.
int rotary_bwd_groups(int tokens) {
  const int tiles = (tokens + kRotaryTile - 1) / kRotaryTile;
  return tiles < 1 ? 1 : (tiles < 512 ? tiles : 512);
}

hipError_t launch_rotary(const RotaryArgs &a, int in_dtype, bool backward, hipStream_t stream) {
  if (a.tokens == 0 && !backward) return hipSuccess;
  return in_dtype == CKDA_BF16 ? launch_t<__hip_bfloat16>(a, backward, stream)
                               : launch_t<float>(a, backward, stream);
}

}  // namespace ckda
