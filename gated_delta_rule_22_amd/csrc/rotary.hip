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
// two) share a row.  A workgroup takes kTok tokens at a time and computes the
// tokens' cosines and sines once into LDS for all of their heads: an angle
// costs an fp64 product (pos * f in turns, reduced exactly, so that positions
// of a million and more lose nothing) and an fp32 sincospi, about as much work
// as the rest of a pair.
#include "ckda_internal.h"

namespace ckda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;          // rd <= 256

// 2V channels of a row: V first and V second elements of its pairs.
template <int V> struct Unit { float a[V], b[V]; };


template <int V> __device__ __forceinline__ void load_vec(const __hip_bfloat16 *p, float *x) {
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else if constexpr (V == 4) {
    const float4 f = load4_f32(p);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(p[i]);
  }
}
template <int V> __device__ __forceinline__ void load_vec(const float *p, float *x) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = load4_f32(p + i);
      x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = p[i];
  }
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

// Offsets within a row of a unit's first and second V channels in memory, and
// whether they are rotated.  In the interleaved layout (and behind the rotated
// part) the 2V channels are contiguous and the pairs are (even, odd).
struct Place { int p0, p1, pair; bool rot; };
template <int V> __device__ __forceinline__ Place place(int u, int rd, bool half) {
  const int ur = rd / (2 * V);
  Place pl;
  pl.rot = u < ur;
  pl.pair = u * V;
  if (pl.rot && half) {
    pl.p0 = u * V;
    pl.p1 = rd / 2 + u * V;
  } else {
    pl.p0 = 2 * V * u;
    pl.p1 = 2 * V * u + V;
  }
  return pl;
}

// Raw 2V channels to pairs: in the half layout the two vectors are the pairs'
// first and second elements; otherwise channels alternate.
template <int V, typename T>
__device__ __forceinline__ Unit<V> load_unit(const T *row, const Place &pl, bool half) {
  Unit<V> r;
  float x[2 * V];
  load_vec<V>(row + pl.p0, x);
  load_vec<V>(row + pl.p1, x + V);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r.a[i] = half ? x[i] : x[2 * i];
    r.b[i] = half ? x[V + i] : x[2 * i + 1];
  }
  return r;
}
template <int V, typename T>
__device__ __forceinline__ void store_unit(T *row, const Place &pl, bool half, const Unit<V> &r) {
  float x[2 * V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[half ? i : 2 * i] = r.a[i];
    x[half ? V + i : 2 * i + 1] = r.b[i];
  }
  store_vec<V>(row + pl.p0, x);
  store_vec<V>(row + pl.p1, x + V);
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

// cos and sin (times `scale`) of kTok tokens' angles into LDS.
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

// kTok: 4 tokens share a workgroup where there are many (fewer, fuller
// workgroups); 1 where there are few, so that they spread over the chip.
template <typename T, int V, bool kNorm, int kTok>
__global__ __launch_bounds__(kThreads) void rotary_fwd_kernel(RotaryArgs a) {
  constexpr int kU = V == 1 ? 2 : 1;     // units a lane holds (V = 1: up to 128 pairs a row)
  __shared__ float2 s_cs[kTok][kMaxPairs];
  const int t0 = blockIdx.x * kTok;
  const int nt = min(kTok, a.tokens - t0);
  if (a.rd) angles(s_cs, a.pos, a.freqs, t0, nt, a.rd / 2, a.rotary_scale);
  __syncthreads();

  const int G = a.lanes, units = a.d / (2 * V);
  const int lane = threadIdx.x % G, group = threadIdx.x / G, groups = kThreads / G;
  const int heads = a.Hq + a.Hk;
  Place pl[kU];
  bool on[kU], half[kU];
  Unit<V> wq[kU], wk[kU];
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    const int u = lane + j * G;
    on[j] = u < units;
    pl[j] = place<V>(on[j] ? u : 0, a.rd, a.half);
    half[j] = a.half && pl[j].rot;
    if (on[j] && a.wq) wq[j] = load_unit<V>(a.wq, pl[j], half[j]);
    if (on[j] && a.wk) wk[j] = load_unit<V>(a.wk, pl[j], half[j]);
  }
  for (int r = group; r < nt * heads; r += groups) {
    const int t = r / heads, h = r - t * heads;
    const bool isq = h < a.Hq;
    const size_t tok = (size_t)(t0 + t);
    const T *row = isq ? static_cast<const T *>(a.q) + tok * a.ldq + (size_t)h * a.d
                       : static_cast<const T *>(a.k) + tok * a.ldk + (size_t)(h - a.Hq) * a.d;
    T *dst = isq ? static_cast<T *>(a.qo) + tok * a.ldqo + (size_t)h * a.d
                 : static_cast<T *>(a.ko) + tok * a.ldko + (size_t)(h - a.Hq) * a.d;
    Unit<V> x[kU];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (on[j]) {
        x[j] = load_unit<V>(row, pl[j], half[j]);
        if (kNorm)
#pragma unroll
          for (int i = 0; i < V; ++i) ss += x[j].a[i] * x[j].a[i] + x[j].b[i] * x[j].b[i];
      }
    float f = isq ? a.q_scale : 1.f;
    if (kNorm) {
      for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
      f *= 1.f / sqrtf(ss * a.norm_scale + a.eps);
    }
    const bool has_w = isq ? a.wq != nullptr : a.wk != nullptr;
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (on[j]) {
        const Unit<V> &w = isq ? wq[j] : wk[j];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[j].a[i] *= has_w ? f * w.a[i] : f;
          x[j].b[i] *= has_w ? f * w.b[i] : f;
        }
        rotate<V>(x[j], s_cs[t], pl[j], a.inverse);
        store_unit<V>(dst, pl[j], half[j], x[j]);
      }
  }
}

// Sums over a workgroup's row groups, in a fixed order, of each lane's 2V
// weight-gradient terms; one row of d per workgroup goes to the workspace.
template <int V, int kU>
__device__ __forceinline__ void write_partial(const Unit<V> *acc, const Place *pl, const bool *on,
                                              const bool *half, float *s_red, int group,
                                              int groups, int d, float *dst) {
  // Row groups write their terms in turn into kSlots rows of LDS, then add up.
  for (int g = 0; g < groups; ++g) {
    if (group == g)
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (on[j])
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int ca = half[j] ? pl[j].p0 + i : pl[j].p0 + 2 * i;
            const int cb = half[j] ? pl[j].p1 + i : pl[j].p0 + 2 * i + 1;
            s_red[ca] = (g ? s_red[ca] : 0.f) + acc[j].a[i];
            s_red[cb] = (g ? s_red[cb] : 0.f) + acc[j].b[i];
          }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < d; c += kThreads) dst[c] = s_red[c];
  __syncthreads();
}

template <typename T, int V, bool kNorm>
__global__ __launch_bounds__(kThreads) void rotary_bwd_kernel(RotaryArgs a) {
  constexpr int kU = V == 1 ? 2 : 1, kTok = 4;
  __shared__ float2 s_cs[kTok][kMaxPairs];
  __shared__ float s_red[2 * kMaxPairs];
  const int G = a.lanes, units = a.d / (2 * V);
  const int lane = threadIdx.x % G, group = threadIdx.x / G, groups = kThreads / G;
  const int heads = a.Hq + a.Hk;
  Place pl[kU];
  bool on[kU], half[kU];
  Unit<V> wq[kU], wk[kU], dwq[kU], dwk[kU];
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    const int u = lane + j * G;
    on[j] = u < units;
    pl[j] = place<V>(on[j] ? u : 0, a.rd, a.half);
    half[j] = a.half && pl[j].rot;
    if (on[j] && a.wq) wq[j] = load_unit<V>(a.wq, pl[j], half[j]);
    if (on[j] && a.wk) wk[j] = load_unit<V>(a.wk, pl[j], half[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) dwq[j].a[i] = dwq[j].b[i] = dwk[j].a[i] = dwk[j].b[i] = 0.f;
  }
  const int tiles = (a.tokens + kTok - 1) / kTok;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int t0 = tile * kTok, nt = min(kTok, a.tokens - t0);
    if (a.rd) angles(s_cs, a.pos, a.freqs, t0, nt, a.rd / 2, a.rotary_scale);
    __syncthreads();
    for (int r = group; r < nt * heads; r += groups) {
      const int t = r / heads, h = r - t * heads;
      const bool isq = h < a.Hq;
      const size_t tok = (size_t)(t0 + t);
      const size_t hh = (size_t)(isq ? h : h - a.Hq) * a.d;
      const T *row = static_cast<const T *>(isq ? a.q : a.k) + tok * (isq ? a.ldq : a.ldk) + hh;
      const T *up = static_cast<const T *>(isq ? a.dq : a.dk) + tok * (isq ? a.lddq : a.lddk) + hh;
      T *dst = static_cast<T *>(isq ? a.qo : a.ko) + tok * (isq ? a.ldqo : a.ldko) + hh;
      Unit<V> x[kU], y[kU];
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (on[j]) {
          x[j] = load_unit<V>(row, pl[j], half[j]);
          y[j] = load_unit<V>(up, pl[j], half[j]);
          if (kNorm)
#pragma unroll
            for (int i = 0; i < V; ++i) ss += x[j].a[i] * x[j].a[i] + x[j].b[i] * x[j].b[i];
        }
      float rs = 1.f;
      if (kNorm) {
        for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
        rs = 1.f / sqrtf(ss * a.norm_scale + a.eps);
      }
      const float f = isq ? a.q_scale : 1.f;
      const bool has_w = isq ? a.wq != nullptr : a.wk != nullptr;
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (on[j]) {
          rotate<V>(y[j], s_cs[t], pl[j], true);
          const Unit<V> &w = isq ? wq[j] : wk[j];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            x[j].a[i] *= rs;
            x[j].b[i] *= rs;
            y[j].a[i] *= f;
            y[j].b[i] *= f;
            const float ta = y[j].a[i] * x[j].a[i], tb = y[j].b[i] * x[j].b[i];
            if (has_w) {
              // selects, not a branch: the sums stay in registers
              dwq[j].a[i] += isq ? ta : 0.f;
              dwq[j].b[i] += isq ? tb : 0.f;
              dwk[j].a[i] += isq ? 0.f : ta;
              dwk[j].b[i] += isq ? 0.f : tb;
              y[j].a[i] *= w.a[i];
              y[j].b[i] *= w.b[i];
            }
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
          store_unit<V>(dst, pl[j], half[j], y[j]);
        }
    }
    __syncthreads();                     // s_cs is rewritten for the next tile
  }
  float *part = a.partial + (size_t)blockIdx.x * 2 * a.d;
  if (a.wq) write_partial<V, kU>(dwq, pl, on, half, s_red, group, groups, a.d, part);
  if (a.wk) write_partial<V, kU>(dwk, pl, on, half, s_red, group, groups, a.d, part + a.d);
}

// dw[c] = the sum of the workgroups' rows, always in the same order: 16
// threads a column, each over every 16th row, then their 16 sums.
__global__ __launch_bounds__(kThreads) void weight_sum_kernel(const float *part, int rows, int d,
                                                              float *dwq, float *dwk) {
  __shared__ float s[16][17];
  const int cx = threadIdx.x % 16, ry = threadIdx.x / 16;
  const int c = blockIdx.x * 16 + cx;    // column of the pair of rows [dwq | dwk]
  float sum = 0.f;
  const bool want = c < 2 * d && (c < d ? dwq : dwk) != nullptr;
  if (want)
    for (int r = ry; r < rows; r += 16) sum += part[(size_t)r * 2 * d + c];
  s[ry][cx] = sum;
  __syncthreads();
  if (ry == 0 && want) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][cx];
    (c < d ? dwq : dwk)[c < d ? c : c - d] = t;
  }
}

// Channels per thread: the widest V such that every vector of V channels that
// a thread touches is whole pairs of the row and aligned.
template <typename T> int unit_width(const RotaryArgs &a) {
  for (int V = 8; V > 1; V >>= 1) {
    if (V == 2) continue;                // V = 4 or 8 vectors, else single pairs
    bool ok = a.d % (2 * V) == 0 && (a.rd / 2) % V == 0;
    const size_t ld[] = {a.ldq, a.ldk, a.ldqo, a.ldko, a.lddq, a.lddk};
    for (size_t l : ld) ok = ok && l % V == 0;
    const void *ps[] = {a.q, a.k, a.qo, a.ko, a.dq, a.dk};
    const size_t bytes = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
    for (const void *p : ps) ok = ok && reinterpret_cast<uintptr_t>(p) % bytes == 0;
    ok = ok && reinterpret_cast<uintptr_t>(a.wq) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(a.wk) % 16 == 0;
    if (ok) return V;
  }
  return 1;
}

template <typename T, int V> hipError_t launch_v(RotaryArgs a, bool backward, hipStream_t st) {
  const int units = a.d / (2 * V);
  int G = 1;
  while (G < units && G < 64) G *= 2;
  a.lanes = G;
  if (backward) {
    const dim3 grid(rotary_bwd_groups(a.tokens));
    if (a.norm) hipLaunchKernelGGL((rotary_bwd_kernel<T, V, true>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((rotary_bwd_kernel<T, V, false>), grid, dim3(kThreads), 0, st, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (a.dwq || a.dwk) {
      hipLaunchKernelGGL(weight_sum_kernel, dim3((2 * a.d + 15) / 16), dim3(kThreads), 0, st,
                         a.partial, (int)grid.x, a.d, a.dwq, a.dwk);
    }
    return hipGetLastError();
  }
  if (a.tokens >= 4096) {
    const dim3 grid((a.tokens + 3) / 4);
    if (a.norm) hipLaunchKernelGGL((rotary_fwd_kernel<T, V, true, 4>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((rotary_fwd_kernel<T, V, false, 4>), grid, dim3(kThreads), 0, st, a);
  } else {
    const dim3 grid(a.tokens);
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

// Workgroups of the backward: each keeps its weight-gradient sums over many
// tiles of 4 tokens, so their number is bounded (one row of the workspace
// each) and fixed by the number of tokens alone.
int rotary_bwd_groups(int tokens) {
  const int tiles = (tokens + 3) / 4;
  return tiles < 1 ? 1 : (tiles < 1024 ? tiles : 1024);
}

hipError_t launch_rotary(const RotaryArgs &a, int in_dtype, bool backward, hipStream_t stream) {
  if (a.tokens == 0 && !backward) return hipSuccess;
  return in_dtype == CKDA_BF16 ? launch_t<__hip_bfloat16>(a, backward, stream)
                               : launch_t<float>(a, backward, stream);
}

}  // namespace ckda
