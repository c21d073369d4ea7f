// Host-side helpers shared by the entry points: argument checks and debug mode.
#pragma once

#include <stdlib.h>
#include <string.h>

#include "ckda_internal.h"

namespace ckda {

inline bool dims_ok(int d) { return d == 64 || d == 128; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline bool debug_mode() {
  const char *e = getenv("CKDA_DEBUG");
  return e && *e && strcmp(e, "0") != 0;
}

// Debug mode: the host copy of cu_seqlens must be non-decreasing from 0 to T.
// Copied in pieces through a stack buffer, so the check allocates nothing.
inline int debug_check_cu(const int32_t *cu_seqlens, int N, int T, hipStream_t st) {
  constexpr int kPiece = 256;
  int32_t h[kPiece];
  int32_t prev = 0;
  for (int i0 = 0; i0 <= N; i0 += kPiece) {
    const int n = (N + 1 - i0) < kPiece ? (N + 1 - i0) : kPiece;
    if (hipMemcpyAsync(h, cu_seqlens + i0, (size_t)n * sizeof(int32_t), hipMemcpyDeviceToHost,
                       st) != hipSuccess ||
        hipStreamSynchronize(st) != hipSuccess)
      return CKDA_ERR_LAUNCH;
    for (int i = 0; i < n; ++i) {
      if ((i0 + i == 0 && h[i] != 0) || h[i] < prev) return CKDA_ERR_SHAPE;
      prev = h[i];
    }
  }
  return prev == T ? CKDA_OK : CKDA_ERR_SHAPE;
}

// Debug-mode steps shared by the forward and the backward, after validation.
inline int debug_prologue(const int32_t *cu_seqlens, int N, int T, void *workspace, size_t bytes,
                   hipStream_t st) {
  if (!debug_mode()) return CKDA_OK;
  if (cu_seqlens)
    if (int s = debug_check_cu(cu_seqlens, N, T, st)) return s;
  if (workspace && launch_poison(workspace, bytes & ~(size_t)3, st) != hipSuccess)
    return CKDA_ERR_LAUNCH;
  return CKDA_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace ckda
