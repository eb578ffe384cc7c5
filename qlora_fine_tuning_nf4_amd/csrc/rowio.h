// N consecutive row elements of any dtype as fp32, for the elementwise and row
// kernels.  Rows may start at any element: the loads and stores name only the
// element's alignment, which this target serves with full-width instructions
// from any address.
//
// A lane holds eight elements side by side.  Streaming (non-temporal) stores
// are used where that is one 16-byte store, so that an instruction covers
// whole cache lines: fp32 rows, two stores 32 bytes apart, are written the
// ordinary way (512 MiB filled so: 85 us, streaming 229 us; four elements a lane
// instead cost more in the 16-bit rows beside them: residual norm of 4096 x 8192
// 112 us against 82).
#pragma once
#include "common.h"

namespace ql {

typedef u32x4_t u32x4_a2_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_a2_t __attribute__((aligned(2)));

enum { kElF32 = 0, kElBf16 = 1, kElF16 = 2 };   // QLORA_F32, QLORA_BF16, QLORA_F16

template <int T>
constexpr int kElBytes = T == kElF32 ? 4 : 2;
constexpr int kVec = 8;

template <int T, int N>
struct Raw {
  uint32_t w[N * kElBytes<T> / 4];
};

// Row r of a matrix with row stride ld: uniform where r is, which leaves the
// lanes one 32-bit offset.
template <int T>
QL_DEV const char* row_of(const void* p, int64_t r, int64_t ld) {
  return reinterpret_cast<const char*>(p) + r * ld * kElBytes<T>;
}
template <int T>
QL_DEV char* row_of(void* p, int64_t r, int64_t ld) {
  return reinterpret_cast<char*>(p) + r * ld * kElBytes<T>;
}

template <int T>
QL_DEV float load1(const void* p, int64_t i) {
  if constexpr (T == kElF32)
    return gptr(reinterpret_cast<const float*>(p))[i];
  else
    return w16<T == kElF16>(gptr(reinterpret_cast<const uint16_t*>(p))[i]);
}

template <int T>
QL_DEV void store1(void* p, int64_t i, float v) {
  if constexpr (T == kElF32)
    gptr_w(reinterpret_cast<float*>(p))[i] = v;
  else
    gptr_w(reinterpret_cast<uint16_t*>(p))[i] = to16<T == kElF16>(v);
}

// Elements [i, i + N) of a row p; those from i + left on are zero (left >= 1).  STREAM:
// the data is not read again (acted on if it is one load).
template <int T, int N, bool STREAM = false>
QL_DEV Raw<T, N> loadv(const void* p, int i, int left) {
  constexpr int W = N * kElBytes<T> / 4;
  static_assert(W % 4 == 0);
  Raw<T, N> r;
  if (left >= N) {
    const char* at = reinterpret_cast<const char*>(p) + (uint32_t)(i * kElBytes<T>);
#pragma unroll
    for (int h = 0; h < W / 4; ++h) {
      const QL_GLOBAL u32x4_a2_t* q = (const QL_GLOBAL u32x4_a2_t*)(at + 16 * h);
      const u32x4_t v = STREAM && W == 4 ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[4 * h + j] = v[j];
    }
  } else if constexpr (T == kElF32) {
    // the row's last element stands in for those past it: all loads are in
    // flight together
    const QL_GLOBAL uint32_t* q = gptr(reinterpret_cast<const uint32_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < N; ++j) r.w[j] = q[min(j, left - 1)];
#pragma unroll
    for (int j = 1; j < N; ++j) r.w[j] = j < left ? r.w[j] : 0u;
  } else {
    const QL_GLOBAL uint16_t* q = gptr(reinterpret_cast<const uint16_t*>(p) + i);
    uint32_t h[N];
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = q[min(j, left - 1)];
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
      r.w[j] = h[2 * j] * (2 * j < left) | (2 * j + 1 < left ? h[2 * j + 1] << 16 : 0u);
  }
  return r;
}

template <int T, int N>
QL_DEV float el(const Raw<T, N>& r, int j) {
  if constexpr (T == kElF32)
    return __builtin_bit_cast(float, r.w[j]);
  else
    return (j & 1) ? hi16<T == kElF16>(r.w[j >> 1]) : lo16<T == kElF16>(r.w[j >> 1]);
}

// Elements [i, i + min(left, N)) of a row p.  STREAM: written past the caches, if
// it is one store.
template <int T, int N, bool STREAM = false>
QL_DEV void storev(void* p, int i, int left, const float (&f)[N]) {
  constexpr int W = N * kElBytes<T> / 4;
  static_assert(W % 4 == 0);
  if (left >= N) {
    uint32_t w[W];
#pragma unroll
    for (int j = 0; j < W; ++j)
      w[j] = T == kElF32 ? __builtin_bit_cast(uint32_t, f[j]) : pack16x2<T == kElF16>(f[2 * j % N], f[(2 * j + 1) % N]);
    char* at = reinterpret_cast<char*>(p) + (uint32_t)(i * kElBytes<T>);
#pragma unroll
    for (int h = 0; h < W / 4; ++h) {
      QL_GLOBAL u32x4_a2_t* q = (QL_GLOBAL u32x4_a2_t*)(at + 16 * h);
      const u32x4_t v = {w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]};
      if (STREAM && W == 4) __builtin_nontemporal_store((u32x4_a2_t)v, q);
      else *q = v;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (j < left) store1<T>(p, i + j, f[j]);
}

}  // namespace ql
