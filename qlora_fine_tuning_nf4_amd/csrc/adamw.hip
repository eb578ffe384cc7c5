// AdamW over all tensors of a plan in one launch, and the global gradient
// norm.  Both are streams over memory: 28 bytes a value with fp32 moments and
// fp32 gradients, 16 with 8-bit moments (2 more with a 16-bit copy).
// Measured: 8.4M values of 256 tensors, fp32 moments and bf16 copies 41 us (6.1
// TB/s; 52 with the norm and its clip factor before it), 56M of 280 tensors with 8-bit
// moments 164 us (6.2 TB/s), one tensor of 131M with bf16 gradients 347 us
// (6.1 TB/s).
//
// The plan's tensors are cut into chunks of 1024 consecutive values, each
// within one tensor; a workgroup looks its chunk up in the plan's map (one
// 8-byte entry), a wave takes one 256-value block of the state and a lane four
// consecutive values.  That is one 16-byte load per fp32 operand and lane, and
// with 8-bit moments makes a block's largest value one reduction within the
// wave.  Nothing is read twice, so loads and stores are non-temporal.  Short
// workgroups and streaming accesses are what the memory takes best here: 131M
// values with 8-bit moments 355 us, chunks of 2048 361, of 4096 391; with ordinary
// accesses 365, 378 and 402.
#include <algorithm>

#include "rowio.h"
#include "train_kernels.h"

namespace ql {

namespace {

typedef f32x4_t f32x4_a4_t __attribute__((aligned(4)));

// Values [i, i + 4) of p as fp32 (those from i + left on are zero).
template <int T>
QL_DEV f32x4_t load4(const void* p, int64_t i, int left) {
  f32x4_t o = {0.f, 0.f, 0.f, 0.f};
  if (left >= 4) {
    if constexpr (T == kElF32) {
      const QL_GLOBAL f32x4_a4_t* q = (const QL_GLOBAL f32x4_a4_t*)(reinterpret_cast<const float*>(p) + i);
      o = __builtin_nontemporal_load(q);
    } else {
      const QL_GLOBAL u32x2_a2_t* q = (const QL_GLOBAL u32x2_a2_t*)(reinterpret_cast<const uint16_t*>(p) + i);
      const u32x2_t v = __builtin_nontemporal_load(q);
      constexpr bool F = T == kElF16;
      o = f32x4_t{lo16<F>(v[0]), hi16<F>(v[0]), lo16<F>(v[1]), hi16<F>(v[1])};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) o[j] = load1<T>(p, i + j);
  }
  return o;
}

template <int T>
QL_DEV void store4(void* p, int64_t i, int left, f32x4_t f) {
  if (left >= 4) {
    if constexpr (T == kElF32) {
      __builtin_nontemporal_store((f32x4_a4_t)f, (QL_GLOBAL f32x4_a4_t*)(reinterpret_cast<float*>(p) + i));
    } else {
      const u32x2_t v = {pack16x2<T == kElF16>(f[0], f[1]), pack16x2<T == kElF16>(f[2], f[3])};
      __builtin_nontemporal_store((u32x2_a2_t)v, (QL_GLOBAL u32x2_a2_t*)(reinterpret_cast<uint16_t*>(p) + i));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) store1<T>(p, i + j, f[j]);
  }
}

QL_DEV uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// 8-bit codes of a non-negative x on the grid of an 8-bit float whose largest
// value stands for the block's maximum: y = x * inv is scaled by 2^-(126 +
// emin), emin the grid's smallest normal exponent, which turns the grid's
// subnormals into binary32's own, so that code = bits >> drop for both; the
// random bits below the kept ones make the cut stochastic.  y <= top, which
// is on the grid, so the carry never passes the largest code.  An x that is not
// finite gets the largest code (inf * inv is inf or NaN, and the minimum is top).
QL_DEV uint32_t code8(float x, float inv, float top, float power, int drop, uint32_t rnd) {
  const float y = fminf(x * inv, top) * power;
  return (__builtin_bit_cast(uint32_t, y) + rnd) >> drop;
}

constexpr float kTopM = 448.f, kTopV = 57344.f;             // largest e4m3 / e5m2 value
constexpr float kTiny = 7.70371977754894341222391177034e-34f;   // 2^-110: 57344 / kTiny is finite

// Largest of a wave's values (none negative), uniform: DPP shifts within rows of
// 16, then the rows' maxima passed on, in lane 63.
template <int CTRL, int ROWS>
QL_DEV float dpp_max(float v) {
  const int s = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false);
  return fmaxf(v, __builtin_bit_cast(float, s));
}
QL_DEV float wave_largest(float v) {
  v = dpp_max<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);   // row_bcast 15 into rows 1 and 3
  v = dpp_max<0x143, 0xC>(v);   // row_bcast 31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

QL_DEV float of_lane(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// One chunk a workgroup.  Bound by memory (6.0 TB/s over 131M values with
// 8-bit moments and bf16 gradients, what a copy reaches), with the vector ALU
// not far behind: about 80 instructions a value, two of them quarter-rate
// products of the rounding bits, one a root and one a reciprocal.  So the
// block's two divisions share one instruction sequence, and nothing is
// selected per value that the state's zero padding or a uniform branch settles.
template <int PT, int GT, int CT, bool S8>
__global__ __launch_bounds__(256) void k_adamw(const OptEntry* __restrict__ tab,
                                               const OptChunk* __restrict__ map,
                                               qlora_opt_state in, qlora_opt_state out,
                                               AdamwScalars k, const float* __restrict__ gscale) {
  const OptChunk ch = map[blockIdx.x];
  const OptEntry e = tab[ch.tensor];
  const float c = gscale ? *gscale : 1.f;
  const float lr = k.lr * e.lr_mul;
  const float keep = 1.f - lr * (k.wd * e.wd_mul), rate = k.lr_bc1 * e.lr_mul;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  static_assert(kOptChunk == 4 * QLORA_ADAMW_BLOCK);
  const int64_t b0 = (int64_t)ch.index * kOptChunk + wave * QLORA_ADAMW_BLOCK;   // first value of the wave's block
  if (b0 >= e.n) return;
  const int64_t i = b0 + 4 * lane;
  const int left = (int)min((int64_t)4, e.n - i);
  const int64_t blk = e.block0 + b0 / QLORA_ADAMW_BLOCK;
  const int64_t si = blk * QLORA_ADAMW_BLOCK + 4 * lane;
  const f32x4_t p = load4<PT>(e.p, i, left);
  const f32x4_t g = load4<GT>(e.g, i, left);
  f32x4_t m, v;
  uint32_t mq = 0, vq = 0;
  float ms = 0.f, vs = 0.f;
  if constexpr (S8) {
    mq = __builtin_nontemporal_load((const QL_GLOBAL uint32_t*)((const uint8_t*)in.m + si));
    vq = __builtin_nontemporal_load((const QL_GLOBAL uint32_t*)((const uint8_t*)in.v + si));
    ms = gptr(in.m_scale)[blk];
    vs = gptr(in.v_scale)[blk];
    m = f32x4_t{__builtin_amdgcn_cvt_f32_fp8(mq, 0), __builtin_amdgcn_cvt_f32_fp8(mq, 1),
                __builtin_amdgcn_cvt_f32_fp8(mq, 2), __builtin_amdgcn_cvt_f32_fp8(mq, 3)};
    v = f32x4_t{__builtin_amdgcn_cvt_f32_bf8(vq, 0), __builtin_amdgcn_cvt_f32_bf8(vq, 1),
                __builtin_amdgcn_cvt_f32_bf8(vq, 2), __builtin_amdgcn_cvt_f32_bf8(vq, 3)};
  } else {
    m = __builtin_nontemporal_load((const QL_GLOBAL f32x4_t*)((const float*)in.m + si));
    v = __builtin_nontemporal_load((const QL_GLOBAL f32x4_t*)((const float*)in.v + si));
  }
  f32x4_t pn = p;
  if (fabsf(c) < __builtin_inff()) {
    {
      // each product and sum of the moments is rounded by itself: their 8-bit
      // codes are then the same whatever computes them
#pragma clang fp contract(off)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (S8) {
          m[j] = m[j] * ms;
          v[j] = v[j] * vs;
        }
        const float gj = g[j] * c;
        m[j] = m[j] * k.b1 + gj * k.c1;
        v[j] = v[j] * k.b2 + (gj * gj) * k.c2;
      }
    }
    if (k.small_eps) {
#pragma unroll
      for (int j = 0; j < 4; ++j) pn[j] = p[j] * keep - rate * (m[j] / (sqrtf(v[j]) * k.rs_bc2 + k.eps));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float den = __builtin_amdgcn_sqrtf(v[j]) * k.rs_bc2 + k.eps;
        // the update needs a relative accuracy far below its share of p: the
        // one-ulp root and reciprocal are enough
        pn[j] = p[j] * keep - rate * (m[j] * __builtin_amdgcn_rcpf(den));
      }
    }
    if constexpr (S8) {
      // (values past the tensor's end are zero in the state and have no gradient)
      float am = 0.f, av = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        am = fmaxf(am, fabsf(m[j]));
        av = fmaxf(av, v[j]);
      }
      am = wave_largest(am);
      av = wave_largest(av);
      // (both uniform: compared as integers on the scalar unit)
      if (max(__builtin_bit_cast(uint32_t, am), __builtin_bit_cast(uint32_t, av)) >= 0x7F800000u) {
        // infinities stay out of the scales, as NaNs do: one value must not take its block along
        float fm = 0.f, fv = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          fm = fmaxf(fm, fabsf(m[j]) < __builtin_inff() ? fabsf(m[j]) : 0.f);
          fv = fmaxf(fv, v[j] < __builtin_inff() ? v[j] : 0.f);
        }
        am = wave_largest(fm);
        av = wave_largest(fv);
      }
      const bool some_m = am >= kTiny, some_v = av >= kTiny;
      // top / largest: the lower lanes divide for m, the upper ones for v
      const bool low = lane < 32;
      const float inv = (low ? kTopM : kTopV) / (low ? am : av);
      const float im = some_m ? of_lane(inv, 0) : 0.f, iv = some_v ? of_lane(inv, 63) : 0.f;
      const uint32_t least_v = some_v ? 1u : 0u;
      const uint32_t kb = mix32(k.key + 0x510E527Fu * (uint32_t)blk);
      const uint32_t x0 = kb + 0x9E3779B9u * (uint32_t)(4 * lane + 1);
      mq = vq = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t r = mix32(x0 + 0x9E3779B9u * (uint32_t)j);
        const float mj = m[j], vj = v[j];
        uint32_t cm = code8(fabsf(mj), im, kTopM, 0x1p-120f, 20, (r & 0xFFFFu) << 4 | 8u);
        uint32_t cv = code8(vj, iv, kTopV, 0x1p-112f, 21, (r >> 16) << 5 | 16u);
        cm |= (__builtin_bit_cast(uint32_t, mj) >> 24) & 0x80u;
        cv = max(cv, min(__builtin_bit_cast(uint32_t, vj), least_v));   // a positive moment stays positive
        mq |= cm << (8 * j);
        vq |= cv << (8 * j);
      }
      ms = some_m ? am * (1.f / kTopM) : 0.f;
      vs = some_v ? av * (1.f / kTopV) : 0.f;
    }
  }
  store4<PT>(e.po, i, left, pn);
  if constexpr (CT != kElF32)
    if (e.copy) store4<CT>(e.copy, i, left, pn);
  if constexpr (S8) {
    __builtin_nontemporal_store(mq, (QL_GLOBAL uint32_t*)((uint8_t*)out.m + si));
    __builtin_nontemporal_store(vq, (QL_GLOBAL uint32_t*)((uint8_t*)out.v + si));
    if (lane == 0) {
      gptr_w(out.m_scale)[blk] = ms;
      gptr_w(out.v_scale)[blk] = vs;
    }
  } else {
    __builtin_nontemporal_store(m, (QL_GLOBAL f32x4_t*)((float*)out.m + si));
    __builtin_nontemporal_store(v, (QL_GLOBAL f32x4_t*)((float*)out.v + si));
  }
}

// Norm of all gradients and its clip factor.  Every workgroup leaves the sum of
// squares of its chunks; the one that arrives last, by a count kept in the
// plan's table, adds the sums in the order of their index.  The count wraps to zero
// with the last arrival: a call finds it at zero whatever came before, also after
// calls that overlapped (whose own results are then undefined).  No workgroup
// waits for another.  The sums cross XCDs, whose
// L2s are not coherent: they are written and read with device-scope atomics,
// which act at the level the XCDs share, and the count is raised only after
// the write is done (the wait on the vector-memory counter).  A release fence
// would do the same and write the whole L2 back besides: 45 us instead of 9
// over 1024 workgroups.
//
// 256 threads walk a stretch of consecutive chunks, looking the plan up only
// where the tensor changes, with eight 16-byte loads in flight (56M fp32 values
// 41 us, with a lookup a chunk 49). Four such groups a workgroup and at
// most one workgroup a CU, since the arrivals queue up at one address (about
// 10 ns each).
constexpr int kNormThreads = 1024;
constexpr int kNormAhead = 8;
constexpr int kNormSide = 4;   // groups of a workgroup

template <int GT>
__global__ __launch_bounds__(kNormThreads) void k_grad_norm(const OptEntry* __restrict__ tab,
                                                            const OptChunk* __restrict__ map, int64_t chunks,
                                                            float max_norm, float* __restrict__ out,
                                                            float* part, uint32_t* arrived) {
  static_assert(kNormWgs <= kNormThreads);
  __shared__ float s[kNormThreads / 64];
  __shared__ bool last;
  const int side = __builtin_amdgcn_readfirstlane(threadIdx.x / (kNormThreads / kNormSide));
  constexpr int V = 16 / kElBytes<GT>, kGroup = kNormThreads / kNormSide;   // values of a load, threads of a group
  const int mine = V * (threadIdx.x % kGroup);
  const int64_t groups = (int64_t)gridDim.x * kNormSide, per = (chunks + groups - 1) / groups;
  int64_t q = ((int64_t)blockIdx.x * kNormSide + side) * per;
  const int64_t q1 = min(chunks, q + per);
  float acc[kNormAhead] = {};
  while (q < q1) {
    const OptChunk ch = map[q];
    const int64_t n = tab[ch.tensor].n, i0 = (int64_t)ch.index * kOptChunk;
    const int64_t run = min(q1 - q, (n - i0 + kOptChunk - 1) / kOptChunk);
    const int64_t count = min(n - i0, run * kOptChunk);
    const char* data = (const char*)tab[ch.tensor].g + i0 * kElBytes<GT>;
    for (int64_t r = mine; r < count; r += V * kGroup * kNormAhead) {
      Raw<GT, V> g[kNormAhead] = {};
#pragma unroll
      for (int u = 0; u < kNormAhead; ++u) {
        const int64_t i = r + u * V * kGroup;
        if (i < count) g[u] = loadv<GT, V>(data + i * kElBytes<GT>, 0, (int)min((int64_t)V, count - i));
      }
#pragma unroll
      for (int u = 0; u < kNormAhead; ++u)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[u] += el(g[u], j) * el(g[u], j);
    }
    q += run;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto block_sum = [&](float v) {   // in every thread
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) s[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 64; ++i) v += s[i];
    return v;
  };
  float total = acc[0];
#pragma unroll
  for (int u = 1; u < kNormAhead; ++u) total += acc[u];
  const float sum = block_sum(total);
  if (threadIdx.x == 0) {
    __hip_atomic_store(part + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    QL_VMCNT(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    last = atomicInc(arrived, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  const float all = block_sum(
      threadIdx.x < gridDim.x ? __hip_atomic_load(part + threadIdx.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.f);
  if (threadIdx.x == 0) {
    const float norm = sqrtf(all);
    float f = max_norm > 0.f ? fminf(1.f, max_norm / (norm + 1e-6f)) : 1.f;
    if (!(norm < __builtin_inff())) f = __builtin_nanf("");
    out[0] = norm;
    out[1] = f;
  }
}

template <int PT, int GT, int CT>
hipError_t adamw_types(const OptEntry* tab, const OptChunk* map, int64_t chunks, int bits,
                       const qlora_opt_state& in, const qlora_opt_state& out, const AdamwScalars& k,
                       const float* gs, hipStream_t s) {
  // a launch holds fewer than 2^32 threads
  constexpr int64_t kMost = int64_t(1) << 23;
  for (int64_t at = 0; at < chunks; at += kMost) {
    const unsigned wgs = (unsigned)std::min(kMost, chunks - at);
    if (bits == 8)
      k_adamw<PT, GT, CT, true><<<wgs, 256, 0, s>>>(tab, map + at, in, out, k, gs);
    else
      k_adamw<PT, GT, CT, false><<<wgs, 256, 0, s>>>(tab, map + at, in, out, k, gs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int PT, int GT>
hipError_t adamw_copy(int ct, const OptEntry* tab, const OptChunk* map, int64_t chunks, int bits,
                      const qlora_opt_state& in, const qlora_opt_state& out, const AdamwScalars& k,
                      const float* gs, hipStream_t s) {
  if constexpr (PT == kElF32) {   // copies are of fp32 values only
    if (ct == QLORA_BF16) return adamw_types<PT, GT, kElBf16>(tab, map, chunks, bits, in, out, k, gs, s);
    if (ct == QLORA_F16) return adamw_types<PT, GT, kElF16>(tab, map, chunks, bits, in, out, k, gs, s);
  }
  return adamw_types<PT, GT, kElF32>(tab, map, chunks, bits, in, out, k, gs, s);
}

template <int PT>
hipError_t adamw_grad(int gt, int ct, const OptEntry* tab, const OptChunk* map, int64_t chunks,
                      int bits, const qlora_opt_state& in, const qlora_opt_state& out,
                      const AdamwScalars& k, const float* gs, hipStream_t s) {
  if (gt == QLORA_F32) return adamw_copy<PT, kElF32>(ct, tab, map, chunks, bits, in, out, k, gs, s);
  if (gt == QLORA_BF16) return adamw_copy<PT, kElBf16>(ct, tab, map, chunks, bits, in, out, k, gs, s);
  return adamw_copy<PT, kElF16>(ct, tab, map, chunks, bits, in, out, k, gs, s);
}

}  // namespace

hipError_t launch_adamw(const OptEntry* tab, const OptChunk* map, int64_t chunks, int p_dtype,
                        int g_dtype, int copy_dtype, int state_bits, const qlora_opt_state& in,
                        const qlora_opt_state& out, const AdamwScalars& k, const float* gs,
                        hipStream_t s) {
  if (chunks == 0) return hipSuccess;
  if (p_dtype == QLORA_F32)
    return adamw_grad<kElF32>(g_dtype, copy_dtype, tab, map, chunks, state_bits, in, out, k, gs, s);
  if (p_dtype == QLORA_BF16)
    return adamw_grad<kElBf16>(g_dtype, copy_dtype, tab, map, chunks, state_bits, in, out, k, gs, s);
  return adamw_grad<kElF16>(g_dtype, copy_dtype, tab, map, chunks, state_bits, in, out, k, gs, s);
}

hipError_t launch_grad_norm(const OptEntry* tab, const OptChunk* map, int64_t chunks, int g_dtype,
                            float max_norm, float* out, float* part, uint32_t* arrived, hipStream_t s) {
  const int wgs = (int)std::max<int64_t>(1, std::min<int64_t>((chunks + kNormSide - 1) / kNormSide, kNormWgs));
  if (g_dtype == QLORA_F32)
    k_grad_norm<kElF32><<<wgs, kNormThreads, 0, s>>>(tab, map, chunks, max_norm, out, part, arrived);
  else if (g_dtype == QLORA_BF16)
    k_grad_norm<kElBf16><<<wgs, kNormThreads, 0, s>>>(tab, map, chunks, max_norm, out, part, arrived);
  else
    k_grad_norm<kElF16><<<wgs, kNormThreads, 0, s>>>(tab, map, chunks, max_norm, out, part, arrived);
  return hipGetLastError();
}

}  // namespace ql
