// The residual norm of a block and its gradient, a row at a time:
//   p = rms(y) w_post,  h = x + s g p,  z = rms(h) w_pre
// Both directions make one pass over the rows: a row stays in registers
// between its loads and its stores, so each operand crosses memory once and
// the kernels are bound by that traffic.
//
// A row of d values is held by G threads, 16 values each, G the power of two
// from 64 up that covers it: a row of up to 1024 values needs no barrier, a
// wider one exchanges its waves' sums through LDS, one barrier for each sum
// that the next step depends on (two a row in both directions).  A workgroup
// walks the rows, several side by side where they are narrow, with the
// weights, and in the backward the column sums, in registers.  Rows too wide
// for that, or narrower than a vector (k_*_wide), are read once for each
// dependent step, the later times from L2.
//
// The weight of the post norm and a per-channel gate enter every formula as
// their product, and the column sums of their gradients are the same sum
//   T[c] = sum_t D rms(y):   dw_post = s g T,   dgate = s w_post T
// (with a gate that changes from row to row: T = sum_t g D rms(y), dw_post = s T),
// so one register array serves both.
//
// Sums and products take rows already divided by their root mean square, a
// value of the size of 1, and the backward factors the root out last: a square
// or cube of it would leave binary32's range long before the result does (rows of
// 1e15, or of 1e-14 with eps = 0).
//
// Measured: forward of 4096 x 8192 (bf16, fp32 residual) 76 us, 5.3 TB/s;
// 16384 x 4096 (bf16) 95 us, 5.7 TB/s; one row 3.3 us on the device.  Backward
// of 16384 x 4096 with all gradients 154 us, 5.2 TB/s (HBM traffic equal to the
// operands; 520 vector instructions a row and wave, a third of the issue
// slots).  Bound by memory in large calls; in small ones by the dependent
// steps of a row (load, two sums, store: 3 to 4 us) and the launches.
#include <type_traits>

#include "rowio.h"
#include "train_kernels.h"

namespace ql {

namespace {

// Sum over a wave, the same in every lane: DPP shifts within rows of 16, then
// the rows' sums passed on, total in lane 63.
template <int CTRL, int ROWS>
QL_DEV float dpp_add(float v) {
  const int s = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(float, s);
}
QL_DEV float wave_total(float v) {
  v = dpp_add<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);   // row_bcast 15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);   // row_bcast 31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sum of each of v[0..N) over the G threads of a row.  `slot` alternates, so
// that one barrier a call is enough: a wave reaches its next write to the same
// slots only after another barrier.
template <int G, int N, int W>
QL_DEV void row_sum(float (&v)[N], float (*slots)[W][N], int& slot) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_total(v[i]);
  if constexpr (G > 64) {
    constexpr int R = G / 64;   // waves of a row
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, w0 = wave & ~(R - 1);
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) slots[slot][wave][i] = v[i];
    // only the LDS writes have to be done: a full barrier would also wait for
    // the row's stores and the next row's loads
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    QL_LGKMCNT0();
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < R; ++w) s += slots[slot][w0 + w][i];
      v[i] = s;
    }
    slot ^= 1;
  }
}

// 1 / sqrt(x) to one ulp.  The instruction takes a subnormal x for zero: such an x (rows of
// 1e-19 and less with eps = 0) is scaled by a power of four first.
QL_DEV float inv_root(float x) {
  const bool tiny = x < 0x1p-126f;
  const float r = __builtin_amdgcn_rsqf(tiny ? x * 0x1p64f : x);
  return tiny ? r * 0x1p32f : r;
}

// o *= (or =, SET) w_offset + w for N weights; a missing weight counts as 1.
template <int AT, bool SET, int N>
QL_DEV void mul_weight(float (&o)[N], const void* w, bool f32, float offset, int64_t c, int left) {
  if (!w) {
    if (SET)
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = 1.f;
    return;
  }
  float f[N];
  if (AT == kElF32 || f32) {
    const Raw<kElF32, N> r = loadv<kElF32, N>(w, c, left);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = offset + el(r, j);
  } else {
    const Raw<AT, N> r = loadv<AT, N>(w, c, left);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = offset + el(r, j);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] = SET ? f[j] : o[j] * f[j];
}

template <int AT>
QL_DEV float load_param(const void* p, bool f32, int64_t i) {
  return (AT == kElF32 || f32) ? load1<kElF32>(p, i) : load1<AT>(p, i);
}

// What both directions know of a call.
struct Mode {
  bool branch, post, pre, wf32;
  int gate;
  float inv_d;
};
QL_DEV Mode mode_of(const qlora_resnorm& a) {
  const bool branch = a.y != nullptr;
  return {branch, branch && a.post, a.pre != 0, a.param_dtype == kElF32, branch ? a.gate_kind : QLORA_GATE_NONE,
          1.f / (float)a.d};
}
QL_DEV Mode mode_of(const qlora_resnorm_grad& a) {
  const bool branch = a.y != nullptr;
  return {branch, branch && a.post, a.dz != nullptr, a.param_dtype == kElF32,
          branch ? a.gate_kind : QLORA_GATE_NONE, 1.f / (float)a.d};
}

// w_post times a per-channel gate, N columns.
template <int AT, int N, typename Args>
QL_DEV void branch_weight(float (&o)[N], const Args& a, const Mode& k, int c, int left) {
  mul_weight<AT, true>(o, k.post ? a.w_post : nullptr, k.wf32, a.w_offset, c, left);
  if (k.gate == QLORA_GATE_CHANNEL) mul_weight<AT, false>(o, a.gate, k.wf32, 0.f, c, left);
}

constexpr int kHeld = 16, kRowVecs = kHeld / kVec;   // values, vectors a thread holds of a row

// work(row, operands) for every row of the workgroup, the operands by
// load(row, operands): columns past the row's end stay zero.  Side by side with
// the last rows work is called for rows past the end too, with zeros or an
// earlier row's operands, so that the barriers are met: nothing of such a row
// may reach a sum over rows, not even multiplied by zero (its values may not be finite).
// AHEAD: the next row is loaded while this one is worked on.
template <bool AHEAD, int RPW, typename Row, typename Load, typename Work>
QL_DEV void each_row(int64_t m, int sub, Load load, Work work) {
  const int64_t hop = (int64_t)gridDim.x * RPW;
  int64_t row0 = (int64_t)blockIdx.x * RPW;
  if constexpr (AHEAD) {
    Row ra = {}, rb = {};
    load(row0 + sub, ra);
    while (row0 < m) {
      load(row0 + sub + hop, rb);
      work(row0 + sub, ra);
      row0 += hop;
      if (row0 >= m) break;
      load(row0 + sub + hop, ra);
      work(row0 + sub, rb);
      row0 += hop;
    }
  } else {
    Row r = {};
    for (; row0 < m; row0 += hop) {
      load(row0 + sub, r);
      work(row0 + sub, r);
    }
  }
}

// The columns of a thread: kRowVecs vectors.  TAIL: where the row ends inside
// one, it lies over the row's last kVec values instead and leaves out the first `skip`, which the
// thread before holds: every load is a whole vector inside the row.
template <int NV, bool TAIL>
struct Columns {
  int col[NV], skip[TAIL ? NV : 1];
  bool in[NV];
  QL_DEV Columns(int d, int g, int t) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      col[v] = (v * g + t) * kVec;
      in[v] = col[v] < d;
      if constexpr (TAIL) {
        skip[v] = max(0, min(kVec, col[v] + kVec - d));
        col[v] -= skip[v];
      }
    }
  }
  // zeros in the place of the values left out, and of their weights: an infinite
  // weight of the thread before times zero would be no number
  template <int T>
  QL_DEV Raw<T, kVec> only_mine(int v, Raw<T, kVec> r) const {
    if constexpr (TAIL) {
      if constexpr (T == kElF32) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) r.w[j] = j < skip[v] ? 0u : r.w[j];
      } else {
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j)
          r.w[j] &= (2 * j < skip[v] ? 0u : 0xFFFFu) | (2 * j + 1 < skip[v] ? 0u : 0xFFFF0000u);
      }
    }
    return r;
  }
  QL_DEV void only_mine(int v, float (&w)[kVec]) const {
    if constexpr (TAIL)
#pragma unroll
      for (int j = 0; j < kVec; ++j) w[j] = j < skip[v] ? 0.f : w[j];
  }
  template <int T, bool STREAM>
  QL_DEV Raw<T, kVec> load(int v, const char* row) const {
    return only_mine<T>(v, loadv<T, kVec, STREAM>(row, col[v], kVec));
  }
  template <int T, bool STREAM = true>
  QL_DEV void store(int v, void* row, const float (&f)[kVec]) const {
    if constexpr (TAIL)
      if (skip[v] > 0) {
#pragma unroll
        for (int j = 1; j < kVec; ++j)
          if (j >= skip[v]) store1<T>(row, col[v] + j, f[j]);
        return;
      }
    storev<T, kVec, STREAM>(row, col[v], kVec, f);
  }
};

// FULL: a gate value for every element.  TAIL: d is not a multiple of kVec.
// STREAM: loads past the caches (see kStreamBytes).
template <int AT, int RT, int G, bool FULL, bool TAIL, bool STREAM>
__global__ __launch_bounds__(resnorm_fwd_block(G)) void k_resnorm_fwd(qlora_resnorm a) {
  constexpr int EV = kVec, NV = kRowVecs;
  constexpr int TPB = resnorm_fwd_block(G), RPW = TPB / G;   // rows a workgroup holds at a time
  __shared__ float slots[2][TPB / 64][1];
  int slot = 0;
  const int t = threadIdx.x & (G - 1);
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  const Mode k = mode_of(a);
  float wb[NV][EV] = {}, wpre[NV][EV] = {};
  const Columns<NV, TAIL> at_col((int)a.d, G, t);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!at_col.in[v]) continue;
    if (k.branch) branch_weight<AT, EV>(wb[v], a, k, at_col.col[v], EV);
    if (k.pre) mul_weight<AT, true, EV>(wpre[v], a.w_pre, k.wf32, a.w_offset, at_col.col[v], EV);
    at_col.only_mine(v, wb[v]);
    at_col.only_mine(v, wpre[v]);
  }

  struct Row {
    Raw<RT, EV> x[NV];
    Raw<AT, EV> y[NV], g[FULL ? NV : 1];
  };
  auto load_row = [&](int64_t row, Row& r) {
    if (row >= a.m) return;
    const char* x = row_of<RT>(a.x, row, a.ldx);
    const char* y = row_of<AT>(a.y, row, a.ldy);
    const char* g = row_of<AT>(a.gate, row, a.ldg);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at_col.in[v]) continue;
      if (k.branch) r.y[v] = at_col.template load<AT, STREAM>(v, y);
      r.x[v] = at_col.template load<RT, STREAM>(v, x);
      if (FULL) r.g[v] = at_col.template load<AT, STREAM>(v, g);
    }
  };
  auto work = [&](int64_t row, const Row& r) {
    const bool live = row < a.m;
    float sg = a.scale;
    if (k.gate == QLORA_GATE_TOKEN && live) sg *= load_param<AT>(a.gate, k.wf32, row);
    if (k.post) {
      float s[1] = {0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < EV; ++j) s[0] += el(r.y[v], j) * el(r.y[v], j);
      row_sum<G>(s, slots, slot);
      sg *= inv_root(s[0] * k.inv_d + a.eps);
    }
    float h[NV][EV];
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < EV; ++j) {
        float b = el(r.y[v], j) * (sg * wb[v][j]);
        if (FULL) b *= el(r.g[v], j);
        h[v][j] = el(r.x[v], j) + b;
        s[0] += h[v][j] * h[v][j];
      }
    if (live && k.branch) {
      char* o = row_of<RT>(a.h, row, a.ldh);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (at_col.in[v]) at_col.template store<RT>(v, o, h[v]);
    }
    if (!k.pre) return;
    row_sum<G>(s, slots, slot);
    if (!live) return;
    const float rh = inv_root(s[0] * k.inv_d + a.eps);
    char* o = row_of<AT>(a.z, row, a.ldz);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < EV; ++j) h[v][j] *= rh * wpre[v][j];
      if (at_col.in[v]) at_col.template store<AT>(v, o, h[v]);
    }
  };
  each_row<!FULL, RPW, Row>(a.m, sub, load_row, work);
}

// Threads to a row that the register kernels do not hold: 1024 where it is
// wide (4096 x 16384 bf16 forward 157 us; backward with column sums 328 us),
// one wave where it is narrower than a vector (16384 x 5 forward 22 us, with
// 1024 threads 217).
constexpr int kWideThreads = 1024, kNarrowThreads = 64;

// A workgroup to a row; each dependent step reads the row again.
template <int AT, int RT, int WT>
__global__ __launch_bounds__(WT) void k_resnorm_fwd_wide(qlora_resnorm a) {
  constexpr int EV = kVec;
  __shared__ float slots[2][WT / 64][1];
  int slot = 0;
  const Mode k = mode_of(a);
  const int d = (int)a.d;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
    float sg = a.scale;
    if (k.gate == QLORA_GATE_TOKEN) sg *= load_param<AT>(a.gate, k.wf32, row);
    if (k.post) {
      float s[1] = {0.f};
      for (int c = threadIdx.x * EV; c < d; c += WT * EV) {
        const Raw<AT, EV> y = loadv<AT, EV>(row_of<AT>(a.y, row, a.ldy), c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) s[0] += el(y, j) * el(y, j);
      }
      row_sum<WT>(s, slots, slot);
      sg *= inv_root(s[0] * k.inv_d + a.eps);
    }
    auto residual = [&](int c, float (&h)[EV]) {
      const Raw<RT, EV> x = loadv<RT, EV>(row_of<RT>(a.x, row, a.ldx), c, d - c);
#pragma unroll
      for (int j = 0; j < EV; ++j) h[j] = el(x, j);
      if (!k.branch) return;
      float w[EV];
      branch_weight<AT, EV>(w, a, k, c, d - c);
      if (k.gate == QLORA_GATE_FULL) {
        const Raw<AT, EV> g = loadv<AT, EV>(row_of<AT>(a.gate, row, a.ldg), c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) w[j] *= el(g, j);
      }
      const Raw<AT, EV> y = loadv<AT, EV>(row_of<AT>(a.y, row, a.ldy), c, d - c);
#pragma unroll
      for (int j = 0; j < EV; ++j) h[j] += el(y, j) * sg * w[j];
    };
    float rh = 0.f;
    if (k.pre) {
      float s[1] = {0.f};
      for (int c = threadIdx.x * EV; c < d; c += WT * EV) {
        float h[EV];
        residual(c, h);
#pragma unroll
        for (int j = 0; j < EV; ++j) s[0] += (c + j < d) ? h[j] * h[j] : 0.f;
      }
      row_sum<WT>(s, slots, slot);
      rh = inv_root(s[0] * k.inv_d + a.eps);
    }
    for (int c = threadIdx.x * EV; c < d; c += WT * EV) {
      float h[EV], w[EV];
      residual(c, h);
      if (k.branch) storev<RT, EV, true>(row_of<RT>(a.h, row, a.ldh), c, d - c, h);
      if (k.pre) {
        mul_weight<AT, true, EV>(w, a.w_pre, k.wf32, a.w_offset, c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) h[j] *= rh * w[j];
        storev<AT, EV, true>(row_of<AT>(a.z, row, a.ldz), c, d - c, h);
      }
    }
  }
}

// One row's operands, as loaded; zeros where there is none.
template <int AT, int RT, bool FULL>
struct GradRow {
  Raw<AT, kVec> dz[kRowVecs], y[kRowVecs], g[FULL ? kRowVecs : 1];
  Raw<RT, kVec> dh[kRowVecs], h[kRowVecs];
};

template <int AT, int RT, int G, bool FULL, bool TAIL, bool STREAM>
__global__ __launch_bounds__(kResnormBwdBlock) void k_resnorm_bwd(qlora_resnorm_grad a, float* part) {
  constexpr int EV = kVec, NV = kRowVecs;
  constexpr int TPB = kResnormBwdBlock, RPW = TPB / G;
  // the next row is loaded while this one is worked on, where the registers
  // hold both (16-bit residual, no gate row)
  constexpr bool AHEAD = RT != kElF32 && !FULL;
  __shared__ float slots3[2][TPB / 64][3];
  __shared__ float slots2[2][TPB / 64][2];
  __shared__ float sums[RPW > 1 ? RPW - 1 : 1][2][kHeld][RPW > 1 ? G : 1];
  int slot3 = 0, slot2 = 0;
  const int t = threadIdx.x & (G - 1);
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  const Mode k = mode_of(a);

  float wb[NV][EV] = {}, wpre[NV][EV] = {}, apre[NV][EV] = {}, at[NV][EV] = {};
  const Columns<NV, TAIL> at_col((int)a.d, G, t);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!at_col.in[v]) continue;
    if (k.branch) branch_weight<AT, EV>(wb[v], a, k, at_col.col[v], EV);
    if (k.pre) mul_weight<AT, true, EV>(wpre[v], a.w_pre, k.wf32, a.w_offset, at_col.col[v], EV);
    at_col.only_mine(v, wb[v]);
    at_col.only_mine(v, wpre[v]);
  }
  using Row = GradRow<AT, RT, FULL>;
  auto load_row = [&](int64_t row, Row& r) {
    if (row >= a.m) return;
    const char* dz = row_of<AT>(a.dz, row, a.lddz);
    const char* h = row_of<RT>(a.h, row, a.ldh);
    const char* dh = row_of<RT>(a.dh, row, a.lddh);
    const char* y = row_of<AT>(a.y, row, a.ldy);
    const char* g = row_of<AT>(a.gate, row, a.ldg);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at_col.in[v]) continue;
      if (k.pre) r.dz[v] = at_col.template load<AT, STREAM>(v, dz);
      if (k.pre) r.h[v] = at_col.template load<RT, STREAM>(v, h);
      if (a.dh) r.dh[v] = at_col.template load<RT, STREAM>(v, dh);
      if (k.branch) r.y[v] = at_col.template load<AT, STREAM>(v, y);
      if (FULL) r.g[v] = at_col.template load<AT, STREAM>(v, g);
    }
  };
  auto work = [&](int64_t row, const Row& r) {
    const bool live = row < a.m;
    float s3[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < EV; ++j) {
        const float hv = el(r.h[v], j), yv = el(r.y[v], j);
        s3[0] += hv * hv;
        s3[1] += el(r.dz[v], j) * wpre[v][j] * hv;
        s3[2] += yv * yv;
      }
    row_sum<G>(s3, slots3, slot3);
    const float rsh = k.pre ? inv_root(s3[0] * k.inv_d + a.eps) : 0.f;
    const float ch = s3[1] * rsh * k.inv_d;   // mean(A rms(h))
    const float rsy = k.post ? inv_root(s3[2] * k.inv_d + a.eps) : 1.f;
    float gt = 1.f;
    if (k.gate == QLORA_GATE_TOKEN && live) gt = load_param<AT>(a.gate, k.wf32, row);

    float D[NV][EV];
    float s2[2] = {0.f, 0.f};   // sums of D p and, with the full gate, g D p
    char* dx = row_of<RT>(a.dx, row, a.lddx);
    char* dgate = FULL ? row_of<AT>(a.dgate, row, a.lddg) : nullptr;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float dg[EV];
#pragma unroll
      for (int j = 0; j < EV; ++j) {
        const float hn = el(r.h[v], j) * rsh, z = el(r.dz[v], j);
        const float x = el(r.dh[v], j) + (z * wpre[v][j] - hn * ch) * rsh;
        const float xy = x * (el(r.y[v], j) * rsy), dp = xy * wb[v][j];
        D[v][j] = x;
        s2[0] += dp;
        float g = gt;
        if constexpr (FULL) {
          g = el(r.g[v], j);
          s2[1] += dp * g;
          dg[j] = a.scale * dp;
        }
        if (live) {
          apre[v][j] += z * hn;
          at[v][j] += xy * g;
        }
      }
      if (live && at_col.in[v]) {
        at_col.template store<RT>(v, dx, D[v]);
        if constexpr (FULL)
          if (a.dgate) at_col.template store<AT>(v, dgate, dg);
      }
    }
    if (!k.branch) return;
    if ((k.post && a.dy) || (k.gate == QLORA_GATE_TOKEN && a.dgate)) row_sum<G>(s2, slots2, slot2);
    if (k.gate == QLORA_GATE_TOKEN && a.dgate && live && t == 0)
      gptr_w(reinterpret_cast<float*>(a.dgate))[row] = a.scale * s2[0];
    if (!a.dy || !live) return;
    // dy = ry s (g D w - rms(y) mean(g D p)), the mean without a post norm left out
    const float sgt = a.scale * gt * rsy, cy = k.post ? s2[FULL] * k.inv_d : 0.f;
    char* dy = row_of<AT>(a.dy, row, a.lddy);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < EV; ++j) {
        D[v][j] *= wb[v][j];
        if constexpr (FULL) D[v][j] *= el(r.g[v], j);
      }
      if (k.post)
#pragma unroll
        for (int j = 0; j < EV; ++j) D[v][j] -= el(r.y[v], j) * rsy * cy;
#pragma unroll
      for (int j = 0; j < EV; ++j) D[v][j] *= sgt;
      if (at_col.in[v]) at_col.template store<AT>(v, dy, D[v]);
    }
  };

  each_row<AHEAD, RPW, Row>(a.m, sub, load_row, work);

  if (part) {
    // the sums of the rows held side by side, joined in order
    if constexpr (RPW > 1) {
      if (sub > 0)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < EV; ++j) {
            sums[sub - 1][0][v * EV + j][t] = apre[v][j];
            sums[sub - 1][1][v * EV + j][t] = at[v][j];
          }
      __syncthreads();
      if (sub > 0) return;
      for (int i = 0; i < RPW - 1; ++i)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < EV; ++j) {
            apre[v][j] += sums[i][0][v * EV + j][t];
            at[v][j] += sums[i][1][v * EV + j][t];
          }
    }
    float* o = part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!at_col.in[v]) continue;
      at_col.template store<kElF32, false>(v, o, apre[v]);
      at_col.template store<kElF32, false>(v, o + a.d, at[v]);
    }
  }
}

// Wide rows.  With `stat` only the row's statistics are written (and a token
// gate's gradient): k_resnorm_cols then forms the outputs along with the column sums.
template <int AT, int RT, int WT>
__global__ __launch_bounds__(WT) void k_resnorm_bwd_wide(qlora_resnorm_grad a, f32x4_t* stat) {
  constexpr int EV = kVec;
  __shared__ float slots3[2][WT / 64][3];
  __shared__ float slots2[2][WT / 64][2];
  int slot3 = 0, slot2 = 0;
  const Mode k = mode_of(a);
  const int d = (int)a.d;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
    float s3[3] = {0.f, 0.f, 0.f};
    for (int c = threadIdx.x * EV; c < d; c += WT * EV) {
      if (k.pre) {
        float w[EV];
        mul_weight<AT, true, EV>(w, a.w_pre, k.wf32, a.w_offset, c, d - c);
        const Raw<AT, EV> dz = loadv<AT, EV>(row_of<AT>(a.dz, row, a.lddz), c, d - c);
        const Raw<RT, EV> h = loadv<RT, EV>(row_of<RT>(a.h, row, a.ldh), c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) {
          s3[0] += el(h, j) * el(h, j);
          s3[1] += el(dz, j) * w[j] * el(h, j);
        }
      }
      if (k.post) {
        const Raw<AT, EV> y = loadv<AT, EV>(row_of<AT>(a.y, row, a.ldy), c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) s3[2] += el(y, j) * el(y, j);
      }
    }
    row_sum<WT>(s3, slots3, slot3);
    const float rsh = k.pre ? inv_root(s3[0] * k.inv_d + a.eps) : 0.f;
    const float ch = s3[1] * rsh * k.inv_d;   // mean(A rms(h))
    const float rsy = k.post ? inv_root(s3[2] * k.inv_d + a.eps) : 1.f;
    float gt = 1.f;
    if (k.gate == QLORA_GATE_TOKEN) gt = load_param<AT>(a.gate, k.wf32, row);
    auto upstream = [&](int c, float (&D)[EV]) {
#pragma unroll
      for (int j = 0; j < EV; ++j) D[j] = 0.f;
      if (a.dh) {
        const Raw<RT, EV> dh = loadv<RT, EV>(row_of<RT>(a.dh, row, a.lddh), c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) D[j] = el(dh, j);
      }
      if (k.pre) {
        float w[EV];
        mul_weight<AT, true, EV>(w, a.w_pre, k.wf32, a.w_offset, c, d - c);
        const Raw<AT, EV> dz = loadv<AT, EV>(row_of<AT>(a.dz, row, a.lddz), c, d - c);
        const Raw<RT, EV> h = loadv<RT, EV>(row_of<RT>(a.h, row, a.ldh), c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) D[j] += (el(dz, j) * w[j] - el(h, j) * rsh * ch) * rsh;
      }
    };
    float s2[2] = {0.f, 0.f};
    if (k.branch && ((k.post && a.dy) || (k.gate == QLORA_GATE_TOKEN && a.dgate))) {
      for (int c = threadIdx.x * EV; c < d; c += WT * EV) {
        float D[EV], w[EV];
        upstream(c, D);
        branch_weight<AT, EV>(w, a, k, c, d - c);
        const Raw<AT, EV> y = loadv<AT, EV>(row_of<AT>(a.y, row, a.ldy), c, d - c);
        Raw<AT, EV> g;
        if (k.gate == QLORA_GATE_FULL) g = loadv<AT, EV>(row_of<AT>(a.gate, row, a.ldg), c, d - c);
#pragma unroll
        for (int j = 0; j < EV; ++j) {
          const float dp = (c + j < d) ? D[j] * (el(y, j) * rsy) * w[j] : 0.f;
          s2[0] += dp;
          if (k.gate == QLORA_GATE_FULL) s2[1] += dp * el(g, j);
        }
      }
      row_sum<WT>(s2, slots2, slot2);
      if (k.gate == QLORA_GATE_TOKEN && a.dgate && threadIdx.x == 0)
        gptr_w(reinterpret_cast<float*>(a.dgate))[row] = a.scale * s2[0];
    }
    const float sgt = a.scale * gt * rsy;
    const float cy = k.post ? (k.gate == QLORA_GATE_FULL ? s2[1] : s2[0]) * k.inv_d : 0.f;
    if (stat) {
      if (threadIdx.x == 0) stat[row] = f32x4_t{rsh, ch, rsy, cy};
      continue;
    }
    for (int c = threadIdx.x * EV; c < d; c += WT * EV) {
      float D[EV], w[EV], dg[EV];
      upstream(c, D);
      Raw<AT, EV> y, g;
      if (k.branch) {
        branch_weight<AT, EV>(w, a, k, c, d - c);
        y = loadv<AT, EV>(row_of<AT>(a.y, row, a.ldy), c, d - c);
        if (k.gate == QLORA_GATE_FULL) g = loadv<AT, EV>(row_of<AT>(a.gate, row, a.ldg), c, d - c);
      }
      storev<RT, EV, true>(row_of<RT>(a.dx, row, a.lddx), c, d - c, D);
      if (!k.branch) continue;
#pragma unroll
      for (int j = 0; j < EV; ++j) {
        dg[j] = a.scale * D[j] * (el(y, j) * rsy) * w[j];
        D[j] *= w[j];
        if (k.gate == QLORA_GATE_FULL) D[j] *= el(g, j);
        D[j] = (k.post ? D[j] - el(y, j) * rsy * cy : D[j]) * sgt;
      }
      if (k.gate == QLORA_GATE_FULL && a.dgate) storev<AT, EV, true>(row_of<AT>(a.dgate, row, a.lddg), c, d - c, dg);
      if (a.dy) storev<AT, EV, true>(row_of<AT>(a.dy, row, a.lddy), c, d - c, D);
    }
  }
}

// Outputs and column sums of wide rows from the rows' statistics: a thread
// owns eight columns, a workgroup a run of rows.
template <int AT, int RT>
__global__ __launch_bounds__(256) void k_resnorm_cols(qlora_resnorm_grad a, const f32x4_t* stat,
                                                      float* part, int64_t rows_per_wg) {
  constexpr int EV = kVec;
  const int c = (int)(blockIdx.x * 256 + threadIdx.x) * EV, left = (int)a.d - c;
  if (left <= 0) return;
  const Mode k = mode_of(a);
  const bool full = k.gate == QLORA_GATE_FULL;
  float wb[EV], wpre[EV], sr[EV] = {}, st[EV] = {};
  branch_weight<AT, EV>(wb, a, k, c, left);
  mul_weight<AT, true, EV>(wpre, k.pre ? a.w_pre : nullptr, k.wf32, a.w_offset, c, left);
  const int64_t r1 = min(a.m, ((int64_t)blockIdx.y + 1) * rows_per_wg);
#pragma unroll 2
  for (int64_t r = (int64_t)blockIdx.y * rows_per_wg; r < r1; ++r) {
    const f32x4_t s = stat[r];
    Raw<AT, EV> dz = {}, y = {}, g = {};
    Raw<RT, EV> dh = {}, h = {};
    if (k.pre) dz = loadv<AT, EV, true>(row_of<AT>(a.dz, r, a.lddz), c, left);
    if (k.pre) h = loadv<RT, EV, true>(row_of<RT>(a.h, r, a.ldh), c, left);
    if (a.dh) dh = loadv<RT, EV, true>(row_of<RT>(a.dh, r, a.lddh), c, left);
    if (k.branch) y = loadv<AT, EV, true>(row_of<AT>(a.y, r, a.ldy), c, left);
    if (full) g = loadv<AT, EV, true>(row_of<AT>(a.gate, r, a.ldg), c, left);
    const float gt = k.gate == QLORA_GATE_TOKEN ? load_param<AT>(a.gate, k.wf32, r) : 1.f;
    float D[EV], dg[EV];
#pragma unroll
    for (int j = 0; j < EV; ++j) {
      const float hn = el(h, j) * s[0];
      D[j] = el(dh, j) + (el(dz, j) * wpre[j] - hn * s[1]) * s[0];
      sr[j] += el(dz, j) * hn;
    }
    storev<RT, EV, true>(row_of<RT>(a.dx, r, a.lddx), c, left, D);
    if (!k.branch) continue;
#pragma unroll
    for (int j = 0; j < EV; ++j) {
      const float yn = el(y, j) * s[2], xy = D[j] * yn;
      st[j] += xy * (full ? el(g, j) : gt);
      dg[j] = a.scale * xy * wb[j];
      D[j] *= wb[j];
      if (full) D[j] *= el(g, j);
      D[j] = (k.post ? D[j] - yn * s[3] : D[j]) * (a.scale * gt * s[2]);
    }
    if (full && a.dgate) storev<AT, EV, true>(row_of<AT>(a.dgate, r, a.lddg), c, left, dg);
    if (a.dy) storev<AT, EV, true>(row_of<AT>(a.dy, r, a.lddy), c, left, D);
  }
  float* o = part + (int64_t)blockIdx.y * 2 * a.d;
  storev<kElF32, EV>(o, c, left, sr);
  storev<kElF32, EV>(o + a.d, c, left, st);
}

// dw_pre = sum of part[.][0][c], T = sum of part[.][1][c] and from it dw_post
// and the channel gate's gradient: a wave adds every 16th part of 64 columns,
// then the 16 waves' sums are joined in order.
template <int AT>
__global__ __launch_bounds__(1024) void k_resnorm_join(qlora_resnorm_grad a, const float* __restrict__ part,
                                                       int nparts) {
  __shared__ float s[16][64];
  const Mode k = mode_of(a);
  float* gc = k.gate == QLORA_GATE_CHANNEL ? (float*)a.dgate : nullptr;
  const bool second = blockIdx.y == 1;
  if (second ? !a.dw_post && !gc : !a.dw_pre) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float acc = 0.f;
  if (c < a.d) {
    const float* p = part + (int64_t)blockIdx.y * a.d + c;
#pragma unroll 4
    for (int i = w; i < nparts; i += 16) acc += p[(int64_t)i * 2 * a.d];
  }
  s[w][lane] = acc;
  __syncthreads();
  if (w != 0 || c >= a.d) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += s[i][lane];
  if (!second) {
    a.dw_pre[c] = v;
    return;
  }
  v *= a.scale;
  if (a.dw_post) a.dw_post[c] = k.gate == QLORA_GATE_CHANNEL ? v * load_param<AT>(a.gate, k.wf32, c) : v;
  if (gc) gc[c] = k.post && a.w_post ? v * (a.w_offset + load_param<AT>(a.w_post, k.wf32, c)) : v;
}

__global__ void k_zero_f32(float* o0, float* o1, float* o2, int64_t d) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  if (o0) o0[c] = 0.f;
  if (o1) o1[c] = 0.f;
  if (o2) o2[c] = 0.f;
}

// f(workgroups, threads to a row) for rows outside the register kernels.
template <typename F>
void wide_launch(int64_t m, int64_t d, F f) {
  if (d > kResnormMaxInRow)
    f((unsigned)std::min<int64_t>(m, kResnormWideWgs), std::integral_constant<int, kWideThreads>{});
  else
    f((unsigned)std::min<int64_t>(m, 16 * kResnormWideWgs), std::integral_constant<int, kNarrowThreads>{});
}

// A call that moves more than this reads past the caches: 16384 x 4096 bf16
// (537 MB forward, 805 MB backward) 94 against 99 us and 153 against 157; one
// that moves less may find its operands there: 16384 x 1024 26 against 23 us forward,
// 2048 x 4096 29 against 26 backward.
constexpr int64_t kStreamBytes = int64_t(256) << 20;

template <int AT, int RT, int G, bool FULL, bool TAIL, bool STREAM>
void fwd_rows(const qlora_resnorm& a, hipStream_t s) {
  constexpr int block = resnorm_fwd_block(G);
  const int64_t wgs = std::min<int64_t>((a.m + block / G - 1) / (block / G), kResnormFwdWgs);
  k_resnorm_fwd<AT, RT, G, FULL, TAIL, STREAM><<<(unsigned)wgs, block, 0, s>>>(a);
}

template <int AT, int RT, bool FULL, bool TAIL, bool STREAM>
void fwd_width(const qlora_resnorm& a, hipStream_t s) {
  switch (resnorm_threads(a.d)) {
    case 64: return fwd_rows<AT, RT, 64, FULL, TAIL, STREAM>(a, s);
    case 128: return fwd_rows<AT, RT, 128, FULL, TAIL, STREAM>(a, s);
    case 256: return fwd_rows<AT, RT, 256, FULL, TAIL, STREAM>(a, s);
    default: return fwd_rows<AT, RT, 512, FULL, TAIL, STREAM>(a, s);
  }
}

template <int AT, int RT>
hipError_t fwd_types(const qlora_resnorm& a, hipStream_t s) {
  const bool full = a.gate_kind == QLORA_GATE_FULL, tail = a.d % kVec != 0;
  const int64_t row_bytes = a.d * 2 * (kElBytes<AT> + kElBytes<RT>);
  if (resnorm_wide(a.d))
    wide_launch(a.m, a.d, [&](unsigned wgs, auto wt) { k_resnorm_fwd_wide<AT, RT, wt.value><<<wgs, wt.value, 0, s>>>(a); });
  else if (full)
    tail ? fwd_width<AT, RT, true, true, false>(a, s) : fwd_width<AT, RT, true, false, false>(a, s);
  else if (tail)
    fwd_width<AT, RT, false, true, false>(a, s);
  else if (a.m > kStreamBytes / row_bytes)
    fwd_width<AT, RT, false, false, true>(a, s);
  else
    fwd_width<AT, RT, false, false, false>(a, s);
  return hipGetLastError();
}

template <int AT, int RT, bool FULL, bool TAIL, bool STREAM>
void bwd_width(const ResnormBwdPlan& p, const qlora_resnorm_grad& a, float* part, hipStream_t s) {
  constexpr int block = kResnormBwdBlock;
  switch (resnorm_threads(a.d)) {
    case 64: k_resnorm_bwd<AT, RT, 64, FULL, TAIL, STREAM><<<p.wgs, block, 0, s>>>(a, part); return;
    case 128: k_resnorm_bwd<AT, RT, 128, FULL, TAIL, STREAM><<<p.wgs, block, 0, s>>>(a, part); return;
    case 256: k_resnorm_bwd<AT, RT, 256, FULL, TAIL, STREAM><<<p.wgs, block, 0, s>>>(a, part); return;
    default: k_resnorm_bwd<AT, RT, 512, FULL, TAIL, STREAM><<<p.wgs, block, 0, s>>>(a, part); return;
  }
}

template <int AT, int RT>
hipError_t bwd_types(const ResnormBwdPlan& p, const qlora_resnorm_grad& a, void* ws, hipStream_t s) {
  const bool cols = a.dw_post || a.dw_pre || (a.dgate && a.gate_kind == QLORA_GATE_CHANNEL);
  const bool full = a.gate_kind == QLORA_GATE_FULL, tail = a.d % kVec != 0;
  float* part = cols ? (float*)((char*)ws + p.part_off) : nullptr;
  int nparts = p.wgs;
  if (resnorm_wide(a.d)) {
    f32x4_t* stat = cols ? (f32x4_t*)((char*)ws + p.stat_off) : nullptr;
    wide_launch(a.m, a.d, [&](unsigned wgs, auto wt) { k_resnorm_bwd_wide<AT, RT, wt.value><<<wgs, wt.value, 0, s>>>(a, stat); });
    if (cols) {
      const int64_t rpg = (a.m + p.wgs - 1) / p.wgs;
      nparts = (int)((a.m + rpg - 1) / rpg);
      const dim3 grid((unsigned)((a.d + 256 * kVec - 1) / (256 * kVec)), (unsigned)nparts);
      k_resnorm_cols<AT, RT><<<grid, 256, 0, s>>>(a, stat, part, rpg);
    }
  } else if (full) {
    tail ? bwd_width<AT, RT, true, true, false>(p, a, part, s) : bwd_width<AT, RT, true, false, false>(p, a, part, s);
  } else if (tail) {
    bwd_width<AT, RT, false, true, false>(p, a, part, s);
  } else if (a.m > kStreamBytes / (a.d * 3 * (kElBytes<AT> + kElBytes<RT>))) {
    bwd_width<AT, RT, false, false, true>(p, a, part, s);
  } else {
    bwd_width<AT, RT, false, false, false>(p, a, part, s);
  }
  if (cols) k_resnorm_join<AT><<<dim3((unsigned)((a.d + 63) / 64), 2), 1024, 0, s>>>(a, part, nparts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_resnorm_fwd(const qlora_resnorm& a, hipStream_t s) {
  if (a.act_dtype == QLORA_F32) return fwd_types<kElF32, kElF32>(a, s);
  if (a.act_dtype == QLORA_BF16)
    return a.res_dtype == QLORA_F32 ? fwd_types<kElBf16, kElF32>(a, s) : fwd_types<kElBf16, kElBf16>(a, s);
  return a.res_dtype == QLORA_F32 ? fwd_types<kElF16, kElF32>(a, s) : fwd_types<kElF16, kElF16>(a, s);
}

hipError_t launch_resnorm_zero(float* o0, float* o1, float* o2, int64_t d, hipStream_t s) {
  k_zero_f32<<<(unsigned)((d + 255) / 256), 256, 0, s>>>(o0, o1, o2, d);
  return hipGetLastError();
}

hipError_t launch_resnorm_bwd(const ResnormBwdPlan& p, const qlora_resnorm_grad& a, void* ws,
                              hipStream_t s) {
  if (a.act_dtype == QLORA_F32) return bwd_types<kElF32, kElF32>(p, a, ws, s);
  if (a.act_dtype == QLORA_BF16)
    return a.res_dtype == QLORA_F32 ? bwd_types<kElBf16, kElF32>(p, a, ws, s)
                                    : bwd_types<kElBf16, kElBf16>(p, a, ws, s);
  return a.res_dtype == QLORA_F32 ? bwd_types<kElF16, kElF32>(p, a, ws, s)
                                  : bwd_types<kElF16, kElF16>(p, a, ws, s);
}

}  // namespace ql
