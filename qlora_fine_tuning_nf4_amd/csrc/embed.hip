// Token embedding: out[t] = s E[id_t], and its gradient dE[v] = s sum dY[t]
// over the tokens t of row v.
//
// The forward is a gather: a thread moves vectors of eight values, four in
// flight.  The gradient sorts the tokens by id and adds up runs of equal ids:
//  * k_embed_sort -- groups the tokens by row.  Workgroup b of W (a power of
//    two, one a CU or more) owns the rows v = b mod W, so that the frequent
//    tokens, which sit together at the low ids, are spread.  Every workgroup
//    reads all ids (from L2): its 16 waves count the ids of its rows in strips
//    of the token sequence, a prefix over rows and strips gives each (strip,
//    row) its place, and a second look at the ids puts them there.  The tokens
//    of a row keep their order, and workgroups exchange nothing.
//  * k_embed_sum -- a wave adds `chunk` consecutive sorted tokens, 512
//    columns at a time, so that a token with thousands of occurrences costs
//    no more than thousands of different ones.  A run within the chunk is
//    written; the two ends of a run that crosses chunks are left as fp32 partial sums.
//    The same launch writes the zero rows.
//  * k_embed_join -- adds those partial sums in order.
//
// Measured: lookup of 20001 rows of 8192 fp32 values to bf16 103 us (5.1 TB/s
// with every table row counted once; repeats come from the caches), 16 rows
// 4 us on the device.  Gradient of 32768 tokens of 4096 into a bf16 table of
// 32000 rows 147 us: sort 28, sum and zero rows 111 (4.8 TB/s), join 9; of
// 2048 tokens into an fp32 table 113 us: sort 7, sum and zero rows 100 (5.4
// TB/s, nearly all of it zero rows), join 7.  The sort is bound by the latency of
// cold ids and of its own code, the join by four dependent loads.
#include <algorithm>

#include "rowio.h"
#include "train_kernels.h"

namespace ql {

namespace {

template <bool I64>
QL_DEV int64_t load_id(const void* ids, int64_t t) {
  if constexpr (I64)
    return gptr(reinterpret_cast<const int64_t*>(ids))[t];
  else
    return gptr(reinterpret_cast<const int32_t*>(ids))[t];
}

// Table row of token t, or -1 outside the table.
template <bool I64>
QL_DEV int load_row(const void* ids, int64_t t, int vocab) {
  const int64_t v = load_id<I64>(ids, t);
  return v >= 0 && v < vocab ? (int)v : -1;
}

// Vectors a thread holds in flight: 64 bytes (20001 x 8192 bf16: 84 us, with 32
// bytes 88, with 16 101; from fp32 106, with 128 bytes 111).
template <int ET>
constexpr int kFwdVecs = 8 / kElBytes<ET>;

template <int ET, int OT, bool I64>
__global__ __launch_bounds__(256) void k_embed_fwd(const void* __restrict__ E, int vocab, int d,
                                                   int64_t lde, const void* __restrict__ ids,
                                                   uint32_t total, float scale,
                                                   void* __restrict__ out, int64_t ldo,
                                                   uint32_t nvec) {
  constexpr int EV = kVec;
  const uint32_t first = blockIdx.x * (256 * kFwdVecs<ET>) + threadIdx.x;
  Raw<ET, EV> r[kFwdVecs<ET>];
  int64_t row[kFwdVecs<ET>];
  int col[kFwdVecs<ET>], src[kFwdVecs<ET>];
#pragma unroll
  for (int i = 0; i < kFwdVecs<ET>; ++i) {
    const uint32_t q = first + i * 256;
    src[i] = -1;
    row[i] = -1;
    if (q < total) {
      row[i] = q / nvec;
      col[i] = (int)(q - (uint32_t)row[i] * nvec) * EV;
      src[i] = load_row<I64>(ids, row[i], vocab);
    }
  }
#pragma unroll
  for (int i = 0; i < kFwdVecs<ET>; ++i)
    if (src[i] >= 0) r[i] = loadv<ET, EV>(row_of<ET>(E, src[i], lde), col[i], d - col[i]);
#pragma unroll
  for (int i = 0; i < kFwdVecs<ET>; ++i) {
    if (row[i] < 0) continue;
    float f[EV];
#pragma unroll
    for (int j = 0; j < EV; ++j) f[j] = src[i] >= 0 ? el(r[i], j) * scale : 0.f;
    storev<OT, EV, true>(row_of<OT>(out, row[i], ldo), col[i], d - col[i], f);
  }
}

// Zeros to a row of d values, by a wave.
template <int GT>
QL_DEV void zero_row(char* row, int d, int lane) {
  constexpr int ZV = 16 / kElBytes<GT>;
  float zero[ZV];
#pragma unroll
  for (int j = 0; j < ZV; ++j) zero[j] = 0.f;
  for (int c = lane * ZV; c < d; c += 64 * ZV) storev<GT, ZV>(row, c, d - c, zero);
}

constexpr int kSortWaves = 16;
constexpr int kSortSteps = 32;   // 64-id steps a wave holds in LDS
constexpr int kSortLoads = 16;   // of them loaded at once

// A token with a row in the table: the row, the token's position.
struct Token {
  int row, pos;
};

// tokens[i] for i < seen[0], the number of tokens with a row in the table: grouped by
// row, the tokens of a row in order.
// has[v]: whether row v has a token (has may be NULL).
template <bool I64>
__global__ __launch_bounds__(64 * kSortWaves) void k_embed_sort(const void* __restrict__ ids, int m,
                                                                int vocab, int range, int log_w,
                                                                Token* __restrict__ tokens,
                                                                int* __restrict__ seen,
                                                                uint8_t* __restrict__ has) {
  __shared__ int cnt[kSortWaves][kEmbedRange];
  __shared__ int16_t loc[kSortWaves][kSortSteps][64];   // index of the id's row in the range, or -1
  __shared__ int below_w[kSortWaves], scan_w[kSortWaves];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x, wmask = (1 << log_w) - 1;
  const int strip = ((m + kSortWaves - 1) / kSortWaves + 63) & ~63;
  const int t0 = min(m, w * strip), t1 = min(m, t0 + strip);
  for (int r = lane; r < range; r += 64) cnt[w][r] = 0;
  // steps [t, t + 64 kSortSteps) into loc; the steps that hold an id of the
  // range as a bit mask (the others' loc is not written)
  int below = 0;
  auto load_steps = [&](int t, bool count) {
    uint32_t hits = 0;
#pragma unroll 1   // code this short stays ahead of the instruction cache
    for (int h = 0; h < kSortSteps && t + 64 * h < t1; h += kSortLoads) {
      int rows[kSortLoads];
#pragma unroll
      for (int u = 0; u < kSortLoads; ++u) {
        const int at = t + 64 * (h + u) + lane;
        rows[u] = at < t1 ? load_row<I64>(ids, at, vocab) : -1;
      }
#pragma unroll
      for (int u = 0; u < kSortLoads; ++u) {
        const int own = rows[u] & wmask;
        const bool mine = rows[u] >= 0 && own == b;
        below += __popcll(__ballot(rows[u] >= 0 && own < b));
        const uint64_t set = __ballot(mine);
        if (set) {
          const int l = mine ? rows[u] >> log_w : -1;
          hits |= 1u << (h + u);
          loc[w][h + u][lane] = (int16_t)l;
          if (count) {
            // many hits are mostly one frequent token: its lanes add up first
            const int first = __builtin_ctzll(set);
            const uint64_t same = __ballot(l == __builtin_amdgcn_readlane(l, first));
            if (lane == first || (mine && !((same >> lane) & 1)))
              atomicAdd(&cnt[w][l], lane == first ? __popcll(same) : 1);
          }
        }
      }
    }
    return hits;
  };
  uint32_t hits = 0;
  for (int t = t0; t < t1; t += 64 * kSortSteps) hits = load_steps(t, true);
  if (lane == 0) below_w[w] = below;
  __syncthreads();
  // thread r < range: row r's total over the strips, then its start
  const int r = threadIdx.x;
  int total = 0;
  if (r < range)
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) total += cnt[i][r];
  int incl = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) scan_w[w] = incl;
  __syncthreads();
  int start = incl - total;
#pragma unroll
  for (int i = 0; i < kSortWaves; ++i) {
    start += below_w[i];
    if (i < w) start += scan_w[i];
  }
  if (r < range) {
    const int v = (r << log_w) + b;
    if (has && v < vocab) has[v] = total > 0;
    if (b == wmask && r == range - 1) seen[0] = start + total;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
      const int n = cnt[i][r];
      cnt[i][r] = start;
      start += n;
    }
  }
  __syncthreads();
  // second look, in order (a strip that fits is still in LDS)
  int row = -1, place = 0;
  for (int t = t0; t < t1; t += 64 * kSortSteps) {
    if (strip > 64 * kSortSteps) hits = load_steps(t, false);
    uint32_t steps = hits;
    int next = steps ? loc[w][__builtin_ctz(steps)][lane] : -1;
    while (steps) {
      const int u = __builtin_ctz(steps), l = next;
      steps &= steps - 1;
      if (steps) next = loc[w][__builtin_ctz(steps)][lane];
      for (uint64_t open = __ballot(l >= 0); open;) {
        const int l0 = __builtin_amdgcn_readlane(l, __builtin_ctzll(open));
        const uint64_t same = __ballot(l == l0);
        open &= ~same;
        // the place of the row met last stays in a register: a frequent
        // token's next hit waits for nothing
        if (l0 != row) {
          if (row >= 0) cnt[w][row] = place;
          place = __builtin_amdgcn_readfirstlane(cnt[w][l0]);
          row = l0;
        }
        if (l == l0) {
          const uint32_t at = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, place));
          tokens[at] = Token{(l0 << log_w) + b, t + 64 * u + lane};
        }
        place += __popcll(same);
      }
    }
  }
}

// Adds f to (or puts it into) N values of the gradient table.
template <int GT, int N>
QL_DEV void putv(void* row, int i, int left, float (&f)[N], bool accumulate) {
  if (accumulate) {
    const Raw<GT, N> o = loadv<GT, N>(row, i, left);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] += el(o, j);
  }
  storev<GT, N, true>(row, i, left, f);
}

struct EmbedSum {
  const void* dY;
  int64_t lddy, ldde;
  void* dE;
  const Token* tokens;
  const int* seen;
  const uint8_t* has;   // a row has a token (NULL when accumulating)
  float* part;       // [chunks][2][d]: the chunk's first run's and last run's partial sums
  float scale;
  int m, d, fill, chunk, accumulate;   // fill: the rows zeroed here where they have no token
};

// Waves [0, sum_units) add up; the rest write the rows without a token.
template <int YT, int GT>
__global__ __launch_bounds__(256) void k_embed_sum(EmbedSum a, int64_t sum_units, int slices,
                                                   int fill_rows) {
  constexpr int EV = kVec, NV = kSumCols / (64 * EV);
  const int lane = threadIdx.x & 63;
  const int64_t unit =
      (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit < sum_units) {
    const int n = gptr(a.seen)[0];
    const int64_t ch = unit / slices;
    const int c0 = (int)(unit - ch * slices) * kSumCols + lane * EV;   // vector v: 64 EV v further on
    const int64_t i0 = ch * a.chunk;
    const int i1 = (int)min((int64_t)n, i0 + a.chunk);
    if (i0 >= n) return;
    // lane i holds the chunk's i-th token
    const int len = i1 - (int)i0;
    const Token mine = lane < len ? a.tokens[i0 + lane] : Token{-1, 0};
    const int before = i0 > 0 ? a.tokens[i0 - 1].row : -1;
    const int after = i1 < n ? a.tokens[i1].row : -1;
    int cur = __builtin_amdgcn_readlane(mine.row, 0);
    float acc[NV][EV];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < EV; ++j) acc[v][j] = 0.f;
    auto flush = [&](bool last) {
      const bool from = cur == before, to = last && cur == after;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = c0 + 64 * EV * v, left = a.d - c;
        if (left <= 0) continue;
#pragma unroll
        for (int j = 0; j < EV; ++j) acc[v][j] *= a.scale;
        if (from || to)
          storev<kElF32, EV>(row_of<kElF32>(a.part, ch * 2 + (from ? 0 : 1), a.d), c, left, acc[v]);
        else
          putv<GT, EV>(row_of<GT>(a.dE, cur, a.ldde), c, left, acc[v], a.accumulate);
#pragma unroll
        for (int j = 0; j < EV; ++j) acc[v][j] = 0.f;
      }
    };
    constexpr int U = 8;
    for (int i = 0; i < len; i += U) {
      Raw<YT, EV> r[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t p = __builtin_amdgcn_readlane(mine.pos, min(i + u, len - 1));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = c0 + 64 * EV * v;
          if (c < a.d) r[u][v] = loadv<YT, EV, true>(row_of<YT>(a.dY, p, a.lddy), c, a.d - c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u < len) {
          const int k = __builtin_amdgcn_readlane(mine.row, i + u);
          if (k != cur) {
            flush(false);
            cur = k;
          }
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < EV; ++j) acc[v][j] += el(r[u][v], j);
        }
      }
    }
    flush(true);
    return;
  }
  // rows [v0, v0 + fill_rows) of the fill, at most 64
  const int64_t v0 = (unit - sum_units) * fill_rows;
  if (v0 >= a.fill) return;
  uint64_t empty = __ballot(lane < fill_rows && v0 + lane < a.fill && !a.has[v0 + lane]);
  for (; empty; empty &= empty - 1)
    zero_row<GT>(row_of<GT>(a.dE, v0 + __builtin_ctzll(empty), a.ldde), a.d, lane);
}

constexpr int kJoinWaves = 4;

// The runs that cross chunks: the chunk where a run begins adds its own end
// and the first runs of the chunks that follow.  The waves take equal
// stretches of them, whose sums are joined in order.
template <int GT>
__global__ __launch_bounds__(64 * kJoinWaves) void k_embed_join(EmbedSum a) {
  __shared__ float s[kJoinWaves][8][64];
  const int64_t ch = blockIdx.x;
  const int64_t i0 = ch * a.chunk, i1 = i0 + a.chunk;
  if (i1 >= a.m) return;
  const int n = a.seen[0], v = a.tokens[i1 - 1].row, next = a.tokens[i1].row;
  const int first = a.tokens[i0].row, before = a.tokens[i0 > 0 ? i0 - 1 : 0].row;
  if (i1 >= n || next != v) return;                    // nothing crosses the chunk's end
  if (first == v && i0 > 0 && before == v) return;     // began in an earlier chunk
  // the chunks that begin inside the run
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t end = ch + 1;
  while (true) {
    const int64_t q = end + lane;
    const uint64_t more = __ballot(q * a.chunk < n && a.tokens[q * a.chunk].row == v);
    end += __popcll(more);
    if (more != ~0ull) break;
  }
  const int c = blockIdx.y * kSumCols + lane * 8, left = a.d - c;
  const int64_t per = (end - ch - 1 + kJoinWaves - 1) / kJoinWaves;
  const int64_t q0 = ch + 1 + w * per, q1 = min(end, q0 + per);
  float acc[8] = {};
  if (left > 0) {
    if (w == 0) {
      const Raw<kElF32, 8> t = loadv<kElF32, 8>(row_of<kElF32>(a.part, ch * 2 + 1, a.d), c, left);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = el(t, j);
    }
    constexpr int U = 8;
    for (int64_t q = q0; q < q1; q += U) {
      Raw<kElF32, 8> h[U];
#pragma unroll
      for (int u = 0; u < U; ++u) h[u] = loadv<kElF32, 8>(row_of<kElF32>(a.part, min(q + u, q1 - 1) * 2, a.d), c, left);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (q + u < q1)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += el(h[u], j);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) s[w][j][lane] = acc[j];
  __syncthreads();
  if (w != 0 || left <= 0) return;
  for (int i = 1; i < kJoinWaves; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += s[i][j][lane];
  putv<GT, 8>(row_of<GT>(a.dE, v, a.ldde), c, left, acc, a.accumulate);
}

template <int ET, int OT>
hipError_t fwd_ids(const void* E, int64_t vocab, int64_t d, int64_t lde, const void* ids, bool ids64,
                   int64_t m, float scale, void* out, int64_t ldo, hipStream_t s) {
  constexpr int EV = kVec;
  const uint32_t nvec = (uint32_t)((d + EV - 1) / EV);
  // a launch holds less than 2^32 threads: at most 2^31 vectors each
  const int64_t most = (int64_t(1) << 31) / nvec;
  for (int64_t r = 0; r < m; r += most) {
    const uint32_t total = (uint32_t)(std::min(most, m - r) * nvec);
    const unsigned wgs = (total + 256 * kFwdVecs<ET> - 1) / (256 * kFwdVecs<ET>);
    const char* id = (const char*)ids + r * (ids64 ? 8 : 4);
    char* o = (char*)out + r * ldo * kElBytes<OT>;
    if (ids64)
      k_embed_fwd<ET, OT, true><<<wgs, 256, 0, s>>>(E, (int)vocab, (int)d, lde, id, total, scale, o, ldo, nvec);
    else
      k_embed_fwd<ET, OT, false><<<wgs, 256, 0, s>>>(E, (int)vocab, (int)d, lde, id, total, scale, o, ldo, nvec);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int YT, int GT>
hipError_t bwd_types(const EmbedBwdPlan& p, EmbedSum a, const void* ids, bool ids64, int64_t vocab, char* ws,
                     hipStream_t s) {
  Token* tokens = (Token*)(ws + p.tokens_off);
  int* seen = (int*)(ws + p.seen_off);
  uint8_t* has = a.accumulate ? nullptr : (uint8_t*)(ws + p.has_off);
  if (ids64)
    k_embed_sort<true><<<1u << p.log_w, 64 * kSortWaves, 0, s>>>(ids, a.m, (int)vocab, p.range, p.log_w, tokens, seen, has);
  else
    k_embed_sort<false><<<1u << p.log_w, 64 * kSortWaves, 0, s>>>(ids, a.m, (int)vocab, p.range, p.log_w, tokens, seen, has);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.tokens = tokens;
  a.seen = seen;
  a.has = has;
  a.part = (float*)(ws + p.part_off);
  a.chunk = p.chunk;
  a.fill = a.accumulate ? 0 : (int)vocab;
  const int slices = (a.d + kSumCols - 1) / kSumCols;
  const int64_t units = p.chunks * slices;
  // fill units of about 32 KB
  const int rows = (int)std::max<int64_t>(1, std::min<int64_t>(64, 32768 / ((int64_t)a.d * kElBytes<GT>)));
  const int64_t fill = ((int64_t)a.fill + rows - 1) / rows;
  if (units + fill > 0)
    k_embed_sum<YT, GT><<<(unsigned)((units + fill + 3) / 4), 256, 0, s>>>(a, units, slices, rows);
  if (p.chunks > 1) k_embed_join<GT><<<dim3((unsigned)p.chunks, (unsigned)slices), 64 * kJoinWaves, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(const void* E, int e_dtype, int64_t vocab, int64_t d, int64_t lde,
                            const void* ids, bool ids64, int64_t m, float scale, void* out,
                            int out_dtype, int64_t ldo, hipStream_t s) {
#define QL_FWD(ET, OT) return fwd_ids<ET, OT>(E, vocab, d, lde, ids, ids64, m, scale, out, ldo, s)
  if (e_dtype == QLORA_F32) {
    if (out_dtype == QLORA_F32) QL_FWD(kElF32, kElF32);
    if (out_dtype == QLORA_BF16) QL_FWD(kElF32, kElBf16);
    QL_FWD(kElF32, kElF16);
  }
  if (e_dtype == QLORA_BF16) {
    if (out_dtype == QLORA_F32) QL_FWD(kElBf16, kElF32);
    QL_FWD(kElBf16, kElBf16);
  }
  if (out_dtype == QLORA_F32) QL_FWD(kElF16, kElF32);
  QL_FWD(kElF16, kElF16);
#undef QL_FWD
}

hipError_t launch_embed_bwd(const EmbedBwdPlan& p, const void* dY, int dy_dtype, int64_t m,
                            int64_t d, int64_t lddy, const void* ids, bool ids64, int64_t vocab,
                            float scale, void* dE, int de_dtype, int64_t ldde, bool accumulate,
                            void* ws, hipStream_t s) {
  EmbedSum a{};
  a.dY = dY;
  a.lddy = lddy;
  a.ldde = ldde;
  a.dE = dE;
  a.scale = scale;
  a.m = (int)m;
  a.d = (int)d;
  a.accumulate = accumulate;
  char* b = (char*)ws;
  if (dy_dtype == QLORA_F32) return bwd_types<kElF32, kElF32>(p, a, ids, ids64, vocab, b, s);
  if (dy_dtype == QLORA_BF16)
    return de_dtype == QLORA_F32 ? bwd_types<kElBf16, kElF32>(p, a, ids, ids64, vocab, b, s)
                                 : bwd_types<kElBf16, kElBf16>(p, a, ids, ids64, vocab, b, s);
  return de_dtype == QLORA_F32 ? bwd_types<kElF16, kElF32>(p, a, ids, ids64, vocab, b, s)
                               : bwd_types<kElF16, kElF16>(p, a, ids, ids64, vocab, b, s);
}

}  // namespace ql
