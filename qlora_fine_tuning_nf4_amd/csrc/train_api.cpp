// C ABI of the fine-tuning operators (include/qlora_train.h): argument checks,
// workspace layout, launches.  Everything is checked before the first HIP
// call; on error nothing is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "train_kernels.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up16(size_t b) { return (b + 15) & ~size_t(15); }

bool dtype_ok(int t) { return t == QLORA_F32 || t == QLORA_BF16 || t == QLORA_F16; }
size_t bytes_of(int t) { return t == QLORA_F32 ? 4 : 2; }
bool el_aligned(const void* p, int t) { return aligned(p, bytes_of(t)); }

// ---- embedding

bool embed_shape_ok(int64_t m, int64_t vocab, int64_t d) {
  return m >= 0 && m <= QLORA_EMBED_MAX_M && vocab >= 1 && vocab <= QLORA_EMBED_MAX_V && d >= 1 &&
         d <= QLORA_EMBED_MAX_D;
}

// Row strides: at least the row, and far enough below 2^63 bytes in all.
bool ld_ok(int64_t ld, int64_t d) { return ld >= d && ld < (int64_t(1) << 31); }

// ---- residual norm: what the two directions check alike

int check_norm(int64_t m, int64_t d, int act, int res, int param, bool branch, int pre, int gate,
               float eps, float scale, float offset) {
  if (m < 0 || m > QLORA_MAX_M || d < 1 || d > QLORA_RESNORM_MAX_D) return QLORA_ERR_SHAPE;
  if (!dtype_ok(act) || (res != QLORA_F32 && res != act) || (param != QLORA_F32 && param != act))
    return QLORA_ERR_DTYPE;
  if (!branch && !pre) return QLORA_ERR_ARG;
  if (branch && (gate < QLORA_GATE_NONE || gate > QLORA_GATE_FULL)) return QLORA_ERR_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(scale) || !std::isfinite(offset))
    return QLORA_ERR_ARG;
  return QLORA_OK;
}

// ---- AdamW

bool handle_ok(const qlora_adamw* p) {
  return p->count >= 1 && p->count <= QLORA_ADAMW_MAX_TENSORS && p->blocks >= 0 &&
         p->blocks < (int64_t(1) << 31) && p->chunks >= 0 && p->chunks <= p->blocks &&
         (p->state_bits == 8 || p->state_bits == 32) && dtype_ok(p->p_dtype) &&
         dtype_ok(p->g_dtype) && (p->copy_dtype == QLORA_F32 || dtype_ok(p->copy_dtype));
}

size_t map_off(int64_t count) { return ql::kOptHead + up16(sizeof(ql::OptEntry) * (size_t)count); }

bool plan_sizes(const int64_t* n, int count, size_t stride, int64_t* blocks, int64_t* chunks) {
  int64_t b = 0, c = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t ni = *reinterpret_cast<const int64_t*>(reinterpret_cast<const char*>(n) + stride * (size_t)i);
    if (ni < 0 || ni >= (int64_t(1) << 31) * QLORA_ADAMW_BLOCK) return false;
    b += cdiv(ni, QLORA_ADAMW_BLOCK);
    c += cdiv(ni, ql::kOptChunk);
    if (b >= (int64_t(1) << 31)) return false;
  }
  *blocks = b;
  *chunks = c;
  return true;
}

uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

bool finite_nonneg(double x) { return std::isfinite(x) && x >= 0; }

}  // namespace

namespace ql {

EmbedBwdPlan embed_bwd_plan(int64_t m, int64_t vocab, int64_t d) {
  EmbedBwdPlan p;
  // one workgroup a CU, more when its share would pass kEmbedRange rows
  p.log_w = 8;
  while (cdiv(vocab, int64_t(1) << p.log_w) > kEmbedRange) ++p.log_w;
  p.range = (int)cdiv(vocab, int64_t(1) << p.log_w);
  const int64_t slices = cdiv(d, kSumCols);
  // Tokens a wave of the sum takes: fewer in small calls, until there are a thousand waves' worth.
  // 32768 tokens x 256, 1000 rows: 39 us, with four thousand 50 (more partial sums to join); 32768 x
  // 4096 149, with sixteen thousand 159.  At least 8: 300 tokens x 1000 15 us, with at least 16 17;
  // 8192 x 512 25, with at least 4 28.
  int chunk = 64;
  while (chunk > 8 && cdiv(m, chunk) * slices < 1024) chunk /= 2;
  p.chunk = chunk;
  p.chunks = cdiv(m, chunk);
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  p.tokens_off = 0;
  p.seen_off = up(8 * (size_t)m);
  p.has_off = p.seen_off + 256;
  p.part_off = p.has_off + up((size_t)vocab);
  p.total = p.part_off + (p.chunks > 1 ? sizeof(float) * 2 * (size_t)p.chunks * (size_t)d : 0);
  return p;
}

ResnormBwdPlan resnorm_bwd_plan(int64_t m, int64_t d) {
  ResnormBwdPlan p;
  const bool wide = resnorm_wide(d);
  const int64_t side = wide ? 1 : kResnormBwdBlock / resnorm_threads(d);   // rows a workgroup holds at a time
  // wide rows: 4096 x 16384 328 us with 128, 370 with 256 (more column sums to join); rows under a
  // vector: 16384 x 5 96 us with 1024, 136 with 256 (one thread walks a part's rows)
  const int64_t most = d < 8 ? 1024 : wide ? 128 : 256;
  p.wgs = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(m, side), most));
  p.part_off = 0;
  p.stat_off = up16(sizeof(float) * (size_t)p.wgs * 2 * (size_t)d);
  p.total = p.stat_off + (wide ? 4 * sizeof(float) * (size_t)m : 0);
  return p;
}

}  // namespace ql

extern "C" {

int qlora_embed_fwd(const void* E, int e_dtype, int64_t vocab, int64_t d, int64_t lde,
                    const void* ids, int id_bits, int64_t m, float scale, void* out, int out_dtype,
                    int64_t ldo, void* stream) {
  if (!embed_shape_ok(m, vocab, d) || !ld_ok(lde, d) || !ld_ok(ldo, d)) return QLORA_ERR_SHAPE;
  if (!dtype_ok(e_dtype) || !dtype_ok(out_dtype)) return QLORA_ERR_DTYPE;
  if (out_dtype != e_dtype && out_dtype != QLORA_F32 && e_dtype != QLORA_F32) return QLORA_ERR_DTYPE;
  if (id_bits != 32 && id_bits != 64) return QLORA_ERR_ARG;
  if (m == 0) return QLORA_OK;
  if (!E || !ids || !out) return QLORA_ERR_NULL;
  if (!el_aligned(E, e_dtype) || !el_aligned(out, out_dtype) || !aligned(ids, id_bits / 8))
    return QLORA_ERR_ALIGN;
  if (ql::launch_embed_fwd(E, e_dtype, vocab, d, lde, ids, id_bits == 64, m, scale, out, out_dtype, ldo,
                           (hipStream_t)stream) != hipSuccess)
    return QLORA_ERR_HIP;
  return QLORA_OK;
}

size_t qlora_embed_workspace_bytes(int64_t m, int64_t vocab, int64_t d) {
  if (!embed_shape_ok(m, vocab, d)) return 0;
  return ql::embed_bwd_plan(m, vocab, d).total;
}

int qlora_embed_bwd(const void* dY, int dy_dtype, int64_t m, int64_t d, int64_t lddy,
                    const void* ids, int id_bits, int64_t vocab, float scale, void* dE,
                    int de_dtype, int64_t ldde, int accumulate, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!embed_shape_ok(m, vocab, d) || !ld_ok(lddy, d) || !ld_ok(ldde, d)) return QLORA_ERR_SHAPE;
  if (!dtype_ok(dy_dtype) || (de_dtype != QLORA_F32 && de_dtype != dy_dtype)) return QLORA_ERR_DTYPE;
  if (id_bits != 32 && id_bits != 64) return QLORA_ERR_ARG;
  if (!dE || (m > 0 && (!dY || !ids))) return QLORA_ERR_NULL;
  if (!el_aligned(dE, de_dtype) || (m > 0 && (!el_aligned(dY, dy_dtype) || !aligned(ids, id_bits / 8))))
    return QLORA_ERR_ALIGN;
  const ql::EmbedBwdPlan p = ql::embed_bwd_plan(m, vocab, d);
  if (!workspace || workspace_bytes < p.total) return QLORA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return QLORA_ERR_ALIGN;
  if (m == 0 && accumulate) return QLORA_OK;
  if (ql::launch_embed_bwd(p, dY, dy_dtype, m, d, lddy, ids, id_bits == 64, vocab, scale, dE, de_dtype,
                           ldde, accumulate != 0, workspace, (hipStream_t)stream) != hipSuccess)
    return QLORA_ERR_HIP;
  return QLORA_OK;
}

int qlora_resnorm_fwd(const qlora_resnorm* p, void* stream) {
  if (!p) return QLORA_ERR_NULL;
  qlora_resnorm a = *p;
  const bool branch = a.y != nullptr || a.m == 0;   // an empty y may have no address
  if (int e = check_norm(a.m, a.d, a.act_dtype, a.res_dtype, a.param_dtype, branch, a.pre, a.gate_kind,
                         a.eps, a.scale, a.w_offset))
    return e;
  if (a.m == 0) return QLORA_OK;
  if (!branch) a.post = a.gate_kind = 0;
  const int gate = a.gate_kind;
  if (!ld_ok(a.ldx, a.d) || (branch && (!ld_ok(a.ldy, a.d) || !ld_ok(a.ldh, a.d))) ||
      (a.pre && !ld_ok(a.ldz, a.d)) || (gate == QLORA_GATE_FULL && !ld_ok(a.ldg, a.d)))
    return QLORA_ERR_SHAPE;
  if (!a.x || (branch && !a.h) || (a.pre && !a.z) || (gate && !a.gate)) return QLORA_ERR_NULL;
  if (!el_aligned(a.x, a.res_dtype) || (branch && (!el_aligned(a.y, a.act_dtype) || !el_aligned(a.h, a.res_dtype))) ||
      (a.pre && (!el_aligned(a.z, a.act_dtype) || !el_aligned(a.w_pre, a.param_dtype))) ||
      (a.post && !el_aligned(a.w_post, a.param_dtype)) ||
      (gate && !el_aligned(a.gate, gate == QLORA_GATE_FULL ? a.act_dtype : a.param_dtype)))
    return QLORA_ERR_ALIGN;
  if (ql::launch_resnorm_fwd(a, (hipStream_t)stream) != hipSuccess) return QLORA_ERR_HIP;
  return QLORA_OK;
}

size_t qlora_resnorm_workspace_bytes(int64_t m, int64_t d) {
  if (m < 0 || m > QLORA_MAX_M || d < 1 || d > QLORA_RESNORM_MAX_D) return 0;
  return ql::resnorm_bwd_plan(m, d).total;
}

int qlora_resnorm_bwd(const qlora_resnorm_grad* p, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (!p) return QLORA_ERR_NULL;
  qlora_resnorm_grad a = *p;
  const bool branch = a.y != nullptr || a.m == 0;   // an empty y may have no address
  if (int e = check_norm(a.m, a.d, a.act_dtype, a.res_dtype, a.param_dtype, branch, a.pre, a.gate_kind,
                         a.eps, a.scale, a.w_offset))
    return e;
  // what the call does not compute
  if (!branch) {
    a.post = a.gate_kind = 0;
    a.dy = nullptr;
  }
  const int gate = a.gate_kind;
  if (!gate) a.dgate = nullptr;
  if (!a.post) a.dw_post = nullptr;
  if (!a.pre) {
    a.dz = nullptr;
    a.dw_pre = nullptr;
  }
  if (a.m == 0) {
    float* gc = gate == QLORA_GATE_CHANNEL ? (float*)a.dgate : nullptr;
    if (!aligned(a.dw_post, 4) || !aligned(a.dw_pre, 4) || !aligned(gc, 4)) return QLORA_ERR_ALIGN;
    if ((a.dw_post || a.dw_pre || gc) &&
        ql::launch_resnorm_zero(a.dw_post, a.dw_pre, gc, a.d, (hipStream_t)stream) != hipSuccess)
      return QLORA_ERR_HIP;
    return QLORA_OK;
  }
  if (!ld_ok(a.lddx, a.d) || (a.dz && !ld_ok(a.lddz, a.d)) || (a.dh && !ld_ok(a.lddh, a.d)) ||
      (a.dz && !ld_ok(a.ldh, a.d)) || (branch && !ld_ok(a.ldy, a.d)) || (a.dy && !ld_ok(a.lddy, a.d)) ||
      (gate == QLORA_GATE_FULL && (!ld_ok(a.ldg, a.d) || (a.dgate && !ld_ok(a.lddg, a.d)))))
    return QLORA_ERR_SHAPE;
  if (!a.dx || (a.pre && !a.dz) || (!a.pre && !a.dh) || (a.pre && !a.h) || (gate && !a.gate))
    return QLORA_ERR_NULL;
  if (!el_aligned(a.dx, a.res_dtype) || !el_aligned(a.dh, a.res_dtype) || !el_aligned(a.dz, a.act_dtype) ||
      !el_aligned(a.h, a.res_dtype) || !el_aligned(a.y, a.act_dtype) || !el_aligned(a.dy, a.act_dtype) ||
      !el_aligned(a.w_post, a.param_dtype) || !el_aligned(a.w_pre, a.param_dtype) ||
      !aligned(a.dw_post, 4) || !aligned(a.dw_pre, 4) ||
      (gate && !el_aligned(a.gate, gate == QLORA_GATE_FULL ? a.act_dtype : a.param_dtype)) ||
      !aligned(a.dgate, gate == QLORA_GATE_FULL ? bytes_of(a.act_dtype) : 4))
    return QLORA_ERR_ALIGN;
  const ql::ResnormBwdPlan w = ql::resnorm_bwd_plan(a.m, a.d);
  if (a.dw_post || a.dw_pre || (a.dgate && gate == QLORA_GATE_CHANNEL)) {
    if (!workspace || workspace_bytes < w.total) return QLORA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return QLORA_ERR_ALIGN;
  }
  if (ql::launch_resnorm_bwd(w, a, workspace, (hipStream_t)stream) != hipSuccess) return QLORA_ERR_HIP;
  return QLORA_OK;
}

size_t qlora_adamw_table_bytes(const int64_t* n, int count) {
  int64_t blocks = 0, chunks = 0;
  if (!n || count < 1 || count > QLORA_ADAMW_MAX_TENSORS ||
      !plan_sizes(n, count, sizeof(int64_t), &blocks, &chunks))
    return 0;
  return map_off(count) + up16(sizeof(ql::OptChunk) * (size_t)chunks);
}

int qlora_adamw_init(qlora_adamw* plan, const qlora_opt_tensor* tensors, int count, int p_dtype,
                     int g_dtype, int copy_dtype, int state_bits, void* table, size_t table_bytes) {
  if (!plan || !tensors || !table) return QLORA_ERR_NULL;
  if (count < 1 || count > QLORA_ADAMW_MAX_TENSORS) return QLORA_ERR_ARG;
  if (state_bits != 8 && state_bits != 32) return QLORA_ERR_ARG;
  if (!dtype_ok(p_dtype) || !dtype_ok(g_dtype)) return QLORA_ERR_DTYPE;
  if (!aligned(table, 16)) return QLORA_ERR_ALIGN;
  int64_t blocks = 0, chunks = 0;
  if (!plan_sizes(&tensors[0].n, count, sizeof(qlora_opt_tensor), &blocks, &chunks)) return QLORA_ERR_SHAPE;
  bool copies = false;
  for (int i = 0; i < count; ++i) {
    const qlora_opt_tensor& t = tensors[i];
    if (!std::isfinite(t.lr_mul) || !std::isfinite(t.wd_mul)) return QLORA_ERR_ARG;
    if (t.n > 0 && (!t.p || !t.g || !t.p_out)) return QLORA_ERR_NULL;
    if (!el_aligned(t.p, p_dtype) || !el_aligned(t.p_out, p_dtype) || !el_aligned(t.g, g_dtype) ||
        !aligned(t.copy, 2))
      return QLORA_ERR_ALIGN;
    copies = copies || t.copy;
  }
  if (copies && (p_dtype != QLORA_F32 || (copy_dtype != QLORA_BF16 && copy_dtype != QLORA_F16)))
    return QLORA_ERR_DTYPE;
  const size_t off = map_off(count), total = off + up16(sizeof(ql::OptChunk) * (size_t)chunks);
  if (table_bytes < total) return QLORA_ERR_WORKSPACE;
  char* host = new (std::nothrow) char[total]();
  if (!host) return QLORA_ERR_WORKSPACE;
  ql::OptEntry* e = reinterpret_cast<ql::OptEntry*>(host + ql::kOptHead);
  ql::OptChunk* c = reinterpret_cast<ql::OptChunk*>(host + off);
  int64_t b = 0;
  for (int i = 0; i < count; ++i) {
    const qlora_opt_tensor& t = tensors[i];
    e[i] = ql::OptEntry{t.p, t.g, t.p_out, t.copy, t.n, b, t.lr_mul, t.wd_mul, 0};
    b += cdiv(t.n, QLORA_ADAMW_BLOCK);
    for (int64_t j = 0; j < cdiv(t.n, ql::kOptChunk); ++j) *c++ = ql::OptChunk{i, (int32_t)j};
  }
  const hipError_t err = hipMemcpy(table, host, total, hipMemcpyHostToDevice);
  delete[] host;
  if (err != hipSuccess) return QLORA_ERR_HIP;
  *plan = qlora_adamw{table, count, p_dtype, g_dtype, copies ? copy_dtype : QLORA_F32, state_bits, blocks, chunks};
  return QLORA_OK;
}

size_t qlora_grad_norm_workspace_bytes(const qlora_adamw* plan) {
  return plan ? sizeof(float) * ql::kNormWgs : 0;
}

int qlora_grad_norm(const qlora_adamw* plan, float max_norm, float* out, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!plan || !out || !plan->table) return QLORA_ERR_NULL;
  if (!handle_ok(plan) || std::isnan(max_norm)) return QLORA_ERR_ARG;
  if (!workspace || workspace_bytes < sizeof(float) * ql::kNormWgs) return QLORA_ERR_WORKSPACE;
  if (!aligned(out, 4) || !aligned(workspace, 16)) return QLORA_ERR_ALIGN;
  char* t = (char*)plan->table;
  if (ql::launch_grad_norm((const ql::OptEntry*)(t + ql::kOptHead), (const ql::OptChunk*)(t + map_off(plan->count)),
                           plan->chunks, plan->g_dtype, max_norm, out, (float*)workspace,
                           (uint32_t*)t, (hipStream_t)stream) != hipSuccess)
    return QLORA_ERR_HIP;
  return QLORA_OK;
}

int qlora_adamw_step(const qlora_adamw* plan, const qlora_opt_state* in, const qlora_opt_state* out,
                     const qlora_adamw_hyper* h, const float* grad_scale, void* stream) {
  if (!plan || !in || !out || !h || !plan->table) return QLORA_ERR_NULL;
  if (!handle_ok(plan)) return QLORA_ERR_ARG;
  if (h->step < 1 || !(h->beta1 >= 0 && h->beta1 < 1) || !(h->beta2 >= 0 && h->beta2 < 1) ||
      !finite_nonneg(h->lr) || !finite_nonneg(h->eps) || !finite_nonneg(h->weight_decay))
    return QLORA_ERR_ARG;
  const bool s8 = plan->state_bits == 8;
  for (const qlora_opt_state* s : {in, out}) {
    if (plan->blocks == 0) break;
    if (!s->m || !s->v || (s8 && (!s->m_scale || !s->v_scale))) return QLORA_ERR_NULL;
    if (!aligned(s->m, s8 ? 4 : 16) || !aligned(s->v, s8 ? 4 : 16) ||
        (s8 && (!aligned(s->m_scale, 4) || !aligned(s->v_scale, 4))))
      return QLORA_ERR_ALIGN;
  }
  if (!aligned(grad_scale, 4)) return QLORA_ERR_ALIGN;
  const double bc1 = 1 - std::pow(h->beta1, (double)h->step), bc2 = 1 - std::pow(h->beta2, (double)h->step);
  ql::AdamwScalars k;
  k.b1 = (float)h->beta1;
  k.c1 = (float)(1 - h->beta1);
  k.b2 = (float)h->beta2;
  k.c2 = (float)(1 - h->beta2);
  k.lr = (float)h->lr;
  k.wd = (float)h->weight_decay;
  k.lr_bc1 = (float)(h->lr / bc1);
  k.rs_bc2 = (float)(1 / std::sqrt(bc2));
  k.eps = (float)h->eps;
  k.small_eps = k.eps < 0x1p-39f * k.rs_bc2;
  k.key = mix32(h->seed + 0x9E3779B9u * (uint32_t)h->step);
  const char* t = (const char*)plan->table;
  if (ql::launch_adamw((const ql::OptEntry*)(t + ql::kOptHead), (const ql::OptChunk*)(t + map_off(plan->count)), plan->chunks,
                       plan->p_dtype, plan->g_dtype, plan->copy_dtype, plan->state_bits, *in, *out, k,
                       grad_scale, (hipStream_t)stream) != hipSuccess)
    return QLORA_ERR_HIP;
  return QLORA_OK;
}

}  // extern "C"
