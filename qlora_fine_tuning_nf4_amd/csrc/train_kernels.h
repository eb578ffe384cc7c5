// Launchers of the fine-tuning operators (include/qlora_train.h), called by
// train_api.cpp after it has checked every argument.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/qlora_train.h"

namespace ql {

// ---- embedding (embed.hip)
hipError_t launch_embed_fwd(const void* E, int e_dtype, int64_t vocab, int64_t d, int64_t lde,
                            const void* ids, bool ids64, int64_t m, float scale, void* out,
                            int out_dtype, int64_t ldo, hipStream_t s);

// Sizes of the gradient's launches and the layout of its workspace.
struct EmbedBwdPlan {
  int log_w;            // 2^log_w workgroups of the sort: each owns every 2^log_w-th row,
  int range;            // this many at most (up to kEmbedRange)
  int chunk;            // sorted tokens a wave adds up
  int64_t chunks;       // ceil(m / chunk)
  size_t tokens_off, seen_off, has_off, part_off, total;   // byte offsets
};
constexpr int kEmbedRange = 512;
constexpr int kSumCols = 512;   // columns a wave of the sum holds
EmbedBwdPlan embed_bwd_plan(int64_t m, int64_t vocab, int64_t d);
hipError_t launch_embed_bwd(const EmbedBwdPlan& p, const void* dY, int dy_dtype, int64_t m,
                            int64_t d, int64_t lddy, const void* ids, bool ids64, int64_t vocab,
                            float scale, void* dE, int de_dtype, int64_t ldde, bool accumulate,
                            void* ws, hipStream_t s);

// ---- residual norm (norm.hip)
hipError_t launch_resnorm_fwd(const qlora_resnorm& a, hipStream_t s);
// Rows up to kResnormMaxInRow wide are held in registers, the backward's column
// sums too: its `wgs` workgroups leave 2 x d floats each.  Wider rows take four
// statistics a row and a second pass.
constexpr int64_t kResnormMaxInRow = 8192;
inline bool resnorm_wide(int64_t d) { return d > kResnormMaxInRow || d < 8; }
// Threads that hold a row of d values between them.
inline int resnorm_threads(int64_t d) {
  int g = 64;
  while (g < 512 && (int64_t)g * 16 < d) g *= 2;
  return g;
}
constexpr int resnorm_fwd_block(int g) { return g < 256 ? 256 : g; }   // threads of a workgroup
constexpr int kResnormBwdBlock = 512;
// Two workgroups a CU: the rows beyond are walked, their operands loaded ahead.
constexpr int kResnormFwdWgs = 512;
constexpr int kResnormWideWgs = 2048;
struct ResnormBwdPlan {
  int wgs;
  size_t part_off, stat_off, total;
};
ResnormBwdPlan resnorm_bwd_plan(int64_t m, int64_t d);
hipError_t launch_resnorm_bwd(const ResnormBwdPlan& p, const qlora_resnorm_grad& a, void* ws,
                              hipStream_t s);

// Zeros to up to three [d] outputs (NULL: none).
hipError_t launch_resnorm_zero(float* o0, float* o1, float* o2, int64_t d, hipStream_t s);

// ---- AdamW (adamw.hip)
struct OptEntry {          // one tensor, in the device table
  const void* p;
  const void* g;
  void* po;
  void* copy;
  int64_t n;
  int64_t block0;          // its first block of the state
  float lr_mul, wd_mul;
  int64_t pad;
};
struct OptChunk {          // kOptChunk consecutive values of one tensor
  int32_t tensor, index;
};
constexpr int64_t kOptChunk = 1024;
// The table: a 16-byte head (the count of k_grad_norm, zero between calls), the
// entries, the chunks.
constexpr size_t kOptHead = 16;
struct AdamwScalars {
  float b1, c1, b2, c2;    // beta, 1 - beta
  float lr, wd, lr_bc1, rs_bc2, eps;   // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  // The root and reciprocal instructions take subnormals for zero.  A subnormal v, whose root is
  // below 2^-63, may count as zero where eps is 2^24 times what that root adds to the
  // denominator; below that eps the update takes the full root and division (131M values with
  // 8-bit moments 380 us, otherwise 353).
  bool small_eps;
  uint32_t key;            // step key of the rounding bits
};
constexpr int kNormWgs = 256;   // most workgroups, and partial sums, of the gradient norm
hipError_t launch_grad_norm(const OptEntry* tab, const OptChunk* map, int64_t chunks, int g_dtype,
                            float max_norm, float* out, float* part, uint32_t* arrived, hipStream_t s);
hipError_t launch_adamw(const OptEntry* tab, const OptChunk* map, int64_t chunks, int p_dtype,
                        int g_dtype, int copy_dtype, int state_bits, const qlora_opt_state& in,
                        const qlora_opt_state& out, const AdamwScalars& k, const float* grad_scale,
                        hipStream_t s);

}  // namespace ql
