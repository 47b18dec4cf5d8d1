// C ABI of AdamW over many tensors: the table of the tensors, checked on the host,
// and the launches.  Nothing here allocates or throws.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/lora.h"
#include "lora_kernels.h"

namespace {

using lora::AdamwTensor;
using lora::kAdamwBlock;
using lora::kAdamwChunk;
using lora::kAdamwTensorBytes;
static_assert(LORA_ADAMW_BLOCK == kAdamwBlock, "block");

// The smallest eps: the smallest normal number, whose reciprocal is finite.  8-bit second
// moments whose blocks are below 2^-100 become zeros, roots of up to 2^-50 that bias corrections
// of the first steps raise to 2^-45: nothing beside an eps of 2^-40, all there is beside a
// smaller one.
constexpr float kMinEps = 0x1p-126f, kMinEps8 = 0x1p-40f;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool valid_dtype(int32_t d) { return d == LORA_F32 || d == LORA_BF16; }

bool valid_sizes(const lora_adamw_tensor *t, int32_t n) {
  if (!t || n < 1 || n > LORA_ADAMW_MAX_TENSORS) return false;
  for (int32_t i = 0; i < n; ++i)
    if (t[i].numel < 0 || t[i].numel > LORA_ADAMW_MAX_NUMEL) return false;
  return true;
}
int64_t chunks_of(int64_t numel) { return (numel + kAdamwChunk - 1) / kAdamwChunk; }

// A range of bytes, with bit 0 of its (16-byte aligned) start set where it is written.
struct Range {
  uint64_t begin, end;
};

lora_status check_opt(const lora_adamw *o) {
  if (!o) return LORA_ERR_NULL;
  if (o->n_tensors < 1 || o->n_tensors > LORA_ADAMW_MAX_TENSORS) return LORA_ERR_SHAPE;
  if (!valid_dtype(o->param_dtype) || !valid_dtype(o->grad_dtype)) return LORA_ERR_DTYPE;
  if (o->state_bits != 8 && o->state_bits != 32) return LORA_ERR_DTYPE;
  if (o->masters && o->param_dtype != LORA_BF16) return LORA_ERR_SHAPE;
  if (o->state_numel < 0 || o->state_numel % kAdamwBlock) return LORA_ERR_SHAPE;
  if (o->table_bytes < o->n_tensors * kAdamwTensorBytes || o->table_bytes % 4) return LORA_ERR_SHAPE;
  if (!o->table || !o->step) return LORA_ERR_NULL;
  if (!aligned(o->table, 16) || !aligned(o->step, 4)) return LORA_ERR_ALIGN;
  if (o->state_numel > 0) {
    if (!o->m || !o->v || (o->state_bits == 8 && (!o->m_scale || !o->v_scale))) return LORA_ERR_NULL;
    if (!aligned(o->m, 16) || !aligned(o->v, 16) || !aligned(o->m_scale, 16) ||
        !aligned(o->v_scale, 16))
      return LORA_ERR_ALIGN;
  }
  return LORA_OK;
}

}  // namespace

extern "C" {

int64_t lora_adamw_state_numel(const lora_adamw_tensor *tensors, int32_t n_tensors) {
  if (!valid_sizes(tensors, n_tensors)) return -1;
  int64_t total = 0;
  for (int32_t i = 0; i < n_tensors; ++i)
    total += (tensors[i].numel + kAdamwBlock - 1) / kAdamwBlock * kAdamwBlock;
  return total;
}

int64_t lora_adamw_table_bytes(const lora_adamw_tensor *tensors, int32_t n_tensors) {
  if (!valid_sizes(tensors, n_tensors)) return -1;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n_tensors; ++i) chunks += chunks_of(tensors[i].numel);
  return n_tensors * kAdamwTensorBytes + chunks * 4;
}

lora_status lora_adamw_table(const lora_adamw_tensor *tensors, int32_t n_tensors,
                             int32_t param_dtype, int32_t grad_dtype, void *table) {
  if (!tensors || !table) return LORA_ERR_NULL;
  if (!valid_sizes(tensors, n_tensors)) return LORA_ERR_SHAPE;
  if (!valid_dtype(param_dtype) || !valid_dtype(grad_dtype)) return LORA_ERR_DTYPE;
  if (!aligned(table, 16)) return LORA_ERR_ALIGN;
  const int64_t pb = param_dtype == LORA_BF16 ? 2 : 4, gb = grad_dtype == LORA_BF16 ? 2 : 4;
  // what is written may overlap nothing (the ranges are sorted in the table's memory)
  Range *const r = static_cast<Range *>(table);
  static_assert(3 * sizeof(Range) <= kAdamwTensorBytes, "the ranges fit");
  int64_t nr = 0;
  bool with = false, without = false;
  auto add = [&](const void *p, int64_t bytes, bool written) {
    const uint64_t b = reinterpret_cast<uintptr_t>(p);
    r[nr++] = Range{b | (written ? 1u : 0u), b + (uint64_t)bytes};
  };
  for (int32_t i = 0; i < n_tensors; ++i) {
    const lora_adamw_tensor &t = tensors[i];
    if (t.numel == 0) continue;
    if (!t.param || !t.grad) return LORA_ERR_NULL;
    if (!aligned(t.param, 16) || !aligned(t.grad, 16) || !aligned(t.master, 16))
      return LORA_ERR_ALIGN;
    (t.master ? with : without) = true;
    add(t.param, t.numel * pb, true);
    add(t.grad, t.numel * gb, false);
    if (t.master) add(t.master, t.numel * 4, true);
  }
  if (with && (without || param_dtype != LORA_BF16)) return LORA_ERR_SHAPE;
  std::sort(r, r + nr, [](const Range &a, const Range &b) { return (a.begin & ~1ull) < (b.begin & ~1ull); });
  uint64_t end_written = 0, end_any = 0;
  for (int64_t i = 0; i < nr; ++i) {
    const uint64_t b = r[i].begin & ~1ull;
    const bool written = r[i].begin & 1u;
    if (b < end_written || (written && b < end_any)) return LORA_ERR_SHAPE;
    end_any = std::max(end_any, r[i].end);
    if (written) end_written = std::max(end_written, r[i].end);
  }
  AdamwTensor *const out = static_cast<AdamwTensor *>(table);
  int32_t *const map = reinterpret_cast<int32_t *>(out + n_tensors);
  int64_t start = 0, chunk = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const lora_adamw_tensor &t = tensors[i];
    out[i] = AdamwTensor{t.param, t.grad, t.master, t.numel, start, chunk};
    start += (t.numel + kAdamwBlock - 1) / kAdamwBlock * kAdamwBlock;
    for (int64_t c = chunks_of(t.numel); c > 0; --c) map[chunk++] = i;
  }
  return LORA_OK;
}

lora_status lora_adamw_step(const lora_adamw *opt, double lr, const float *lr_dev, double beta1,
                            double beta2, double eps, double weight_decay,
                            const float *grad_scale, const int32_t *active, uint32_t seed,
                            void *stream) {
  const lora_status st = check_opt(opt);
  if (st != LORA_OK) return st;
  // (comparisons that a NaN fails)
  if (!std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
      !((float)eps >= (opt->state_bits == 8 ? kMinEps8 : kMinEps) && std::isfinite((float)eps)) ||
      !(weight_decay >= 0.0 && std::isfinite(weight_decay)))
    return LORA_ERR_SHAPE;
  if (!aligned(lr_dev, 4) || !aligned(grad_scale, 4) || !aligned(active, 4)) return LORA_ERR_ALIGN;
  lora::AdamwArgs a{};
  a.n_tensors = opt->n_tensors;
  a.param_dtype = opt->param_dtype;
  a.grad_dtype = opt->grad_dtype;
  a.bits = opt->state_bits;
  a.master = opt->masters != 0;
  a.n_chunks = (opt->table_bytes - opt->n_tensors * kAdamwTensorBytes) / 4;
  a.tensors = static_cast<const AdamwTensor *>(opt->table);
  a.chunk_tensor = reinterpret_cast<const int32_t *>(a.tensors + opt->n_tensors);
  a.m = opt->m;
  a.v = opt->v;
  a.m_scale = opt->m_scale;
  a.v_scale = opt->v_scale;
  a.step = opt->step;
  a.active = active;
  a.lr_dev = lr_dev;
  a.grad_scale = grad_scale;
  a.lr = lr;
  a.beta1 = beta1;
  a.beta2 = beta2;
  a.weight_decay = weight_decay;
  a.eps = (float)eps;
  a.seed = seed;
  return lora::launch_adamw(a, static_cast<hipStream_t>(stream)) == hipSuccess ? LORA_OK
                                                                               : LORA_ERR_HIP;
}

lora_status lora_adamw_read(const lora_adamw *opt, int32_t dtype, void *m_out, void *v_out,
                            void *stream) {
  const lora_status st = check_opt(opt);
  if (st != LORA_OK) return st;
  if (opt->state_bits != 8 || !valid_dtype(dtype)) return LORA_ERR_DTYPE;
  if (opt->state_numel == 0) return LORA_OK;
  if (!m_out || !v_out) return LORA_ERR_NULL;
  if (!aligned(m_out, 16) || !aligned(v_out, 16)) return LORA_ERR_ALIGN;
  return lora::launch_adamw_read(opt->m, opt->v, opt->m_scale, opt->v_scale, opt->state_numel,
                                 dtype, m_out, v_out,
                                 static_cast<hipStream_t>(stream)) == hipSuccess
             ? LORA_OK
             : LORA_ERR_HIP;
}

}  // extern "C"
