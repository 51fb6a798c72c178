// Host-only argument checks and host-side scalars of the C ABI.
#include "validate.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>

namespace zero {

int set_err(Err& e, int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(e.msg, sizeof e.msg, fmt, ap);
  va_end(ap);
  return status;
}

bool overlaps(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

static Range range_of(const void* p, int64_t bytes) {
  uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}

static bool mul_overflows(int64_t a, int64_t b) {
  return a != 0 && b > INT64_MAX / a;
}

int check_reduce_scatter(const void* const* rank_grads, const float* rank_weights,
                         int n_ranks, int64_t numel, float* const* shards_out, int n_shards,
                         int accumulate, Err& e, int elem_bytes) {
  if (!rank_grads || !rank_weights || !shards_out)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter: NULL pointer table or weights");
  if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter: n_ranks=%d outside [1,%d]", n_ranks, ZERO_MAX_RANKS);
  if (n_shards < 1 || n_shards > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter: n_shards=%d outside [1,%d]", n_shards, ZERO_MAX_RANKS);
  if (numel < 0) return set_err(e, ZERO_ERR_ARG, "reduce_scatter: numel=%lld < 0", (long long)numel);
  if (accumulate != 0 && accumulate != 1)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter: accumulate must be 0 or 1");
  if (numel % n_shards != 0)
    return set_err(e, ZERO_ERR_SIZE, "reduce_scatter: numel=%lld not divisible by n_shards=%d",
                   (long long)numel, n_shards);
  if (mul_overflows(numel, 4)) return set_err(e, ZERO_ERR_SIZE, "reduce_scatter: numel too large");
  const int64_t shard = numel / n_shards;
  // an empty reduction touches no buffer, so its pointers may be NULL (as
  // PyTorch's empty tensors are)
  if (numel == 0) return ZERO_OK;
  for (int r = 0; r < n_ranks; ++r) {
    if (!rank_grads[r]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter: rank_grads[%d] is NULL", r);
    if (reinterpret_cast<uintptr_t>(rank_grads[r]) & static_cast<uintptr_t>(elem_bytes - 1))
      return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter: rank_grads[%d] not %d-byte aligned", r, elem_bytes);
  }
  for (int k = 0; k < n_shards; ++k) {
    if (!shards_out[k]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter: shards_out[%d] is NULL", k);
    if (reinterpret_cast<uintptr_t>(shards_out[k]) & 3u)
      return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter: shards_out[%d] not 4-byte aligned", k);
  }
  for (int k = 0; k < n_shards; ++k) {
    Range ok = range_of(shards_out[k], shard * 4);
    for (int j = k + 1; j < n_shards; ++j)
      if (overlaps(ok, range_of(shards_out[j], shard * 4)))
        return set_err(e, ZERO_ERR_ARG, "reduce_scatter: shards_out[%d] and [%d] overlap", k, j);
    for (int r = 0; r < n_ranks; ++r)
      if (overlaps(ok, range_of(rank_grads[r], numel * elem_bytes)))
        return set_err(e, ZERO_ERR_ARG, "reduce_scatter: shards_out[%d] overlaps rank_grads[%d]", k, r);
  }
  return ZERO_OK;
}

int check_reduce_scatter_adam(const uint16_t* const* rank_grads, const float* rank_weights,
                              int n_ranks, int64_t numel, int n_shards, float* const* master,
                              float* const* exp_avg, float* const* exp_avg_sq,
                              uint16_t* const* bf16_out, const float* const* grad_acc,
                              float* const* grad_out, const zero_adam_hparams* hp, Err& e) {
  int st = check_adam_hparams(hp, e);
  if (st) return st;
  return check_reduce_scatter_adam_buffers(rank_grads, rank_weights, n_ranks, numel, n_shards, master,
                                           exp_avg, exp_avg_sq, bf16_out, grad_acc, grad_out, e);
}

int check_reduce_scatter_adam_dev(const uint16_t* const* rank_grads, const float* rank_weights,
                                  int n_ranks, int64_t numel, int n_shards, float* const* master,
                                  float* const* exp_avg, float* const* exp_avg_sq,
                                  uint16_t* const* bf16_out, const float* const* grad_acc,
                                  float* const* grad_out, const zero_adam_scalars* scalars_dev, Err& e) {
  int st = check_reduce_scatter_adam_buffers(rank_grads, rank_weights, n_ranks, numel, n_shards, master,
                                             exp_avg, exp_avg_sq, bf16_out, grad_acc, grad_out, e);
  if (st) return st;
  if (!scalars_dev) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: NULL device scalars");
  if (reinterpret_cast<uintptr_t>(scalars_dev) & 3u)
    return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_adam: device scalars not 4-byte aligned");
  if (numel == 0) return ZERO_OK;
  const int64_t shard = numel / n_shards;
  const Range sc = range_of(scalars_dev, sizeof(zero_adam_scalars));
  for (int k = 0; k < n_shards; ++k) {
    const Range outs[5] = {range_of(master[k], shard * 4), range_of(exp_avg[k], shard * 4),
                           range_of(exp_avg_sq[k], shard * 4), range_of(bf16_out[k], shard * 2),
                           range_of(grad_out ? grad_out[k] : nullptr, grad_out ? shard * 4 : 0)};
    for (const Range& r : outs)
      if (overlaps(sc, r))
        return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: device scalars overlap an output of owner %d", k);
  }
  return ZERO_OK;
}

int check_reduce_scatter_adam_buffers(const uint16_t* const* rank_grads, const float* rank_weights,
                                      int n_ranks, int64_t numel, int n_shards, float* const* master,
                                      float* const* exp_avg, float* const* exp_avg_sq,
                                      uint16_t* const* bf16_out, const float* const* grad_acc,
                                      float* const* grad_out, Err& e) {
  if (!rank_grads || !rank_weights || !master || !exp_avg || !exp_avg_sq || !bf16_out)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: NULL pointer table or weights");
  if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: n_ranks=%d outside [1,%d]", n_ranks, ZERO_MAX_RANKS);
  if (n_shards < 1 || n_shards > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: n_shards=%d outside [1,%d]", n_shards, ZERO_MAX_RANKS);
  if (numel < 0) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: numel < 0");
  if (numel % n_shards != 0)
    return set_err(e, ZERO_ERR_SIZE, "reduce_scatter_adam: numel=%lld not divisible by n_shards=%d",
                   (long long)numel, n_shards);
  if (mul_overflows(numel, 4)) return set_err(e, ZERO_ERR_SIZE, "reduce_scatter_adam: numel too large");
  if (numel == 0) return ZERO_OK;
  const int64_t shard = numel / n_shards;
  // outputs: per owner master, m, v, bf16 and (optionally) grad_out; inputs:
  // the rank contributions and the accumulators.  acc_of_out[i] / acc_of_in[j]
  // name the owner whose grad_out / grad_acc the range is (-1 otherwise).
  Range outs[ZERO_MAX_RANKS * 5], ins[ZERO_MAX_RANKS * 2];
  int out_owner[ZERO_MAX_RANKS * 5], in_owner[ZERO_MAX_RANKS * 2];
  int no = 0, ni = 0;
  for (int r = 0; r < n_ranks; ++r) {
    if (!rank_grads[r]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: rank_grads[%d] is NULL", r);
    if (reinterpret_cast<uintptr_t>(rank_grads[r]) & 1u)
      return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_adam: rank_grads[%d] not 2-byte aligned", r);
    in_owner[ni] = -1;
    ins[ni++] = range_of(rank_grads[r], numel * 2);
  }
  for (int k = 0; k < n_shards; ++k) {
    const void* f32s[3] = {master[k], exp_avg[k], exp_avg_sq[k]};
    for (const void* q : f32s) {
      if (!q) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: NULL state of owner %d", k);
      if (reinterpret_cast<uintptr_t>(q) & 3u)
        return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_adam: FP32 state of owner %d misaligned", k);
      out_owner[no] = -1;
      outs[no++] = range_of(q, shard * 4);
    }
    if (!bf16_out[k]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: bf16_out[%d] is NULL", k);
    if (reinterpret_cast<uintptr_t>(bf16_out[k]) & 1u)
      return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_adam: bf16_out[%d] misaligned", k);
    out_owner[no] = -1;
    outs[no++] = range_of(bf16_out[k], shard * 2);
    if (grad_out) {
      if (!grad_out[k]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: grad_out[%d] is NULL", k);
      if (reinterpret_cast<uintptr_t>(grad_out[k]) & 3u)
        return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_adam: grad_out[%d] misaligned", k);
      out_owner[no] = k;
      outs[no++] = range_of(grad_out[k], shard * 4);
    }
    if (grad_acc) {
      if (!grad_acc[k]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: grad_acc[%d] is NULL", k);
      if (reinterpret_cast<uintptr_t>(grad_acc[k]) & 3u)
        return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_adam: grad_acc[%d] misaligned", k);
      in_owner[ni] = k;
      ins[ni++] = range_of(grad_acc[k], shard * 4);
    }
  }
  for (int i = 0; i < no; ++i) {
    for (int j = i + 1; j < no; ++j)
      if (overlaps(outs[i], outs[j]))
        return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: two output buffers overlap");
    for (int j = 0; j < ni; ++j) {
      // the one permitted alias: grad_out[k] == grad_acc[k] exactly (each
      // element is read, then written, by the same lane)
      const bool in_place = out_owner[i] >= 0 && out_owner[i] == in_owner[j] &&
                            outs[i].lo == ins[j].lo && outs[i].hi == ins[j].hi;
      if (!in_place && overlaps(outs[i], ins[j]))
        return set_err(e, ZERO_ERR_ARG, "reduce_scatter_adam: an output overlaps an input");
    }
  }
  return ZERO_OK;
}

int check_grad_norm(const float* const* shards, int n_shards, int64_t shard_numel,
                    const double* workspace, int64_t workspace_len, const double* norm_sq_out,
                    float max_norm, const float* clip_coef_out, Err& e) {
  if (!shards || !workspace || !norm_sq_out)
    return set_err(e, ZERO_ERR_ARG, "grad_norm: NULL shard table, workspace or output");
  if (n_shards < 1 || n_shards > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "grad_norm: n_shards=%d outside [1,%d]", n_shards, ZERO_MAX_RANKS);
  if (shard_numel < 0) return set_err(e, ZERO_ERR_ARG, "grad_norm: shard_numel < 0");
  if (mul_overflows(shard_numel, 4)) return set_err(e, ZERO_ERR_SIZE, "grad_norm: shard_numel too large");
  if (workspace_len < static_cast<int64_t>(n_shards) * ZERO_NORM_BLOCKS)
    return set_err(e, ZERO_ERR_SIZE, "grad_norm: workspace needs n_shards*%d doubles", ZERO_NORM_BLOCKS);
  if (clip_coef_out && !(max_norm > 0.0f))
    return set_err(e, ZERO_ERR_ARG, "grad_norm: max_norm must be > 0 when a clip coefficient is requested");
  const uintptr_t a8 = reinterpret_cast<uintptr_t>(workspace) | reinterpret_cast<uintptr_t>(norm_sq_out);
  if (a8 & 7u) return set_err(e, ZERO_ERR_ALIGN, "grad_norm: workspace or output not 8-byte aligned");
  if (clip_coef_out && (reinterpret_cast<uintptr_t>(clip_coef_out) & 3u))
    return set_err(e, ZERO_ERR_ALIGN, "grad_norm: clip_coef_out not 4-byte aligned");
  Range outs[3] = {range_of(workspace, workspace_len * 8), range_of(norm_sq_out, 8),
                   range_of(clip_coef_out, clip_coef_out ? 4 : 0)};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(outs[i], outs[j])) return set_err(e, ZERO_ERR_ARG, "grad_norm: outputs overlap");
  for (int k = 0; k < n_shards; ++k) {
    if (shard_numel > 0 && !shards[k]) return set_err(e, ZERO_ERR_ARG, "grad_norm: shards[%d] is NULL", k);
    if (reinterpret_cast<uintptr_t>(shards[k]) & 3u)
      return set_err(e, ZERO_ERR_ALIGN, "grad_norm: shards[%d] not 4-byte aligned", k);
    for (int i = 0; i < 3; ++i)
      if (overlaps(outs[i], range_of(shards[k], shard_numel * 4)))
        return set_err(e, ZERO_ERR_ARG, "grad_norm: an output overlaps shards[%d]", k);
  }
  return ZERO_OK;
}

int check_adam_hparams(const zero_adam_hparams* hp, Err& e) {
  if (!hp) return set_err(e, ZERO_ERR_ARG, "adam: NULL hyper-parameters");
  if (hp->step < 1) return set_err(e, ZERO_ERR_ARG, "adam: step=%lld < 1", (long long)hp->step);
  if (!(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) || !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f))
    return set_err(e, ZERO_ERR_ARG, "adam: betas must lie in [0, 1)");
  return ZERO_OK;
}

int check_adam(const float* master, const float* exp_avg, const float* exp_avg_sq,
               const uint16_t* bf16_out, const float* grad, int64_t n,
               const zero_adam_hparams* hp, Err& e) {
  int st = check_adam_hparams(hp, e);
  if (st) return st;
  return check_adam_buffers(master, exp_avg, exp_avg_sq, bf16_out, grad, n, e);
}

int check_scalars_fetch(const zero_adam_scalars* ring_host, int ring_len, const uint32_t* cursor_dev,
                        const zero_adam_scalars* scalars_dev, Err& e) {
  if (!ring_host || !cursor_dev || !scalars_dev) return set_err(e, ZERO_ERR_ARG, "scalars_fetch: NULL pointer");
  if (ring_len < 1 || ring_len > (1 << 16) || (ring_len & (ring_len - 1)) != 0)
    return set_err(e, ZERO_ERR_ARG, "scalars_fetch: ring_len=%d is not a power of two in 1..65536", ring_len);
  if ((reinterpret_cast<uintptr_t>(ring_host) | reinterpret_cast<uintptr_t>(cursor_dev) |
       reinterpret_cast<uintptr_t>(scalars_dev)) & 3u)
    return set_err(e, ZERO_ERR_ALIGN, "scalars_fetch: pointers must be 4-byte aligned");
  const Range ring = range_of(ring_host, static_cast<int64_t>(ring_len) * sizeof(zero_adam_scalars));
  const Range cur = range_of(cursor_dev, sizeof(uint32_t));
  const Range out = range_of(scalars_dev, sizeof(zero_adam_scalars));
  if (overlaps(cur, out) || overlaps(ring, out) || overlaps(ring, cur))
    return set_err(e, ZERO_ERR_ARG, "scalars_fetch: ring, cursor and scalars must not overlap");
  return ZERO_OK;
}

int check_adam_dev(const float* master, const float* exp_avg, const float* exp_avg_sq,
                   const uint16_t* bf16_out, const float* grad, int64_t n,
                   const zero_adam_scalars* scalars_dev, Err& e) {
  int st = check_adam_buffers(master, exp_avg, exp_avg_sq, bf16_out, grad, n, e);
  if (st) return st;
  if (!scalars_dev) return set_err(e, ZERO_ERR_ARG, "adam: NULL device scalars");
  if (reinterpret_cast<uintptr_t>(scalars_dev) & 3u)
    return set_err(e, ZERO_ERR_ALIGN, "adam: device scalars not 4-byte aligned");
  if (n == 0) return ZERO_OK;
  const Range sc = range_of(scalars_dev, sizeof(zero_adam_scalars));
  const Range outs[4] = {range_of(master, n * 4), range_of(exp_avg, n * 4), range_of(exp_avg_sq, n * 4),
                         range_of(bf16_out, n * 2)};
  for (const Range& r : outs)
    if (overlaps(sc, r)) return set_err(e, ZERO_ERR_ARG, "adam: device scalars overlap a buffer the update writes");
  return ZERO_OK;
}

int check_adam_buffers(const float* master, const float* exp_avg, const float* exp_avg_sq,
                       const uint16_t* bf16_out, const float* grad, int64_t n, Err& e) {
  if (n < 0) return set_err(e, ZERO_ERR_ARG, "adam: n=%lld < 0", (long long)n);
  if (n == 0) return ZERO_OK;  // touches no buffer; NULL pointers allowed
  if (!master || !exp_avg || !exp_avg_sq || !bf16_out || !grad)
    return set_err(e, ZERO_ERR_ARG, "adam: NULL buffer");
  if (mul_overflows(n, 4)) return set_err(e, ZERO_ERR_SIZE, "adam: n too large");
  const void* f32s[4] = {master, exp_avg, exp_avg_sq, grad};
  for (const void* p : f32s)
    if (reinterpret_cast<uintptr_t>(p) & 3u)
      return set_err(e, ZERO_ERR_ALIGN, "adam: FP32 buffer not 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(bf16_out) & 1u)
    return set_err(e, ZERO_ERR_ALIGN, "adam: bf16_out not 2-byte aligned");
  Range rs[5] = {range_of(master, n * 4), range_of(exp_avg, n * 4), range_of(exp_avg_sq, n * 4),
                 range_of(grad, n * 4), range_of(bf16_out, n * 2)};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (overlaps(rs[i], rs[j])) return set_err(e, ZERO_ERR_ARG, "adam: buffers %d and %d overlap", i, j);
  return ZERO_OK;
}

int check_adam_scale(const float* grad_scale, const float* master, const float* exp_avg,
                     const float* exp_avg_sq, const uint16_t* bf16_out, int64_t n, Err& e) {
  if (!grad_scale) return set_err(e, ZERO_ERR_ARG, "adam: NULL grad_scale");
  if (reinterpret_cast<uintptr_t>(grad_scale) & 3u)
    return set_err(e, ZERO_ERR_ALIGN, "adam: grad_scale not 4-byte aligned");
  // every workgroup reads the scale while others write the state: it must not
  // lie inside a buffer the update writes
  const Range sc = range_of(grad_scale, 4);
  const Range outs[4] = {range_of(master, n * 4), range_of(exp_avg, n * 4), range_of(exp_avg_sq, n * 4),
                         range_of(bf16_out, n * 2)};
  for (const Range& r : outs)
    if (overlaps(sc, r)) return set_err(e, ZERO_ERR_ARG, "adam: grad_scale overlaps a buffer the update writes");
  return ZERO_OK;
}

int check_all_gather(const void* const* shards, int n_shards, int64_t shard_bytes,
                     const void* full_view, Err& e) {
  if (!shards) return set_err(e, ZERO_ERR_ARG, "all_gather: NULL shard table");
  if (n_shards < 1 || n_shards > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "all_gather: n_shards=%d outside [1,%d]", n_shards, ZERO_MAX_RANKS);
  if (shard_bytes < 0) return set_err(e, ZERO_ERR_ARG, "all_gather: shard_bytes < 0");
  if (shard_bytes == 0) return ZERO_OK;  // touches no buffer; NULL pointers allowed
  if (!full_view) return set_err(e, ZERO_ERR_ARG, "all_gather: NULL view");
  if (mul_overflows(shard_bytes, n_shards)) return set_err(e, ZERO_ERR_SIZE, "all_gather: size overflow");
  Range view = range_of(full_view, shard_bytes * n_shards);
  for (int k = 0; k < n_shards; ++k) {
    if (!shards[k]) return set_err(e, ZERO_ERR_ARG, "all_gather: shards[%d] is NULL", k);
    if (overlaps(view, range_of(shards[k], shard_bytes)))
      return set_err(e, ZERO_ERR_ARG, "all_gather: shards[%d] overlaps the view", k);
  }
  return ZERO_OK;
}

int check_offload_create(int n_ranks, int64_t shard_numel, int64_t chunk_numel,
                         const float* host_shard, uint16_t* const slot_contrib[2],
                         float* const slot_f32[2], Err& e) {
  if (!host_shard || !slot_contrib || !slot_f32 || !slot_contrib[0] || !slot_contrib[1] ||
      !slot_f32[0] || !slot_f32[1])
    return set_err(e, ZERO_ERR_ARG, "offload_create: NULL buffer");
  if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "offload_create: n_ranks=%d outside [1,%d]", n_ranks, ZERO_MAX_RANKS);
  if (shard_numel < 1 || chunk_numel < 1)
    return set_err(e, ZERO_ERR_ARG, "offload_create: sizes must be positive");
  if (mul_overflows(chunk_numel, 2 * (int64_t)n_ranks) || mul_overflows(shard_numel, 4))
    return set_err(e, ZERO_ERR_SIZE, "offload_create: size overflow");
  if ((shard_numel - 1) / chunk_numel + 1 > ZERO_OFFLOAD_MAX_CHUNKS)
    return set_err(e, ZERO_ERR_SIZE, "offload_create: more than %d chunks", ZERO_OFFLOAD_MAX_CHUNKS);
  for (int s = 0; s < 2; ++s) {
    if (reinterpret_cast<uintptr_t>(slot_contrib[s]) & 1u || reinterpret_cast<uintptr_t>(slot_f32[s]) & 3u)
      return set_err(e, ZERO_ERR_ALIGN, "offload_create: slot %d misaligned", s);
  }
  if (reinterpret_cast<uintptr_t>(host_shard) & 3u)
    return set_err(e, ZERO_ERR_ALIGN, "offload_create: host shard misaligned");
  Range rs[4] = {range_of(slot_contrib[0], chunk_numel * 2 * n_ranks),
                 range_of(slot_contrib[1], chunk_numel * 2 * n_ranks),
                 range_of(slot_f32[0], chunk_numel * 4), range_of(slot_f32[1], chunk_numel * 4)};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(rs[i], rs[j])) return set_err(e, ZERO_ERR_ARG, "offload_create: slots overlap");
  return ZERO_OK;
}

int adam_scalars(const zero_adam_hparams* hp, zero_adam_scalars* out, Err& e) {
  int st = check_adam_hparams(hp, e);
  if (st) return st;
  if (!out) return set_err(e, ZERO_ERR_ARG, "adam_scalars: NULL output");
  const float b1 = hp->beta1, b2 = hp->beta2;
  out->lr = hp->lr;
  out->beta1 = b1;
  out->beta2 = b2;
  out->one_minus_beta1 = 1.0f - b1;  // binary32 subtraction, exact for b1 in [1/2, 1]
  out->one_minus_beta2 = 1.0f - b2;
  out->bias_correction1 = static_cast<float>(1.0 - std::pow(static_cast<double>(b1), static_cast<double>(hp->step)));
  out->bias_correction2 = static_cast<float>(1.0 - std::pow(static_cast<double>(b2), static_cast<double>(hp->step)));
  out->eps = hp->eps;
  out->weight_decay = hp->weight_decay;
  return ZERO_OK;
}

int rank_weights(const int64_t* counts, int n_ranks, float* out, Err& e) {
  if (!out) return set_err(e, ZERO_ERR_ARG, "rank_weights: NULL output");
  if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "rank_weights: n_ranks=%d outside [1,%d]", n_ranks, ZERO_MAX_RANKS);
  if (!counts) {
    for (int r = 0; r < n_ranks; ++r) out[r] = static_cast<float>(1.0 / static_cast<double>(n_ranks));
    return ZERO_OK;
  }
  int64_t total = 0;
  for (int r = 0; r < n_ranks; ++r) {
    if (counts[r] < 0) return set_err(e, ZERO_ERR_ARG, "rank_weights: counts[%d] < 0", r);
    if (counts[r] > INT64_MAX - total) return set_err(e, ZERO_ERR_SIZE, "rank_weights: sum overflows");
    total += counts[r];
  }
  if (total == 0) return set_err(e, ZERO_ERR_ARG, "rank_weights: counts sum to 0");
  for (int r = 0; r < n_ranks; ++r)
    out[r] = static_cast<float>(static_cast<double>(counts[r]) / static_cast<double>(total));
  return ZERO_OK;
}

int shard_layout(const int64_t* numels, int n_tensors, int n_shards, int64_t* psi,
                 int64_t* psi_pad, int64_t* shard_numel, Err& e) {
  if (!psi || !psi_pad || !shard_numel || (n_tensors > 0 && !numels) || n_tensors < 0)
    return set_err(e, ZERO_ERR_ARG, "shard_layout: NULL pointer or negative n_tensors");
  if (n_shards < 1 || n_shards > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "shard_layout: n_shards=%d outside [1,%d]", n_shards, ZERO_MAX_RANKS);
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    if (numels[i] < 0) return set_err(e, ZERO_ERR_ARG, "shard_layout: numels[%d] < 0", i);
    if (numels[i] > INT64_MAX / 8 - total) return set_err(e, ZERO_ERR_SIZE, "shard_layout: overflow");
    total += numels[i];
  }
  const int64_t q = static_cast<int64_t>(n_shards) * 256;
  const int64_t pad = ((total + q - 1) / q) * q;
  *psi = total;
  *psi_pad = pad;
  *shard_numel = pad / n_shards;
  return ZERO_OK;
}

int check_muon_hparams(const zero_muon_hparams* hp, Err& e) {
  if (!hp) return set_err(e, ZERO_ERR_ARG, "muon: NULL hyper-parameters");
  if (!(hp->momentum >= 0.0f && hp->momentum < 1.0f))
    return set_err(e, ZERO_ERR_ARG, "muon: momentum must lie in [0, 1)");
  if (hp->nesterov != 0 && hp->nesterov != 1)
    return set_err(e, ZERO_ERR_ARG, "muon: nesterov must be 0 or 1");
  return ZERO_OK;
}

// An optional device float: 4-byte aligned and outside the written ranges
// (every workgroup reads it while others write).
static int check_device_float(const float* p, const char* name, const Range* outs, int n_outs, Err& e) {
  if (!p) return ZERO_OK;
  if (reinterpret_cast<uintptr_t>(p) & 3u) return set_err(e, ZERO_ERR_ALIGN, "muon: %s not 4-byte aligned", name);
  for (int i = 0; i < n_outs; ++i)
    if (overlaps(range_of(p, 4), outs[i]))
      return set_err(e, ZERO_ERR_ARG, "muon: %s overlaps a buffer the call writes", name);
  return ZERO_OK;
}

int check_muon_momentum(const float* momentum, const uint16_t* direction_out, const float* grad,
                        const float* grad_scale, int64_t n, const zero_muon_hparams* hp, Err& e) {
  int st = check_muon_hparams(hp, e);
  if (st) return st;
  if (n < 0) return set_err(e, ZERO_ERR_ARG, "muon: n=%lld < 0", (long long)n);
  if (n == 0) return ZERO_OK;  // touches no buffer; NULL pointers allowed
  if (!momentum || !direction_out || !grad) return set_err(e, ZERO_ERR_ARG, "muon: NULL buffer");
  if (mul_overflows(n, 4)) return set_err(e, ZERO_ERR_SIZE, "muon: n too large");
  if ((reinterpret_cast<uintptr_t>(momentum) | reinterpret_cast<uintptr_t>(grad)) & 3u)
    return set_err(e, ZERO_ERR_ALIGN, "muon: FP32 buffer not 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(direction_out) & 1u)
    return set_err(e, ZERO_ERR_ALIGN, "muon: direction_out not 2-byte aligned");
  const Range outs[2] = {range_of(momentum, n * 4), range_of(direction_out, n * 2)};
  const Range in = range_of(grad, n * 4);
  if (overlaps(outs[0], outs[1]) || overlaps(outs[0], in) || overlaps(outs[1], in))
    return set_err(e, ZERO_ERR_ARG, "muon: momentum, direction and gradient overlap");
  return check_device_float(grad_scale, "grad_scale", outs, 2, e);
}

int check_reduce_scatter_muon(const uint16_t* const* rank_grads, const float* rank_weights, int n_ranks,
                              int64_t numel, int n_shards, float* const* momentum,
                              uint16_t* const* direction_out, const float* const* grad_acc,
                              const zero_muon_hparams* hp, Err& e) {
  int st = check_muon_hparams(hp, e);
  if (st) return st;
  if (!rank_grads || !rank_weights || !momentum || !direction_out)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: NULL pointer table or weights");
  if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: n_ranks=%d outside [1,%d]", n_ranks, ZERO_MAX_RANKS);
  if (n_shards < 1 || n_shards > ZERO_MAX_RANKS)
    return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: n_shards=%d outside [1,%d]", n_shards, ZERO_MAX_RANKS);
  if (numel < 0) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: numel < 0");
  if (numel % n_shards != 0)
    return set_err(e, ZERO_ERR_SIZE, "reduce_scatter_muon: numel=%lld not divisible by n_shards=%d",
                   (long long)numel, n_shards);
  if (mul_overflows(numel, 4)) return set_err(e, ZERO_ERR_SIZE, "reduce_scatter_muon: numel too large");
  if (numel == 0) return ZERO_OK;
  const int64_t shard = numel / n_shards;
  Range outs[ZERO_MAX_RANKS * 2], ins[ZERO_MAX_RANKS * 2];
  int no = 0, ni = 0;
  for (int r = 0; r < n_ranks; ++r) {
    if (!rank_grads[r]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: rank_grads[%d] is NULL", r);
    if (reinterpret_cast<uintptr_t>(rank_grads[r]) & 1u)
      return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_muon: rank_grads[%d] not 2-byte aligned", r);
    ins[ni++] = range_of(rank_grads[r], numel * 2);
  }
  for (int k = 0; k < n_shards; ++k) {
    if (!momentum[k] || !direction_out[k])
      return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: NULL momentum or direction of owner %d", k);
    if (reinterpret_cast<uintptr_t>(momentum[k]) & 3u)
      return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_muon: momentum[%d] not 4-byte aligned", k);
    if (reinterpret_cast<uintptr_t>(direction_out[k]) & 1u)
      return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_muon: direction_out[%d] not 2-byte aligned", k);
    outs[no++] = range_of(momentum[k], shard * 4);
    outs[no++] = range_of(direction_out[k], shard * 2);
    if (grad_acc) {
      if (!grad_acc[k]) return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: grad_acc[%d] is NULL", k);
      if (reinterpret_cast<uintptr_t>(grad_acc[k]) & 3u)
        return set_err(e, ZERO_ERR_ALIGN, "reduce_scatter_muon: grad_acc[%d] not 4-byte aligned", k);
      ins[ni++] = range_of(grad_acc[k], shard * 4);
    }
  }
  for (int i = 0; i < no; ++i) {
    for (int j = i + 1; j < no; ++j)
      if (overlaps(outs[i], outs[j]))
        return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: two output buffers overlap");
    for (int j = 0; j < ni; ++j)
      if (overlaps(outs[i], ins[j]))
        return set_err(e, ZERO_ERR_ARG, "reduce_scatter_muon: an output overlaps an input");
  }
  return ZERO_OK;
}

int check_muon_shard(const float* master, const uint16_t* bf16_out, const uint16_t* update,
                     const float* lr_dev, int64_t n, const zero_muon_hparams* hp, Err& e) {
  int st = check_muon_hparams(hp, e);
  if (st) return st;
  if (n < 0) return set_err(e, ZERO_ERR_ARG, "muon: n=%lld < 0", (long long)n);
  if (n == 0) return ZERO_OK;  // touches no buffer; NULL pointers allowed
  if (!master || !bf16_out || !update) return set_err(e, ZERO_ERR_ARG, "muon: NULL buffer");
  if (mul_overflows(n, 4)) return set_err(e, ZERO_ERR_SIZE, "muon: n too large");
  if (reinterpret_cast<uintptr_t>(master) & 3u)
    return set_err(e, ZERO_ERR_ALIGN, "muon: master not 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(bf16_out) | reinterpret_cast<uintptr_t>(update)) & 1u)
    return set_err(e, ZERO_ERR_ALIGN, "muon: BF16 buffer not 2-byte aligned");
  const Range outs[2] = {range_of(master, n * 4), range_of(bf16_out, n * 2)};
  const Range in = range_of(update, n * 2);
  if (overlaps(outs[0], outs[1]) || overlaps(outs[0], in) || overlaps(outs[1], in))
    return set_err(e, ZERO_ERR_ARG, "muon: master, working weights and update overlap");
  return check_device_float(lr_dev, "lr_dev", outs, 2, e);
}

int check_ns_shape(int64_t n_mats, int64_t rows, int64_t cols, Err& e) {
  if (n_mats < 0 || rows < 0 || cols < 0) return set_err(e, ZERO_ERR_ARG, "newton_schulz: negative size");
  if (n_mats > ZERO_NS_MAX_MATS)
    return set_err(e, ZERO_ERR_SIZE, "newton_schulz: n_mats=%lld above %d", (long long)n_mats, ZERO_NS_MAX_MATS);
  if (rows > ZERO_NS_MAX_SIDE || cols > ZERO_NS_MAX_SIDE)
    return set_err(e, ZERO_ERR_SIZE, "newton_schulz: a side above %d", ZERO_NS_MAX_SIDE);
  // The workspace: per matrix three X and four k x k matrices padded to 64 and one X
  // padded to 256, two-byte values, and 4 KiB at most of sums and alignment; once, 256 rows.
  static_assert((ZERO_NS_MAX_SIDE + int64_t(256)) * (ZERO_NS_MAX_SIDE + int64_t(256)) * 16 + 4096 <
                    INT64_MAX / (ZERO_NS_MAX_MATS + int64_t(1)),
                "its bytes fit 64 bits within the limits");
  return ZERO_OK;
}

// The largest |p(s)| and |p(s)/s| of p(s) = a s + b s^3 + c s^5 over 0 <= s <= top.
static void ns_step_bound(double a, double b, double c, double top, double* p_max, double* r_max) {
  auto p = [&](double s) { return std::fabs(((c * s * s + b) * s * s + a) * s); };
  auto r = [&](double x) { return std::fabs((c * x + b) * x + a); };
  double pm = p(top), rm = std::fmax(r(0.0), r(top * top));
  if (c != 0.0) {
    const double x = -b / (2.0 * c);  // vertex of a + b x + c x^2, x = s^2
    if (x > 0.0 && x < top * top) rm = std::fmax(rm, r(x));
  }
  // stationary points: a + 3 b x + 5 c x^2 = 0, from the root that adds up: with c
  // next to 0 the other sum would lose the point near -a / 3b
  double x[2] = {-1.0, -1.0};
  const double d = 9.0 * b * b - 20.0 * a * c;
  if (d >= 0.0) {
    const double q = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));
    if (c != 0.0) x[0] = q / (5.0 * c);
    if (q != 0.0) x[1] = a / q;
  }
  for (double v : x)
    if (v > 0.0 && v < top * top) pm = std::fmax(pm, p(std::sqrt(v)));
  *p_max = pm;
  *r_max = rm;
}

// How far the steps raise roundings, in units of an operand's rounding (half a step,
// relative), over singular values that start at 2^-10 to 1:
//   value  a result's singular value, relative (at least to 1/8): each step's factor is
//          off by as much of |a| + 2 |b| s^2 + 3 |c| s^4 (C and, twice, A), and what
//          was there is taken on with the polynomial's slope;
//   turn   a result's singular vectors: the factor's diagonal, |a|, or of the first two
//          steps together |a a'|, is rounded entry by entry, against what the
//          factor makes of s;
//   rest   the directions of no singular value, where X's roundings lie, those of X
//          after two steps carried (see newton_schulz.hip): the sum over the later
//          X of the products of |a| that follow.
struct NsRaised {
  float value, turn, rest;
};

// In five steps the quintic 3.4445, -4.7750, 2.0315 raises roundings by (208, 24, 15),
// in six by (300, 28, 56); five steps that start at 4.1 to 2.8 s, by (86, 55, 11).  With
// one FP16 value (11 bits) per operand their results are at most 2.2e-2 off, over
// spectra of every kind.  Seven quintics, (504, 31, 197): 5e-2.  Five steps that are
// each the best for what the last one leaves, (663, 117, 10): 7e-2, and 2.5e-1 from
// FP32.  The limits lie between.  With pairs of FP16 values (22 bits) the latter come
// out within the result's rounding to BF16, for three times the products and their
// step by step form: 4096 x 4096 in seven steps 5.2 ms instead of 1.84, 32 of
// 512 x 1024 1.03 ms instead of 0.43.
constexpr float kNsPairsValue = 500.0f, kNsPairsTurn = 64.0f, kNsPairsRest = 60.0f;
// With 22 bits this much is 2^-6 of the result.  Sixteen quintics raise by 1.1e4; a set
// that takes singular values to where the next polynomial's slope is 10, and so on, by
// 2.9e5: there a single rounding decides whether the results grow.
constexpr float kNsMostRaised = 65536.0f;

// Singular values 2^(-10 i / 63).
struct NsSamples {
  static constexpr int kCount = 64;
  float s[kCount];
  constexpr NsSamples() : s() {
    double v = 1.0;
    for (int i = 0; i < kCount; ++i, v *= 0.895770256) s[i] = static_cast<float>(v);
  }
};

static NsRaised ns_raised(const float* coefs, int steps) {
  static constexpr NsSamples samples;
  constexpr int kSamples = NsSamples::kCount;
  float s[kSamples], first[kSamples], err[kSamples], turn[kSamples];   // floats: four at a time
  for (int i = 0; i < kSamples; ++i) {
    s[i] = first[i] = samples.s[i];
    err[i] = turn[i] = 0.0f;
  }
  NsRaised r = {0.0f, 0.0f, 0.0f};
  for (int t = 0; t < steps; ++t) {
    const float a = coefs[3 * t], b = coefs[3 * t + 1], c = coefs[3 * t + 2];
    const float fa = std::fabs(a), fb = 2.0f * std::fabs(b), fc = 3.0f * std::fabs(c);
    const bool pair = t == 0 && steps > 1;   // its factor is rounded with the next step's
    const float lead = t == 1 ? fa * std::fabs(coefs[0]) : fa;
    for (int i = 0; i < kSamples; ++i) {
      const float x = s[i] * s[i], from = t == 1 ? first[i] : s[i];
      const float next = std::fabs((a + (b + c * x) * x) * s[i]);
      err[i] = std::fabs(a + (3.0f * b + 5.0f * c * x) * x) * err[i] + (fa + (fb + fc * x) * x) * s[i];
      first[i] = s[i];
      s[i] = next;
      if (!pair) turn[i] += lead * from / (next > 0.0625f ? next : 0.0625f);
    }
    if (t >= 2) r.rest = t == 2 ? 0.0f : (r.rest + 1.0f) * fa;
  }
  for (int i = 0; i < kSamples; ++i) {
    const float rel = err[i] / (s[i] > 0.125f ? s[i] : 0.125f);
    if (!(rel <= r.value)) r.value = rel;
    if (!(turn[i] <= r.turn)) r.turn = turn[i];
  }
  return r;
}

int check_ns_coefs(const float* coefs, int steps, Err& e, bool* pairs) {
  if (!coefs) return set_err(e, ZERO_ERR_ARG, "newton_schulz: NULL coefficients");
  if (steps < 1 || steps > ZERO_NS_MAX_STEPS)
    return set_err(e, ZERO_ERR_ARG, "newton_schulz: steps=%d outside [1,%d]", steps, ZERO_NS_MAX_STEPS);
  // The singular values start in [0, 1].  The kernels hold X, A and C in FP16
  // with fixed power-of-two scales that leave room for singular values up to
  // ZERO_NS_MAX_SIGMA and a step's gain |p(s)/s| up to ZERO_NS_MAX_GAIN.
  double top = 1.0;
  for (int t = 0; t < steps; ++t) {
    const double a = coefs[3 * t], b = coefs[3 * t + 1], c = coefs[3 * t + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
      return set_err(e, ZERO_ERR_ARG, "newton_schulz: coefficients of step %d are not finite", t);
    double p_max, r_max;
    ns_step_bound(a, b, c, top, &p_max, &r_max);
    if (!(p_max <= ZERO_NS_MAX_SIGMA) || !(r_max <= ZERO_NS_MAX_GAIN))
      return set_err(e, ZERO_ERR_ARG, "newton_schulz: step %d takes singular values to %g with a gain of %g (limits %d and %d)",
                     t, p_max, r_max, ZERO_NS_MAX_SIGMA, ZERO_NS_MAX_GAIN);
    top = p_max;
  }
  const NsRaised r = ns_raised(coefs, steps);
  if (pairs) *pairs = r.value > kNsPairsValue || r.turn > kNsPairsTurn || r.rest > kNsPairsRest;
  if (!(r.value <= kNsMostRaised))
    return set_err(e, ZERO_ERR_ARG, "newton_schulz: the steps raise a rounding to %g of itself (limit %g): no room "
                   "between the values they reach and where they grow", r.value, kNsMostRaised);
  return ZERO_OK;
}

// Bytes from a matrix stack's first element to the end of its last.
static int64_t stack_bytes(int64_t mats, int64_t rows, int64_t cols, int64_t row_stride, int64_t mat_stride,
                           int64_t elem) {
  return ((mats - 1) * mat_stride + (rows - 1) * row_stride + cols) * elem;
}

// Whether two matrices share an element: matrices one after the other do not, nor,
// say, column ranges of one wider buffer.  Matrix i's first row starts i * mat_stride
// past that of matrix 0, whose rows start every row_stride >= cols and are cols long:
// only the last row at or before it and the next one can come close.
static bool matrices_meet(int64_t mats, int64_t rows, int64_t cols, int64_t row_stride, int64_t mat_stride) {
  if (mats == 1) return false;
  const int64_t last = (rows - 1) * row_stride;   // of matrix 0, its last row's start
  for (int64_t i = 1; i < mats; ++i) {
    const int64_t at = i * mat_stride;
    if (at >= last + cols) return false;          // and so are all that follow
    if (rows == 1) return true;
    const int64_t row = at / row_stride, past = at - row * row_stride;
    if (past < cols || (row + 1 < rows && row_stride - past < cols)) return true;
  }
  return false;
}

static int check_ns_strides(const char* name, int64_t mats, int64_t rows, int64_t cols, int64_t row_stride,
                            int64_t mat_stride, Err& e) {
  if (rows > 1 && row_stride < cols)
    return set_err(e, ZERO_ERR_SIZE, "newton_schulz: %s row stride %lld below cols", name, (long long)row_stride);
  if (row_stride < 0 || mat_stride < 0 || mul_overflows(rows, row_stride) ||
      mul_overflows(mats, mat_stride) || rows * row_stride > INT64_MAX / 16 - mats * mat_stride)
    return set_err(e, ZERO_ERR_SIZE, "newton_schulz: %s strides out of range", name);
  if (matrices_meet(mats, rows, cols, row_stride, mat_stride))
    return set_err(e, ZERO_ERR_SIZE, "newton_schulz: %s matrices overlap", name);
  return ZERO_OK;
}

int check_newton_schulz(const void* in, int in_dtype, int64_t in_row_stride, int64_t in_mat_stride,
                        const uint16_t* out, int64_t out_row_stride, int64_t out_mat_stride,
                        int64_t n_mats, int64_t rows, int64_t cols, const float* coefs, int steps,
                        float scale, const void* workspace, int64_t workspace_bytes,
                        int64_t workspace_need, Err& e, bool* pairs) {
  int st = check_ns_coefs(coefs, steps, e, pairs);
  if (st) return st;
  if (in_dtype != ZERO_BF16 && in_dtype != ZERO_FP32)
    return set_err(e, ZERO_ERR_ARG, "newton_schulz: in_dtype=%d is neither ZERO_BF16 nor ZERO_FP32", in_dtype);
  if (!std::isfinite(scale)) return set_err(e, ZERO_ERR_ARG, "newton_schulz: scale is not finite");
  st = check_ns_shape(n_mats, rows, cols, e);
  if (st) return st;
  if (n_mats == 0 || rows == 0 || cols == 0) return ZERO_OK;  // touches no buffer; NULL pointers allowed
  if (!in || !out || !workspace) return set_err(e, ZERO_ERR_ARG, "newton_schulz: NULL buffer");
  st = check_ns_strides("input", n_mats, rows, cols, in_row_stride, in_mat_stride, e);
  if (!st) st = check_ns_strides("output", n_mats, rows, cols, out_row_stride, out_mat_stride, e);
  if (st) return st;
  const int64_t esz = in_dtype == ZERO_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(in) & static_cast<uintptr_t>(esz - 1))
    return set_err(e, ZERO_ERR_ALIGN, "newton_schulz: input not %d-byte aligned", (int)esz);
  if (reinterpret_cast<uintptr_t>(out) & 1u)
    return set_err(e, ZERO_ERR_ALIGN, "newton_schulz: output not 2-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return set_err(e, ZERO_ERR_ALIGN, "newton_schulz: workspace not 256-byte aligned");
  if (workspace_bytes < workspace_need)
    return set_err(e, ZERO_ERR_SIZE, "newton_schulz: workspace of %lld bytes, %lld needed",
                   (long long)workspace_bytes, (long long)workspace_need);
  const Range ri = range_of(in, stack_bytes(n_mats, rows, cols, in_row_stride, in_mat_stride, esz));
  const Range ro = range_of(out, stack_bytes(n_mats, rows, cols, out_row_stride, out_mat_stride, 2));
  const Range rw = range_of(workspace, workspace_need);
  if (overlaps(ri, ro) || overlaps(ri, rw) || overlaps(ro, rw))
    return set_err(e, ZERO_ERR_ARG, "newton_schulz: input, output and workspace overlap");
  return ZERO_OK;
}

}  // namespace zero
