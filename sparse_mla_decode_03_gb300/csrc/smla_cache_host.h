// Checks of arguments that the paged-cache calls share, and the layout of their workspace.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/smla.h"
#include "smla_internal.h"

namespace smla {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline int check_cache(const smla_cache_params* c) {
  if (c == nullptr || c->num_pages < 1 || c->page_size < 1 || c->num_seqs < 1 || c->max_pages < 1)
    return SMLA_ERR_INVALID_ARG;
  if (!row_stride_ok(c->kv_row_stride)) return SMLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c->num_pages) * c->page_size > (int64_t{1} << 31) || c->num_seqs > 65535)
    return SMLA_ERR_UNSUPPORTED_SHAPE;
  return SMLA_OK;
}

inline bool ints_ok(const void* p) { return p != nullptr && aligned(p, 4); }
inline bool pool_ok(const void* p, const smla_cache_params* c) {
  return p != nullptr && aligned(p, is_row4(c->kv_row_stride) ? 16 : 8);
}

// Workspace: three lists of num_pages entries, one of num_seqs.
inline size_t list_bytes(const smla_cache_params* c) { return round256(size_t{4} * c->num_pages); }

inline int check_workspace(const smla_cache_params* c, const void* ws, size_t bytes) {
  if (ws == nullptr || !aligned(ws, 256)) return SMLA_ERR_INVALID_ARG;
  size_t need = 0;
  const int st = smla_cache_workspace_size(c, &need);
  if (st != SMLA_OK) return st;
  return bytes < need ? SMLA_ERR_WORKSPACE_TOO_SMALL : SMLA_OK;
}

// The device check and the status word; the last step before a launch.
inline int ready(int** status) {
  const int st = check_device();
  if (st != SMLA_OK) return st;
  return status_word_address(status) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

inline int done(cudaError_t e) { return e == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA; }

}  // namespace smla
