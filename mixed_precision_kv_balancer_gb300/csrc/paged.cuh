// The paged cache as the kernels see it, and its host-side checks (internal; not part of the C ABI).
#pragma once

#include "common.cuh"
#include "page_index.h"

namespace mikv {

struct Pool {
  uint8_t *k, *v;            // [layers][n_pages][Hkv][ps][row_bytes]
  uint8_t *km, *vm;          // INT8: [layers][n_pages][Hkv][ps][kMetaBytes], else null
  int32_t *table, *lens, *refs;
  int32_t layers, n_pages, Hkv, max_seqs, max_pages, cap, row_bytes, type;
  FastDiv ps;

  __host__ __device__ __forceinline__ size_t layer_rows() const {
    return static_cast<size_t>(n_pages) * Hkv * ps.d;
  }
  // The sequence's length, held inside what its table row can name.
  __device__ __forceinline__ int32_t len_of(int32_t seq) const { return min(max(lens[seq], 0), cap); }
  __device__ __forceinline__ bool has(int32_t page) const {
    return static_cast<uint32_t>(page) < static_cast<uint32_t>(n_pages);
  }
};

constexpr int kMetaBytes = kD / kGS * 4;  // fp16 (scale, zero) per group of a row

// Fills `out` from the C struct after checking it; `what` names the caller.
int check_pages(const mikv_pages* p, const char* what, Pool* out);
// Checks a strided view of [B][H][T][D] 16-bit rows.
int check_rows(const mikv_rows* r, const char* what, const char* name);

// Wait-status words of the files that read pages or wait on mbarriers.
int paged_attention_status(unsigned* out, bool clear);
int paged_rows_status(unsigned* out, bool clear);
int window_attention_status(unsigned* out, bool clear);

// A strided view with its data typed as bytes; strides in bytes.
struct RowView {
  uint8_t* p;
  int64_t sb, sh, st;
  __device__ __forceinline__ uint8_t* row(int b, int h, int64_t t) const { return p + b * sb + h * sh + t * st; }
};
inline RowView row_view(const mikv_rows& r) {
  return {static_cast<uint8_t*>(r.data), r.stride_b * 2, r.stride_h * 2, r.stride_t * 2};
}

}  // namespace mikv
