// Rows into pages and back: append and gather of the paged cache.
//
// A CTA moves 64 tokens of one (sequence, key head): its first threads look their pages up,
// then every thread copies 16-byte pieces with several loads in flight.  Both operators are
// bound by HBM: each row is read and written once.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "quant_device.cuh"
#include "tcgen05.cuh"

namespace mikv {

int paged_rows_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 64;

// Pool rows of tokens slot0 .. slot0 + rows - 1 of sequence s, head h, into `at`.
__device__ __forceinline__ void find_rows(const Pool& p, int32_t s, int h, int slot0, int rows, uint32_t* at) {
  if (static_cast<int>(threadIdx.x) < kRowTokens) {
    uint32_t r = kNoRow;
    if (static_cast<int>(threadIdx.x) < rows) {
      const uint32_t slot = slot0 + threadIdx.x, q = div_of(slot, p.ps);
      r = pool_row(p.table[static_cast<size_t>(s) * p.max_pages + q], p.n_pages, p.Hkv, h, p.ps.d, slot - q * p.ps.d);
      if (r == kNoRow) tc::report_giveup(tc::kBadPage);
    }
    at[threadIdx.x] = r;
  }
  __syncthreads();
}

// CTA (chunk, head, row i): source tokens chunk * 64 .. of row i to slots start + t of its
// sequence.  Rows of a sequence that an earlier row of the call names are skipped.
template <bool Q8>
__global__ void __launch_bounds__(kRowThreads) paged_append_kernel(const Pool p, int layer, RowView k, RowView v, int T,
                                                                   const int32_t* __restrict__ seqs,
                                                                   const int32_t* __restrict__ start,
                                                                   const int32_t* __restrict__ counts) {
  __shared__ uint32_t at[kRowTokens];
  __shared__ int twice;
  const int i = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * kRowTokens;
  const int count = counts ? min(counts[i], T) : T;
  if (t0 >= count) return;
  const int32_t s = seqs ? seqs[i] : i;
  if (static_cast<uint32_t>(s) >= static_cast<uint32_t>(p.max_seqs)) return;
  const int len = p.len_of(s);
  const int first = start ? start[i] : len - count;
  if (first < 0) return;                                 // a refused reservation, or more tokens than slots
  if (threadIdx.x == 0) twice = 0;
  __syncthreads();
  if (seqs)
    for (int j = threadIdx.x; j < i; j += kRowThreads)
      if (seqs[j] == s) twice = 1;
  __syncthreads();
  if (twice) return;
  const int64_t slot0 = static_cast<int64_t>(first) + t0;
  const int rows = static_cast<int>(min(static_cast<int64_t>(min(kRowTokens, count - t0)), len - slot0));
  if (rows <= 0) return;                                 // slots past the sequence's length
  find_rows(p, s, h, static_cast<int>(slot0), rows, at);
  const size_t lrow = p.layer_rows() * layer;
  if (!Q8) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = threadIdx.x + u * kRowThreads, r = c >> 4;
      if (r < rows && at[r] != kNoRow) {
        a[u] = *reinterpret_cast<const uint4*>(k.row(i, h, t0 + r) + (c & 15) * 16);
        b[u] = *reinterpret_cast<const uint4*>(v.row(i, h, t0 + r) + (c & 15) * 16);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = threadIdx.x + u * kRowThreads, r = c >> 4;
      if (r < rows && at[r] != kNoRow) {
        const size_t off = (lrow + at[r]) * (kD * 2) + (c & 15) * 16;
        *reinterpret_cast<uint4*>(p.k + off) = a[u];
        *reinterpret_cast<uint4*>(p.v + off) = b[u];
      }
    }
  } else {
    // one warp per token, 4 channels a lane: the quantiser of the contiguous cache
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 2
    for (int r = w; r < rows; r += kRowThreads / 32) {
      if (at[r] == kNoRow) continue;  // uniform over the warp
      const Row4 xk = load_fp16x4(reinterpret_cast<const __half*>(k.row(i, h, t0 + r)) + lane * 4);
      const Row4 xv = load_fp16x4(reinterpret_cast<const __half*>(v.row(i, h, t0 + r)) + lane * 4);
      uint32_t mk, mv;
      const uint32_t ck = quantize4(xk, 8, mk), cv = quantize4(xv, 8, mv);
      const size_t row = lrow + at[r];
      store_codes(p.k + row * kD, lane, 8, ck);
      store_codes(p.v + row * kD, lane, 8, cv);
      store_meta(reinterpret_cast<__half2*>(p.km + row * kMetaBytes), lane, mk);
      store_meta(reinterpret_cast<__half2*>(p.vm + row * kMetaBytes), lane, mv);
    }
  }
}

// 8 codes to 8 fp16 values fp16(s * code + z), one fp32 rounding before the last.
__device__ __forceinline__ uint4 values_of(uint2 c, __half2 m) {
  const float s = __low2float(m), z = __high2float(m);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = (j < 2 ? c.x : c.y) >> (16 * (j & 1));
    const __half lo = __float2half_rn(__fadd_rn(__fmul_rn(s, static_cast<float>(x & 0xffu)), z));
    const __half hi = __float2half_rn(__fadd_rn(__fmul_rn(s, static_cast<float>((x >> 8) & 0xffu)), z));
    w[j] = pack_half2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// CTA (chunk, head, row i): slots chunk * 64 .. of row i's sequence, as far as it reaches, to
// rows of k and v.  Rows past the sequence's end keep what they hold.
template <bool Q8>
__global__ void __launch_bounds__(kRowThreads) paged_gather_kernel(const Pool p, int layer, RowView k, RowView v, int T,
                                                                   const int32_t* __restrict__ seqs) {
  __shared__ uint32_t at[kRowTokens];
  const int i = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * kRowTokens;
  const int32_t s = seqs ? seqs[i] : i;
  if (static_cast<uint32_t>(s) >= static_cast<uint32_t>(p.max_seqs)) return;
  const int rows = min(kRowTokens, min(p.len_of(s), T) - t0);
  if (rows <= 0) return;
  find_rows(p, s, h, t0, rows, at);
  const size_t lrow = p.layer_rows() * layer;
  uint4 a[4], b[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = threadIdx.x + u * kRowThreads, r = c >> 4, piece = c & 15;
    if (r >= rows || at[r] == kNoRow) {
      a[u] = b[u] = make_uint4(0, 0, 0, 0);  // a slot without a page reads as zeros
    } else if (!Q8) {
      const size_t off = (lrow + at[r]) * (kD * 2) + piece * 16;
      a[u] = *reinterpret_cast<const uint4*>(p.k + off);
      b[u] = *reinterpret_cast<const uint4*>(p.v + off);
    } else {
      const size_t row = lrow + at[r];
      const __half2* mk = reinterpret_cast<const __half2*>(p.km + row * kMetaBytes);
      const __half2* mv = reinterpret_cast<const __half2*>(p.vm + row * kMetaBytes);
      a[u] = values_of(*reinterpret_cast<const uint2*>(p.k + row * kD + piece * 8), mk[piece >> 3]);
      b[u] = values_of(*reinterpret_cast<const uint2*>(p.v + row * kD + piece * 8), mv[piece >> 3]);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = threadIdx.x + u * kRowThreads, r = c >> 4, piece = c & 15;
    if (r < rows) {
      *reinterpret_cast<uint4*>(k.row(i, h, t0 + r) + piece * 16) = a[u];
      *reinterpret_cast<uint4*>(v.row(i, h, t0 + r) + piece * 16) = b[u];
    }
  }
}

// What both calls check; MIKV_OK with *go false where there is nothing to do.
int check_move(const char* what, const mikv_pages* pages, int layer, const mikv_rows* k, const mikv_rows* v, int n, int T,
               const int32_t* seqs, Pool* p, bool* go) {
  *go = false;
  if (int e = check_pages(pages, what, p)) return e;
  if (layer < 0 || layer >= p->layers) return fail(MIKV_ESHAPE, "%s: layer=%d of %d", what, layer, p->layers);
  if (n < 0 || n > 65535 || T < 0 || (!seqs && n > p->max_seqs)) return fail(MIKV_ESHAPE, "%s: n=%d T=%d", what, n, T);
  if (n == 0 || T == 0) return MIKV_OK;
  if (int e = check_rows(k, what, "k")) return e;
  if (int e = check_rows(v, what, "v")) return e;
  *go = true;
  return MIKV_OK;
}
dim3 move_grid(const Pool& p, int n, int T) { return dim3((T + kRowTokens - 1) / kRowTokens, p.Hkv, n); }

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" int mikv_paged_append(const mikv_pages* pages, int layer, const mikv_rows* k, const mikv_rows* v, int n, int T,
                                 const int32_t* seqs, const int32_t* start, const int32_t* counts, void* stream) {
  clear_error();
  Pool p;
  bool go;
  if (int e = check_move("paged_append", pages, layer, k, v, n, T, seqs, &p, &go)) return e;
  if (!go) return MIKV_OK;
  const auto kern = p.type == MIKV_PAGES_INT8 ? paged_append_kernel<true> : paged_append_kernel<false>;
  kern<<<move_grid(p, n, T), kRowThreads, 0, as_stream(stream)>>>(p, layer, row_view(*k), row_view(*v), T, seqs, start, counts);
  return check_launch("paged_append_kernel");
}

extern "C" int mikv_paged_gather(const mikv_pages* pages, int layer, const int32_t* seqs, int n, int T, const mikv_rows* k_out,
                                 const mikv_rows* v_out, void* stream) {
  clear_error();
  Pool p;
  bool go;
  if (int e = check_move("paged_gather", pages, layer, k_out, v_out, n, T, seqs, &p, &go)) return e;
  if (!go) return MIKV_OK;
  const auto kern = p.type == MIKV_PAGES_INT8 ? paged_gather_kernel<true> : paged_gather_kernel<false>;
  kern<<<move_grid(p, n, T), kRowThreads, 0, as_stream(stream)>>>(p, layer, row_view(*k_out), row_view(*v_out), T, seqs);
  return check_launch("paged_gather_kernel");
}
