// Attention of the rows of a packed batch over the paged cache: chunks of prompts and single tokens
// side by side, under a sliding window with sinks.
//
// Mathematics: one pass over the visible keys, out = sum_j p_j v_j / sum_j p_j with p_j = exp2(l_j - m)
// and a running maximum m.  First form: a CTA per (row, query head), whose warps take every fourth
// group of 32 keys, a key a lane, and join at the end.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int chunk_attention_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kCaThreads = 128;
constexpr int kCaWarps = kCaThreads / 32;

struct ChunkArgs {
  Pool p;
  RowView q, out;
  float* lse;
  const int32_t *seqs, *start, *row_start;
  int layer, n, rows, Hq, rep, window, sinks;
  float scale;
};

template <int TYPE>
__device__ __forceinline__ float elem(const uint8_t* x, const uint8_t* meta, size_t row, int c) {
  if (TYPE == MIKV_PAGES_INT8) {
    const __half2 m = reinterpret_cast<const __half2*>(meta + row * kMetaBytes)[c / kGS];
    return __half2float(__float2half_rn(fmaf(__low2float(m), static_cast<float>(x[row * kD + c]), __high2float(m))));
  }
  const uint16_t h = reinterpret_cast<const uint16_t*>(x)[row * kD + c];
  return TYPE == MIKV_PAGES_BF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
}

template <int TYPE>
__global__ void __launch_bounds__(kCaThreads) chunk_rows_kernel(const ChunkArgs a) {
  __shared__ float s_q[kD], s_o[kCaWarps][kD], s_m[kCaWarps], s_l[kCaWarps];
  const int r = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int lo = 0, hi = a.n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.row_start[mid + 1] > r)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo >= a.n || a.row_start[lo] > r) return;
  const int first = max(a.row_start[lo], 0), count = min(a.row_start[lo + 1], a.rows) - first;
  const int32_t s = a.seqs ? a.seqs[lo] : lo;
  int64_t pos = -1;
  int32_t len = 0;
  if (static_cast<uint32_t>(s) < static_cast<uint32_t>(a.p.max_seqs)) {
    len = a.p.len_of(s);
    const int32_t from = a.start ? a.start[lo] : len - count;
    if (!a.start || from >= 0) pos = static_cast<int64_t>(from) + (r - first);
  }
  const int end = static_cast<int>(min(pos + 1, static_cast<int64_t>(len)));
  const uint16_t x = reinterpret_cast<const uint16_t*>(a.q.row(0, h, r))[tid];
  s_q[tid] = TYPE == MIKV_PAGES_BF16 ? __uint_as_float(static_cast<uint32_t>(x) << 16) : __half2float(__ushort_as_half(x));
  __syncthreads();
  const size_t layer0 = a.p.layer_rows() * a.layer;
  float m = -INFINITY, l = 0.f, o[4] = {};
  for (int j0 = w * 32; j0 < end; j0 += kCaThreads) {
    const int j = j0 + lane;
    const bool seen = j < end && (a.window == 0 || j > pos - a.window || j < a.sinks);
    uint32_t row = kNoRow;
    if (seen) {
      const uint32_t pg = div_of(j, a.p.ps);
      row = pool_row(a.p.table[static_cast<size_t>(s) * a.p.max_pages + pg], a.p.n_pages, a.p.Hkv, h / a.rep, a.p.ps.d, j - pg * a.p.ps.d);
      if (row == kNoRow) tc::report_giveup(tc::kBadPage);
    }
    float d = -INFINITY;
    if (row != kNoRow) {
      d = 0.f;
      for (int c = 0; c < kD; ++c) d += s_q[c] * elem<TYPE>(a.p.k, a.p.km, layer0 + row, c);
      d *= a.scale;
    }
    float mx = d;
#pragma unroll
    for (int e = 16; e; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float f = exp2f(m - mn), p = exp2f(d - mn);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] *= f;
    for (int e = 0; e < 32; ++e) {
      const uint32_t re = __shfl_sync(0xffffffffu, row, e);
      const float pe = __shfl_sync(0xffffffffu, p, e);
      if (re == kNoRow) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] += pe * elem<TYPE>(a.p.v, a.p.vm, layer0 + re, lane * 4 + c);
    }
  }
#pragma unroll
  for (int e = 16; e; e >>= 1) l += __shfl_xor_sync(0xffffffffu, l, e);
#pragma unroll
  for (int c = 0; c < 4; ++c) s_o[w][lane * 4 + c] = o[c];
  if (lane == 0) {
    s_m[w] = m;
    s_l[w] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, v = 0.f;
  for (int e = 0; e < kCaWarps; ++e) top = fmaxf(top, s_m[e]);
  if (top != -INFINITY)
    for (int e = 0; e < kCaWarps; ++e) {
      const float f = exp2f(s_m[e] - top);
      sum += s_l[e] * f;
      v += s_o[e][tid] * f;
    }
  v = sum > 0.f ? v / sum : 0.f;
  uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.row(0, h, r));
  dst[tid] = TYPE == MIKV_PAGES_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
  if (tid == 0 && a.lse)
    a.lse[static_cast<size_t>(r) * a.Hq + h] = sum > 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_chunk_attention_workspace_bytes(const mikv_pages* p, int n, int rows, int Hq) {
  Pool pool;
  if (check_pages(p, "chunk_attention", &pool) || n < 1 || n > 4096 || rows < 1 || Hq < 1 || Hq % p->Hkv) return 0;
  return 16;
}

extern "C" int mikv_chunk_attention(const mikv_rows* q, const mikv_pages* pages, int layer, const int32_t* seqs, const int32_t* start,
                                    const int32_t* row_start, int n, int rows, int Hq, int window, int sinks, const mikv_rows* out,
                                    float* lse, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  ChunkArgs a;
  if (int e = check_pages(pages, "chunk_attention", &a.p)) return e;
  if (layer < 0 || layer >= a.p.layers) return fail(MIKV_ESHAPE, "chunk_attention: layer=%d of %d", layer, a.p.layers);
  if (n < 0 || n > 4096 || rows < 0 || (!seqs && n > a.p.max_seqs)) return fail(MIKV_ESHAPE, "chunk_attention: n=%d rows=%d", n, rows);
  if (Hq < 1 || Hq % a.p.Hkv || Hq / a.p.Hkv > 1024) return fail(MIKV_ESHAPE, "chunk_attention: Hq=%d Hkv=%d", Hq, a.p.Hkv);
  if (window < 0 || sinks < 0) return fail(MIKV_EINVAL, "chunk_attention: window=%d sinks=%d", window, sinks);
  if (n == 0 || rows == 0) return MIKV_OK;
  if (int e = check_rows(q, "chunk_attention", "q")) return e;
  if (int e = check_rows(out, "chunk_attention", "out")) return e;
  const int64_t st = out->stride_t, sh = out->stride_h;   // rows apart: the heads of a row side by side, or the rows of a head
  if ((Hq == 1 || st < (Hq - 1) * sh + kD || sh < kD) && (rows == 1 || sh < (rows - 1) * st + kD || st < kD) &&
      !(Hq == 1 && (rows == 1 || st >= kD)) && !(rows == 1 && sh >= kD))
    return fail(MIKV_EINVAL, "chunk_attention: rows of out overlap");
  if (!row_start || !ws) return fail(MIKV_EINVAL, "chunk_attention: null pointer");
  if (reinterpret_cast<uintptr_t>(ws) & 31u) return fail(MIKV_EALIGN, "chunk_attention: workspace must be 32-byte aligned");
  const size_t need = mikv_chunk_attention_workspace_bytes(pages, n, rows, Hq);
  if (ws_bytes < need) return fail(MIKV_ESHAPE, "chunk_attention: workspace %zu < %zu", ws_bytes, need);
  a.q = row_view(*q);
  a.out = row_view(*out);
  a.lse = lse;
  a.seqs = seqs;
  a.start = start;
  a.row_start = row_start;
  a.layer = layer;
  a.n = n;
  a.rows = rows;
  a.Hq = Hq;
  a.rep = Hq / a.p.Hkv;
  a.window = window;
  a.sinks = sinks;
  a.scale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
  const auto kern = a.p.type == MIKV_PAGES_INT8   ? chunk_rows_kernel<MIKV_PAGES_INT8>
                    : a.p.type == MIKV_PAGES_BF16 ? chunk_rows_kernel<MIKV_PAGES_BF16>
                                                  : chunk_rows_kernel<MIKV_PAGES_FP16>;
  kern<<<dim3(rows, Hq), kCaThreads, 0, as_stream(stream)>>>(a);
  return check_launch("chunk_rows_kernel");
}
