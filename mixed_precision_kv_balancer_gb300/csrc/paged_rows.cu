// Rows into pages and back: append and gather of the paged cache.
//
// A CTA moves 32 tokens of one (sequence, key head): its first warp looks their pages up, and
// every thread copies four 16-byte pieces of keys and of values, all requested before the first
// is written.  Both operators are bound by HBM: each row is read and written once.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int paged_rows_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kRowThreads = 128;
constexpr int kRowTokens = 32;

// Pool rows of tokens slot0 .. slot0 + rows - 1 of sequence s, head h, into `at`.  Rows to be written
// (WRITE) have none on a page that several sequences own: what the others read stays as it is (one more
// dependent read; a token for each of 64 sequences, in a graph: 2.1 -> 2.3 us).
template <bool WRITE>
__device__ __forceinline__ void find_rows(const Pool& p, int32_t s, int h, int slot0, int rows, uint32_t* at) {
  if (static_cast<int>(threadIdx.x) < kRowTokens) {
    uint32_t r = kNoRow;
    if (static_cast<int>(threadIdx.x) < rows) {
      const uint32_t slot = slot0 + threadIdx.x, q = div_of(slot, p.ps);
      const int32_t page = p.table[static_cast<size_t>(s) * p.max_pages + q];
      r = pool_row(page, p.n_pages, p.Hkv, h, p.ps.d, slot - q * p.ps.d);
      if (r == kNoRow) {
        tc::report_giveup(tc::kBadPage);
      } else if (WRITE && p.refs[page] > 1) {
        tc::report_giveup(tc::kSharedPage);
        r = kNoRow;
      }
    }
    at[threadIdx.x] = r;
  }
  __syncthreads();
}

// The smaller one, or NaN where one is no number (fminf gives the other).
__device__ __forceinline__ float min_or_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The quantiser of the contiguous cache at 8 bits on 8 fp16 channels a lane, 8 lanes a group, with
// its arithmetic: s = fp16(fl(fl(mx - mn) / 255)), z = fp16(mn), code = clamp(rint_even(fl(fl(x - z) / s))),
// 0 where the quotient is no number.  NaN does not count for mn and mx.
__device__ __forceinline__ uint2 quantize8(const uint4& x, uint32_t& meta) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = *reinterpret_cast<const __half2*>(&in[j]);
    f[2 * j] = __low2float(h);
    f[2 * j + 1] = __high2float(h);
  }
  float mn = f[0], mx = f[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    mn = fminf(mn, f[j]);
    mx = fmaxf(mx, f[j]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 255.f)), zh = __float2half_rn(mn);
  const float s = __half2float(sh), z = __half2float(zh);
  meta = pack_half2(sh, zh);
  uint32_t c[2] = {0, 0};
  if (s != 0.f) {
    // A product with the reciprocal is within 2^-13 of the quotient (at most 300 after the clamp),
    // so both round to the same code unless the product lies that near to a half: then, and for
    // what is no number, the division decides (its conversion gives 0).  1.5 * 2^23 added leaves rint in the last bits.
    const float r = __frcp_rn(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = __fsub_rn(f[j], z), t = min_or_nan(__fmul_rn(d, r), 300.f);
      const float big = __fadd_rn(t, 12582912.f);
      int q = __float_as_int(big) - 0x4B400000;
      if (!(fabsf(t - (big - 12582912.f)) < 0.49f)) q = __float2int_rn(__fdiv_rn(d, s));
      c[j >> 2] |= static_cast<uint32_t>(min(max(q, 0), 255)) << (8 * (j & 3));
    }
  }
  return make_uint2(c[0], c[1]);
}

// CTA (chunk, head, row i): source tokens chunk * 32 .. of row i to slots start + t of its
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
  // the source rows are requested before anything is looked up; piece c of a row: 16 bytes
  uint4 a[4], b[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = threadIdx.x + u * kRowThreads, r = c >> 4;
    a[u] = b[u] = make_uint4(0, 0, 0, 0);
    if (t0 + r < count) {
      a[u] = *reinterpret_cast<const uint4*>(k.row(i, h, t0 + r) + (c & 15) * 16);
      b[u] = *reinterpret_cast<const uint4*>(v.row(i, h, t0 + r) + (c & 15) * 16);
    }
  }
  const int32_t s = seqs ? seqs[i] : i;
  if (static_cast<uint32_t>(s) >= static_cast<uint32_t>(p.max_seqs)) return;
  const int len = p.len_of(s);
  const int first = start ? start[i] : len - count;
  if (first < 0) return;                                 // a refused reservation, or more tokens than slots
  if (seqs) {
    if (threadIdx.x == 0) twice = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < i; j += kRowThreads)
      if (seqs[j] == s) twice = 1;
    __syncthreads();
    if (twice) return;
  }
  const int64_t slot0 = static_cast<int64_t>(first) + t0;
  const int rows = static_cast<int>(min(static_cast<int64_t>(min(kRowTokens, count - t0)), len - slot0));
  if (rows <= 0) return;                                 // slots past the sequence's length
  find_rows<true>(p, s, h, static_cast<int>(slot0), rows, at);
  const size_t lrow = p.layer_rows() * layer;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = threadIdx.x + u * kRowThreads, r = c >> 4, piece = c & 15;
    const bool ok = r < rows && at[r] != kNoRow;
    const size_t row = lrow + (ok ? at[r] : 0);
    if (!Q8) {
      if (ok) {
        *reinterpret_cast<uint4*>(p.k + row * (kD * 2) + piece * 16) = a[u];
        *reinterpret_cast<uint4*>(p.v + row * (kD * 2) + piece * 16) = b[u];
      }
    } else {   // 16 lanes a row: all of a warp quantise
      uint32_t mk, mv;
      const uint2 ck = quantize8(a[u], mk), cv = quantize8(b[u], mv);
      if (ok) {
        *reinterpret_cast<uint2*>(p.k + row * kD + piece * 8) = ck;
        *reinterpret_cast<uint2*>(p.v + row * kD + piece * 8) = cv;
        if ((piece & 7) == 0) {
          reinterpret_cast<uint32_t*>(p.km + row * kMetaBytes)[piece >> 3] = mk;
          reinterpret_cast<uint32_t*>(p.vm + row * kMetaBytes)[piece >> 3] = mv;
        }
      }
    }
  }
}

// 8 codes to 8 fp16 values fp16(s * code + z), one fp32 rounding before the last (s * code is exact:
// 11 + 8 bits).  A code becomes fp32 as the last bits of 2^23 + code: two full-rate operations,
// where a conversion would take a quarter-rate one.
__device__ __forceinline__ uint4 values_of(uint2 c, __half2 m) {
  const float s = __low2float(m), z = __high2float(m);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      f[e] = fmaf(s, __uint_as_float(__byte_perm(j < 2 ? c.x : c.y, 0x4B000000u, 0x7440u + 2 * (j & 1) + e)) - 8388608.f, z);
    const __half2 h = __floats2half2_rn(f[0], f[1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// CTA (chunk, head, row i): slots chunk * 32 .. of row i's sequence, as far as it reaches, to
// rows of k and v.  Rows past the sequence's end keep what they hold.
template <bool Q8>
__global__ void __launch_bounds__(kRowThreads, 8) paged_gather_kernel(const Pool p, int layer, RowView k, RowView v, int T,
                                                                   const int32_t* __restrict__ seqs) {
  __shared__ uint32_t at[kRowTokens];
  const int i = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * kRowTokens;
  const int32_t s = seqs ? seqs[i] : i;
  if (static_cast<uint32_t>(s) >= static_cast<uint32_t>(p.max_seqs)) return;
  const int rows = min(kRowTokens, min(p.len_of(s), T) - t0);
  if (rows <= 0) return;
  find_rows<false>(p, s, h, t0, rows, at);
  const size_t lrow = p.layer_rows() * layer;
  uint4 a[4], b[4];
  bool ok[4];
  uint2 ca[4], cb[4];
  __half2 ma[4], mb[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {   // all requested before the first is used; without a page, row 0 of the layer
    const int c = threadIdx.x + u * kRowThreads, r = c >> 4, piece = c & 15;
    ok[u] = r < rows && at[r] != kNoRow;
    const size_t row = lrow + (ok[u] ? at[r] : 0);
    if (!Q8) {
      a[u] = *reinterpret_cast<const uint4*>(p.k + row * (kD * 2) + piece * 16);
      b[u] = *reinterpret_cast<const uint4*>(p.v + row * (kD * 2) + piece * 16);
    } else {
      ca[u] = *reinterpret_cast<const uint2*>(p.k + row * kD + piece * 8);
      cb[u] = *reinterpret_cast<const uint2*>(p.v + row * kD + piece * 8);
      ma[u] = reinterpret_cast<const __half2*>(p.km + row * kMetaBytes)[piece >> 3];
      mb[u] = reinterpret_cast<const __half2*>(p.vm + row * kMetaBytes)[piece >> 3];
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (Q8) {
      a[u] = values_of(ca[u], ma[u]);
      b[u] = values_of(cb[u], mb[u]);
    }
    if (!ok[u]) a[u] = b[u] = make_uint4(0, 0, 0, 0);  // a slot without a page reads as zeros
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
