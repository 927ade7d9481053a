// Channel-wise bounds of the keys of a page, in 8 bits: what a block's score is made of.
//
// Mathematics: over the filled slots of a page, lo_c = min_j k_jc and hi_c = max_j k_jc; with
// s = fl(max_c max(|lo_c|, |hi_c|) / 127) they are held as floor(fl(lo_c / s)) and ceil(fl(hi_c / s)),
// so that s * code encloses every key (up to the rounding of the two divisions).  Bound by HBM and
// L2: each touched page's keys are read once (they were written a moment ago), 260 bytes are
// written a page and key head.  The page is read again as a whole rather than merged with the
// bounds that it had: a page that was given back, copied or cut down needs no case of its own.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int page_bounds_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kBoundThreads = 128;
constexpr int kBoundWarps = kBoundThreads / 32;
constexpr int kBoundRows = 8;     // packed rows of a CTA

// Four channels of a stored key, exactly (INT8: fl(s * code + z), s * code is exact).
template <int TYPE>
__device__ __forceinline__ void key4(const Pool& p, size_t row, int lane, float (&x)[4]) {
  if (TYPE == MIKV_PAGES_INT8) {
    const uint32_t c = reinterpret_cast<const uint32_t*>(p.k + row * kD)[lane];
    const __half2 m = reinterpret_cast<const __half2*>(p.km + row * kMetaBytes)[lane >> 4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf(__low2float(m), static_cast<float>((c >> (8 * e)) & 255u), __high2float(m));
  } else {
    const uint2 v = reinterpret_cast<const uint2*>(p.k + row * (kD * 2))[lane];
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (TYPE == MIKV_PAGES_BF16) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      } else {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[e]);
        x[2 * e] = __low2float(h);
        x[2 * e + 1] = __high2float(h);
      }
    }
  }
}

// CTA (rows, head): the pages that kBoundRows packed rows lie on, each once: by the first of the rows
// that follow one another on it.
template <int TYPE>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const Pool p, int layer, const int32_t* __restrict__ row_seq,
                                                                    const int32_t* __restrict__ row_pos, int rows,
                                                                    int8_t* __restrict__ bounds, float* __restrict__ scales) {
  __shared__ float4 s_lo[kBoundWarps][32], s_hi[kBoundWarps][32];
  __shared__ int s_bad[kBoundWarps];
  const int h = blockIdx.y, r0 = blockIdx.x * kBoundRows, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const size_t layer_row = p.layer_rows() * layer;
  // lane e of every warp looks at row r0 + e
  int32_t page = -1, fill = 0;
  if (lane < kBoundRows && r0 + lane < rows) {
    const int r = r0 + lane;
    const int32_t s = row_seq[r], at = row_pos[r];
    if (static_cast<uint32_t>(s) < static_cast<uint32_t>(p.max_seqs) && at >= 0) {
      const int32_t len = p.len_of(s);
      const uint32_t b = div_of(static_cast<uint32_t>(at), p.ps);
      const bool again = r > 0 && row_seq[r - 1] == s && row_pos[r - 1] >= 0 && div_of(static_cast<uint32_t>(row_pos[r - 1]), p.ps) == b;
      if (at < len && !again) {
        page = p.table[static_cast<size_t>(s) * p.max_pages + b];
        fill = min(static_cast<int32_t>(p.ps.d), len - static_cast<int32_t>(b * p.ps.d));
        if (!p.has(page)) {
          if (threadIdx.x < 32) tc::report_giveup(tc::kBadPage);
          page = -1;
        }
      }
    }
  }
  for (uint32_t live = __ballot_sync(0xffffffffu, page >= 0); live; live &= live - 1) {
    const int e = __ffs(live) - 1;
    const int32_t pg = __shfl_sync(0xffffffffu, page, e), n = __shfl_sync(0xffffffffu, fill, e);
    const size_t unit = static_cast<size_t>(layer) * p.n_pages * p.Hkv + static_cast<size_t>(pg) * p.Hkv + h;
    const size_t row0 = unit * p.ps.d;
    float lo[4], hi[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      lo[c] = INFINITY;
      hi[c] = -INFINITY;
    }
    bool bad = false;   // a key that is no finite number
#pragma unroll 4
    for (int j = w; j < n; j += kBoundWarps) {
      float x[4];
      key4<TYPE>(p, row0 + j, lane, x);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lo[c] = fminf(lo[c], x[c]);
        hi[c] = fmaxf(hi[c], x[c]);
        bad |= !(fabsf(x[c]) <= 3.402823466e38f);
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    __syncthreads();   // the last page's values have been read
    s_lo[w][lane] = make_float4(lo[0], lo[1], lo[2], lo[3]);
    s_hi[w][lane] = make_float4(hi[0], hi[1], hi[2], hi[3]);
    if (lane == 0) s_bad[w] = bad;
    __syncthreads();
    if (w > 0) continue;
    float top = 0.f;
#pragma unroll
    for (int k = 1; k < kBoundWarps; ++k) {
      const float4 a = s_lo[k][lane], b = s_hi[k][lane];
      lo[0] = fminf(lo[0], a.x), lo[1] = fminf(lo[1], a.y), lo[2] = fminf(lo[2], a.z), lo[3] = fminf(lo[3], a.w);
      hi[0] = fmaxf(hi[0], b.x), hi[1] = fmaxf(hi[1], b.y), hi[2] = fmaxf(hi[2], b.z), hi[3] = fmaxf(hi[3], b.w);
      bad |= s_bad[k] != 0;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) top = fmaxf(top, fmaxf(fabsf(lo[c]), fabsf(hi[c])));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = bad ? INFINITY : __fdiv_rn(top, 127.f);
    uint32_t cl = 0, ch = 0;
    if (!bad && scale > 0.f) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int a = static_cast<int>(fminf(fmaxf(floorf(__fdiv_rn(lo[c], scale)), -127.f), 127.f));
        const int b = static_cast<int>(fminf(fmaxf(ceilf(__fdiv_rn(hi[c], scale)), -127.f), 127.f));
        cl |= (static_cast<uint32_t>(a) & 255u) << (8 * c);
        ch |= (static_cast<uint32_t>(b) & 255u) << (8 * c);
      }
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(bounds + unit * (2 * kD));
    dst[lane] = cl;
    dst[kD / 4 + lane] = ch;
    if (lane == 0) scales[unit] = scale;
  }
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" int mikv_page_bounds(const mikv_pages* pages, int layer, const int32_t* row_seq, const int32_t* row_pos, int rows,
                                int8_t* bounds, float* scales, void* stream) {
  clear_error();
  Pool p;
  if (int e = check_pages(pages, "page_bounds", &p)) return e;
  if (layer < 0 || layer >= p.layers) return fail(MIKV_ESHAPE, "page_bounds: layer=%d of %d", layer, p.layers);
  if (rows < 0) return fail(MIKV_ESHAPE, "page_bounds: rows=%d", rows);
  if (rows == 0) return MIKV_OK;
  if (!row_seq || !row_pos || !bounds || !scales) return fail(MIKV_EINVAL, "page_bounds: null pointer");
  if (!aligned16(bounds)) return fail(MIKV_EALIGN, "page_bounds: bounds must be 16-byte aligned");
  const auto kern = p.type == MIKV_PAGES_INT8   ? page_bounds_kernel<MIKV_PAGES_INT8>
                    : p.type == MIKV_PAGES_BF16 ? page_bounds_kernel<MIKV_PAGES_BF16>
                                                : page_bounds_kernel<MIKV_PAGES_FP16>;
  kern<<<dim3((rows - 1) / kBoundRows + 1, p.Hkv), kBoundThreads, 0, as_stream(stream)>>>(p, layer, row_seq, row_pos, rows, bounds, scales);
  return check_launch("page_bounds_kernel");
}
