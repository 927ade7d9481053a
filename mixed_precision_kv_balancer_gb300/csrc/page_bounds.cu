// Channel-wise bounds of the keys of a page, in 8 bits: what a block's score is made of.
//
// Mathematics: over the filled slots of a page, lo_c = min_j k_jc and hi_c = max_j k_jc; with
// s = fl(max_c max(|lo_c|, |hi_c|) / 127) they are held as floor(fl(lo_c / s)) and ceil(fl(hi_c / s)),
// so that s * code encloses every key (up to the rounding of the two divisions).  Bound by HBM and
// L2: each touched page's keys are read once (they were written a moment ago), 260 bytes are
// written a page and key head.  The page is read again as a whole rather than merged with the
// bounds that it had: a page that was given back, copied or cut down needs no case of its own.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int page_bounds_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kBoundThreads = 256;
constexpr int kBoundWarps = kBoundThreads / 32;
constexpr int kWarpRows = 128;     // a page of more rows is shared by the CTA's warps

// The smaller and larger values of pairs; what is no number stays.
template <bool BF>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t y;
  if (BF)
    asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
template <bool BF>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t y;
  if (BF)
    asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A lane's bounds: 8 channels of every second row (16-bit types: pairs, exactly as stored), or 16 of every fourth (INT8).
template <int TYPE>
struct Bounds {
  static constexpr bool q8 = TYPE == MIKV_PAGES_INT8, bf = TYPE == MIKV_PAGES_BF16;
  static constexpr int lanes = q8 ? 8 : 16, at_once = 32 / lanes, channels = kD / lanes, batch = q8 ? 4 : 8;
  float lo[channels], hi[channels];

  // Rows j, j + step, ... below n of the page whose rows begin at `row0`, `batch` of them requested together.
  __device__ __forceinline__ void rows(const Pool& p, size_t row0, int j, int step, int n) {
    const int piece = (threadIdx.x & 31) % lanes;
    if (q8) {
#pragma unroll
      for (int c = 0; c < channels; ++c) {
        lo[c] = INFINITY;
        hi[c] = -INFINITY;
      }
      for (; j < n; j += batch * step) {
        uint4 x[batch];
        __half2 m[batch];
#pragma unroll
        for (int e = 0; e < batch; ++e) {
          const size_t row = row0 + (j + e * step < n ? j + e * step : j);   // (a row again changes nothing)
          x[e] = reinterpret_cast<const uint4*>(p.k + row * kD)[piece];
          m[e] = reinterpret_cast<const __half2*>(p.km + row * kMetaBytes)[piece >> 2];
        }
#pragma unroll
        for (int e = 0; e < batch; ++e) {
          const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
          const float s = __low2float(m[e]), z = __high2float(m[e]);
#pragma unroll
          for (int c = 0; c < channels; ++c) {   // fl(s * code + z): s * code is exact; a code as the last bits of 2^23 + code
            const float v = fmaf(s, __uint_as_float(__byte_perm(w[(c >> 2) & 3], 0x4B000000u, 0x7440u + (c & 3))) - 8388608.f, z);
            lo[c] = min_nan(lo[c], v);
            hi[c] = max_nan(hi[c], v);
          }
        }
      }
    } else {
      constexpr uint32_t kInf = bf ? 0x7f807f80u : 0x7c007c00u, kNegInf = kInf | 0x80008000u;
      uint32_t l[4], h[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        l[c] = kInf;
        h[c] = kNegInf;
      }
      for (; j < n; j += batch * step) {
        uint4 x[batch];
#pragma unroll
        for (int e = 0; e < batch; ++e) x[e] = reinterpret_cast<const uint4*>(p.k + (row0 + (j + e * step < n ? j + e * step : j)) * (kD * 2))[piece];
#pragma unroll
        for (int e = 0; e < batch; ++e) {
          const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            l[c] = min2<bf>(l[c], w[c]);
            h[c] = max2<bf>(h[c], w[c]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < channels; ++c) {
        lo[c] = wide(l[(c >> 1) & 3] >> (16 * (c & 1)));
        hi[c] = wide(h[(c >> 1) & 3] >> (16 * (c & 1)));
      }
    }
  }
  __device__ __forceinline__ static float wide(uint32_t x) {
    return bf ? __uint_as_float(x << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(x)));
  }
  // Over the lanes that hold the same channels.
  __device__ __forceinline__ void join_lanes() {
#pragma unroll
    for (int o = lanes; o < 32; o <<= 1)
#pragma unroll
      for (int c = 0; c < channels; ++c) {
        lo[c] = min_nan(lo[c], __shfl_xor_sync(0xffffffffu, lo[c], o));
        hi[c] = max_nan(hi[c], __shfl_xor_sync(0xffffffffu, hi[c], o));
      }
  }
  // Codes and scale, by a whole warp.
  __device__ __forceinline__ void store(int8_t* codes, float* scale_out) const {
    const int lane = threadIdx.x & 31, piece = lane % lanes;
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < channels; ++c) top = max_nan(top, max_nan(fabsf(lo[c]), fabsf(hi[c])));
#pragma unroll
    for (int o = 1; o < lanes; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool bad = !(top <= 3.402823466e38f);   // a key that is no finite number
    const float scale = bad ? INFINITY : __fdiv_rn(top, 127.f);
    // every lane has the bounds of its channels' lanes: four channels each
    const int group = lane / lanes;
    float l4[4], h4[4];
#pragma unroll
    for (int c = 0; c < channels; ++c)
      if (c / 4 == group) {
        l4[c % 4] = lo[c];
        h4[c % 4] = hi[c];
      }
    uint32_t out[2] = {0, 0};
    if (!bad && scale > 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int a = static_cast<int>(fminf(fmaxf(floorf(__fdiv_rn(l4[e], scale)), -127.f), 127.f));
        const int b = static_cast<int>(fminf(fmaxf(ceilf(__fdiv_rn(h4[e], scale)), -127.f), 127.f));
        out[0] |= (static_cast<uint32_t>(a) & 255u) << (8 * e);
        out[1] |= (static_cast<uint32_t>(b) & 255u) << (8 * e);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) *reinterpret_cast<uint32_t*>(codes + k * kD + piece * channels + group * 4) = out[k];
    if (lane == 0) *scale_out = scale;
  }
};

// CTA: the pages that ROWS packed rows lie on, each once: by the first of the rows that follow one another on it.
// A warp has a key head of a page to itself, unless the page is long.  (A CTA of 8 rows that took its pages one after the
// other was bound by its reads' latency: 16 pages of 16 rows took 11.7 us, 3.6 this way.)
template <int TYPE, int ROWS>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const Pool p, int layer, const int32_t* __restrict__ row_seq,
                                                                    const int32_t* __restrict__ row_pos, int rows,
                                                                    int8_t* __restrict__ bounds, float* __restrict__ scales) {
  using B = Bounds<TYPE>;
  __shared__ float s_lo[kBoundWarps][kD], s_hi[kBoundWarps][kD];
  const int r0 = blockIdx.x * ROWS, lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // lane e of every warp looks at row r0 + e
  int32_t page = -1, fill = 0;
  if (lane < ROWS && r0 + lane < rows) {
    const int r = r0 + lane;
    const int32_t s = row_seq[r], at = row_pos[r], s1 = r > 0 ? row_seq[r - 1] : -1, at1 = r > 0 ? row_pos[r - 1] : -1;
    if (static_cast<uint32_t>(s) < static_cast<uint32_t>(p.max_seqs) && at >= 0) {
      const uint32_t b = div_of(static_cast<uint32_t>(at), p.ps);
      const int32_t len = p.len_of(s);
      const bool again = s1 == s && at1 >= 0 && at1 < len && div_of(static_cast<uint32_t>(at1), p.ps) == b;
      if (!again && at < p.cap) {
        page = p.table[static_cast<size_t>(s) * p.max_pages + b];
        fill = min(static_cast<int32_t>(p.ps.d), len - static_cast<int32_t>(b * p.ps.d));
        if (at >= len) {
          page = -1;
        } else if (!p.has(page)) {
          if (threadIdx.x < 32) tc::report_giveup(tc::kBadPage);
          page = -1;
        }
      }
    }
  }
  const bool shared = p.ps.d > kWarpRows;
  int item = w;   // (page, key head) of this CTA, counted through all of its pages
  for (uint32_t live = __ballot_sync(0xffffffffu, page >= 0); live; live &= live - 1) {
    const int e = __ffs(live) - 1;
    const int32_t pg = __shfl_sync(0xffffffffu, page, e), n = __shfl_sync(0xffffffffu, fill, e);
    int h = shared ? 0 : item;
    for (; h < p.Hkv; h += shared ? 1 : warps) {
      const size_t unit = (static_cast<size_t>(layer) * p.n_pages + pg) * p.Hkv + h;
      const int j = lane / B::lanes, step = B::at_once;
      B b;
      b.rows(p, unit * p.ps.d, shared ? w * step + j : j, shared ? warps * step : step, n);
      b.join_lanes();
      if (shared) {
        __syncthreads();   // the last values have been read
        if (lane < B::lanes)
#pragma unroll
          for (int c = 0; c < B::channels; ++c) {
            s_lo[w][lane * B::channels + c] = b.lo[c];
            s_hi[w][lane * B::channels + c] = b.hi[c];
          }
        __syncthreads();
        if (w > 0) continue;
        for (int v = 1; v < warps; ++v)
#pragma unroll
          for (int c = 0; c < B::channels; ++c) {
            b.lo[c] = min_nan(b.lo[c], s_lo[v][lane % B::lanes * B::channels + c]);
            b.hi[c] = max_nan(b.hi[c], s_hi[v][lane % B::lanes * B::channels + c]);
          }
      }
      b.store(bounds + unit * (2 * kD), scales + unit);
    }
    item = h - p.Hkv;
  }
}

template <int TYPE>
void launch_bounds(const Pool& p, int layer, const int32_t* row_seq, const int32_t* row_pos, int rows, int8_t* bounds, float* scales,
                   cudaStream_t st) {
  // Few rows are mostly of as many sequences, each with a page of its own; of many, most share a page with the row before.
  // (One / two rows a CTA, 8 key heads, 16-bit pages of 64 rows: 64 tokens 4.4 / 6.4 us, 256 5.0 / 6.3, 1024 11.8 / 11.7; chunks of 512
  // rows 5.1 / 4.9, four of them 6.3 / 5.7, eight of 1024 12.1 / 9.0, four of 4096 19.6 / 12.9.  INT8: 64 tokens 6.6 / 10.3, 1024
  // 19.9 / 22.4, eight chunks of 1024 18.4 / 14.6.)
  const int each = rows <= 1024 ? 1 : 2;
  const int warps = static_cast<int>(p.ps.d) > kWarpRows ? kBoundWarps : std::min(kBoundWarps, each * p.Hkv);
  const auto kern = each == 1 ? page_bounds_kernel<TYPE, 1> : page_bounds_kernel<TYPE, 2>;
  kern<<<(rows - 1) / each + 1, warps * 32, 0, st>>>(p, layer, row_seq, row_pos, rows, bounds, scales);
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
  const cudaStream_t st = as_stream(stream);
  switch (p.type) {
    case MIKV_PAGES_FP16: launch_bounds<MIKV_PAGES_FP16>(p, layer, row_seq, row_pos, rows, bounds, scales, st); break;
    case MIKV_PAGES_BF16: launch_bounds<MIKV_PAGES_BF16>(p, layer, row_seq, row_pos, rows, bounds, scales, st); break;
    default: launch_bounds<MIKV_PAGES_INT8>(p, layer, row_seq, row_pos, rows, bounds, scales, st);
  }
  return check_launch("page_bounds_kernel");
}
