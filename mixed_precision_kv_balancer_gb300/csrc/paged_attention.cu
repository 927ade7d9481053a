// Attention of one new token per sequence over a paged cache, split over the cache's length.
//
// Mathematics: out_h = sum_j p_j v_j / sum_j p_j with p_j = exp(l_j - m), one pass over the
// visible slots with a running maximum and sum.  A unit is one (sequence, key head, group of up
// to 16 of its query heads): the group's queries meet each key once, as the 16 rows of an
// mma.sync m16n8k16 whose columns are slots (q . K^T) and then channels (P . V), so every
// cached row is read from HBM once.  Bound by HBM: 512 (16-bit) or 272 (INT8) bytes per slot
// and key head against 4 * 16 * 128 products, 16 flop a byte.
//
// Split: the visible slots of all units, cut into tiles, form one line; CTA c takes the c-th of
// `grid` equal parts of it, whatever the sequences' lengths, so ragged batches stay balanced and
// the grid does not depend on lengths that only the device knows.  A unit that one CTA holds
// whole is finished there; the others' partial sums go to the workspace and are joined, in
// order, by a second kernel.
//
// Inside a CTA four warps take 16 (16-bit) or 32 (INT8) slots each of every tile, through rings
// of their own in shared memory (16-byte cp.async, rows of any page, zero-filled where no slot
// is), and are joined at a unit's end.
//
// Precision: scores, maximum, sum and accumulators are fp32.  The weights p meet the values as
// two 16-bit parts (p = hi + lo, 16 to 22 bits), so they add nothing to the rounding of the
// output; fp16 weights carry a factor 2^15, so that many small ones beside one large one stay
// out of fp16's subnormal range (down to 2^-29 of the largest).  INT8 codes enter the products
// as exact integers: q . (s c + z) = s (q . c) + z sum(q) per group of 64 channels (fp16), and
// sum_j p_j (s_j c_j + z_j) = sum_j (p_j s_j) (c_j - 128) + sum_j p_j (z_j + 128 s_j), where the
// weights p_j s_j and the codes are bf16, whose range takes any scale.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int paged_attention_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kPaThreads = 128;
constexpr int kPaWarps = 4;
constexpr int kPaRows = 16;       // query heads of a unit: the mma's M
constexpr int kPaCtasPerSM = 2;

template <int TYPE>
struct Shape {
  static constexpr bool q8 = TYPE == MIKV_PAGES_INT8;
  static constexpr int tw = q8 ? 32 : 16;             // slots of one warp's stage
  static constexpr int tile = tw * kPaWarps;          // slots of a tile
  static constexpr int row = q8 ? kD : kD * 2;        // bytes of a stored row
  static constexpr int shift = TYPE == MIKV_PAGES_FP16 ? 15 : 0;  // the weights' factor, log2
  static constexpr int pv = q8 ? MIKV_PAGES_BF16 : TYPE;          // type of the weights and values in products
  static constexpr int stages = 3;
  static constexpr int k_bytes = tw * row;
  static constexpr int meta = q8 ? tw * kMetaBytes : 0;
  static constexpr int stage = 2 * k_bytes + 2 * meta + 16;  // + the mask of valid slots
  static constexpr int smem = kPaWarps * stages * stage;
};

struct AttendArgs {
  Pool p;
  const uint16_t* q;
  const int32_t* seqs;
  int layer, n, Hq, rep, groups, heads;   // query heads per key head; groups of `heads` of them
  int window, sinks;
  uint16_t* out;
  float* lse;
  float* part;    // [2 * grid][kPartFloats]
  float scale;    // log2(e) / sqrt(D)
};
constexpr int kPartFloats = kPaRows * kD + 2 * kPaRows;  // O, then m, then l

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

template <int TYPE>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (TYPE == MIKV_PAGES_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// Two values as a pair of 16-bit parts: hi = round(x), lo = round(x - hi).
template <int TYPE>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  if (TYPE == MIKV_PAGES_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x0 - __low2float(h), x1 - __high2float(h));
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    const __half2 h = __floats2half2_rn(x0, x1);
    const __half2 l = __floats2half2_rn(x0 - __low2float(h), x1 - __high2float(h));
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}
template <int TYPE>
__device__ __forceinline__ uint16_t to_out(float x) {
  if (TYPE == MIKV_PAGES_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return __half_as_ushort(__float2half_rn(x));
}

// Visible slots of row b's sequence; none for a sequence number out of range.
__device__ __forceinline__ Visible row_visible(const AttendArgs& a, int b, int32_t& seq) {
  seq = a.seqs ? a.seqs[b] : b;
  if (static_cast<uint32_t>(seq) >= static_cast<uint32_t>(a.p.max_seqs)) return {0, 0, 0};
  return visible_slots(a.p.len_of(seq), a.window, a.sinks);
}
template <int TILE>
__device__ __forceinline__ int row_tiles(const AttendArgs& a, int b) {
  int32_t s;
  return (row_visible(a, b, s).count + TILE - 1) / TILE;
}

// Sums over the block's threads below this one (inclusive) and over all of them.
__device__ __forceinline__ int64_t scan64(int64_t v, int64_t* warp_sums, int64_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kPaWarps; ++i) {
    if (i < w) before += warp_sums[i];
    total += warp_sums[i];
  }
  return v + before;
}

// CTAs that get a part: with fewer tiles than CTAs one each, so that no part is empty.
__device__ __forceinline__ int workers_of(int64_t total, int grid) { return static_cast<int>(min(total, static_cast<int64_t>(grid))); }

// One warp's accumulators over its slots of a unit.
template <int TYPE, bool WIDE>
struct Acc {
  float o[kD / 8][4];   // 16 rows x 128 channels, mma layout (INT8: even and odd channels apart)
  float m[2], l[2];     // rows g and g + 8: maximum (log2 units) and this thread's part of the sum
  float z[2][2];        // INT8: sum of p (z + 128 s) per row and group, this thread's part
};

// Shared-memory address of 16-byte piece c of row r of a stage's keys or values.
template <bool Q8>
__device__ __forceinline__ uint32_t k_at(uint32_t s, int r, int c) {
  return Q8 ? s + r * kD + ((c ^ ((r & 1) << 2)) << 4) : s + r * (kD * 2) + ((c ^ (r & 7)) << 4);
}
template <bool Q8>
__device__ __forceinline__ uint32_t v_at(uint32_t s, int r, int c) {
  return s + r * (Q8 ? kD : kD * 2) + ((c ^ (r & 7)) << 4);
}

// The pool row of visible slot `i`, kNoRow past the last one or where the table names no page.
__device__ __forceinline__ uint32_t slot_row(const Pool& p, const int32_t* row, const Visible& vis, int h, int64_t i) {
  if (i >= vis.count) return kNoRow;
  const uint32_t slot = visible_slot(vis, static_cast<int32_t>(i)), pg = div_of(slot, p.ps);
  const uint32_t r = pool_row(__ldg(row + pg), p.n_pages, p.Hkv, h, p.ps.d, slot - pg * p.ps.d);
  if (r == kNoRow) tc::report_giveup(tc::kBadPage);
  return r;
}

// Starts the copies of one stage: lane l < tw holds the pool row of the stage's slot l.
template <int TYPE>
__device__ __forceinline__ void issue(const Pool& p, size_t lrow, uint32_t st, uint32_t my_row, uint64_t policy) {
  using S = Shape<TYPE>;
  const int lane = threadIdx.x & 31;
  constexpr int per_row = S::row / 16;       // lanes of one row
  constexpr int at_once = 32 / per_row;      // rows of one warp-wide copy
  const uint8_t* kb = p.k + lrow * S::row;
  const uint8_t* vb = p.v + lrow * S::row;
#pragma unroll
  for (int j = 0; j < S::tw / at_once; ++j) {
    const int r = j * at_once + lane / per_row, c = lane % per_row;
    const uint32_t src = __shfl_sync(0xffffffffu, my_row, r);
    const bool ok = src != kNoRow;
    const size_t off = ok ? static_cast<size_t>(src) * S::row + c * 16 : 0;
    cp_async16_once(k_at<S::q8>(st, r, c), kb + off, ok, policy);
    cp_async16_once(v_at<S::q8>(st + S::k_bytes, r, c), vb + off, ok, policy);
  }
  if (S::q8) {
    const bool ok = my_row != kNoRow;
    const size_t off = ok ? (lrow + my_row) * kMetaBytes : 0;
    cp_async8(st + 2 * S::k_bytes + lane * kMetaBytes, p.km + off, ok);
    cp_async8(st + 2 * S::k_bytes + S::meta + lane * kMetaBytes, p.vm + off, ok);
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, my_row != kNoRow);
  if (lane == 0) asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(st + 2 * S::k_bytes + 2 * S::meta), "r"(mask));
}

__device__ __forceinline__ float meta_s(uint32_t m) { return __half2float(__ushort_as_half(m & 0xffffu)); }
__device__ __forceinline__ float meta_z(uint32_t m) { return __half2float(__ushort_as_half(m >> 16)); }
// The codes in two bytes of x (`sel` puts them under 0x64) as an fp16 pair: 0x64cc is 1024 + c.
__device__ __forceinline__ uint32_t codes_f16(uint32_t x, uint32_t sel) {
  const uint32_t w = __byte_perm(x, 0x64646464u, sel), bias = 0x64006400u;
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Codes minus 128 as a bf16 pair: 0x4300 is 128 and its last seven bits count ones, so
// (128 + c mod 128) - (c < 128 ? 256 : 128) = c - 128; 0x4380 is 256.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t x, uint32_t sel) {
  const uint32_t w = __byte_perm(x, 0x43434343u, sel);
  const uint32_t a = w & 0xff7fff7fu, b = (~w & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One stage: scores of its slots, the running softmax, and their values.
// `qf`: the queries as A fragments; `qsum`: INT8, sums of the query's two groups for rows g, g + 8.
template <int TYPE, bool WIDE>
__device__ __forceinline__ void consume(uint32_t st, const uint32_t (&qf)[kD / 16][4], const float (&qsum)[2][2], float scale,
                                        Acc<TYPE, WIDE>& acc) {
  using S = Shape<TYPE>;
  constexpr int NT = S::tw / 8;
  constexpr int R = WIDE ? 2 : 1;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t mask = lds32(st + 2 * S::k_bytes + 2 * S::meta);
  float s[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (!S::q8) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k2 = 0; k2 < kD / 32; ++k2) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(k_at<S::q8>(st, nt * 8 + (lane & 7), k2 * 4 + (lane >> 3)), b0, b1, b2, b3);
        mma<TYPE>(d, qf[2 * k2], b0, b1);
        mma<TYPE>(d, qf[2 * k2 + 1], b2, b3);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s[nt][j] = d[j] * scale;
    } else {
      float d[2][4] = {};
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        const uint4 c = lds128(k_at<S::q8>(st, nt * 8 + g, grp * 4 + t));
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma<TYPE>(d[grp], qf[grp * 4 + kk], codes_f16(w[kk], 0x4140u), codes_f16(w[kk], 0x4342u));
      }
      const uint32_t ms = st + 2 * S::k_bytes + (nt * 8 + 2 * t) * kMetaBytes;
      const uint2 m0 = lds64(ms), m1 = lds64(ms + kMetaBytes);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint2 mm = (j & 1) ? m1 : m0;
        const int r = j >> 1;
        s[nt][j] = scale * (meta_s(mm.x) * d[0][j] + meta_z(mm.x) * qsum[r][0] + (meta_s(mm.y) * d[1][j] + meta_z(mm.y) * qsum[r][1]));
      }
    }
  }
  if (mask != (S::tw == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!((mask >> (nt * 8 + 2 * t + (j & 1))) & 1u)) s[nt][j] = -INFINITY;
  }
  float sub[2], alpha[2];
  bool grew = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float mx = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * r], s[nt][2 * r + 1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(acc.m[r], mx);
    // nothing seen yet: all weights are exp2(-inf) = 0
    alpha[r] = mn == -INFINITY ? 0.f : ex2(acc.m[r] - mn);
    sub[r] = mn == -INFINITY ? 0.f : mn - S::shift;
    grew |= mn > acc.m[r];
    acc.m[r] = mn;
  }
  if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      acc.l[r] *= alpha[r];
      if (S::q8) {
        acc.z[r][0] *= alpha[r];
        acc.z[r][1] *= alpha[r];
      }
#pragma unroll
      for (int i = 0; i < kD / 8; ++i) {
        acc.o[i][2 * r] *= alpha[r];
        acc.o[i][2 * r + 1] *= alpha[r];
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2 * R; ++j) {
      s[nt][j] = ex2(s[nt][j] - sub[j >> 1]);
      acc.l[j >> 1] += s[nt][j];
    }
  const uint32_t vs = st + S::k_bytes;
#pragma unroll
  for (int kt = 0; kt < S::tw / 16; ++kt) {
    if (!S::q8) {
      uint32_t hi[4] = {}, lo[4] = {};
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int r = 0; r < R; ++r)
          split_pair<TYPE>(s[2 * kt + half][2 * r], s[2 * kt + half][2 * r + 1], hi[half * 2 + r], lo[half * 2 + r]);
#pragma unroll
      for (int c = 0; c < kD / 8; c += 2) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(v_at<S::q8>(vs, kt * 16 + (lane & 15), c + (lane >> 4)), b0, b1, b2, b3);
        mma<TYPE>(acc.o[c], hi, b0, b1);
        mma<TYPE>(acc.o[c], lo, b0, b1);
        mma<TYPE>(acc.o[c + 1], hi, b2, b3);
        mma<TYPE>(acc.o[c + 1], lo, b2, b3);
      }
    } else {
      uint32_t hi[2][4] = {}, lo[2][4] = {};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t ms = st + 2 * S::k_bytes + S::meta + ((2 * kt + half) * 8 + 2 * t) * kMetaBytes;
        const uint2 m0 = lds64(ms), m1 = lds64(ms + kMetaBytes);
#pragma unroll
        for (int grp = 0; grp < 2; ++grp) {
          const uint32_t w0 = grp ? m0.y : m0.x, w1 = grp ? m1.y : m1.x;
          const float s0 = meta_s(w0), s1 = meta_s(w1);
          const float z0 = fmaf(128.f, s0, meta_z(w0)), z1 = fmaf(128.f, s1, meta_z(w1));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float p0 = s[2 * kt + half][2 * r], p1 = s[2 * kt + half][2 * r + 1];
            split_pair<S::pv>(p0 * s0, p1 * s1, hi[grp][half * 2 + r], lo[grp][half * 2 + r]);
            acc.z[r][grp] += p0 * z0 + p1 * z1;
          }
        }
      }
      // b16 pairs of codes, transposed: word = (slot 2t: channels 2g, 2g+1; slot 2t+1: the same)
#pragma unroll
      for (int c = 0; c < kD / 16; c += 2) {   // 16-channel blocks
        uint32_t x[4];
        ldsm_x4_t(v_at<S::q8>(vs, kt * 16 + (lane & 15), c + (lane >> 4)), x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int grp = (c + b) >> 2;
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t sel = odd ? 0x4341u : 0x4240u;
            const uint32_t b0 = codes_bf16(x[2 * b], sel), b1 = codes_bf16(x[2 * b + 1], sel);
            mma<S::pv>(acc.o[2 * (c + b) + odd], hi[grp], b0, b1);
            mma<S::pv>(acc.o[2 * (c + b) + odd], lo[grp], b0, b1);
          }
        }
      }
    }
  }
}

// The four warps' accumulators, joined: row r's maximum, sum and channel d.  `sm` floats:
// [warp][16][128] O, then [warp][16] m, then [warp][16] l.
template <int TYPE, bool WIDE>
__device__ __forceinline__ void store_acc(float* sm, Acc<TYPE, WIDE>& acc) {
  using S = Shape<TYPE>;
  constexpr int R = WIDE ? 2 : 1;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float* so = sm + w * kPaRows * kD;
  float* smax = sm + kPaWarps * kPaRows * kD;
  float* ssum = smax + kPaWarps * kPaRows;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = g + 8 * r;
    float l = acc.l[r];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    float z[2] = {0.f, 0.f};
    if (S::q8) {
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        z[grp] = acc.z[r][grp];
        z[grp] += __shfl_xor_sync(0xffffffffu, z[grp], 1);
        z[grp] += __shfl_xor_sync(0xffffffffu, z[grp], 2);
      }
    }
    if (t == 0) {
      smax[w * kPaRows + row] = acc.m[r];
      ssum[w * kPaRows + row] = l;
    }
    if (!S::q8) {
#pragma unroll
      for (int c = 0; c < kD / 8; ++c)
        *reinterpret_cast<float2*>(so + row * kD + c * 8 + 2 * t) = make_float2(acc.o[c][2 * r], acc.o[c][2 * r + 1]);
    } else {
#pragma unroll
      for (int b = 0; b < kD / 16; ++b) {
        const float zz = z[b >> 2];
        const float4 x = make_float4(acc.o[2 * b][2 * r] + zz, acc.o[2 * b + 1][2 * r] + zz, acc.o[2 * b][2 * r + 1] + zz,
                                     acc.o[2 * b + 1][2 * r + 1] + zz);
        *reinterpret_cast<float4*>(so + row * kD + b * 16 + 4 * t) = x;
      }
    }
  }
}

template <int TYPE>
__device__ __forceinline__ float lse_of(float m, float l) {
  return (m + (log2f(l) - Shape<TYPE>::shift)) * 0.6931471805599453f;
}

// CTA c of the split.
template <int TYPE, bool WIDE>
__global__ void __launch_bounds__(kPaThreads, kPaCtasPerSM) paged_partial_kernel(const AttendArgs a) {
  using S = Shape<TYPE>;
  constexpr int R = WIDE ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sums[kPaWarps];
  __shared__ int64_t s_base;
  __shared__ int s_seq;
  pdl_trigger();
  const Pool& p = a.p;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int units = p.Hkv * a.groups;
  // this CTA's part of the line of tiles, and the sequence it begins in
  int64_t mine = 0, total;
  for (int b = tid; b < a.n; b += kPaThreads) mine += row_tiles<S::tile>(a, b);
  scan64(mine * units, warp_sums, total);
  const int workers = workers_of(total, gridDim.x);
  if (static_cast<int>(blockIdx.x) >= workers) return;
  const int64_t begin = split_begin(total, workers, blockIdx.x), end = split_begin(total, workers, blockIdx.x + 1);
  int64_t before = 0;
  for (int b0 = 0;; b0 += kPaThreads) {   // ends: the last tile is below `total`
    const int b = b0 + tid;
    const int64_t v = b < a.n ? static_cast<int64_t>(row_tiles<S::tile>(a, b)) * units : 0;
    int64_t sum;
    const int64_t incl = before + scan64(v, warp_sums, sum);
    if (begin < incl && begin >= incl - v) {
      s_base = incl - v;
      s_seq = b;
    }
    before += sum;
    if (begin < before) break;
  }
  __syncthreads();
  int64_t base = s_base;
  int b = s_seq;

  const uint32_t ring = smem_u32(smem) + w * S::stages * S::stage;
  const size_t lrow = p.layer_rows() * a.layer;
  const uint64_t policy = l2_evict_first_policy();
  for (int64_t cur = begin; cur < end;) {
    int32_t seq;
    const Visible vis = row_visible(a, b, seq);
    const int tiles = (vis.count + S::tile - 1) / S::tile;
    if (tiles == 0) {
      ++b;
      continue;
    }
    const int u = static_cast<int>((cur - base) / tiles), t0 = static_cast<int>((cur - base) % tiles);
    const int count = static_cast<int>(min(static_cast<int64_t>(tiles - t0), end - cur));
    const int h = u / a.groups, head0 = h * a.rep + (u % a.groups) * a.heads;
    const int rows = min(a.heads, a.rep - (u % a.groups) * a.heads);
    const int32_t* table = p.table + static_cast<size_t>(seq) * p.max_pages;
    // slots of this warp: i0 + tile * S::tile + lane
    const int64_t i0 = static_cast<int64_t>(t0) * S::tile + w * S::tw + lane;
    const auto find = [&](int it) {
      return (lane < S::tw && it < count) ? slot_row(p, table, vis, h, i0 + static_cast<int64_t>(it) * S::tile) : kNoRow;
    };
#pragma unroll
    for (int it = 0; it < S::stages - 1; ++it) {
      const uint32_t r = find(it);
      if (it < count) issue<TYPE>(p, lrow, ring + it * S::stage, r, policy);
      cp_async_commit();
    }
    uint32_t next = find(S::stages - 1);
    // the queries, as A fragments (INT8: channels in the order the codes are read)
    uint32_t qf[kD / 16][4];
    float qsum[2][2] = {};
#pragma unroll
    for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = g + 8 * (j & 1);
        const int ch = S::q8 ? 64 * (ks >> 2) + 16 * t + 4 * (ks & 3) + 2 * (j >> 1) : 16 * ks + 8 * (j >> 1) + 2 * t;
        uint32_t x = 0;
        if (row < rows)
          x = *reinterpret_cast<const uint32_t*>(a.q + (static_cast<size_t>(b) * a.Hq + head0 + row) * kD + ch);
        qf[ks][j] = x;
        if (S::q8) {
          const __half2 x2 = *reinterpret_cast<const __half2*>(&x);
          qsum[j & 1][ks >> 2] += __low2float(x2) + __high2float(x2);
        }
      }
    if (S::q8) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int grp = 0; grp < 2; ++grp) {
          qsum[r][grp] += __shfl_xor_sync(0xffffffffu, qsum[r][grp], 1);
          qsum[r][grp] += __shfl_xor_sync(0xffffffffu, qsum[r][grp], 2);
        }
    }
    Acc<TYPE, WIDE> acc;
#pragma unroll
    for (int i = 0; i < kD / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc.o[i][j] = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      acc.m[r] = -INFINITY;
      acc.l[r] = acc.z[r][0] = acc.z[r][1] = 0.f;
    }
    int rd = 0, wr = S::stages - 1;
    for (int it = 0; it < count; ++it) {
      cp_async_wait<S::stages - 2>();
      __syncwarp();   // the stage has landed for all lanes, and the one to be refilled is read
      if (it + S::stages - 1 < count) issue<TYPE>(p, lrow, ring + wr * S::stage, next, policy);
      cp_async_commit();
      next = find(it + S::stages);
      consume<TYPE, WIDE>(ring + rd * S::stage, qf, qsum, a.scale, acc);
      rd = rd + 1 == S::stages ? 0 : rd + 1;
      wr = wr + 1 == S::stages ? 0 : wr + 1;
    }
    cp_async_wait<0>();
    __syncthreads();   // every warp is done with its ring: its space holds the accumulators now
    float* sm = reinterpret_cast<float*>(smem);
    store_acc<TYPE, WIDE>(sm, acc);
    __syncthreads();
    const float* smax = sm + kPaWarps * kPaRows * kD;
    const float* ssum = smax + kPaWarps * kPaRows;
    const bool whole = t0 == 0 && count == tiles;
    float* part = a.part + (static_cast<size_t>(blockIdx.x) * 2 + (cur == begin ? 0 : 1)) * kPartFloats;
#pragma unroll 1
    for (int row = 0; row < min(rows, 8 * R); ++row) {
      float m = smax[row], l = 0.f, o = 0.f;
#pragma unroll
      for (int i = 1; i < kPaWarps; ++i) m = fmaxf(m, smax[i * kPaRows + row]);
      const float sub = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int i = 0; i < kPaWarps; ++i) {
        const float f = ex2(smax[i * kPaRows + row] - sub);
        l += f * ssum[i * kPaRows + row];
        o += f * sm[(i * kPaRows + row) * kD + tid];
      }
      if (whole) {
        const size_t at = static_cast<size_t>(b) * a.Hq + head0 + row;
        a.out[at * kD + tid] = to_out<TYPE>(l == 0.f ? 0.f : o / l);   // all pages bad: nothing seen
        if (tid == 0 && a.lse) a.lse[at] = lse_of<TYPE>(m, l);
      } else {
        part[row * kD + tid] = o;
        if (tid == 0) {
          part[kPaRows * kD + row] = m;
          part[kPaRows * kD + kPaRows + row] = l;
        }
      }
    }
    __syncthreads();   // the ring may be refilled
    cur += count;
    if (cur - base == static_cast<int64_t>(tiles) * units) {
      base = cur;
      ++b;
    }
  }
}

// CTA (unit, row b): joins the parts of a unit that several CTAs held, in their order, and
// answers for the units without a visible slot.
template <int TYPE>
__global__ void __launch_bounds__(kPaThreads) paged_merge_kernel(const AttendArgs a, int grid) {
  using S = Shape<TYPE>;
  __shared__ int64_t warp_sums[kPaWarps];
  const int units = a.p.Hkv * a.groups, b = blockIdx.y, u = blockIdx.x, tid = threadIdx.x;
  const int h = u / a.groups, head0 = h * a.rep + (u % a.groups) * a.heads;
  const int rows = min(a.heads, a.rep - (u % a.groups) * a.heads);
  int64_t mine = 0, below = 0, total, base;
  for (int i = tid; i < a.n; i += kPaThreads) {
    const int x = row_tiles<S::tile>(a, i);
    mine += x;
    if (i < b) below += x;
  }
  scan64(mine * units, warp_sums, total);
  scan64(below * units, warp_sums, base);
  const int tiles = row_tiles<S::tile>(a, b);
  pdl_wait();
  const size_t at = static_cast<size_t>(b) * a.Hq + head0;
  if (tiles == 0) {
    for (int row = 0; row < rows; ++row) {
      a.out[(at + row) * kD + tid] = 0;
      if (tid == 0 && a.lse) a.lse[at + row] = -INFINITY;
    }
    return;
  }
  const int workers = workers_of(total, grid);
  const int64_t first = base + static_cast<int64_t>(u) * tiles;
  const int c0 = split_owner(total, workers, first), c1 = split_owner(total, workers, first + tiles - 1);
  if (c0 == c1) return;
  const int skip = split_begin(total, workers, c0) < first ? 1 : 0;   // c0 holds it as its second part
  const float* p0 = a.part + (static_cast<size_t>(c0) * 2 + skip) * kPartFloats;
  for (int row = 0; row < rows; ++row) {
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const float* q = c == c0 ? p0 : a.part + static_cast<size_t>(c) * 2 * kPartFloats;
      const float mc = q[kPaRows * kD + row], lc = q[kPaRows * kD + kPaRows + row], oc = q[row * kD + tid];
      const float mn = fmaxf(m, mc), sub = mn == -INFINITY ? 0.f : mn;
      const float f = ex2(m - sub), fc = ex2(mc - sub);
      l = l * f + lc * fc;
      o = o * f + oc * fc;
      m = mn;
    }
    a.out[(at + row) * kD + tid] = to_out<TYPE>(l == 0.f ? 0.f : o / l);
    if (tid == 0 && a.lse) a.lse[at + row] = lse_of<TYPE>(m, l);
  }
}

// CTAs of the split: two per SM, or one per tile where that is fewer.
int grid_of(const mikv_pages* p, int n, int Hq, int window, int sinks) {
  const int tile = p->type == MIKV_PAGES_INT8 ? Shape<MIKV_PAGES_INT8>::tile : Shape<MIKV_PAGES_FP16>::tile;
  const int rep = Hq / p->Hkv, groups = (rep + kPaRows - 1) / kPaRows;
  int64_t slots = static_cast<int64_t>(p->max_pages) * p->page_size;
  if (window > 0) slots = std::min(slots, static_cast<int64_t>(window) + sinks);
  const int64_t tiles = (slots + tile - 1) / tile;
  const int64_t most = static_cast<int64_t>(kPaCtasPerSM) * kNumSMs;
  return static_cast<int>(std::max<int64_t>(1, std::min(most, tiles * n * p->Hkv * groups)));
}

template <int TYPE, bool WIDE>
int launch(const AttendArgs& a, int grid, cudaStream_t st) {
  const auto kern = paged_partial_kernel<TYPE, WIDE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<TYPE>::smem);
  if (e != cudaSuccess) return check_launch_after(e, "paged_partial_kernel");
  kern<<<grid, kPaThreads, Shape<TYPE>::smem, st>>>(a);
  if (int r = check_launch("paged_partial_kernel")) return r;
  return check_launch_after(launch_after(paged_merge_kernel<TYPE>, dim3(a.p.Hkv * a.groups, a.n), dim3(kPaThreads), 0, st, a, grid),
                            "paged_merge_kernel");
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_paged_attention_workspace_bytes(const mikv_pages* p, int n, int Hq, int window, int sinks) {
  Pool pool;
  if (check_pages(p, "paged_attention", &pool) || n < 1 || n > 65535 || Hq < 1 || Hq % p->Hkv || window < 0 || sinks < 0) return 0;
  return static_cast<size_t>(grid_of(p, n, Hq, window, sinks)) * 2 * kPartFloats * sizeof(float);
}

extern "C" int mikv_paged_attention(const void* q, const mikv_pages* pages, int layer, const int32_t* seqs, int n, int Hq,
                                    int window, int sinks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  AttendArgs a;
  if (int e = check_pages(pages, "paged_attention", &a.p)) return e;
  if (layer < 0 || layer >= a.p.layers) return fail(MIKV_ESHAPE, "paged_attention: layer=%d of %d", layer, a.p.layers);
  if (n < 0 || n > 65535 || (!seqs && n > a.p.max_seqs)) return fail(MIKV_ESHAPE, "paged_attention: n=%d", n);
  if (Hq < 1 || Hq % a.p.Hkv || Hq / a.p.Hkv > 1024) return fail(MIKV_ESHAPE, "paged_attention: Hq=%d Hkv=%d", Hq, a.p.Hkv);
  if (window < 0 || sinks < 0) return fail(MIKV_EINVAL, "paged_attention: window=%d sinks=%d", window, sinks);
  if (n == 0) return MIKV_OK;
  if (!q || !out || !ws) return fail(MIKV_EINVAL, "paged_attention: null pointer");
  if (!aligned16(q) || !aligned16(out) || !aligned16(ws)) return fail(MIKV_EALIGN, "paged_attention: 16-byte alignment");
  const int grid = grid_of(pages, n, Hq, window, sinks);
  const size_t need = static_cast<size_t>(grid) * 2 * kPartFloats * sizeof(float);
  if (ws_bytes < need) return fail(MIKV_ESHAPE, "paged_attention: workspace %zu < %zu", ws_bytes, need);
  a.q = static_cast<const uint16_t*>(q);
  a.seqs = seqs;
  a.layer = layer;
  a.n = n;
  a.Hq = Hq;
  a.rep = Hq / a.p.Hkv;
  a.groups = (a.rep + kPaRows - 1) / kPaRows;
  a.heads = (a.rep + a.groups - 1) / a.groups;
  a.window = window;
  a.sinks = sinks;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.scale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
  const cudaStream_t st = as_stream(stream);
  const bool wide = a.heads > 8;
  switch (a.p.type) {
    case MIKV_PAGES_FP16: return wide ? launch<MIKV_PAGES_FP16, true>(a, grid, st) : launch<MIKV_PAGES_FP16, false>(a, grid, st);
    case MIKV_PAGES_BF16: return wide ? launch<MIKV_PAGES_BF16, true>(a, grid, st) : launch<MIKV_PAGES_BF16, false>(a, grid, st);
    default: return wide ? launch<MIKV_PAGES_INT8, true>(a, grid, st) : launch<MIKV_PAGES_INT8, false>(a, grid, st);
  }
}
