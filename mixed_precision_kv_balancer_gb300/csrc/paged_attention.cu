// Attention of one new token per sequence over a paged cache, split over the cache's length.
//
// Mathematics: out_h = sum_j p_j v_j / sum_j p_j with p_j = exp(l_j - m), one pass over the
// visible slots with a running maximum and sum.  A unit is one (sequence, key head, group of up
// to 16 of its query heads): the group's queries meet each cached row once.  Bound by HBM: 512
// (16-bit) or 272 (INT8) bytes per slot and key head against 4 * 16 * 128 products, 16 flop a
// byte; mma.sync suffices, with 16 slots (or channels) as its M and 8 query heads as its N:
// S = K Q^T, then O^T += V^T P^T, so that scores, weights and sums of a head stay in one lane's
// columns and up to 8 heads waste nothing.
//
// Split: the visible slots of all units, cut into tiles of 16 (INT8: 32), form one line; warp c of
// the grid takes the c-th of equal parts of it, whatever the sequences' lengths, so ragged batches
// stay balanced and the grid does not depend on lengths that only the device knows.  A unit that
// one warp holds whole is finished there; the others' partial sums go to the workspace and are
// joined, in order, by a second kernel.  Warps never wait for one another: each streams its part
// through a ring of its own in shared memory (16-byte cp.async, rows of any page, zero-filled
// where no slot is) and requests tiles ahead of the one it works on across the units' ends.
//
// Precision: scores, maximum, sum and accumulators are fp32.  The weights p meet the values as
// two 16-bit parts (p = hi + lo, 16 to 22 bits), so they add nothing to the rounding of the
// output; fp16 weights carry a factor 2^15, so that many small ones beside one large one stay
// out of fp16's subnormal range (down to 2^-29 of the largest).  INT8 codes enter the products
// as exact integers: q . (s c + z) = s (q . c) + z sum(q) per group of 64 channels (fp16), and
// sum_j p_j (s_j c_j + z_j) = sum_j (p_j s_j) (c_j - 128) + sum_j p_j (z_j + 128 s_j), where the
// weights p_j s_j carry the factor 2^15 / cap, cap the power of two above every s_j so far (the
// sums are rescaled where it moves).
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int paged_attention_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kPaThreads = 128;
constexpr int kPaWarps = 4;
constexpr int kPaRows = 16;       // query heads of a unit at most: two column blocks of the mma
constexpr int kPaCtasPerSM = 2;
constexpr int kMergeWarps = 16;   // of one head's join, where it has many parts

template <int TYPE>
struct Shape {
  static constexpr bool q8 = TYPE == MIKV_PAGES_INT8;
  static constexpr int tw = q8 ? 32 : 16;             // slots of a tile
  static constexpr int row = q8 ? kD : kD * 2;        // bytes of a stored row
  static constexpr int shift = TYPE == MIKV_PAGES_FP16 ? 15 : 0;  // the weights' factor, log2
  static constexpr int stages = 3;
  static constexpr int k_bytes = tw * row;
  static constexpr int meta = q8 ? tw * kMetaBytes : 0;
  // + the mask of valid slots; stages begin at multiples of 256 bytes, so that swizzled addresses
  // are one exclusive or
  static constexpr int stage = (2 * k_bytes + 2 * meta + 16 + 255) / 256 * 256;
  static constexpr int smem = kPaWarps * stages * stage + 256;
};

struct AttendArgs {
  Pool p;
  const uint16_t* q;
  const int32_t* seqs;
  int layer, n, Hq, rep, groups, heads;   // query heads per key head; groups of `heads` of them
  int window, sinks;
  uint16_t* out;
  float* lse;
  float* part;    // [2 * warps of the grid][kPartFloats]
  float scale;    // log2(e) / sqrt(D)
  // picked blocks: n = packed rows * key heads, and a "row" below is one of these; sel [n][keep], n_sel [n]
  const int32_t *row_seq, *row_pos, *sel, *n_sel;
  int keep;
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

// Visible slots of row b's sequence; none for a sequence number out of range.  Picked blocks (SEL): all
// slots of the row's blocks are numbered, of which those up to `skip`, the last position, are seen.
template <bool SEL>
__device__ __forceinline__ Visible row_visible(const AttendArgs& a, int b, int32_t& seq) {
  if (SEL) {
    const int r = b / a.p.Hkv;
    seq = a.row_seq ? a.row_seq[r] : r;
    if (static_cast<uint32_t>(seq) >= static_cast<uint32_t>(a.p.max_seqs)) return {0, 0, 0};
    const int32_t last = a.p.len_of(seq) - 1, at = a.row_pos ? min(a.row_pos[r], last) : last;
    if (at < 0) return {0, 0, 0};
    return {min(max(a.n_sel[b], 0), a.keep) * static_cast<int32_t>(a.p.ps.d), 0, at};
  }
  seq = a.seqs ? a.seqs[b] : b;
  if (static_cast<uint32_t>(seq) >= static_cast<uint32_t>(a.p.max_seqs)) return {0, 0, 0};
  return visible_slots(a.p.len_of(seq), a.window, a.sinks);
}
template <int TILE, bool SEL>
__device__ __forceinline__ int row_tiles(const AttendArgs& a, int b) {
  int32_t s;
  return (row_visible<SEL>(a, b, s).count + TILE - 1) / TILE;
}

// Sums over the block's threads below this one (inclusive) and over all of them.
template <int W = kPaWarps>
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
  for (int i = 0; i < W; ++i) {
    if (i < w) before += warp_sums[i];
    total += warp_sums[i];
  }
  return v + before;
}

// Warps that get a part: with fewer tiles than warps one each, so that no part is empty.
__device__ __forceinline__ int workers_of(int64_t total, int warps) { return static_cast<int>(min(total, static_cast<int64_t>(warps))); }

// One warp's accumulators of a unit.  Column block nh, thread column j: query head 8 nh + 2 t + j.
template <int NH>
struct Acc {
  float o[kD / 16][NH][4];   // O^T: 16 channels x 8 heads, mma layout
  float m[NH][2];            // maximum, log2 units (the same in the 8 lanes of a column)
  float l[NH][2];            // this thread's part of the sum
  float z[NH][2][2];         // INT8: this thread's part of sum p (z + 128 s), per group of channels
  float cap[2];              // INT8: power of two not below any scale of a value so far, per group
};

// Shared-memory address of 16-byte piece c of row r of a stage's keys or values, as k_row ^ (c << 4), v_row ^ (c << 4).
template <bool Q8>
__device__ __forceinline__ uint32_t k_row(uint32_t s, int r) {
  return Q8 ? s + r * kD + ((r & 1) << 6) : s + r * (kD * 2) + ((r & 7) << 4);
}
template <bool Q8>
__device__ __forceinline__ uint32_t v_row(uint32_t s, int r) {
  return s + r * (Q8 ? kD : kD * 2) + ((r & 7) << 4);
}

// The pool row of visible slot `i`, kNoRow past the last one or where the table names no page.
__device__ __forceinline__ uint32_t slot_row(const Pool& p, const int32_t* row, const Visible& vis, int h, int64_t i) {
  if (i >= vis.count) return kNoRow;
  const uint32_t slot = visible_slot(vis, static_cast<int32_t>(i)), pg = div_of(slot, p.ps);
  const uint32_t r = pool_row(__ldg(row + pg), p.n_pages, p.Hkv, h, p.ps.d, slot - pg * p.ps.d);
  if (r == kNoRow) tc::report_giveup(tc::kBadPage);
  return r;
}

// The same of numbered slot `i` of picked blocks; a block that is none of the row's counts as a bad page.
__device__ __forceinline__ uint32_t picked_row(const Pool& p, const int32_t* row, const Visible& vis, const int32_t* sel, int h, int64_t i) {
  if (i >= vis.count) return kNoRow;
  const uint32_t e = div_of(static_cast<uint32_t>(i), p.ps), in = static_cast<uint32_t>(i) - e * p.ps.d;
  const int32_t block = __ldg(sel + e);
  uint32_t r = kNoRow;
  if (static_cast<uint32_t>(block) <= div_of(static_cast<uint32_t>(vis.skip), p.ps)) {
    if (static_cast<int32_t>(block * p.ps.d + in) > vis.skip) return kNoRow;   // behind the row's position
    r = pool_row(__ldg(row + block), p.n_pages, p.Hkv, h, p.ps.d, in);
  }
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
    cp_async16_once(k_row<S::q8>(st, r) ^ (c << 4), kb + off, ok, policy);
    cp_async16_once(v_row<S::q8>(st + S::k_bytes, r) ^ (c << 4), vb + off, ok, policy);
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
// The codes in two bytes of x (`sel` puts them under 0x64) as an fp16 pair, exactly: 0x64cc is
// 1024 + c, and `bias` twice 1024, or 1152 for c - 128.
__device__ __forceinline__ uint32_t codes_f16(uint32_t x, uint32_t sel, uint32_t bias) {
  const uint32_t w = __byte_perm(x, 0x64646464u, sel);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// One tile: scores of its slots, the running softmax, and their values.
// `qf`: the queries as B fragments; `qsum`: INT8, sums of each query's two groups.
template <int TYPE, int NH>
__device__ __forceinline__ void consume(uint32_t st, const uint32_t (&qf)[kD / 16][NH][2], const float (&qsum)[NH][2][2], float scale,
                                        Acc<NH>& acc) {
  using S = Shape<TYPE>;
  constexpr int KT = S::tw / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const uint32_t mask = lds32(st + 2 * S::k_bytes + 2 * S::meta);
  // this lane's row and first piece of the keys (rows 8 and 16 apart swizzle alike)
  const uint32_t kr = S::q8 ? k_row<S::q8>(st, g) ^ ((lane & 3) << 4) : k_row<S::q8>(st, lane & 15) ^ ((lane >> 4) << 4);
  float s[KT][NH][4];   // slots 16 kt + g and + 8, heads as in Acc
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    if (!S::q8) {
      float d[NH][4] = {};
#pragma unroll
      for (int ks = 0; ks < kD / 16; ++ks) {
        uint32_t a[4];
        ldsm_x4((kr ^ (ks << 5)) + kt * 16 * S::row, a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) mma<TYPE>(d[nh], a, qf[ks][nh][0], qf[ks][nh][1]);
      }
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[kt][nh][j] = d[nh][j] * scale;
    } else {
      float d[2][NH][4] = {};
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        // 16 codes of slots g and g + 8; the channels' order is the queries' too
        const uint4 c0 = lds128((kr ^ (grp << 6)) + kt * 16 * S::row);
        const uint4 c1 = lds128((kr ^ (grp << 6)) + (kt * 16 + 8) * S::row);
        const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t a[4] = {codes_f16(w0[kk], 0x4140u, 0x64006400u), codes_f16(w1[kk], 0x4140u, 0x64006400u), codes_f16(w0[kk], 0x4342u, 0x64006400u),
                                 codes_f16(w1[kk], 0x4342u, 0x64006400u)};
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma<TYPE>(d[grp][nh], a, qf[grp * 4 + kk][nh][0], qf[grp * 4 + kk][nh][1]);
        }
      }
      const uint32_t ms = st + 2 * S::k_bytes + (kt * 16 + g) * kMetaBytes;
      const uint2 m[2] = {lds64(ms), lds64(ms + 8 * kMetaBytes)};
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint2 mm = m[j >> 1];
          s[kt][nh][j] = scale * (meta_s(mm.x) * d[0][nh][j] + meta_z(mm.x) * qsum[nh][j & 1][0] +
                                  (meta_s(mm.y) * d[1][nh][j] + meta_z(mm.y) * qsum[nh][j & 1][1]));
        }
    }
  }
  if (mask != (S::tw == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (!((mask >> (kt * 16 + g + 8 * (j >> 1))) & 1u)) s[kt][nh][j] = -INFINITY;
  }
  float sub[NH][2], alpha[NH][2];
  bool grew = false;
#pragma unroll
  for (int nh = 0; nh < NH; ++nh)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = fmaxf(s[0][nh][j], s[0][nh][j + 2]);
#pragma unroll
      for (int kt = 1; kt < KT; ++kt) mx = fmaxf(mx, fmaxf(s[kt][nh][j], s[kt][nh][j + 2]));
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(acc.m[nh][j], mx);
      // nothing seen yet: all weights are exp2(-inf) = 0
      alpha[nh][j] = mn == -INFINITY ? 0.f : ex2(acc.m[nh][j] - mn);
      sub[nh][j] = mn == -INFINITY ? 0.f : mn - S::shift;
      grew |= mn > acc.m[nh][j];
      acc.m[nh][j] = mn;
    }
  if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc.l[nh][j] *= alpha[nh][j];
        if (S::q8) {
          acc.z[nh][j][0] *= alpha[nh][j];
          acc.z[nh][j][1] *= alpha[nh][j];
        }
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt) {
          acc.o[mt][nh][j] *= alpha[nh][j];
          acc.o[mt][nh][j + 2] *= alpha[nh][j];
        }
      }
  }
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[kt][nh][j] = ex2(s[kt][nh][j] - sub[nh][j & 1]);
        acc.l[nh][j & 1] += s[kt][nh][j];
      }
  const uint32_t vr = S::q8 ? v_row<S::q8>(st + S::k_bytes, lane & 15) ^ ((lane >> 4) << 4)
                            : v_row<S::q8>(st + S::k_bytes, (lane & 7) + (lane >> 4) * 8) ^ (((lane >> 3) & 1) << 4);
  uint2 vm[KT][2];   // INT8: (scale, zero) of both groups of the values of slots 16 kt + g and + 8
  float vf[2] = {1.f, 1.f};
  if (S::q8) {
    __half2 top = __float2half2_rn(0.f);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        vm[kt][r] = lds64(st + 2 * S::k_bytes + S::meta + (kt * 16 + g + 8 * r) * kMetaBytes);
        const uint32_t sc = __byte_perm(vm[kt][r].x, vm[kt][r].y, 0x5410u);
        top = __hmax2(top, *reinterpret_cast<const __half2*>(&sc));
      }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) top = __hmax2(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float tops[2] = {__low2float(top), __high2float(top)};
#pragma unroll
    for (int grp = 0; grp < 2; ++grp) {
      if (tops[grp] > acc.cap[grp]) {   // the same in all lanes
        const float cap = __uint_as_float((__float_as_uint(tops[grp]) & 0x7f800000u) + 0x00800000u);   // the power of two above
        const float f = acc.cap[grp] / cap;
        acc.cap[grp] = cap;
#pragma unroll
        for (int mt = grp * 4; mt < grp * 4 + 4; ++mt)
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc.o[mt][nh][j] *= f;
      }
      vf[grp] = 32768.f / acc.cap[grp];
    }
  }
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    // weights as B fragments (slots x heads): pairs of heads, transposed into pairs of slots
    constexpr int G = S::q8 ? 2 : 1;   // INT8: one set per group of channels, scaled
    uint32_t hi[G][NH][2], lo[G][NH][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint2 m = S::q8 ? vm[kt][r] : make_uint2(0, 0);
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        const float sc = S::q8 ? meta_s(grp ? m.y : m.x) : 1.f;
        const float z = S::q8 ? fmaf(128.f, sc, meta_z(grp ? m.y : m.x)) : 0.f;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          const float p0 = s[kt][nh][2 * r], p1 = s[kt][nh][2 * r + 1];
          uint32_t h, l;
          split_pair<TYPE>(S::q8 ? p0 * (sc * vf[grp]) : p0, S::q8 ? p1 * (sc * vf[grp]) : p1, h, l);
          hi[grp][nh][r] = movmatrix_t(h);
          lo[grp][nh][r] = movmatrix_t(l);
          if (S::q8) {
            acc.z[nh][0][grp] += p0 * z;
            acc.z[nh][1][grp] += p1 * z;
          }
        }
      }
    }
    if (!S::q8) {
#pragma unroll
      for (int mt = 0; mt < kD / 16; ++mt) {
        uint32_t a[4];
        ldsm_x4_t((vr ^ (mt << 5)) + kt * 16 * S::row, a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          mma<TYPE>(acc.o[mt][nh], a, hi[0][nh][0], hi[0][nh][1]);
          mma<TYPE>(acc.o[mt][nh], a, lo[0][nh][0], lo[0][nh][1]);
        }
      }
    } else {
      // b16 pairs of codes, transposed: a word holds channels 2g, 2g + 1 of slots 2t and 2t + 1, so
      // row g of the product is channel 2g and row g + 8 channel 2g + 1
#pragma unroll
      for (int mt = 0; mt < kD / 16; mt += 2) {
        uint32_t x[4];
        ldsm_x4_t((vr ^ (mt << 4)) + kt * 16 * S::row, x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int grp = (mt + b) >> 2;
          constexpr uint32_t kBias = 0x64806480u;
          const uint32_t a[4] = {codes_f16(x[2 * b], 0x4240u, kBias), codes_f16(x[2 * b], 0x4341u, kBias),
                                 codes_f16(x[2 * b + 1], 0x4240u, kBias), codes_f16(x[2 * b + 1], 0x4341u, kBias)};
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            mma<TYPE>(acc.o[mt + b][nh], a, hi[grp][nh][0], hi[grp][nh][1]);
            mma<TYPE>(acc.o[mt + b][nh], a, lo[grp][nh][0], lo[grp][nh][1]);
          }
        }
      }
    }
  }
}

template <int TYPE>
__device__ __forceinline__ float lse_of(float m, float l) {
  return (m + (log2f(l) - Shape<TYPE>::shift)) * 0.6931471805599453f;
}
// Sum over the 8 lanes that share a column.
__device__ __forceinline__ float column_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Units of a row: one per key head and group of its query heads; picked blocks: a row has one key head.
template <bool SEL>
__device__ __forceinline__ int units_of(const AttendArgs& a) {
  return SEL ? a.groups : a.p.Hkv * a.groups;
}
// The first query head of unit u of row b, counted through all rows of q, and the heads of the unit.
template <bool SEL>
__device__ __forceinline__ size_t head_of(const AttendArgs& a, int b, int u) {
  if (SEL) return static_cast<size_t>(b) * a.rep + u * a.heads;   // row b / Hkv, key head b % Hkv
  return static_cast<size_t>(b) * a.Hq + u / a.groups * a.rep + u % a.groups * a.heads;
}
__device__ __forceinline__ int heads_of(const AttendArgs& a, int u) { return min(a.heads, a.rep - u % a.groups * a.heads); }

// A warp's place in the line of tiles: tile t of `tiles` of unit u of row b.
struct Cursor {
  int b, u, t, tiles;
  int32_t seq;
  Visible vis;
};
template <int TYPE, bool SEL>
__device__ __forceinline__ void open_row(const AttendArgs& a, Cursor& c) {   // the first row from c.b on that has tiles
  for (;; ++c.b) {
    c.vis = row_visible<SEL>(a, c.b, c.seq);
    c.tiles = (c.vis.count + Shape<TYPE>::tw - 1) / Shape<TYPE>::tw;
    if (c.tiles > 0) return;
  }
}
// To the next unit; the caller knows that there is one.
template <int TYPE, bool SEL>
__device__ __forceinline__ void next_unit(const AttendArgs& a, Cursor& c) {
  c.t = 0;
  if (++c.u == units_of<SEL>(a)) {
    c.u = 0;
    ++c.b;
    open_row<TYPE, SEL>(a, c);
  }
}

// Writes a finished unit, or a part of one for the join (`part` not null).
template <int TYPE, int NH, bool SEL>
__device__ __forceinline__ void store_unit(const AttendArgs& a, int b, int u, Acc<NH>& acc, float* part) {
  using S = Shape<TYPE>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rows = heads_of(a, u);
  const size_t at = head_of<SEL>(a, b, u);
#pragma unroll
  for (int nh = 0; nh < NH; ++nh) {
    float l[2], inv[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      l[j] = column_sum(acc.l[nh][j]);
      if (S::q8) {
#pragma unroll
        for (int grp = 0; grp < 2; ++grp) {
          const float z = column_sum(acc.z[nh][j][grp]);
#pragma unroll
          for (int mt = grp * 4; mt < grp * 4 + 4; ++mt) {
            acc.o[mt][nh][j] = fmaf(acc.o[mt][nh][j], acc.cap[grp] * (1.f / 32768.f), z);
            acc.o[mt][nh][j + 2] = fmaf(acc.o[mt][nh][j + 2], acc.cap[grp] * (1.f / 32768.f), z);
          }
        }
      }
      inv[j] = l[j] == 0.f ? 0.f : 1.f / l[j];   // all pages bad: nothing seen
      const int row = nh * 8 + 2 * t + j;
      if (g == 0 && row < rows) {
        if (part) {
          part[kPaRows * kD + row] = acc.m[nh][j];
          part[kPaRows * kD + kPaRows + row] = l[j];
        } else if (a.lse) {
          a.lse[at + row] = lse_of<TYPE>(acc.m[nh][j], l[j]);
        }
      }
    }
    if (part) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = nh * 8 + 2 * t + j;
        if (row >= rows) continue;
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt) {
          float* dst = part + row * kD + mt * 16;
          if (S::q8) {
            *reinterpret_cast<float2*>(dst + 2 * g) = make_float2(acc.o[mt][nh][j], acc.o[mt][nh][j + 2]);
          } else {
            dst[g] = acc.o[mt][nh][j];
            dst[g + 8] = acc.o[mt][nh][j + 2];
          }
        }
      }
    } else {
      const int row = nh * 8 + g;   // after the transposition
      uint16_t* dst = a.out + (at + row) * kD;
#pragma unroll
      for (int mt = 0; mt < kD / 16; ++mt) {
        const float* o = acc.o[mt][nh];
        const uint32_t x0 = static_cast<uint32_t>(to_out<TYPE>(o[0] * inv[0])) | static_cast<uint32_t>(to_out<TYPE>(o[1] * inv[1])) << 16;
        const uint32_t x1 = static_cast<uint32_t>(to_out<TYPE>(o[2] * inv[0])) | static_cast<uint32_t>(to_out<TYPE>(o[3] * inv[1])) << 16;
        const uint32_t y0 = movmatrix_t(x0), y1 = movmatrix_t(x1);   // head g, rows 2t, 2t + 1 (and + 8) of the product
        if (row >= rows) continue;
        if (S::q8) {
          *reinterpret_cast<uint2*>(dst + mt * 16 + 4 * t) = make_uint2(__byte_perm(y0, y1, 0x5410u), __byte_perm(y0, y1, 0x7632u));
        } else {
          *reinterpret_cast<uint32_t*>(dst + mt * 16 + 2 * t) = y0;
          *reinterpret_cast<uint32_t*>(dst + mt * 16 + 8 + 2 * t) = y1;
        }
      }
    }
  }
}

template <int TYPE, int NH, bool SEL>
__global__ void __launch_bounds__(kPaThreads, kPaCtasPerSM) paged_partial_kernel(const AttendArgs a) {
  using S = Shape<TYPE>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sums[kPaWarps];
  __shared__ int64_t s_incl[kPaThreads];
  pdl_trigger();
  const Pool& p = a.p;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int units = units_of<SEL>(a);
  // this warp's part of the line of tiles, and the row it begins in; consecutive parts lie on
  // different SMs, so that a few of them do not share one
  int64_t mine = tid < a.n ? row_tiles<S::tw, SEL>(a, tid) : 0, total;
  const int64_t head = mine;
  for (int b = tid + kPaThreads; b < a.n; b += kPaThreads) mine += row_tiles<S::tw, SEL>(a, b);
  int64_t incl = scan64(mine * units, warp_sums, total);
  if (total == 0) return;   // nothing is seen: the join answers
  const int workers = workers_of(total, gridDim.x * kPaWarps), c = w * gridDim.x + blockIdx.x;
  const int64_t begin = split_begin(total, workers, c), end = split_begin(total, workers, c + 1);
  const bool idle = c >= workers;
  Cursor at;
  at.b = -1;
  int64_t pass = 0, base = 0;   // tiles before this pass's rows (all warps alike), and before this warp's row
  for (int b0 = 0; b0 < a.n; b0 += kPaThreads) {
    int64_t sum = total;
    if (a.n > kPaThreads) {
      const int b = b0 + tid;
      const int64_t v = b0 == 0 ? head : b < a.n ? row_tiles<S::tw, SEL>(a, b) : 0;
      incl = pass + scan64(v * units, warp_sums, sum);
    }
    __syncthreads();   // the last pass's sums have been read
    s_incl[tid] = incl;
    __syncthreads();
    if (!idle && at.b < 0 && begin < pass + sum) {
      int below = 0;   // rows of this pass that end at or before `begin`
#pragma unroll
      for (int i = 0; i < kPaThreads; i += 32) below += __popc(__ballot_sync(0xffffffffu, s_incl[i + lane] <= begin));
      at.b = b0 + below;
      base = below ? s_incl[below - 1] : pass;
    }
    pass += sum;
    if (__syncthreads_and(idle || at.b >= 0)) break;
  }
  if (idle) return;
  const int n = static_cast<int>(end - begin);   // tiles of this warp: below 2^31 / tw a row, far fewer a warp
  open_row<TYPE, SEL>(a, at);
  at.u = static_cast<int>((begin - base) / at.tiles);
  at.t = static_cast<int>((begin - base) % at.tiles);

  const uint32_t ring = ((smem_u32(smem) + 255u) & ~255u) + w * S::stages * S::stage;
  const size_t lrow = p.layer_rows() * a.layer;
  const uint64_t policy = l2_evict_first_policy();
  Cursor ahead = at;   // the next tile to be requested
  int asked = 0;
  // the pool row of this lane's slot of that tile, and on to the next one
  const auto find = [&] {
    uint32_t r = kNoRow;
    if (asked < n) {
      const int32_t* table = p.table + static_cast<size_t>(ahead.seq) * p.max_pages;
      const int64_t i = static_cast<int64_t>(ahead.t) * S::tw + lane;
      if (lane < S::tw)
        r = SEL ? picked_row(p, table, ahead.vis, a.sel + static_cast<size_t>(ahead.b) * a.keep, ahead.b % p.Hkv, i)
                : slot_row(p, table, ahead.vis, ahead.u / a.groups, i);
      if (++ahead.t == ahead.tiles && asked + 1 < n) next_unit<TYPE, SEL>(a, ahead);
      ++asked;
    }
    return r;
  };
#pragma unroll
  for (int i = 0; i < S::stages - 1; ++i) {
    const uint32_t r = find();
    if (i < n) issue<TYPE>(p, lrow, ring + i * S::stage, r, policy);
    cp_async_commit();
  }
  uint32_t next = find();
  int rd = 0, wr = S::stages - 1, left = n;
  bool first = true;
  while (left > 0) {
    const size_t head0 = head_of<SEL>(a, at.b, at.u);
    const int rows = heads_of(a, at.u);
    // the queries as B fragments (INT8: channels in the order the codes are read)
    uint32_t qf[kD / 16][NH][2];
    float qsum[NH][2][2] = {};
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int ch = S::q8 ? 64 * (ks >> 2) + 16 * t + 4 * (ks & 3) + 2 * j : 16 * ks + 8 * j + 2 * t;
          uint32_t x = 0;
          if (nh * 8 + g < rows)
            x = *reinterpret_cast<const uint32_t*>(a.q + (head0 + nh * 8 + g) * kD + ch);
          qf[ks][nh][j] = x;
          if (S::q8) {
            const __half2 x2 = *reinterpret_cast<const __half2*>(&x);
            sum[ks >> 2] += __low2float(x2) + __high2float(x2);
          }
        }
      if (S::q8) {
#pragma unroll
        for (int grp = 0; grp < 2; ++grp) {
          float x = sum[grp];   // of head g, this lane's channels
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          qsum[nh][0][grp] = __shfl_sync(0xffffffffu, x, 8 * t);       // heads 2t, 2t + 1
          qsum[nh][1][grp] = __shfl_sync(0xffffffffu, x, 8 * t + 4);
        }
      }
    }
    Acc<NH> acc;
    acc.cap[0] = acc.cap[1] = 0x1p-26f;   // below every fp16 number but 0
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
      for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc.o[mt][nh][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc.m[nh][j] = -INFINITY;
        acc.l[nh][j] = acc.z[nh][j][0] = acc.z[nh][j][1] = 0.f;
      }
    }
    const int count = min(at.tiles - at.t, left);
    for (int i = 0; i < count; ++i) {
      cp_async_wait<S::stages - 2>();
      __syncwarp();   // the tile has landed for all lanes, and the one to be refilled is read
      if (left - i > S::stages - 1) issue<TYPE>(p, lrow, ring + wr * S::stage, next, policy);
      cp_async_commit();
      next = find();
      consume<TYPE, NH>(ring + rd * S::stage, qf, qsum, a.scale, acc);
      rd = rd + 1 == S::stages ? 0 : rd + 1;
      wr = wr + 1 == S::stages ? 0 : wr + 1;
    }
    const bool whole = count == at.tiles;
    store_unit<TYPE, NH, SEL>(a, at.b, at.u, acc, whole ? nullptr : a.part + (static_cast<size_t>(c) * 2 + (first ? 0 : 1)) * kPartFloats);
    first = false;
    left -= count;
    if (left > 0) next_unit<TYPE, SEL>(a, at);
  }
}

// One partial result of a query head: maximum, sum, four channels of the lane.
struct Part {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float mb, float lb, const float4& ob) {
    const float mn = fmaxf(m, mb), sub = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - sub), fb = ex2(mb - sub);
    l = l * f + lb * fb;
    o = make_float4(o.x * f + ob.x * fb, o.y * f + ob.y * fb, o.z * f + ob.z * fb, o.w * f + ob.w * fb);
    m = mn;
  }
};

// CTA (unit, row b, query head, or four heads where WARPS is 1): joins the parts of a unit that several
// warps held, in a fixed order, and answers for the units without a visible slot.  Four channels
// a lane; WARPS warps share a head, each with every WARPS-th part, BATCH of them requested together.
template <int TYPE, int WARPS, int BATCH, bool SEL>
__global__ void __launch_bounds__(WARPS > 1 ? WARPS * 32 : kPaThreads) paged_merge_kernel(const AttendArgs a, int warps) {
  using S = Shape<TYPE>;
  constexpr int W = WARPS > 1 ? WARPS : kPaWarps;   // warps of the CTA
  __shared__ int64_t warp_sums[W];
  __shared__ float4 s_o[W][32];
  __shared__ float2 s_ml[W];
  const int units = units_of<SEL>(a), b = blockIdx.y, u = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = heads_of(a, u);
  int64_t mine = 0, below = 0, total, base;
  for (int i = tid; i < a.n; i += W * 32) {
    const int x = row_tiles<S::tw, SEL>(a, i);
    mine += x;
    if (i < b) below += x;
  }
  scan64<W>(mine * units, warp_sums, total);
  scan64<W>(below * units, warp_sums, base);
  const int tiles = row_tiles<S::tw, SEL>(a, b);
  const int workers = workers_of(total, warps);
  const int64_t first = base + static_cast<int64_t>(u) * tiles;
  const int c0 = tiles ? split_owner(total, workers, first) : 0, c1 = tiles ? split_owner(total, workers, first + tiles - 1) : -1;
  const int skip = tiles && split_begin(total, workers, c0) < first ? 1 : 0;   // c0 holds it as its second part
  pdl_wait();
  if (tiles > 0 && c0 == c1) return;   // finished by its warp
  const int row = WARPS > 1 ? blockIdx.z : blockIdx.z * kPaWarps + warp;   // the query head of the group
  if (row < rows) {
    Part sum = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int cb = c0 + (WARPS > 1 ? warp : 0); cb <= c1; cb += BATCH * WARPS) {
      float m[BATCH], l[BATCH];
      float4 o[BATCH];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int c = cb + e * WARPS;
        m[e] = -INFINITY;
        l[e] = 0.f;
        o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c <= c1) {
          const float* q = a.part + (static_cast<size_t>(c) * 2 + (c == c0 ? skip : 0)) * kPartFloats;
          m[e] = q[kPaRows * kD + row];
          l[e] = q[kPaRows * kD + kPaRows + row];
          o[e] = reinterpret_cast<const float4*>(q + row * kD)[lane];
        }
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) sum.add(m[e], l[e], o[e]);
    }
    if (WARPS > 1) {
      s_o[warp][lane] = sum.o;
      if (lane == 0) s_ml[warp] = make_float2(sum.m, sum.l);
      __syncthreads();
      if (warp != 0) return;
#pragma unroll
      for (int e = 1; e < WARPS; ++e) sum.add(s_ml[e].x, s_ml[e].y, s_o[e][lane]);
    }
    const size_t at = head_of<SEL>(a, b, u) + row;
    const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
    *reinterpret_cast<uint2*>(a.out + at * kD + 4 * lane) =
        make_uint2(static_cast<uint32_t>(to_out<TYPE>(sum.o.x * inv)) | static_cast<uint32_t>(to_out<TYPE>(sum.o.y * inv)) << 16,
                   static_cast<uint32_t>(to_out<TYPE>(sum.o.z * inv)) | static_cast<uint32_t>(to_out<TYPE>(sum.o.w * inv)) << 16);
    if (lane == 0 && a.lse) a.lse[at] = lse_of<TYPE>(sum.m, sum.l);
  }
}

// Tiles of the longest unit that the table can hold, and of one that has all its `keep` blocks.
int64_t tiles_in(const mikv_pages* p, int64_t slots) {
  const int tile = p->type == MIKV_PAGES_INT8 ? Shape<MIKV_PAGES_INT8>::tw : Shape<MIKV_PAGES_FP16>::tw;
  return (slots + tile - 1) / tile;
}
int64_t tiles_of(const mikv_pages* p, int window, int sinks) {
  int64_t slots = static_cast<int64_t>(p->max_pages) * p->page_size;
  if (window > 0) slots = std::min(slots, static_cast<int64_t>(window) + sinks);
  return tiles_in(p, slots);
}
int64_t picked_tiles(const mikv_pages* p, int keep) {
  return tiles_in(p, static_cast<int64_t>(std::min(keep, p->max_pages)) * p->page_size);
}
// CTAs of the split: two per SM, or one a tile where that is fewer (one of its warps then has the
// tile, so that few tiles lie on as many SMs).
int grid_of(const mikv_pages* p, int n, int Hq, int64_t tiles) {
  const int rep = Hq / p->Hkv, groups = (rep + kPaRows - 1) / kPaRows;
  const int64_t most = static_cast<int64_t>(kPaCtasPerSM) * kNumSMs;
  return static_cast<int>(std::max<int64_t>(1, std::min(most, tiles * n * p->Hkv * groups)));
}
size_t part_bytes(int grid) { return static_cast<size_t>(grid) * kPaWarps * 2 * kPartFloats * sizeof(float); }

template <int TYPE, int NH, bool SEL>
int launch(const AttendArgs& a, int grid, int64_t tiles, cudaStream_t st) {
  const auto kern = paged_partial_kernel<TYPE, NH, SEL>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<TYPE>::smem);
  if (e != cudaSuccess) return check_launch_after(e, "paged_partial_kernel");
  kern<<<grid, kPaThreads, Shape<TYPE>::smem, st>>>(a);
  if (int r = check_launch("paged_partial_kernel")) return r;
  // Parts that a unit has where all are of one length, and the warps that join a head: one sequence
  // of 65536 slots and one key head, 1216 parts: 661 us with one warp a head, 68 with four, 22 with
  // 16; 16 sequences of 2048 and 8 key heads, 9 parts: 30, 27 and 35 us; one of 77 and 8 key heads, five
  // parts, in a graph: 5.8 us with four, 6.5 with 16.
  const int units = SEL ? a.groups : a.p.Hkv * a.groups;
  const int64_t parts = parts_of_unit(tiles, static_cast<int64_t>(units) * a.n, grid * kPaWarps);
  const int64_t joins = static_cast<int64_t>(units) * a.n * a.heads;   // CTAs of the two wider forms
  const bool many = parts >= 16 && joins <= 2 * kNumSMs, some = !many && parts >= 5 && joins <= 8 * kNumSMs;
  const auto merge = many   ? paged_merge_kernel<TYPE, kMergeWarps, 8, SEL>
                     : some ? paged_merge_kernel<TYPE, kPaWarps, 8, SEL>
                            : paged_merge_kernel<TYPE, 1, 4, SEL>;
  return check_launch_after(launch_after(merge, dim3(units, a.n, many || some ? a.heads : (a.heads + kPaWarps - 1) / kPaWarps),
                                         dim3(many ? kMergeWarps * 32 : kPaThreads), 0, st, a, grid * kPaWarps),
                            "paged_merge_kernel");
}

// What both calls set; the rest is none.
void fill_args(AttendArgs& a, const void* q, int layer, int n, int Hq, void* out, float* lse, void* ws) {
  a.q = static_cast<const uint16_t*>(q);
  a.layer = layer;
  a.n = n;
  a.Hq = Hq;
  a.rep = Hq / a.p.Hkv;
  a.groups = (a.rep + kPaRows - 1) / kPaRows;
  a.heads = (a.rep + a.groups - 1) / a.groups;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.scale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
  a.seqs = a.row_seq = a.row_pos = a.sel = a.n_sel = nullptr;
  a.window = a.sinks = a.keep = 0;
}

template <bool SEL>
int dispatch(const AttendArgs& a, int grid, int64_t tiles, cudaStream_t st) {
  const bool wide = a.heads > 8;
  switch (a.p.type) {
    case MIKV_PAGES_FP16: return wide ? launch<MIKV_PAGES_FP16, 2, SEL>(a, grid, tiles, st) : launch<MIKV_PAGES_FP16, 1, SEL>(a, grid, tiles, st);
    case MIKV_PAGES_BF16: return wide ? launch<MIKV_PAGES_BF16, 2, SEL>(a, grid, tiles, st) : launch<MIKV_PAGES_BF16, 1, SEL>(a, grid, tiles, st);
    default: return wide ? launch<MIKV_PAGES_INT8, 2, SEL>(a, grid, tiles, st) : launch<MIKV_PAGES_INT8, 1, SEL>(a, grid, tiles, st);
  }
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_paged_attention_workspace_bytes(const mikv_pages* p, int n, int Hq, int window, int sinks) {
  Pool pool;
  if (check_pages(p, "paged_attention", &pool) || n < 1 || n > 65535 || Hq < 1 || Hq % p->Hkv || window < 0 || sinks < 0) return 0;
  return part_bytes(grid_of(p, n, Hq, tiles_of(p, window, sinks)));
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
  const int64_t tiles = tiles_of(pages, window, sinks);
  const int grid = grid_of(pages, n, Hq, tiles);
  const size_t need = part_bytes(grid);
  if (ws_bytes < need) return fail(MIKV_ESHAPE, "paged_attention: workspace %zu < %zu", ws_bytes, need);
  fill_args(a, q, layer, n, Hq, out, lse, ws);
  a.seqs = seqs;
  a.window = window;
  a.sinks = sinks;
  return dispatch<false>(a, grid, tiles, as_stream(stream));
}

extern "C" size_t mikv_block_attention_workspace_bytes(const mikv_pages* p, int rows, int Hq, int keep) {
  Pool pool;
  if (check_pages(p, "block_attention", &pool) || rows < 1 || static_cast<int64_t>(rows) * p->Hkv > 65535 || Hq < 1 || Hq % p->Hkv ||
      keep < 1)
    return 0;
  return part_bytes(grid_of(p, rows, Hq, picked_tiles(p, keep)));
}

extern "C" int mikv_block_attention(const void* q, const mikv_pages* pages, int layer, const int32_t* row_seq, const int32_t* row_pos,
                                    const int32_t* sel, const int32_t* n_sel, int rows, int Hq, int keep, void* out, float* lse, void* ws,
                                    size_t ws_bytes, void* stream) {
  clear_error();
  AttendArgs a;
  if (int e = check_pages(pages, "block_attention", &a.p)) return e;
  if (layer < 0 || layer >= a.p.layers) return fail(MIKV_ESHAPE, "block_attention: layer=%d of %d", layer, a.p.layers);
  if (rows < 0 || static_cast<int64_t>(rows) * a.p.Hkv > 65535 || (!row_seq && rows > a.p.max_seqs))
    return fail(MIKV_ESHAPE, "block_attention: rows=%d Hkv=%d", rows, a.p.Hkv);
  if (Hq < 1 || Hq % a.p.Hkv || Hq / a.p.Hkv > 1024) return fail(MIKV_ESHAPE, "block_attention: Hq=%d Hkv=%d", Hq, a.p.Hkv);
  if (keep < 1 || static_cast<int64_t>(keep) * pages->page_size > 0x7fffffffLL - 4096)
    return fail(MIKV_ESHAPE, "block_attention: keep=%d blocks of %d", keep, pages->page_size);
  if (rows == 0) return MIKV_OK;
  if (!q || !sel || !n_sel || !out || !ws) return fail(MIKV_EINVAL, "block_attention: null pointer");
  if (!aligned16(q) || !aligned16(out) || !aligned16(ws)) return fail(MIKV_EALIGN, "block_attention: 16-byte alignment");
  const int64_t tiles = picked_tiles(pages, keep);
  const int grid = grid_of(pages, rows, Hq, tiles);
  const size_t need = part_bytes(grid);
  if (ws_bytes < need) return fail(MIKV_ESHAPE, "block_attention: workspace %zu < %zu", ws_bytes, need);
  fill_args(a, q, layer, rows * a.p.Hkv, Hq, out, lse, ws);
  a.row_seq = row_seq;
  a.row_pos = row_pos;
  a.sel = sel;
  a.n_sel = n_sel;
  a.keep = keep;
  return dispatch<true>(a, grid, tiles, as_stream(stream));
}
