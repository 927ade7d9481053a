// The blocks of its sequence that each row of a packed batch reads, by a score of the keys' bounds.
//
// Mathematics: a query's codes are c = rint(fl(q / s_q)) with s_q = fl(max |q| / 127).  A block's keys
// lie between s_b lo and s_b hi (page_bounds.cu), so no logit of the block exceeds, up to the
// codes' rounding, s_q s_b u / sqrt(D) with the whole number
//   u = sum_c max(c_c lo_c, c_c hi_c) = sum_{c > 0} c_c hi_c + sum_{c < 0} c_c lo_c,
// |u| <= 128 * 127 * 127 < 2^24: u is exact in 32 bits whatever the order of the sum, and the score
// fl(fl(u s_b) s_q) is the same to the bit wherever it is computed, so that the choice is too.  The
// heads of a group read one set of blocks: a block's score is the largest of theirs.
//
// Up to three kernels: the queries' codes, in the order in which the products take them, once a (row, key head), where there
// are many warps that would make them anew; scores of all blocks (bound by HBM: 260 bytes a block and key head; mma.sync on
// fp16 numbers, which hold the codes exactly, as fp32 does the sums, with 16 blocks as its M and 8 query heads as its N;
// four-term integer products took 34 us, 8-bit matrix instructions 37, for 192 units of up to 4096 blocks), and the choice of the `keep` best of each (row, key head), written in the
// blocks' order.  The choice is a search by digits of the scores' bits, but of digits that begin below what all
// of a unit's scores share: scores of one unit lie close together, and counters of their first bits would all be hit at once.
#include <cuda_bf16.h>

#include <algorithm>

#include "block_index.h"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int block_select_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kBsWarps = 4;
constexpr int kBsSteps = 2;                    // of 32 blocks a warp, each with a buffer of its own: all are under way at once
constexpr int kBsBlocks = 32 * kBsSteps;       // blocks of a warp
constexpr int kBsHeads = 8;                    // query heads of a pass
constexpr int kBsSmem = kBsWarps * kBsSteps * 32 * 2 * kD;
static_assert(kBoundBytes == 2 * kD, "bounds of a block");
constexpr int kPickThreads = 512;
constexpr int kPickDigit = 11;                    // bits of a digit
constexpr uint32_t kAlways = 0xffffffffu;   // above every score

struct SelectArgs {
  Pool p;
  const uint16_t* q;
  const int8_t* bounds;
  const float* scales;
  const int32_t *row_seq, *row_pos;
  int layer, rows, rep, keep, first, recent;
  int chunks;            // warps of a (row, key head)
  int64_t warps;         // of all
  int32_t *sel, *n_sel;
  uint32_t* keys;        // [rows][Hkv][max_pages]: scores in the order of whole numbers
  uint4* codes;          // [rows][Hkv][groups][8][32]: the queries' codes by lanes; behind them fp32 scales [rows][Hkv][groups][8]
  int groups;            // of kBsHeads query heads
};

// Blocks that row r can read: all that hold a position up to its own; 0 for a row without a sequence.
__device__ __forceinline__ int32_t blocks_of_row(const SelectArgs& a, int r, int32_t& seq) {
  seq = a.row_seq ? a.row_seq[r] : r;
  if (static_cast<uint32_t>(seq) >= static_cast<uint32_t>(a.p.max_seqs)) return 0;
  const int32_t len = a.p.len_of(seq);
  const int32_t last = a.row_pos ? min(a.row_pos[r], len - 1) : len - 1;
  return pages_of(last + 1, a.p.ps);   // 0 where last < 0
}

__device__ __forceinline__ float to_float(uint32_t h, bool bf) {
  return bf ? __uint_as_float(h << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}
// A number's bits in the order of whole numbers; -0 counts as 0, what is no number as +infinity.
__device__ __forceinline__ uint32_t ordered(float x) {
  x = isnan(x) ? INFINITY : x + 0.f;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Two codes of x (the bytes' first bits turned over, `sel` puts them under 0x64) as an fp16 pair: 0x64cc is 1024 + cc.
__device__ __forceinline__ uint32_t codes_f16(uint32_t x, uint32_t sel) {
  const uint32_t w = __byte_perm(x, 0x64646464u, sel);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float* query_scales(const SelectArgs& a, int unit, int group) {
  float* s = reinterpret_cast<float*>(a.codes + static_cast<size_t>(a.rows) * a.p.Hkv * a.groups * 256);
  return s + (static_cast<size_t>(unit) * a.groups + group) * kBsHeads;
}
// The codes of query heads g0 .. of one (row, key head), by a warp: lane 4 g + t has those of head g0 + g, channels
// 64 k + 16 t .. + 15, in the order in which those of the blocks are read: below 0 (met by lo), then above (by hi).
__device__ __forceinline__ void query_codes(const SelectArgs& a, int unit, int g0, uint32_t (&q)[16][2], float& sq) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool bf = a.p.type == MIKV_PAGES_BF16;
  const bool there = g0 + g < a.rep;
  {
    uint4 v[2][2];
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[k][e] = make_uint4(0, 0, 0, 0);
        if (there)
          v[k][e] = reinterpret_cast<const uint4*>(a.q + (static_cast<size_t>(unit) * a.rep + g0 + g) * kD)[8 * k + 2 * t + e];
      }
    const auto word = [&](int k, int c) {   // channels 2 c, 2 c + 1 of the lane's 16
      const uint4& x = v[k][c >> 2];
      return (c & 3) == 0 ? x.x : (c & 3) == 1 ? x.y : (c & 3) == 2 ? x.z : x.w;
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = fabsf(to_float(word(k, c) >> (16 * e) & 0xffffu, bf));
          top = fmaxf(top, x);
          bad |= !(x <= 3.402823466e38f);
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      bad |= __shfl_xor_sync(0xffffffffu, static_cast<int>(bad), o) != 0;
    }
    sq = bad ? INFINITY : __fdiv_rn(top, 127.f);   // no finite query: its scores are 0 * infinity
    // A product with the reciprocal is within 2^-15 of the quotient, so both round to the same whole number unless the
    // product lies that near to a half: then, and where the reciprocal is no finite number, the division decides.
    const bool some = !bad && sq > 0.f;
    const float inv = some ? __frcp_rn(sq) : 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v0 = to_float(word(k, c) >> (16 * e) & 0xffffu, bf), p = __fmul_rn(v0, inv);
          float r = rintf(p);
          if (!(fabsf(p - r) < 0.49f)) r = rintf(__fdiv_rn(v0, sq));
          x[e] = some ? fminf(fmaxf(r, -127.f), 127.f) : 0.f;
        }
        q[4 * k + (c >> 1)][c & 1] = pack_half2(__float2half_rn(fminf(x[0], 0.f)), __float2half_rn(fminf(x[1], 0.f)));
        q[8 + 4 * k + (c >> 1)][c & 1] = pack_half2(__float2half_rn(fmaxf(x[0], 0.f)), __float2half_rn(fmaxf(x[1], 0.f)));
      }
  }
}
__global__ void __launch_bounds__(kBsWarps * 32) block_query_kernel(const SelectArgs a) {
  const int lane = threadIdx.x & 31;
  pdl_trigger();
  const int id = blockIdx.x * kBsWarps + (threadIdx.x >> 5);
  if (id >= a.rows * a.p.Hkv * a.groups) return;
  const int unit = id / a.groups, g0 = (id - unit * a.groups) * kBsHeads;
  uint32_t q[16][2];
  float sq;
  query_codes(a, unit, g0, q, sq);
  uint4* codes = a.codes + static_cast<size_t>(id) * 256 + lane;
#pragma unroll
  for (int e = 0; e < 8; ++e) codes[e * 32] = make_uint4(q[2 * e][0], q[2 * e][1], q[2 * e + 1][0], q[2 * e + 1][1]);
  if ((lane & 3) == 0) query_scales(a, unit, g0 / kBsHeads)[lane >> 2] = sq;
}

// A warp: kBsBlocks blocks of one (row, key head), 32 a step; the warps of a CTA have the heads of the same blocks side by
// side, whose bounds lie side by side.  OWN: it makes the queries' codes itself.
template <bool OWN>
__global__ void __launch_bounds__(kBsWarps * 32) block_score_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint4 s_b[];   // [warp][step][32 blocks][16 pieces], swizzled by the block
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  pdl_trigger();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kBsWarps + w;
  // (who has nothing to do waits too: the grid is not done before the one before it)
  const auto leave = [] {
    if (!OWN) pdl_wait();
  };
  if (id >= a.warps) return leave();
  const int64_t rest = id / a.p.Hkv;
  const int h = static_cast<int>(id - rest * a.p.Hkv), r = static_cast<int>(rest / a.chunks);
  const int b0 = static_cast<int>(rest - static_cast<int64_t>(r) * a.chunks) * kBsBlocks;
  int32_t seq = a.row_seq ? a.row_seq[r] : r, page[kBsSteps];
  if (static_cast<uint32_t>(seq) >= static_cast<uint32_t>(a.p.max_seqs)) return leave();
  const int32_t* table = a.p.table + static_cast<size_t>(seq) * a.p.max_pages;
#pragma unroll
  for (int i = 0; i < kBsSteps; ++i)   // asked for beside the length that tells whether they count
    page[i] = b0 + 32 * i + lane < a.p.max_pages ? table[b0 + 32 * i + lane] : -1;
  const int32_t nb = blocks_of_row(a, r, seq);
  if (b0 >= nb || nb <= a.keep) return leave();
  const int unit = r * a.p.Hkv + h;
  const size_t layer0 = static_cast<size_t>(a.layer) * a.p.n_pages * a.p.Hkv;
  const int steps = min(kBsSteps, (nb - b0 + 31) / 32);
  const uint32_t buffers = smem_u32(s_b) + w * (kBsSteps * 32 * 2 * kD);
  uint32_t at[kBsSteps];   // (page, key head) of the lane's block, kNoRow without one
#pragma unroll
  for (int i = 0; i < kBsSteps; ++i) {
    const bool ok = b0 + 32 * i + lane < nb && a.p.has(page[i]);
    at[i] = ok ? static_cast<uint32_t>(page[i]) * a.p.Hkv + h : kNoRow;   // (below 2^32, like the pool's rows)
  }
  const auto fetch = [&](int i, uint32_t from) {
    const uint32_t dst = buffers + i * (32 * 2 * kD);
#pragma unroll
    for (int j = 0; j < 16; ++j) {   // two blocks an instruction
      const int e = 2 * j + (lane >> 4), piece = lane & 15;
      const uint32_t src = __shfl_sync(0xffffffffu, from, e);
      const bool ok = src != kNoRow;
      cp_async16(dst + bound_at(e, piece), a.bounds + (layer0 + (ok ? src : 0)) * (2 * kD) + piece * 16, ok);
    }
  };
  float best[kBsSteps];
#pragma unroll
  for (int i = 0; i < kBsSteps; ++i) best[i] = -INFINITY;
  float sb[kBsSteps];
#pragma unroll
  for (int i = 0; i < kBsSteps; ++i) sb[i] = at[i] != kNoRow ? a.scales[layer0 + at[i]] : 0.f;
  for (int g0 = 0; g0 < a.rep; g0 += kBsHeads) {
#pragma unroll
    for (int i = 0; i < kBsSteps; ++i) {
      if (i < steps) fetch(i, at[i]);
      cp_async_commit();
    }
    uint32_t q[16][2];
    float sq;
    if (OWN) {
      query_codes(a, unit, g0, q, sq);
    } else {
      if (g0 == 0) pdl_wait();   // the codes are there
      const uint4* codes = a.codes + (static_cast<size_t>(unit) * a.groups + g0 / kBsHeads) * 256 + lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint4 x = codes[e * 32];
        q[2 * e][0] = x.x;
        q[2 * e][1] = x.y;
        q[2 * e + 1][0] = x.z;
        q[2 * e + 1][1] = x.w;
      }
      sq = query_scales(a, unit, g0 / kBsHeads)[g];
    }
    // scales of the heads whose sums this lane holds
    const float s2[2] = {__shfl_sync(0xffffffffu, sq, 8 * t), __shfl_sync(0xffffffffu, sq, 8 * t + 4)};
#pragma unroll
    for (int i = 0; i < kBsSteps; ++i) {
      if (i >= steps) break;
      static_assert(kBsSteps == 2, "the first step's copies, then all");
      if (i == 0)
        cp_async_wait<1>();
      else
        cp_async_wait<0>();
      __syncwarp();
      const uint32_t src = buffers + i * (32 * 2 * kD);
      float top[2][2];   // blocks 16 mt + g and + 8
      float d[2][2][4] = {};   // two sums each, so that products wait for one another less (whole numbers: any order gives the same)
      const uint32_t at_lane = bound_at(g, t);
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // 64 codes: of lo, lo, hi, hi
        uint4 x[2][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e >> 1][e & 1] = lds128(src + bound_of_lane(at_lane, e, k));
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint4 &y0 = x[mt][0], &y1 = x[mt][1];
            const uint32_t u0 = (s == 0 ? y0.x : s == 1 ? y0.y : s == 2 ? y0.z : y0.w) ^ 0x80808080u;
            const uint32_t u1 = (s == 0 ? y1.x : s == 1 ? y1.y : s == 2 ? y1.z : y1.w) ^ 0x80808080u;
            mma16816(d[mt][s & 1], codes_f16(u0, 0x4140u), codes_f16(u1, 0x4140u), codes_f16(u0, 0x4342u), codes_f16(u1, 0x4342u),
                     q[4 * k + s][0], q[4 * k + s][1]);
          }
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float scale = __shfl_sync(0xffffffffu, sb[i], mt * 16 + half * 8 + g);
          top[mt][half] = -INFINITY;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (g0 + 2 * t + j < a.rep) {
              const float x = __fmul_rn(__fmul_rn(d[mt][0][2 * half + j] + d[mt][1][2 * half + j], scale), s2[j]);
              top[mt][half] = fmaxf(top[mt][half], isnan(x) ? INFINITY : x);
            }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) top[mt][half] = fmaxf(top[mt][half], __shfl_xor_sync(0xffffffffu, top[mt][half], o));
        }
      }
      // block `lane` of the step
      float mine = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __shfl_sync(0xffffffffu, top[e >> 1][e & 1], (lane & 7) * 4);
        if (lane >> 3 == e) mine = x;
      }
      best[i] = fmaxf(best[i], mine);
    }
    __syncwarp();   // the pieces have been read: the next heads' copies may be written over them
  }
#pragma unroll
  for (int i = 0; i < kBsSteps; ++i) {
    const int b = b0 + 32 * i + lane;
    if (b >= nb) break;
    uint32_t key = ordered(best[i]);
    if (at[i] == kNoRow) {   // a block without a page is the last choice
      key = 0;
      tc::report_giveup(tc::kBadPage);
    }
    if (b < a.first || b >= nb - a.recent) key = kAlways;
    a.keys[static_cast<size_t>(unit) * a.p.max_pages + b] = key;
  }
}

// Inclusive sums of two counts (32 bits each) over the block.
__device__ __forceinline__ uint64_t scan2(uint64_t v, uint64_t* warp_sums, uint64_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  total = 0;
  uint64_t before = 0;
#pragma unroll
  for (int i = 0; i < kPickThreads / 32; ++i) {
    if (i < w) before += warp_sums[i];
    total += warp_sums[i];
  }
  return v + before;
}

// CTA (row, key head): the `keep` largest keys, equal ones by their number, in the blocks' order.  KEYS > 0: a thread
// holds KEYS keys that follow one another; 0: keys are read again for every digit, in passes over all of them.
template <int KEYS>
__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const SelectArgs a) {
  constexpr int kBins = 1 << kPickDigit, kOwn = kBins / kPickThreads;   // counters of a thread
  constexpr int kMine = KEYS > 0 ? KEYS : 1;
  __shared__ uint32_t hist[kBins];
  __shared__ uint64_t warp_sums[kPickThreads / 32];
  __shared__ uint32_t s_lo, s_hi, s_bin, s_above, s_count;
  const int tid = threadIdx.x, lane = tid & 31, unit = blockIdx.x, r = unit / a.p.Hkv;
  int32_t seq;
  const int32_t nb = blocks_of_row(a, r, seq), n = min(nb, a.keep);
  int32_t* sel = a.sel + static_cast<size_t>(unit) * a.keep;
  if (tid == 0) a.n_sel[unit] = n;
  for (int i = tid; i < a.keep; i += kPickThreads)
    if (i >= n || nb <= a.keep) sel[i] = i < n ? i : -1;
  pdl_wait();   // (what came before belongs to no kernel of this call, whose first began when all others were done)
  if (nb <= a.keep) return;
  const uint32_t* keys = a.keys + static_cast<size_t>(unit) * a.p.max_pages;
  uint32_t k[kMine];
  if (KEYS > 0) {
#pragma unroll
    for (int e = 0; e < kMine; ++e) k[e] = tid * KEYS + e < nb ? keys[tid * KEYS + e] : 0u;
  }
  // f(key) for every key of this thread
  const auto each = [&](auto f) {
    if (KEYS > 0) {
#pragma unroll
      for (int e = 0; e < kMine; ++e)
        if (tid * KEYS + e < nb) f(k[e]);
    } else {
      for (int i = tid; i < nb; i += kPickThreads) f(keys[i]);
    }
  };
  // what is always taken needs no search; the range of the others
  uint32_t lo = 0xffffffffu, hi = 0;
  int always = 0;
  each([&](uint32_t x) {
    if (x == kAlways) {
      ++always;
    } else {
      lo = min(lo, x);
      hi = max(hi, x);
    }
  });
  if (tid == 0) {
    s_lo = 0xffffffffu;
    s_hi = s_count = 0;
  }
  for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  always = __reduce_add_sync(0xffffffffu, always);
  if (lane == 0) {
    atomicMin(&s_lo, lo);
    atomicMax(&s_hi, hi);
    atomicAdd(&s_count, always);
  }
  __syncthreads();
  lo = s_lo;
  hi = s_hi;
  int need = n - static_cast<int>(s_count);   // of the keys in lo .. hi: at least one is left out
  while (need > 0 && lo < hi) {   // lo .. hi narrows to the smallest key taken
    const int shift = max(0, 32 - __clz(hi - lo) - kPickDigit);
    each([&](uint32_t x) {
      if (x >= lo && x <= hi) atomicAdd(&hist[(x - lo) >> shift], 1u);
    });
    __syncthreads();
    // sums of the counters from the top: thread t has bins kBins - 1 - kOwn t ..
    uint32_t own[kOwn], sum = 0;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      own[e] = hist[kBins - 1 - (tid * kOwn + e)];
      sum += own[e];
    }
    uint64_t total;
    uint32_t above = static_cast<uint32_t>(scan2(sum, warp_sums, total)) - sum;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      if (above < static_cast<uint32_t>(need) && above + own[e] >= static_cast<uint32_t>(need)) {
        s_bin = kBins - 1 - (tid * kOwn + e);
        s_above = above;
        s_count = own[e];
      }
      above += own[e];
      hist[kBins - 1 - (tid * kOwn + e)] = 0;
    }
    __syncthreads();
    need -= static_cast<int>(s_above);
    lo += s_bin << shift;
    hi = min(hi, lo + ((1u << shift) - 1u));
    const bool all = static_cast<int>(s_count) == need;   // the whole bin is taken: no need to look closer
    __syncthreads();
    if (all) {
      need = 0x7fffffff;   // every key from lo on
      break;
    }
  }
  // keys above lo (or, with all of them taken, from lo on), and the first `need` of those equal to it
  if (need == 0) lo = hi;   // only those always taken
  const bool from = need == 0x7fffffff;
  const auto above_it = [&](uint32_t x) { return from ? x >= lo : need == 0 ? x == kAlways : x > lo; };
  const auto equal_it = [&](uint32_t x) { return !from && need > 0 && x == lo; };
  if (KEYS > 0) {
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int e = 0; e < kMine; ++e)
      if (tid * KEYS + e < nb) {
        gt += above_it(k[e]);
        eq += equal_it(k[e]);
      }
    uint64_t total;
    const uint64_t at = scan2((static_cast<uint64_t>(gt) << 32) | eq, warp_sums, total);
    uint32_t g = static_cast<uint32_t>(at >> 32) - gt, q = static_cast<uint32_t>(at) - eq;
#pragma unroll
    for (int e = 0; e < kMine; ++e)
      if (tid * KEYS + e < nb) {
        const bool is_gt = above_it(k[e]), is_eq = equal_it(k[e]) && q < static_cast<uint32_t>(need);
        if (is_gt || is_eq) sel[g + min(q, static_cast<uint32_t>(need))] = tid * KEYS + e;
        g += is_gt;
        q += equal_it(k[e]);
      }
  } else {
    uint64_t before = 0;   // (keys above, keys equal) of the blocks so far
    for (int i0 = 0; i0 < nb; i0 += kPickThreads) {
      const int i = i0 + tid;
      const uint32_t x = i < nb ? keys[i] : 0u;
      const bool gt = i < nb && above_it(x), eq = i < nb && equal_it(x);
      uint64_t total;
      const uint64_t at = before + scan2((static_cast<uint64_t>(gt) << 32) | eq, warp_sums, total);
      const uint32_t g = static_cast<uint32_t>(at >> 32) - gt, q = static_cast<uint32_t>(at) - eq;
      if (gt || (eq && q < static_cast<uint32_t>(need))) sel[g + min(q, static_cast<uint32_t>(need))] = i;
      before += total;
    }
  }
}

int groups_of(int rep) { return (rep + kBsHeads - 1) / kBsHeads; }
size_t key_bytes(const mikv_pages* p, int rows) { return align_up(static_cast<size_t>(rows) * p->Hkv * p->max_pages * 4, 16); }
size_t select_bytes(const mikv_pages* p, int rows, int Hq) {
  return key_bytes(p, rows) + static_cast<size_t>(rows) * p->Hkv * groups_of(Hq / p->Hkv) * (256 * 16 + kBsHeads * 4);
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_block_select_workspace_bytes(const mikv_pages* p, int rows, int Hq) {
  Pool pool;
  if (check_pages(p, "block_select", &pool) || rows < 1 || static_cast<int64_t>(rows) * p->Hkv > 65535 || Hq < 1 || Hq % p->Hkv ||
      Hq / p->Hkv > 1024)
    return 0;
  return select_bytes(p, rows, Hq);
}

extern "C" int mikv_block_select(const void* q, const mikv_pages* pages, int layer, const int8_t* bounds, const float* scales,
                                 const int32_t* row_seq, const int32_t* row_pos, int rows, int Hq, int keep, int first, int recent,
                                 int32_t* sel, int32_t* n_sel, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  SelectArgs a;
  if (int e = check_pages(pages, "block_select", &a.p)) return e;
  if (layer < 0 || layer >= a.p.layers) return fail(MIKV_ESHAPE, "block_select: layer=%d of %d", layer, a.p.layers);
  if (rows < 0 || static_cast<int64_t>(rows) * a.p.Hkv > 65535 || (!row_seq && rows > a.p.max_seqs))
    return fail(MIKV_ESHAPE, "block_select: rows=%d Hkv=%d", rows, a.p.Hkv);
  if (Hq < 1 || Hq % a.p.Hkv || Hq / a.p.Hkv > 1024) return fail(MIKV_ESHAPE, "block_select: Hq=%d Hkv=%d", Hq, a.p.Hkv);
  if (first < 0 || recent < 1 || keep < 1 || first > keep - recent)
    return fail(MIKV_EINVAL, "block_select: keep=%d first=%d recent=%d", keep, first, recent);
  if (rows == 0) return MIKV_OK;
  if (!q || !bounds || !scales || !sel || !n_sel || !ws) return fail(MIKV_EINVAL, "block_select: null pointer");
  if (!aligned16(q) || !aligned16(bounds) || !aligned16(ws)) return fail(MIKV_EALIGN, "block_select: 16-byte alignment");
  const size_t need = select_bytes(pages, rows, Hq);
  if (ws_bytes < need) return fail(MIKV_ESHAPE, "block_select: workspace %zu < %zu", ws_bytes, need);
  a.q = static_cast<const uint16_t*>(q);
  a.bounds = bounds;
  a.scales = scales;
  a.row_seq = row_seq;
  a.row_pos = row_pos;
  a.layer = layer;
  a.rows = rows;
  a.rep = Hq / a.p.Hkv;
  a.keep = keep;
  a.first = first;
  a.recent = recent;
  a.sel = sel;
  a.n_sel = n_sel;
  a.keys = static_cast<uint32_t*>(ws);
  a.codes = reinterpret_cast<uint4*>(static_cast<uint8_t*>(ws) + key_bytes(pages, rows));
  a.groups = groups_of(a.rep);
  a.chunks = (a.p.max_pages - 1) / kBsBlocks + 1;
  a.warps = static_cast<int64_t>(a.chunks) * rows * a.p.Hkv;
  const int64_t ctas = (a.warps - 1) / kBsWarps + 1;
  if (ctas > 0x7fffffffLL) return fail(MIKV_ESHAPE, "block_select: rows=%d max_pages=%d", rows, a.p.max_pages);
  const cudaStream_t st = as_stream(stream);
  // Whether the score kernel makes the queries' codes itself, a launch less, or one before it (8 key heads of 1 to 8 query heads,
  // made in place / before): 40 to 320 warps 11 us either way, 640 11.7 / 12.7, 960 13.3 / 13.4, 2048 19.6 / 16.0, 8192 46.8 / 35.0;
  // where no row has more blocks than it keeps 2.9 / 6.0.  (16 query heads, which every warp makes in two passes: 16.8 / 12.5 from
  // 40 warps on, 30.9 / 20.5 at 2048.)
  const bool own = a.warps <= 8 * kNumSMs;
  const auto score = own ? block_score_kernel<true> : block_score_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(score, cudaFuncAttributeMaxDynamicSharedMemorySize, kBsSmem);
  if (e != cudaSuccess) return check_launch_after(e, "block_score_kernel");
  // The first kernel stays a normal launch: those behind it read the rows, table, lengths and bounds, and write sel and n_sel,
  // before they wait.
  if (own) {
    score<<<static_cast<unsigned>(ctas), kBsWarps * 32, kBsSmem, st>>>(a);
    if (int r = check_launch("block_score_kernel")) return r;
  } else {
    block_query_kernel<<<(rows * a.p.Hkv * a.groups - 1) / kBsWarps + 1, kBsWarps * 32, 0, st>>>(a);
    if (int r = check_launch("block_query_kernel")) return r;
    if (int r = check_launch_after(launch_after(score, dim3(static_cast<unsigned>(ctas)), dim3(kBsWarps * 32), kBsSmem, st, a),
                                   "block_score_kernel"))
      return r;
  }
  const auto pick = a.p.max_pages <= 2 * kPickThreads    ? block_pick_kernel<2>
                    : a.p.max_pages <= 8 * kPickThreads  ? block_pick_kernel<8>
                    : a.p.max_pages <= 32 * kPickThreads ? block_pick_kernel<32>
                                                         : block_pick_kernel<0>;
  return check_launch_after(launch_after(pick, dim3(rows * a.p.Hkv), dim3(kPickThreads), 0, st, a), "block_pick_kernel");
}
