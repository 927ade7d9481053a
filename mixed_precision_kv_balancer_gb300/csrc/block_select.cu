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
// Two kernels: scores of all blocks (bound by HBM: 260 bytes a block and key head, against 64 four-term
// integer products a query head), and the choice of the `keep` best of each (row, key head), written in the
// blocks' order.  The choice is a search by digits of the scores' bits, but of digits that begin below what all
// of a unit's scores share: scores of one unit lie close together, and counters of their first bits would all be hit at once.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int block_select_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kBsThreads = 128;
constexpr int kBsWarps = kBsThreads / 32;
constexpr int kBsSteps = 2;                       // of 32 blocks a warp
constexpr int kBsBlocks = kBsThreads * kBsSteps;  // blocks of a CTA
constexpr int kBsSmem = kBsSteps * kBsWarps * 32 * 2 * kD;   // their bounds
constexpr int kPickThreads = 512;
constexpr int kPickDigit = 11;                    // bits of a digit
constexpr uint32_t kAlways = 0xffffffffu;   // above every score

struct SelectArgs {
  Pool p;
  const uint16_t* q;
  const int8_t* bounds;
  const float* scales;
  const int32_t *row_seq, *row_pos;
  int layer, rows, Hq, rep, keep, first, recent;
  int chunks;            // CTAs of a (row, key head)
  int32_t *sel, *n_sel;
  uint32_t* keys;        // [rows][Hkv][max_pages]: scores in the order of whole numbers
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

// CTA: kBsBlocks blocks of one (row, key head), all requested before anything else is done.  A warp brings the
// bounds of 32 blocks to shared memory in whole lines; then a lane has a block of its own, so that no
// sum crosses lanes.  HEADS query heads a pass.
template <int HEADS>
__global__ void __launch_bounds__(kBsThreads) block_score_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint4 s_b[];                       // [step][warp][32 blocks][16 pieces], swizzled by the block
  __shared__ __align__(16) uint32_t s_q[HEADS][2 * kD / 4];          // codes below 0, codes above 0
  __shared__ float s_scale[HEADS];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int unit = blockIdx.x / a.chunks, b0 = (blockIdx.x - unit * a.chunks) * kBsBlocks;
  const int r = unit / a.p.Hkv, h = unit - r * a.p.Hkv;
  pdl_trigger();
  int32_t seq;
  const int32_t nb = blocks_of_row(a, r, seq);
  if (b0 >= nb || nb <= a.keep) return;
  const bool bf = a.p.type == MIKV_PAGES_BF16;
  const int32_t* table = a.p.table + static_cast<size_t>(seq) * a.p.max_pages;
  const size_t layer0 = static_cast<size_t>(a.layer) * a.p.n_pages * a.p.Hkv;
  const auto block_of = [&](int i) { return b0 + (i * kBsWarps + w) * 32 + lane; };
  const auto pieces = [&](int i) { return s_b + (i * kBsWarps + w) * (32 * 16); };
  bool there[kBsSteps];
  float sb[kBsSteps], best[kBsSteps];
#pragma unroll
  for (int i = 0; i < kBsSteps; ++i) {
    const int b = block_of(i);
    const int32_t page = b < nb ? table[b] : -1;
    there[i] = a.p.has(page);
    const uint32_t at = there[i] ? static_cast<uint32_t>(page) * a.p.Hkv + h : 0;   // (below 2^32, like the pool's rows)
    sb[i] = there[i] ? a.scales[layer0 + at] : 0.f;
    best[i] = -INFINITY;
    uint4* dst = pieces(i);
#pragma unroll
    for (int j = 0; j < 16; ++j) {   // two blocks an instruction
      const int e = 2 * j + (lane >> 4), piece = lane & 15;
      const uint32_t src = __shfl_sync(0xffffffffu, at, e);
      const bool ok = __shfl_sync(0xffffffffu, static_cast<int>(there[i]), e);
      cp_async16(smem_u32(dst + e * 16 + (piece ^ (e & 15))), a.bounds + (layer0 + src) * (2 * kD) + piece * 16, ok);
    }
    cp_async_commit();
  }
  for (int g0 = 0; g0 < a.rep; g0 += HEADS) {
    const int heads = min(HEADS, a.rep - g0);
    if (g0 > 0) __syncthreads();
    for (int e = w; e < heads; e += kBsWarps) {   // a warp per query head: four channels a lane
      const uint2 v = reinterpret_cast<const uint2*>(a.q + (static_cast<size_t>(r) * a.Hq + h * a.rep + g0 + e) * kD)[lane];
      const float x[4] = {to_float(v.x & 0xffffu, bf), to_float(v.x >> 16, bf), to_float(v.y & 0xffffu, bf), to_float(v.y >> 16, bf)};
      float top = 0.f;
      bool bad = false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        top = fmaxf(top, fabsf(x[c]));
        bad |= !(fabsf(x[c]) <= 3.402823466e38f);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      bad = __any_sync(0xffffffffu, bad);
      const float s = bad ? INFINITY : __fdiv_rn(top, 127.f);   // no finite query: its scores are 0 * infinity
      uint32_t neg = 0, pos = 0;
      if (!bad && s > 0.f) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int code = min(max(__float2int_rn(__fdiv_rn(x[c], s)), -127), 127);
          if (code > 0)
            pos |= static_cast<uint32_t>(code) << (8 * c);
          else
            neg |= (static_cast<uint32_t>(code) & 255u) << (8 * c);
        }
      }
      s_q[e][lane] = neg;
      s_q[e][kD / 4 + lane] = pos;
      if (lane == 0) s_scale[e] = s;
    }
    cp_async_wait<0>();
    __syncthreads();
    int u[kBsSteps][HEADS] = {};
#pragma unroll 2
    for (int c = 0; c < 16; ++c) {
      uint4 x[kBsSteps];
#pragma unroll
      for (int i = 0; i < kBsSteps; ++i) x[i] = pieces(i)[lane * 16 + (c ^ (lane & 15))];
#pragma unroll
      for (int e = 0; e < HEADS; ++e) {
        const uint4 y = reinterpret_cast<const uint4*>(s_q[e])[c];
#pragma unroll
        for (int i = 0; i < kBsSteps; ++i) {
          u[i][e] = __dp4a(static_cast<int>(x[i].x), static_cast<int>(y.x), u[i][e]);
          u[i][e] = __dp4a(static_cast<int>(x[i].y), static_cast<int>(y.y), u[i][e]);
          u[i][e] = __dp4a(static_cast<int>(x[i].z), static_cast<int>(y.z), u[i][e]);
          u[i][e] = __dp4a(static_cast<int>(x[i].w), static_cast<int>(y.w), u[i][e]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBsSteps; ++i)
#pragma unroll
      for (int e = 0; e < HEADS; ++e)
        if (e < heads) {
          const float s = __fmul_rn(__fmul_rn(static_cast<float>(u[i][e]), sb[i]), s_scale[e]);
          best[i] = fmaxf(best[i], isnan(s) ? INFINITY : s);
        }
  }
#pragma unroll
  for (int i = 0; i < kBsSteps; ++i) {
    const int b = block_of(i);
    if (b >= nb) break;
    uint32_t key = ordered(best[i]);
    if (!there[i]) {   // a block without a page is the last choice
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
  pdl_wait();
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

size_t key_bytes(const mikv_pages* p, int rows) { return static_cast<size_t>(rows) * p->Hkv * p->max_pages * 4; }

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_block_select_workspace_bytes(const mikv_pages* p, int rows) {
  Pool pool;
  if (check_pages(p, "block_select", &pool) || rows < 1 || static_cast<int64_t>(rows) * p->Hkv > 65535) return 0;
  return align_up(key_bytes(p, rows), 16);
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
  const size_t need = key_bytes(pages, rows);
  if (ws_bytes < need) return fail(MIKV_ESHAPE, "block_select: workspace %zu < %zu", ws_bytes, need);
  a.q = static_cast<const uint16_t*>(q);
  a.bounds = bounds;
  a.scales = scales;
  a.row_seq = row_seq;
  a.row_pos = row_pos;
  a.layer = layer;
  a.rows = rows;
  a.Hq = Hq;
  a.rep = Hq / a.p.Hkv;
  a.keep = keep;
  a.first = first;
  a.recent = recent;
  a.sel = sel;
  a.n_sel = n_sel;
  a.keys = static_cast<uint32_t*>(ws);
  a.chunks = (a.p.max_pages - 1) / kBsBlocks + 1;
  const int64_t ctas = static_cast<int64_t>(a.chunks) * rows * a.p.Hkv;
  if (ctas > 0x7fffffffLL) return fail(MIKV_ESHAPE, "block_select: rows=%d max_pages=%d", rows, a.p.max_pages);
  const cudaStream_t st = as_stream(stream);
  const auto score = a.rep <= 4 ? block_score_kernel<4> : block_score_kernel<8>;
  const cudaError_t e = cudaFuncSetAttribute(score, cudaFuncAttributeMaxDynamicSharedMemorySize, kBsSmem);
  if (e != cudaSuccess) return check_launch_after(e, "block_score_kernel");
  score<<<static_cast<unsigned>(ctas), kBsThreads, kBsSmem, st>>>(a);
  if (int r = check_launch("block_score_kernel")) return r;
  const auto pick = a.p.max_pages <= 2 * kPickThreads    ? block_pick_kernel<2>
                    : a.p.max_pages <= 8 * kPickThreads  ? block_pick_kernel<8>
                    : a.p.max_pages <= 32 * kPickThreads ? block_pick_kernel<32>
                                                         : block_pick_kernel<0>;
  return check_launch_after(launch_after(pick, dim3(rows * a.p.Hkv), dim3(kPickThreads), 0, st, a), "block_pick_kernel");
}
