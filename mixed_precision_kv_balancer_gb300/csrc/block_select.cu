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
// integer products a query head), and the choice of the `keep` best of each (row, key head) by
// a radix search of the scores' bits, written in the blocks' order.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int block_select_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kBsThreads = 128;
constexpr int kBsWarps = kBsThreads / 32;
constexpr int kBsHeads = 8;            // query heads of a pass
constexpr int kBsPass = 2;             // warp-steps of 32 blocks a warp makes
constexpr int kBsBlocks = kBsThreads * kBsPass;   // blocks of a CTA
constexpr int kPickThreads = 512;
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

// CTA: kBsBlocks blocks of one (row, key head).  A warp brings the bounds of 32 blocks to shared memory in
// whole lines; then a lane has a block of its own, so that no sum crosses lanes.
__global__ void __launch_bounds__(kBsThreads) block_score_kernel(const SelectArgs a) {
  __shared__ __align__(16) uint4 s_b[kBsWarps][32 * 16];              // 16 pieces a block, swizzled by the block
  __shared__ __align__(16) uint32_t s_q[kBsHeads][2 * kD / 4];        // codes below 0, codes above 0
  __shared__ float s_scale[kBsHeads];
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
  float best[kBsPass];
#pragma unroll
  for (int i = 0; i < kBsPass; ++i) best[i] = -INFINITY;
  for (int g0 = 0; g0 < a.rep; g0 += kBsHeads) {
    const int heads = min(kBsHeads, a.rep - g0);
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
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBsPass; ++i) {
      const int b = b0 + (i * kBsWarps + w) * 32;
      if (b >= nb) break;
      const int32_t page = b + lane < nb ? table[b + lane] : -1;
      const bool there = a.p.has(page);
      const size_t at = layer0 + static_cast<size_t>(there ? page : 0) * a.p.Hkv + h;
      __syncwarp();   // the last step's pieces have been read
#pragma unroll
      for (int j = 0; j < 16; ++j) {   // two blocks an instruction
        const int e = 2 * j + (lane >> 4), piece = lane & 15;
        const size_t src = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(at), e);
        const bool ok = __shfl_sync(0xffffffffu, static_cast<int>(there), e);
        cp_async16(smem_u32(&s_b[w][e * 16 + (piece ^ (e & 15))]), a.bounds + src * (2 * kD) + piece * 16, ok);
      }
      cp_async_commit();
      const float sb = there ? a.scales[at] : 0.f;
      cp_async_wait<0>();
      __syncwarp();
      int u[kBsHeads];
#pragma unroll
      for (int e = 0; e < kBsHeads; ++e) u[e] = 0;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint4 x = s_b[w][lane * 16 + (c ^ (lane & 15))];
#pragma unroll
        for (int e = 0; e < kBsHeads; ++e) {
          const uint4 y = reinterpret_cast<const uint4*>(s_q[e])[c];
          u[e] = __dp4a(static_cast<int>(x.x), static_cast<int>(y.x), u[e]);
          u[e] = __dp4a(static_cast<int>(x.y), static_cast<int>(y.y), u[e]);
          u[e] = __dp4a(static_cast<int>(x.z), static_cast<int>(y.z), u[e]);
          u[e] = __dp4a(static_cast<int>(x.w), static_cast<int>(y.w), u[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kBsHeads; ++e)
        if (e < heads) {
          const float s = __fmul_rn(__fmul_rn(static_cast<float>(u[e]), sb), s_scale[e]);
          best[i] = fmaxf(best[i], isnan(s) ? INFINITY : s);
        }
      if (g0 + kBsHeads >= a.rep && b + lane < nb) {
        const int x = b + lane;
        uint32_t key = ordered(best[i]);
        if (!there) {   // a block without a page is the last choice
          key = 0;
          tc::report_giveup(tc::kBadPage);
        }
        if (x < a.first || x >= nb - a.recent) key = kAlways;
        a.keys[static_cast<size_t>(unit) * a.p.max_pages + x] = key;
      }
    }
  }
}

// Inclusive sums of two counts over the block.
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

// CTA (row, key head): the `keep` largest keys, equal ones by their number, in the blocks' order.
__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint64_t warp_sums[kPickThreads / 32];
  __shared__ uint32_t s_digit, s_above;
  const int tid = threadIdx.x, unit = blockIdx.x, r = unit / a.p.Hkv;
  int32_t seq;
  const int32_t nb = blocks_of_row(a, r, seq), n = min(nb, a.keep);
  int32_t* sel = a.sel + static_cast<size_t>(unit) * a.keep;
  if (tid == 0) a.n_sel[unit] = n;
  for (int i = tid; i < a.keep; i += kPickThreads)
    if (i >= n || nb <= a.keep) sel[i] = i < n ? i : -1;
  pdl_wait();
  if (nb <= a.keep) return;
  const uint32_t* keys = a.keys + static_cast<size_t>(unit) * a.p.max_pages;
  uint32_t prefix = 0, mask = 0;     // the digits of the smallest key taken, so far
  int need = n;                      // how many keys with that prefix are taken
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kPickThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < nb; i += kPickThreads) {
      const uint32_t k = keys[i];
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 32) {   // eight digits a lane, from the top
      uint32_t own = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) own += hist[255 - (tid * 8 + e)];
      uint32_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += u;
      }
      uint32_t above = incl - own;
      if (above < static_cast<uint32_t>(need) && incl >= static_cast<uint32_t>(need)) {
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = hist[255 - (tid * 8 + e)];
          if (above + c >= static_cast<uint32_t>(need)) {
            s_digit = 255 - (tid * 8 + e);
            s_above = above;
            break;
          }
          above += c;
        }
      }
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    need -= static_cast<int>(s_above);
  }
  uint64_t before = 0;   // (keys above the prefix, keys equal to it) of the blocks so far
  for (int i0 = 0; i0 < nb; i0 += kPickThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < nb ? keys[i] : 0u;
    const bool gt = i < nb && k > prefix, eq = i < nb && k == prefix;
    uint64_t total;
    const uint64_t at = before + scan2((static_cast<uint64_t>(gt) << 32) | eq, warp_sums, total);
    const uint32_t above = static_cast<uint32_t>(at >> 32), equal = static_cast<uint32_t>(at);
    if (gt || (eq && equal <= static_cast<uint32_t>(need)))
      sel[above + min(equal, static_cast<uint32_t>(need)) - 1] = i;
    before += total;
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
  block_score_kernel<<<static_cast<unsigned>(ctas), kBsThreads, 0, st>>>(a);
  if (int e = check_launch("block_score_kernel")) return e;
  return check_launch_after(launch_after(block_pick_kernel, dim3(rows * a.p.Hkv), dim3(kPickThreads), 0, st, a), "block_pick_kernel");
}
