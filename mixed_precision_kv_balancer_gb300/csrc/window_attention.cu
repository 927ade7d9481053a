// Attention of a prompt, or of a chunk of one, under a sliding window with sinks (tcgen05).
//
// Mathematics: one pass over the visible keys, out = sum_j p_j v_j / sum_j p_j with
// p_j = exp2(l_j - m) and a reference m per query row that follows the running maximum: it is
// moved, and the accumulated sums rescaled, only where the maximum has outgrown it by 2^kGrow,
// so almost every tile leaves the accumulators alone.  Bound by the tensor cores (4 * 128 flop
// per visible query-key pair) and, close behind, by the exponentials.
//
// A CTA holds two tiles of 128 query rows over one key head: the same rows of two heads of the
// group, or 256 rows of one head where the group is odd.  Where a chunk has 64 rows or fewer, a
// tile packs the rows of several heads of the group.  Where the items of a call would leave SMs
// idle, each is split over its key tiles and the parts are joined by a second kernel.  Key and value
// tiles of 128 rows come through a ring of five 32 KB buffers (TMA, 128-byte swizzle); tiles
// that none of the rows sees are not read.  Per key tile i and query tile t
//   S_t = Q_t K_i^T     tcgen05, both operands in shared memory, 128 fp32 TMEM columns
//   P_t = exp2(...)     four warps, one query row a thread, written over S_t as 16-bit pairs
//   O_t += P_t V_i      tcgen05, P from TMEM, V as it lies (rows are the contraction)
// The tensor core runs [O_0 += P_0 V_i, S_0 = Q_0 K_i+1] while the warps of tile 1 make their
// weights, and the other way round.  S_t(i + 1) is committed behind O_t(i), so a thread that
// holds new scores may rescale its accumulator row without another wait.
//
// Weights are rounded to the inputs' type once (2^-9 or 2^-12 of each on average); their sum is
// taken before that, in fp32.  fp16 weights carry a factor 2^kShift, which keeps weights down
// to 2^-27 of the row's largest out of fp16's subnormal range; 2^(kShift + kGrow) stays below
// its largest number.
//
// Value rows that no query of the call sees may hold anything (0 * NaN is NaN): the TMA warp
// clears them in shared memory, in the at most three tiles that hold such rows beside others.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int window_attention_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kWaRows = 128;                     // query rows and key rows of a tile
constexpr int kWaNarrow = 32;                    // columns of a tile that holds the last few sinks
constexpr int kWaRing = 5;
constexpr int kMaxRows = 1 << 30;                // of q or k: positions and their differences fit 32 bits
constexpr int kWaThreads = 352;                  // 2 x 4 softmax warps, the TMA warp, 2 MMA warps
constexpr int kWaTmaWarp = 8, kWaMmaWarp = 9;
constexpr int kWaSmem = (2 + kWaRing) * tc::kTileBytes + 1024;
constexpr uint32_t kWaCols = 512;                // S_0, S_1, O_0, O_1: 128 columns each
constexpr uint32_t kWaO = 256;

template <bool BF>
struct Weights {
  static constexpr float shift = BF ? 0.f : 13.f;  // log2 of the weights' factor
  static constexpr float grow = BF ? 8.f : 2.f;    // log2 of the growth that moves the reference
};

struct WindowArgs {
  RowView out;
  float* lse;
  float* part;                   // splits > 1: [splits][B Hq Tq][128] sums, then [splits][B Hq Tq] (maximum, sum)
  const int32_t *q_lens, *k_lens;
  int Hq, rep, Tq, Tk, window, sinks, blocks;
  int64_t rows;                  // B Hq Tq
  int tb, hb, groups;            // a tile: tb rows of each of hb heads; groups = ceil(rep / hb)
  int splits;
  bool pair_heads;               // the CTA's tiles are two groups of heads, else two row blocks of one
  bool wide_out;                 // rows of out begin at multiples of 32 bytes
  int qb, qh, kb, kh, vb, vh;    // 1, or 0 where the view repeats one batch row or head
  float scale;                   // log2(e) / sqrt(D)
};

struct WaBars {
  uint64_t full[kWaRing], empty[kWaRing];   // buffer landed; the products that read it are done
  uint64_t fix[kWaRing];                    // a value tile's hidden rows are cleared
  uint64_t told[2], heard[2];               // the next item is known; every warp has read it
  uint64_t turn[2];                         // the tile's products may be issued
  uint64_t qfree;                           // the products that read the queries are done
  uint64_t q, s[2], p[2][2], o[2];          // queries landed; scores, half the weights, last sums written
};

// The same value in every lane, told to the compiler: what depends on it stays in uniform
// registers, which the matrix instructions read.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// What one CTA works on; every warp computes it alike.
struct Work {
  int ql, kl, off;        // lengths; position of query 0
  int split;
  int group[2], q0[2];    // per tile: group of heads and first row
  int pa[2], pb[2];       // positions of its first and last row
  int begin, end;         // the item's key tiles: of ts of the sinks, then tw0, tw0 + 1, ...
  int ts, tw0;
  int ns;                 // key tiles that hold sinks, of either part of the list
  int from[2], last[2];   // query tile t sees the sinks' key tiles and tiles from .. last; last -1: none
  int nt;                 // query tiles
  __device__ __forceinline__ int j0(int i) const { return (i < ts ? i : tw0 + i - ts) * kWaRows; }
};
// One query tile of it, in registers (an array indexed by a warp's number would not be).
struct Tile {
  bool live;
  int group, q0, pa, pb, from, last;
  // Whether any of its rows sees key tile i.
  __device__ __forceinline__ bool sees(int i, int ns) const { return i <= last && (i < ns || i >= from); }
};
__device__ __forceinline__ Tile tile_of(const Work& w, int t) {
  return {t < w.nt, t ? w.group[1] : w.group[0], t ? w.q0[1] : w.q0[0], t ? w.pa[1] : w.pa[0], t ? w.pb[1] : w.pb[0],
          t ? w.from[1] : w.from[0], t ? w.last[1] : w.last[0]};
}
template <bool SPLIT>
__device__ __forceinline__ Work work_of(const WindowArgs& a, int b, int x) {
  Work w;
  w.ql = a.q_lens ? min(max(uniform(a.q_lens[b]), 0), a.Tq) : a.Tq;
  w.kl = a.k_lens ? min(max(uniform(a.k_lens[b]), 0), a.Tk) : a.Tk;
  w.off = w.kl - w.ql;
  w.split = SPLIT ? x % a.splits : 0;
  if (SPLIT) x /= a.splits;
  const int per = a.pair_heads ? (a.groups + 1) / 2 : a.groups;   // items of one row block
  const int blk = a.blocks - 1 - x / per, u = x % per;            // the last rows, which see the most, first
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    w.group[t] = a.pair_heads ? 2 * u + t : u;
    w.q0[t] = a.pair_heads ? blk * a.tb : (2 * blk + t) * a.tb;
    w.pa[t] = w.off + w.q0[t];
    w.pb[t] = w.off + min(w.q0[t] + a.tb, w.ql) - 1;
  }
  w.nt = w.q0[0] >= w.ql ? 0 : w.q0[1] >= w.ql || w.group[1] >= a.groups ? 1 : 2;
  const int p1 = w.nt == 2 ? w.pb[1] : w.pb[0];           // the largest position (tile 1's rows are not below tile 0's)
  const int lo = a.window > 0 ? max(w.pa[0] - a.window + 1, 0) : 0;
  const int end = p1 < 0 ? 0 : p1 / kWaRows + 1;
  w.tw0 = min(lo / kWaRows, end);
  const int sink_tiles = a.window > 0 ? (min(a.sinks, w.kl) + kWaRows - 1) / kWaRows : 0;
  w.ts = min(sink_tiles, w.tw0);
  const int tiles = w.ts + end - w.tw0;
  // where the window begins among the sinks the list is 0, 1, 2, ... and its first sink_tiles hold
  // sinks, which a later query tile sees though its own window begins behind them
  w.ns = max(w.ts, min(sink_tiles, sink_tiles > w.tw0 ? tiles : w.ts));
  w.begin = SPLIT ? static_cast<int>(static_cast<int64_t>(tiles) * w.split / a.splits) : 0;
  w.end = SPLIT ? static_cast<int>(static_cast<int64_t>(tiles) * (w.split + 1) / a.splits) : tiles;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int e = w.pb[t] < 0 ? -1 : w.pb[t] / kWaRows;
    w.from[t] = w.ts + (a.window > 0 ? max(w.pa[t] - a.window + 1, 0) / kWaRows - w.tw0 : 0);
    int last = t >= w.nt || e < 0 ? -1 : e - w.tw0 + w.ts;
    if (SPLIT) {   // the last one of this part
      last = min(last, w.end - 1);
      if (last < w.from[t]) last = min(last, w.ns - 1);
      if (last < w.begin) last = -1;
    }
    w.last[t] = last;
  }
  return w;
}
// Whether all rows of a query tile see all of the key tile at j0.
__device__ __forceinline__ bool tile_whole(const WindowArgs& a, const Tile& t, int j0) {
  return j0 + kWaRows - 1 <= t.pa && (a.window == 0 || j0 > t.pb - a.window || j0 + kWaRows <= a.sinks);
}
// Whether a key tile counts with its first kWaNarrow columns alone: the sinks' last tile, mostly
// (a window of 1024 with 4 sinks is ten tiles, one of them for the sinks: 79 -> 75 us).
__device__ __forceinline__ bool tile_narrow(const WindowArgs& a, const Work& w, int i) {
  return i < w.ts && a.sinks - w.j0(i) <= kWaNarrow;
}
// Rows [z0, z1) and [z2, 128) of the value tile at j0 that no query of the call sees.
struct Hidden {
  int z0, z1, z2;
  __device__ __forceinline__ bool any() const { return z0 < z1 || z2 < kWaRows; }
};
__device__ __forceinline__ Hidden hidden_rows(const WindowArgs& a, const Work& w, int j0) {
  Hidden h;
  h.z0 = min(max(a.sinks - j0, 0), kWaRows);
  h.z1 = a.window > 0 ? min(max(w.off - a.window + 1 - j0, 0), kWaRows) : 0;
  h.z2 = min(max(w.kl - j0, 0), kWaRows);
  return h;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x0, float x1) {
  if (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(x0, x1);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 fp32 columns of this thread's TMEM lane, without the wait.
__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 32 bytes to a 32-byte boundary.  A thread writes its own row, 32 rows an instruction: what counts
// is the number of instructions (16-byte pieces cost twice the store cycles).
__device__ __forceinline__ void st_global32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
               "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// One thread: rows row0 .. of one (head, batch row) into the tile at `s`, two boxes of 64
// channels; rows past the end are zero-filled.  Completes the boxes' bytes on the mbarrier.
__device__ __forceinline__ void tma_rows(uint32_t s, const CUtensorMap* map, int row0, int h, int b, uint32_t mbar) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(s + j * tc::kKBlock),
        "l"(map), "r"(j * 64), "r"(row0), "r"(h), "r"(b), "r"(mbar)
        : "memory");
}

// The same for a query tile: tb rows of hb heads from head h of the group of key head hk.
__device__ __forceinline__ void tma_queries(uint32_t s, const CUtensorMap* map, int row0, int h, int hk, int b, uint32_t mbar) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::"r"(s + j * tc::kKBlock),
        "l"(map), "r"(j * 64), "r"(row0), "r"(h), "r"(hk), "r"(b), "r"(mbar)
        : "memory");
}

// D[tmem] (+)= A[tmem] . B for one step of 16 along the contraction; B lies with its rows along it.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u));
}
// Descriptor of a value tile as the B operand [128 keys][128 channels], channels contiguous: the
// two 64-channel blocks lie kKBlock apart (leading offset), groups of 8 keys 1024 B apart.
__device__ __forceinline__ uint64_t value_desc(uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(tc::kKBlock >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// The address field of a descriptor counts 16-byte units in its low bits; the tiles lie below
// 256 KB, so a step inside a tile or to another one is an addition.
constexpr uint64_t desc_step(uint32_t bytes) { return bytes >> 4; }

// One thread's row of one query tile.
struct Row {
  float m = -INFINITY, l = 0.f;   // reference (raw scores) and sum of weights
  bool first = true;              // no tile has been accumulated
};

// The n lowest bits set, for any n.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// One tile of scores: COLS columns of this thread's lane at `ts` become weights; the accumulator
// at `to` is rescaled where some row of the warp needs it.
// Each half of the weights is announced (`ready`, one arrival a warp) as soon as it is written.
template <bool BF, int COLS>
__device__ __forceinline__ void softmax_tile(const WindowArgs& a, uint32_t ts, uint32_t to, bool whole, int p, int j0, Row& r,
                                             const uint32_t (&ready)[2]) {
  float s[COLS];
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) ld32(ts + c * 32, s + c * 32);
  wait_ld();
  if (!whole) {
    // the row sees columns lo .. hi and those below sk; 32 columns whole to the warp's rows are left alone
    const int hi = p - j0, lo = a.window > 0 ? hi - a.window + 1 : 0, sk = a.sinks - j0;
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      const uint32_t m = low_bits(hi + 1 - c) & (~low_bits(lo - c) | low_bits(sk - c));
      if (!__all_sync(0xffffffffu, m == 0xffffffffu)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(m & (1u << i))) s[c + i] = -INFINITY;
      }
    }
  }
  float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int c = 4; c < COLS; c += 8)
#pragma unroll
    for (int u = 0; u < 4; ++u) mx[u] = fmaxf(fmaxf(mx[u], s[c + u]), c + 4 + u < COLS ? s[c + 4 + u] : -INFINITY);
  const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  const bool grew = (top - r.m) * a.scale > Weights<BF>::grow;   // from -inf too; never by NaN
  if (__any_sync(0xffffffffu, grew)) {
    // a row whose own maximum has not outgrown its reference keeps it: its result does not hang on
    // the other rows of the warp, which may be rows that do not count
    const float alpha = grew ? ex2((r.m - top) * a.scale) : 1.f;
    if (grew) r.m = top;
    r.l *= alpha;
    if (!r.first) {
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        float o[32];
        uint32_t u[32];
        ld32(to + c, o);
        wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * alpha);
        st16(to + c, u);
        st16(to + c + 16, u + 16);
      }
    }
  }
  r.first = false;
  const float neg = r.m == -INFINITY ? 0.f : Weights<BF>::shift - r.m * a.scale;
  float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
  for (int c = 0; c < COLS; c += 32) {
    uint32_t u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = __ffma2_rn(make_float2(s[c + 2 * i], s[c + 2 * i + 1]), make_float2(a.scale, a.scale), make_float2(neg, neg));
      const float2 e = make_float2(ex2(x.x), ex2(x.y));
      sum[i & 1] = __fadd2_rn(sum[i & 1], e);
      u[i] = pack2<BF>(e.x, e.y);
    }
    st16(ts + c / 2, u);
    if (c % 64 == 32 || COLS == 32) {
      wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {
        tc::mbar_arrive(ready[c / 64]);
        if (COLS == 32) tc::mbar_arrive(ready[1]);
      }
    }
  }
  r.l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// A work item is (pair of query tiles, key head, batch row), one per CTA of the grid; a CTA that
// is done takes over one that has not been launched (cluster launch control), so the SMs stay
// busy whatever the lengths are, and the next item's queries, keys and scores are under way
// while the last sums are written.  Every warp walks the items; lane 0 of the TMA warp asks for
// the next one once it has requested all tiles of this one: two or three key tiles before the
// end, early enough to hide the answer and late enough to keep long items from piling up (asked
// at an item's start, 8192 causal tokens of 32 heads took 394 us instead of 349).
struct Item {
  int x, y, z;
};
__device__ __forceinline__ void ask_next(uint32_t answer, uint32_t mbar) {
  tc::mbar_expect_tx(mbar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(answer),
               "r"(mbar)
               : "memory");
}
// The answer to ask n, by the whole warp: false where nothing is left.
__device__ __forceinline__ bool next_item(WaBars& bar, const uint4* answers, int n, tc::Waits& wait, Item& it) {
  const uint32_t at = smem_u32(&answers[n & 1]);
  wait(smem_u32(&bar.told[n & 1]), (n >> 1) & 1);
  uint32_t x = 0, y = 0, z = 0, ok = 0;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 h;\n ld.shared.b128 h, [%4];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %3, 1, 0, p;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, h;\n}\n"
      : "+r"(x), "+r"(y), "+r"(z), "=r"(ok)
      : "r"(at)
      : "memory");
  tc::fence_proxy_async();   // the answer is read before another overwrites it
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(smem_u32(&bar.heard[n & 1]));
  it = {uniform(x), uniform(y), uniform(z)};
  return __all_sync(0xffffffffu, ok != 0 && wait.ok);
}

template <bool BF, bool SPLIT>
__global__ void __launch_bounds__(kWaThreads, 1)
    window_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const WindowArgs a) {
  extern __shared__ uint8_t smem[];
  __shared__ WaBars bar;
  __shared__ __align__(16) uint4 answers[2];
  __shared__ uint32_t tslot;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWaRing; ++i) {
      tc::mbar_init(smem_u32(&bar.full[i]), 1);
      tc::mbar_init(smem_u32(&bar.empty[i]), 2);
      tc::mbar_init(smem_u32(&bar.fix[i]), 1);
    }
    tc::mbar_init(smem_u32(&bar.q), 1);
    tc::mbar_init(smem_u32(&bar.qfree), 2);
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(smem_u32(&bar.told[t]), 1);
      tc::mbar_init(smem_u32(&bar.heard[t]), kWaThreads / 32);
      tc::mbar_init(smem_u32(&bar.turn[t]), 1);
      tc::mbar_init(smem_u32(&bar.s[t]), 1);
      tc::mbar_init(smem_u32(&bar.p[t][0]), 4);
      tc::mbar_init(smem_u32(&bar.p[t][1]), 4);
      tc::mbar_init(smem_u32(&bar.o[t]), 1);
    }
    tc::mbar_init_fence();
  }
  if (warp == kWaMmaWarp) tc::tmem_alloc(smem_u32(&tslot), kWaCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(tslot);
  if (SPLIT) pdl_trigger();   // the joining kernel may be placed; it waits for this one's end
  const uint32_t sq = tc::smem_base(smem), ring = sq + 2 * tc::kTileBytes;
  tc::Waits wait;
  Item it = {static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y), static_cast<int>(blockIdx.z)};

  if (warp == kWaTmaWarp) {
    int slot = 0, par = 1, qs = 0;   // ring position; parity that an empty buffer shows; query loads
    for (int n = 0;; ++n) {
      const int b = it.z, hk = it.y;
      const Work w = work_of<SPLIT>(a, b, it.x);
      if (w.nt > 0 && w.begin < w.end) {
        if (qs > 0) wait(smem_u32(&bar.qfree), (qs - 1) & 1);
        ++qs;
        if (lane == 0 && wait.ok) {
          tc::mbar_expect_tx(smem_u32(&bar.q), w.nt * a.tb * a.hb * kD * 2);
          tma_queries(sq, &qmap, w.q0[0], w.group[0] * a.hb * a.qh, hk * a.qh, b * a.qb, smem_u32(&bar.q));
          if (w.nt == 2)
            tma_queries(sq + tc::kTileBytes, &qmap, w.q0[1], w.group[1] * a.hb * a.qh, hk * a.qh, b * a.qb, smem_u32(&bar.q));
        }
        for (int c = 2 * w.begin; c < 2 * w.end; ++c) {   // keys of key tile c / 2 (c even), then its values
          const int j0 = w.j0(c >> 1);
          const uint32_t dst = ring + slot * tc::kTileBytes, full = smem_u32(&bar.full[slot]);
          wait(smem_u32(&bar.empty[slot]), par);
          if (lane == 0 && wait.ok) {
            tc::mbar_expect_tx(full, tc::kTileBytes);
            if (c & 1)
              tma_rows(dst, &vmap, j0, hk * a.vh, b * a.vb, full);
            else
              tma_rows(dst, &kmap, j0, hk * a.kh, b * a.kb, full);
          }
          __syncwarp();
          if (c & 1) {
            const Hidden h = hidden_rows(a, w, j0);
            if (h.any()) {
              wait(full, par ^ 1);
              for (int e = lane; e < kWaRows * 16; e += 32) {   // 16-byte pieces, both channel blocks
                const int r = e >> 4, piece = e & 15;
                if ((r >= h.z0 && r < h.z1) || r >= h.z2)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(dst + (piece >> 3) * tc::kKBlock + r * 128 + (piece & 7) * 16),
                               "r"(0)
                               : "memory");
              }
              tc::fence_proxy_async();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(smem_u32(&bar.fix[slot]));
            }
          }
          if (++slot == kWaRing) {
            slot = 0;
            par ^= 1;
          }
        }
      }
      if (n >= 2) wait(smem_u32(&bar.heard[n & 1]), ((n >> 1) - 1) & 1);
      if (lane == 0 && wait.ok) ask_next(smem_u32(&answers[n & 1]), smem_u32(&bar.told[n & 1]));
      if (!next_item(bar, answers, n, wait, it)) break;
    }
    // every buffer's release has arrived before the CTA ends
    for (int c = 0; c < kWaRing; ++c) {
      wait(smem_u32(&bar.empty[slot]), par);
      if (++slot == kWaRing) {
        slot = 0;
        par ^= 1;
      }
    }
    if (qs > 0) wait(smem_u32(&bar.qfree), (qs - 1) & 1);
  } else if (warp >= kWaMmaWarp) {
    // One warp per query tile, so that neither waits in the other's place.  The whole warp walks
    // the steps, so that addresses and descriptors stay uniform; one elected lane issues.
    const int t = warp - kWaMmaWarp;
    bool lead = elect_one();
    constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;
    constexpr uint32_t kScores = tc::idesc_f16(kWaRows, kWaRows) | kType, kFew = tc::idesc_f16(kWaRows, kWaNarrow) | kType;
    constexpr uint32_t kValues = tc::idesc_f16(kWaRows, kD) | kType | (1u << 16);   // B: rows along the contraction
    const uint32_t ts = tmem + t * 128, to = tmem + kWaO + t * 128;
    const uint64_t qd = tc::smem_desc(sq + t * tc::kTileBytes), k0 = tc::smem_desc(ring), v0 = value_desc(ring);
    uint32_t fixed = 0;              // parity of each buffer's next clearing
    int p_par = 0, q_par = 0;        // parity of the next weights, and queries
    int slot = 0, par = 0;           // ring position and parity
    // The two warps issue in turns, one step each: the tiles then stay half a step apart, and one's
    // weights are made while the tensor core works for the other (in step, both would wait).
    int turn = t;   // tile 0 begins without waiting
    const auto take_turn = [&] {
      if (turn > 0) wait(smem_u32(&bar.turn[t]), (turn - 1) & 1);
      ++turn;
    };
    for (int n = 0;; ++n) {
      const Work w = work_of<SPLIT>(a, it.z, it.x);
      if (w.nt > 0 && w.begin < w.end) {
        const Tile tile = tile_of(w, t);
        bool more = false, before = false, clear = false, few = false;
        int vslot = 0, vpar = 0;     // the last step's values
        wait(smem_u32(&bar.q), q_par);
        q_par ^= 1;
        // after a wait that gave up no lane leads, nothing more is issued, and the others' waits run out
        for (int i = w.begin; i <= w.end; ++i) {
          // this step's scores from key tile i, behind the last step's sums over value tile i - 1
          const bool keys = i < w.end, here = keys && tile.sees(i, w.ns);
          const uint64_t kd = k0 + slot * desc_step(tc::kTileBytes), vd = v0 + vslot * desc_step(tc::kTileBytes);
          if (i > w.begin) {
            wait(smem_u32(&bar.full[vslot]), vpar);
            if (clear) {
              wait(smem_u32(&bar.fix[vslot]), (fixed >> vslot) & 1);
              fixed ^= 1u << vslot;
            }
          }
          if (keys) wait(smem_u32(&bar.full[slot]), par);
          if (before) wait(smem_u32(&bar.p[t][0]), p_par);
          take_turn();
          lead &= __all_sync(0xffffffffu, wait.ok) != 0;
          tc::fence_after_sync();
          if (before) {
            const auto sums = [&](int c0, int c1) {
#pragma unroll
              for (int c = c0; c < c1; ++c) mma_ts(to, ts + c * 8, vd + desc_step(c * 2048), kValues, more || c > 0);
            };
            // the tensor core's queue holds about two products: a wait between them leaves it idle
            if (few) {
              wait(smem_u32(&bar.p[t][1]), p_par);
              lead &= __all_sync(0xffffffffu, wait.ok) != 0;
              if (lead) sums(0, kWaNarrow / 16);
            } else if (__all_sync(0xffffffffu, tc::mbar_wait(smem_u32(&bar.p[t][1]), p_par, 1))) {
              tc::fence_after_sync();
              if (lead) sums(0, kWaRows / 16);
            } else {
              if (lead) sums(0, kWaRows / 32);
              wait(smem_u32(&bar.p[t][1]), p_par);
              lead &= __all_sync(0xffffffffu, wait.ok) != 0;
              tc::fence_after_sync();
              if (lead) sums(kWaRows / 32, kWaRows / 16);
            }
            p_par ^= 1;
            more = true;
          }
          const uint32_t scores = keys && tile_narrow(a, w, i) ? kFew : kScores;
          if (lead) {
            if (before && i - 1 == tile.last) tc::commit(smem_u32(&bar.o[t]));
            // the turn passes on a little early: the other warp takes as long to wake as the
            // last products take to issue
            if (here) {
#pragma unroll
              for (int c = 0; c < kD / 16; ++c) {
                const uint64_t off = desc_step((c >> 2) * tc::kKBlock + (c & 3) * 32);
                tc::mma_f16(ts, qd + off, kd + off, scores, c > 0);
                if (c == 4) tc::mbar_arrive(smem_u32(&bar.turn[t ^ 1]));
              }
              tc::commit(smem_u32(&bar.s[t]));
            } else {
              tc::mbar_arrive(smem_u32(&bar.turn[t ^ 1]));
            }
          }
          before = here;
          few = keys && tile_narrow(a, w, i);
          if (lead) {
            if (i > w.begin) tc::commit(smem_u32(&bar.empty[vslot]));
            if (keys) tc::commit(smem_u32(&bar.empty[slot]));
            if (i == w.end - 1) tc::commit(smem_u32(&bar.qfree));   // the last scores
          }
          if (keys) {   // the values of tile i follow its keys in the ring
            clear = hidden_rows(a, w, w.j0(i)).any();
            vslot = slot + 1 == kWaRing ? 0 : slot + 1;
            vpar = vslot == 0 ? par ^ 1 : par;
            slot = vslot + 1 == kWaRing ? 0 : vslot + 1;
            par = slot == 0 ? vpar ^ 1 : vpar;
          }
        }
      }
      if (!next_item(bar, answers, n, wait, it)) break;
    }
  } else {
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;   // the thread's TMEM lane is its row
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + kWaO + t * 128;
    const uint32_t ready[2] = {smem_u32(&bar.p[t][0]), smem_u32(&bar.p[t][1])};
    int s_par = 0, o_par = 0;
    for (int n = 0;; ++n) {
      const int b = it.z;
      const Work w = work_of<SPLIT>(a, b, it.x);
      const Tile tile = tile_of(w, t);
      if (tile.live) {
        const int p = tile.pa + row % a.tb;
        Row r;
        for (int i = w.begin; i < w.end; ++i) {
          if (!tile.sees(i, w.ns)) continue;
          const int j0 = w.j0(i);
          wait(smem_u32(&bar.s[t]), s_par);
          s_par ^= 1;
          tc::fence_after_sync();
          if (tile_narrow(a, w, i))
            softmax_tile<BF, kWaNarrow>(a, ts, to, false, p, j0, r, ready);
          else
            softmax_tile<BF, kWaRows>(a, ts, to, tile_whole(a, tile, j0), p, j0, r, ready);
        }
        if (tile.last >= 0) {
          wait(smem_u32(&bar.o[t]), o_par);
          o_par ^= 1;
        }
        tc::fence_after_sync();
        const int sub = row / a.tb, q = tile.q0 + row - sub * a.tb, h = tile.group * a.hb + sub;   // the row's query and head
        const bool write = sub < a.hb && h < a.rep && q < w.ql;
        const int head = it.y * a.rep + h;
        const int64_t at = (static_cast<int64_t>(b) * a.Hq + head) * a.Tq + q;
        float inv = SPLIT ? 1.f : r.l == 0.f ? 0.f : 1.f / r.l;
        if (!wait.ok) inv = __int_as_float(0x7fffffff);
        uint8_t* dst = !SPLIT ? a.out.row(b, head, q) : reinterpret_cast<uint8_t*>(a.part + (w.split * a.rows + at) * kD);
#pragma unroll 1
        for (int c = 0; c < kD; c += 32) {
          float o[32];
          if (tile.last >= 0) {
            ld32(to + c, o);
            wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (write) {
            uint32_t u[32];
            if (!SPLIT) {
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = pack2<BF>(o[2 * e] * inv, o[2 * e + 1] * inv);
              if (a.wide_out) {
                st_global32(dst + c * 2, u);
                st_global32(dst + c * 2 + 32, u + 8);
              } else {
#pragma unroll
                for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(dst + (c + 2 * e) * 2) = make_uint4(u[e], u[e + 1], u[e + 2], u[e + 3]);
              }
            } else if (tile.last >= 0) {   // a part without a visible key is told by its sum of 0
#pragma unroll
              for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * inv);
#pragma unroll
              for (int e = 0; e < 32; e += 8) st_global32(dst + (c + e) * 4, u + e);
            }
          }
        }
        if (SPLIT && write) {
          float2* ml = reinterpret_cast<float2*>(a.part + a.splits * a.rows * kD);
          ml[w.split * a.rows + at] = make_float2(r.m * a.scale, wait.ok ? r.l : inv);
        } else if (!SPLIT && write && a.lse) {
          const float v = r.l == 0.f ? -INFINITY : (r.m * a.scale + (log2f(r.l) - Weights<BF>::shift)) * 0.6931471805599453f;
          a.lse[at] = wait.ok ? v : inv;
        }
        tc::fence_before_sync();   // the sums are read before the next item's products overwrite them
      }
      if (!next_item(bar, answers, n, wait, it)) break;
    }
  }
  if (!wait.ok) tc::report_giveup(tc::kGiveupWindow);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWaMmaWarp) tc::tmem_dealloc(tmem, kWaCols);
}

// One partial result of a row: maximum (log2 units), sum, four channels of the lane.
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
// Joins the parts of query rows, in a fixed order, four channels a lane.  WARPS warps share a row,
// each with every WARPS-th part, BATCH of them requested together.
template <bool BF, int WARPS, int BATCH>
__global__ void __launch_bounds__(128) window_join_kernel(const WindowArgs a) {
  constexpr int kRows = 4 / WARPS;   // rows of a CTA
  __shared__ float4 s_o[4][32];
  __shared__ float2 s_ml[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = warp % WARPS;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kRows + warp / WARPS;
  pdl_wait();
  bool live = at < a.rows;
  const int64_t row = live ? at : 0;
  const int q = static_cast<int>(row % a.Tq), head = static_cast<int>(row / a.Tq % a.Hq), b = static_cast<int>(row / a.Tq / a.Hq);
  live = live && !(a.q_lens && q >= min(max(a.q_lens[b], 0), a.Tq));
  Part sum = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (live) {
    const float2* ml = reinterpret_cast<const float2*>(a.part + a.splits * a.rows * kD) + row;
    for (int s0 = first; s0 < a.splits; s0 += BATCH * WARPS) {
      float2 x[BATCH];
      float4 os[BATCH];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int s = s0 + e * WARPS;
        x[e] = s < a.splits ? ml[s * a.rows] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        os[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        // a sum of 0: nothing seen there, and no sums written
        if (x[e].y != 0.f) os[e] = reinterpret_cast<const float4*>(a.part + ((s0 + e * WARPS) * a.rows + row) * kD)[lane];
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) sum.add(x[e].x, x[e].y, os[e]);
    }
  }
  if (WARPS > 1) {
    s_o[warp][lane] = sum.o;
    if (lane == 0) s_ml[warp] = make_float2(sum.m, sum.l);
    __syncthreads();
    if (first != 0) return;
#pragma unroll
    for (int e = 1; e < WARPS; ++e) sum.add(s_ml[warp + e].x, s_ml[warp + e].y, s_o[warp + e][lane]);
  }
  if (!live) return;
  const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
  *reinterpret_cast<uint2*>(a.out.row(b, head, q) + lane * 8) =
      make_uint2(pack2<BF>(sum.o.x * inv, sum.o.y * inv), pack2<BF>(sum.o.z * inv, sum.o.w * inv));
  if (lane == 0 && a.lse)
    a.lse[row] = sum.l == 0.f ? -INFINITY : (sum.m + (log2f(sum.l) - Weights<BF>::shift)) * 0.6931471805599453f;
}

// The split of a call: rows and heads of a tile, items, and parts of each item.
struct Plan {
  int tb, hb, groups, blocks, splits;
  bool pair_heads;
  int64_t per_head;   // items of one key head and batch row, without the splits
};
// `pack`: heads of a group may share a tile (their rows are apart in memory).
Plan plan_of(int B, int Hq, int Hkv, int Tq, int Tk, int window, int sinks, bool pack) {
  Plan p;
  const int rep = Hq / Hkv;
  p.hb = pack ? std::min(rep, std::max(1, kWaRows / Tq)) : 1;
  p.tb = p.hb > 1 ? Tq : kWaRows;
  p.groups = (rep + p.hb - 1) / p.hb;
  const int blocks = (Tq + p.tb - 1) / p.tb;
  p.pair_heads = p.groups % 2 == 0 || blocks == 1;
  p.blocks = p.pair_heads ? blocks : (blocks + 1) / 2;
  p.per_head = static_cast<int64_t>(p.blocks) * (p.pair_heads ? (p.groups + 1) / 2 : p.groups);
  // Parts of an item: the number that ends soonest by this estimate, in key tiles of an item's two
  // query tiles (1.4 us each).  An item costs 3 beside its tiles, a part 12 (its sums go out to
  // memory, 128 KB, and come back); the longest item bounds the end, and items of about one length
  // run in whole waves.  Measured: 8192 causal rows of 4 heads, 128 items, 93 us whole and 72 in
  // two parts each; 4096 rows of 8 heads, 128 items, 52 whole and 66 in two; 64 rows of 8 heads
  // behind 16384 keys, 4 items, 26 us in 32 parts and 33 in 64.
  const int64_t items = p.per_head * Hkv * B;
  const int64_t rows = static_cast<int64_t>(p.pair_heads ? 1 : 2) * p.tb;
  double longest = Tk, mean = Tk - 0.5 * std::min(Tq, Tk);
  if (window > 0) {
    longest = std::min<double>(longest, static_cast<double>(window) + sinks + rows);
    mean = std::min(mean, longest);
  }
  longest = std::max(1.0, longest / kWaRows);
  mean = std::max(1.0, mean / kWaRows);
  double best = 1e30;
  for (int s = 1; s == 1 || (s <= 32 && longest / s >= 2.0); ++s) {
    const double cost = s == 1 ? 3 : 12, waves = static_cast<double>(items) * s / kNumSMs;
    const double even = mean > 0.75 * longest ? std::ceil(waves) : waves + 0.5;
    const double est = std::max(longest / s + cost, even * (mean / s + cost));
    if (est < best - 1e-9) {
      best = est;
      p.splits = s;
    }
  }
  return p;
}
size_t part_bytes(const Plan& p, int64_t rows) { return p.splits > 1 ? static_cast<size_t>(p.splits) * rows * (kD + 2) * 4 : 0; }
bool packs(const mikv_rows& q, int Hq) { return Hq == 1 || q.stride_h >= kD; }

// 4-D tensor map (channel, row, head, batch row) of a strided view, box 64 x 128 x 1 x 1 with
// 128-byte swizzle.  A dimension of stride 0 (a repeated head or batch row) has one entry in
// the map; *mb and *mh tell whether the coordinate counts.
int encode_view(CUtensorMap* map, const mikv_rows& r, int T, int H, int B, const char* name, int* mb, int* mh) {
  const auto enc = tc::tensor_map_encoder();
  if (!enc) return fail(MIKV_ECUDA, "window_attention: cuTensorMapEncodeTiled unavailable");
  *mh = H > 1 && r.stride_h != 0;
  *mb = B > 1 && r.stride_b != 0;
  const cuuint64_t row = T > 1 ? static_cast<cuuint64_t>(r.stride_t) * 2 : kD * 2;
  const cuuint64_t dims[4] = {kD, static_cast<cuuint64_t>(T), *mh ? static_cast<cuuint64_t>(H) : 1, *mb ? static_cast<cuuint64_t>(B) : 1};
  const cuuint64_t strides[3] = {row, *mh ? static_cast<cuuint64_t>(r.stride_h) * 2 : row, *mb ? static_cast<cuuint64_t>(r.stride_b) * 2 : row};
  const cuuint32_t box[4] = {64, kWaRows, 1, 1}, estr[4] = {1, 1, 1, 1};
  const CUresult e = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, r.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (e != CUDA_SUCCESS) return fail(MIKV_ECUDA, "window_attention: tensor map of %s (error %d)", name, static_cast<int>(e));
  return MIKV_OK;
}
// The queries' map: (channel, row, head of the group, key head, batch row), box 64 x tb x hb x 1 x 1.
int encode_queries(CUtensorMap* map, const mikv_rows& r, int T, int rep, int Hkv, int B, const Plan& p, int* mb, int* mh) {
  const auto enc = tc::tensor_map_encoder();
  if (!enc) return fail(MIKV_ECUDA, "window_attention: cuTensorMapEncodeTiled unavailable");
  *mh = rep * Hkv > 1 && r.stride_h != 0;
  *mb = B > 1 && r.stride_b != 0;
  const cuuint64_t row = T > 1 ? static_cast<cuuint64_t>(r.stride_t) * 2 : kD * 2;
  const cuuint64_t head = *mh ? static_cast<cuuint64_t>(r.stride_h) * 2 : row;
  const cuuint64_t dims[5] = {kD, static_cast<cuuint64_t>(T), *mh ? static_cast<cuuint64_t>(rep) : 1, *mh ? static_cast<cuuint64_t>(Hkv) : 1,
                              *mb ? static_cast<cuuint64_t>(B) : 1};
  const cuuint64_t strides[4] = {row, head, head * static_cast<cuuint64_t>(*mh ? rep : 1), *mb ? static_cast<cuuint64_t>(r.stride_b) * 2 : row};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(p.tb), static_cast<cuuint32_t>(p.hb), 1, 1}, estr[5] = {1, 1, 1, 1, 1};
  const CUresult e = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, r.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (e != CUDA_SUCCESS) return fail(MIKV_ECUDA, "window_attention: tensor map of q (error %d)", static_cast<int>(e));
  return MIKV_OK;
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_window_attention_workspace_bytes(int B, int Hq, int Hkv, int Tq, int Tk, int window, int sinks) {
  if (B < 1 || B > 65535 || Hkv < 1 || Hkv > 65535 || Hq < 1 || Hq % Hkv || Tq < 1 || Tk < 1 || Tq > kMaxRows || Tk > kMaxRows ||
      window < 0 || sinks < 0)
    return 0;
  size_t most = 0;   // heads that repeat one another's rows are not packed
  for (bool pack : {true, false})
    most = std::max(most, part_bytes(plan_of(B, Hq, Hkv, Tq, Tk, window >= Tk ? 0 : window, std::min(sinks, Tk), pack),
                                     static_cast<int64_t>(B) * Hq * Tq));
  return most;
}

extern "C" int mikv_window_attention(const mikv_rows* q, const mikv_rows* k, const mikv_rows* v, int B, int Hq, int Hkv, int Tq,
                                     int Tk, int D, int type, const int32_t* q_lens, const int32_t* k_lens, int window, int sinks,
                                     const mikv_rows* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (type != MIKV_PAGES_FP16 && type != MIKV_PAGES_BF16) return fail(MIKV_EINVAL, "window_attention: type=%d", type);
  if (D != kD) return fail(MIKV_EUNSUPPORTED, "window_attention: D=%d (only %d)", D, kD);
  if (window < 0 || sinks < 0) return fail(MIKV_EINVAL, "window_attention: window=%d sinks=%d", window, sinks);
  if (B < 0 || B > 65535 || Hkv < 1 || Hkv > 65535 || Hq < 1 || Hq % Hkv || Tq < 1 || Tk < 1 || Tq > kMaxRows || Tk > kMaxRows)
    return fail(MIKV_ESHAPE, "window_attention: B=%d Hq=%d Hkv=%d Tq=%d Tk=%d", B, Hq, Hkv, Tq, Tk);
  if (B == 0) return MIKV_OK;
  if (int e = check_rows(q, "window_attention", "q")) return e;
  if (int e = check_rows(k, "window_attention", "k")) return e;
  if (int e = check_rows(v, "window_attention", "v")) return e;
  if (int e = check_rows(out, "window_attention", "out")) return e;
  if ((Tq > 1 && (q->stride_t < kD || out->stride_t < kD)) || (Tk > 1 && (k->stride_t < kD || v->stride_t < kD)) ||
      (Hq > 1 && out->stride_h < kD) || (B > 1 && out->stride_b < kD))
    return fail(MIKV_EINVAL, "window_attention: rows overlap");
  CUtensorMap qm, km, vm;
  WindowArgs a;
  a.out = row_view(*out);
  a.lse = lse;
  a.q_lens = q_lens;
  a.k_lens = k_lens;
  a.Hq = Hq;
  a.rep = Hq / Hkv;
  a.Tq = Tq;
  a.Tk = Tk;
  a.window = window >= Tk ? 0 : window;   // one that reaches every key is none
  a.sinks = std::min(sinks, Tk);
  a.rows = static_cast<int64_t>(B) * Hq * Tq;
  a.wide_out = ((reinterpret_cast<uintptr_t>(out->data) | static_cast<uintptr_t>(a.out.sb | a.out.sh | a.out.st)) & 31u) == 0;
  a.scale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
  const Plan p = plan_of(B, Hq, Hkv, Tq, Tk, a.window, a.sinks, packs(*q, Hq));
  a.tb = p.tb;
  a.hb = p.hb;
  a.groups = p.groups;
  a.blocks = p.blocks;
  a.pair_heads = p.pair_heads;
  a.splits = p.splits;
  if (p.per_head * p.splits > 0x7fffffffLL) return fail(MIKV_ESHAPE, "window_attention: Tq=%d Hq=%d", Tq, Hq);
  const size_t need = part_bytes(p, a.rows);
  if (need > 0) {
    if (!ws) return fail(MIKV_EINVAL, "window_attention: null workspace");
    if (reinterpret_cast<uintptr_t>(ws) & 31u) return fail(MIKV_EALIGN, "window_attention: workspace must be 32-byte aligned");
    if (ws_bytes < need) return fail(MIKV_ESHAPE, "window_attention: workspace %zu < %zu", ws_bytes, need);
  }
  a.part = static_cast<float*>(ws);
  if (int e = encode_queries(&qm, *q, Tq, a.rep, Hkv, B, p, &a.qb, &a.qh)) return e;
  if (int e = encode_view(&km, *k, Tk, Hkv, B, "k", &a.kb, &a.kh)) return e;
  if (int e = encode_view(&vm, *v, Tk, Hkv, B, "v", &a.vb, &a.vh)) return e;
  const bool bf = type == MIKV_PAGES_BF16;
  const auto kern = bf ? p.splits > 1 ? window_attention_kernel<true, true> : window_attention_kernel<true, false>
                       : p.splits > 1 ? window_attention_kernel<false, true> : window_attention_kernel<false, false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kWaSmem);
  if (e != cudaSuccess) return check_launch_after(e, "window_attention_kernel");
  const cudaStream_t st = as_stream(stream);
  kern<<<dim3(static_cast<unsigned>(p.per_head * p.splits), Hkv, B), kWaThreads, kWaSmem, st>>>(qm, km, vm, a);
  if (int r = check_launch("window_attention_kernel")) return r;
  if (p.splits == 1) return MIKV_OK;
  // Two parts at a time of rows enough to hide it, eight where a row has more; and four warps a row
  // where there are not eight rows an SM (five rows of 8 heads, 32 parts: 18 us with one warp a row,
  // 13 with four; 4096 rows, 9 parts: 30 and 35).
  const bool few = p.splits <= 4, wide = !few && a.rows <= 8 * kNumSMs;
  const auto join = few    ? bf ? window_join_kernel<true, 1, 2> : window_join_kernel<false, 1, 2>
                    : wide ? bf ? window_join_kernel<true, 4, 8> : window_join_kernel<false, 4, 8>
                           : bf ? window_join_kernel<true, 1, 8> : window_join_kernel<false, 1, 8>;
  const int64_t per = wide ? 1 : 4;
  return check_launch_after(launch_after(join, dim3(static_cast<unsigned>((a.rows + per - 1) / per)), dim3(128), 0, st, a),
                            "window_join_kernel");
}
