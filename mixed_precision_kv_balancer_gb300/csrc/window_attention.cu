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
// idle, all their key tiles form one line, of which each CTA takes an equal part, and the items that
// are cut are joined by a second kernel.  Key and value tiles of 128 rows come through a ring of four
// 32 KB buffers (TMA, 128-byte swizzle; a fifth was no faster); tiles that none of the rows sees are not read.  Per key tile i and query tile t
//   S_t = Q_t K_i^T     tcgen05, both operands in shared memory, 128 fp32 TMEM columns
//   P_t = exp2(...)     four warps, one query row a thread, written over S_t as 16-bit pairs
//   O_t += P_t V_i      tcgen05, P from TMEM, V as it lies (rows are the contraction)
// The tensor core runs [O_0 += P_0 V_i, S_0 = Q_0 K_i+1] while the warps of tile 1 make their
// weights, and the other way round.  S_t(i + 1) is committed behind O_t(i), so a thread that
// holds new scores may rescale its accumulator row without another wait.
//
// Weights are rounded to the inputs' type once, which is what the value products take (a second part
// would be half as many products again, and they bound the kernel); their sum is taken before that, in
// fp32.  Error against 64 bits of 8192 causal rows in BF16 2.1e-3, with 32-bit weights 1.6e-3; chunks
// of 500 in FP16 2.9e-4 and 2.1e-4.  fp16 weights carry a factor 2^kShift, which keeps weights down
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
#include "window_index.h"

namespace mikv {

int window_attention_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kWaRows = kKeyRows;                // query rows and key rows of a tile
constexpr int kWaNarrow = 32;                    // columns of a tile that holds the last few sinks
constexpr int kWaRing = 4;
constexpr int kMaxRows = 1 << 30;                // of q or k: positions and their differences fit 32 bits
constexpr int kWaThreads = 352;                  // 2 x 4 softmax warps, the TMA warp, 2 MMA warps
constexpr int kWaTmaWarp = 8, kWaMmaWarp = 9;
constexpr int kWaOut = 4096;                     // a warp's 32 output rows, 64 channels of them
constexpr int kWaSmem = (2 + kWaRing) * tc::kTileBytes + 8 * kWaOut + 1024;
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
  float* part;                   // the line's cut items, see part_sums and part_ml
  const int32_t *q_lens, *k_lens;
  int Hq, rep, Tq, Tk, B, Hkv;
  QueryBlocks qb;                // rows of a tile, the mask
  int hb, groups;                // a tile: qb.tb rows of each of hb heads; groups = ceil(rep / hb)
  int per;                       // items of one row block and key head
  int tile_rows;                 // rows of a tile that can count: min(qb.tb, Tq) hb
  int ctas;                      // of the line
  int share;                     // CTAs an item where each item has as many; 0: equal parts of the line
  bool wide_out;                 // rows of out begin at multiples of 32 bytes
  int qbat, qh, kb, kh, vb, vh;  // 1, or 0 where the view repeats one batch row or head
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

// An item, or the part of one that a CTA of the line takes.
struct Place {
  int b, hk, blk, u;   // batch row, key head, row block, item of these
  int t0, t1;          // the line: its key tiles
  bool whole;          // all of the item
};
// What one CTA works on; every warp computes it alike.
struct Work {
  int ql, kl, off;        // lengths; position of query 0
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
__device__ __forceinline__ int q_len(const WindowArgs& a, int b) { return a.q_lens ? min(max(a.q_lens[b], 0), a.Tq) : a.Tq; }
__device__ __forceinline__ int k_len(const WindowArgs& a, int b) { return a.k_lens ? min(max(a.k_lens[b], 0), a.Tk) : a.Tk; }
template <bool LINE>
__device__ __forceinline__ Work work_of(const WindowArgs& a, const Place& pl) {
  Work w;
  w.ql = uniform(q_len(a, pl.b));
  w.kl = uniform(k_len(a, pl.b));
  w.off = w.kl - w.ql;
  const int tb = a.qb.tb;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    w.group[t] = a.qb.pair_heads ? 2 * pl.u + t : pl.u;
    w.q0[t] = first_row(a.qb, pl.blk) + (a.qb.pair_heads ? 0 : t * tb);
    w.pa[t] = w.off + w.q0[t];
    w.pb[t] = w.off + min(w.q0[t] + tb, w.ql) - 1;
  }
  w.nt = w.q0[0] >= w.ql ? 0 : w.q0[1] >= w.ql || w.group[1] >= a.groups ? 1 : 2;
  const KeyTiles k = key_tiles(a.qb, w.ql, w.kl, pl.blk);
  w.ts = k.ts;
  w.tw0 = k.tw0;
  w.ns = k.ns;
  w.begin = LINE ? min(pl.t0, k.tiles) : 0;
  w.end = LINE ? min(pl.t1, k.tiles) : k.tiles;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int e = w.pb[t] < 0 ? -1 : w.pb[t] / kWaRows;
    w.from[t] = w.ts + (a.qb.window > 0 ? max(w.pa[t] - a.qb.window + 1, 0) / kWaRows - w.tw0 : 0);
    int last = t >= w.nt || e < 0 ? -1 : e - w.tw0 + w.ts;
    if (LINE) {   // the last one of this part
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
  return j0 + kWaRows - 1 <= t.pa && (a.qb.window == 0 || j0 > t.pb - a.qb.window || j0 + kWaRows <= a.qb.sinks);
}
// Whether a key tile counts with its first kWaNarrow columns alone: the sinks' last tile, mostly
// (a window of 1024 with 4 sinks is ten tiles, one of them for the sinks: 79 -> 75 us).
__device__ __forceinline__ bool tile_narrow(const WindowArgs& a, const Work& w, int i) {
  return i < w.ts && a.qb.sinks - w.j0(i) <= kWaNarrow;
}
// Rows [z0, z1) and [z2, 128) of the value tile at j0 that no query of the call sees.
struct Hidden {
  int z0, z1, z2;
  __device__ __forceinline__ bool any() const { return z0 < z1 || z2 < kWaRows; }
};
__device__ __forceinline__ Hidden hidden_rows(const WindowArgs& a, const Work& w, int j0) {
  Hidden h;
  h.z0 = min(max(a.qb.sinks - j0, 0), kWaRows);
  h.z1 = a.qb.window > 0 ? min(max(w.off - a.qb.window + 1 - j0, 0), kWaRows) : 0;
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
    const int hi = p - j0, lo = a.qb.window > 0 ? hi - a.qb.window + 1 : 0, sk = a.qb.sinks - j0;
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
__device__ __forceinline__ void ask_next(uint32_t answer, uint32_t mbar) {
  tc::mbar_expect_tx(mbar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(answer),
               "r"(mbar)
               : "memory");
}
// The answer to ask n, by the whole warp: false where nothing is left.
__device__ __forceinline__ bool heard_next(WaBars& bar, const uint4* answers, int n, tc::Waits& wait, int& at_x, int& at_y, int& at_z) {
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
  at_x = uniform(x);
  at_y = uniform(y);
  at_z = uniform(z);
  return __all_sync(0xffffffffu, ok != 0 && wait.ok);
}

// An entry of the line: the places before it, and those of each of its items.
struct Spot {
  int e, base, places;
};
__device__ __forceinline__ int places_of(const WindowArgs& a, int e) {
  if (e >= a.B * a.qb.blocks) return 0;
  const int b = e / a.qb.blocks;
  return entry_places(a.qb, q_len(a, b), k_len(a, b), a.qb.blocks - 1 - e % a.qb.blocks);
}
// Places of 32 entries, one a lane, and their sums up to it.
struct Sums {
  int v, incl;
};
__device__ __forceinline__ Sums sums_of(const WindowArgs& a, int e0) {
  const int lane = threadIdx.x & 31;
  Sums s;
  s.v = s.incl = places_of(a, e0 + lane);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s.incl, o);
    if (lane >= o) s.incl += u;
  }
  return s;
}
// All places, by a whole warp; the host keeps them below 2^31.  `first`: sums_of the first entries.
__device__ __forceinline__ int line_total(const WindowArgs& a, const Sums& first) {
  int sum = __shfl_sync(0xffffffffu, first.incl, 31);
  for (int e0 = 32; e0 < a.B * a.qb.blocks; e0 += 32) sum += __reduce_add_sync(0xffffffffu, places_of(a, e0 + (threadIdx.x & 31)));
  return uniform(sum) * a.Hkv * a.per;
}
// The entry that holds place `pos` (below the total), by a whole warp.
__device__ __forceinline__ Spot spot_of(const WindowArgs& a, const Sums& first, int pos) {
  const int items = a.Hkv * a.per;
  Spot s = {0, 0, 0};
  for (Sums n = first;; n = sums_of(a, s.e)) {
    const int below = __popc(__ballot_sync(0xffffffffu, s.base + n.incl * items <= pos));   // entries that end at or before it
    if (below < 32 || s.e + 32 >= a.B * a.qb.blocks) {
      const int at = min(below, 31);
      s.places = uniform(__shfl_sync(0xffffffffu, n.v, at));
      s.base = uniform(s.base + (__shfl_sync(0xffffffffu, n.incl, at) - s.places) * items);
      s.e = uniform(s.e + at);
      return s;
    }
    s.base += __shfl_sync(0xffffffffu, n.incl, 31) * items;
    s.e += 32;
  }
}

// What a warp walks: the items that its CTA is given (the grid's, then taken over), or its part of
// the line.
template <bool LINE>
struct Walk {
  int x, y, z;   // the item; the line: the next place, the end
  Spot at;       // the line: the entry of place x
  int t0, t1;    // share > 0: the part of the item
  bool idle;     // the line: nothing for this CTA
  int4 cut;      // the line: the item that begins here and goes on in later CTAs: entry, item, last CTA (-1: none),
                 // whether this CTA's part of it has items before

  __device__ __forceinline__ explicit Walk(const WindowArgs& a) {
    x = blockIdx.x;
    y = blockIdx.y;
    z = blockIdx.z;
    at = {0, 0, 1};
    idle = false;
    cut = {0, 0, -1, 0};
    t0 = t1 = 0;
    if (LINE && a.share > 0) {
      const int items = a.Hkv * a.per, part = x % a.share, item = x / a.share;
      at = {uniform(item / items), 0, 0};
      at.places = uniform(places_of(a, at.e));
      idle = __all_sync(0xffffffffu, at.places == 0);
      if (!idle && part == 0) cut = {at.e, item % items, x + a.share - 1, 0};
      const int tiles = at.places - kItemPlaces;
      t0 = uniform(line_begin(tiles, a.share, part));
      t1 = uniform(line_begin(tiles, a.share, part + 1));
      x = uniform(item % items);
    } else if (LINE) {
      const Sums first = sums_of(a, 0);
      const int total = line_total(a, first), workers = line_workers(total, a.ctas), c = blockIdx.x;
      idle = __all_sync(0xffffffffu, c >= workers || total == 0);
      if (!idle) {
        x = uniform(line_begin(total, workers, c));
        y = uniform(line_begin(total, workers, c + 1));
        at = spot_of(a, first, x);
        const int before = (x - at.base) % at.places;
        if (line_tile(before) == 0) x = uniform(x - before);
        if (y < total) {   // an end among an item's first places is the item's begin
          const Spot s = spot_of(a, first, y);
          const int item = (y - s.base) / s.places, begin = s.base + item * s.places;
          if (line_tile(y - begin) == 0)
            y = uniform(begin);
          else if (begin >= x && threadIdx.x < 32)   // who asks: see part_cut
            cut = {s.e, item, split_owner(total, workers, begin + s.places - 1), begin > x};
        }
        idle = __all_sync(0xffffffffu, x >= y);
      }
    }
  }
  __device__ __forceinline__ Place place(const WindowArgs& a) const {
    if (!LINE) return {z, y, a.qb.blocks - 1 - x / a.per, x % a.per, 0, 0, true};   // the last rows, which see the most, first
    if (a.share > 0) {
      const int b = uniform(at.e / a.qb.blocks), hk = uniform(x / a.per);
      return {b, hk, uniform(a.qb.blocks - 1 - (at.e - b * a.qb.blocks)), uniform(x - hk * a.per), t0, t1, false};
    }
    const int item = (x - at.base) / at.places, in = x - at.base - item * at.places, tiles = at.places - kItemPlaces;
    const int t0 = uniform(line_tile(in)), t1 = uniform(min(tiles, line_tile(in + y - x)));
    const int b = uniform(at.e / a.qb.blocks), hk = uniform(item / a.per);
    return {b, hk, uniform(a.qb.blocks - 1 - (at.e - b * a.qb.blocks)), uniform(item - hk * a.per), t0, t1, t1 - t0 == tiles};
  }
  // On to the next one, by the whole warp; false where there is none.
  __device__ __forceinline__ bool next(const WindowArgs& a, WaBars& bar, const uint4* answers, int n, tc::Waits& wait) {
    if (!LINE) return heard_next(bar, answers, n, wait, x, y, z);
    if (a.share > 0) return false;
    x += at.places - (x - at.base) % at.places;
    if (!__all_sync(0xffffffffu, x < y && wait.ok)) return false;
    if (__all_sync(0xffffffffu, x == at.base + at.places * a.Hkv * a.per)) {
      at.base = x;
      do at.places = uniform(places_of(a, ++at.e));
      while (__all_sync(0xffffffffu, at.places == 0 && at.e < a.B * a.qb.blocks));
    }
    return __all_sync(0xffffffffu, at.places > 0);
  }
};

// A CTA of the line has two slots for parts of items that others hold too, for its first and its last.
// A slot: the rows of two query tiles, 128 sums each, as [query tile][8 channels][row][8], so that the rows of a warp
// are written side by side; the rows' (maximum, sum) behind all slots.
__device__ __forceinline__ float* part_sums(const WindowArgs& a, int slot, int t, int row, int ch) {
  const int64_t tile = static_cast<int64_t>(slot) * 2 + t;
  return a.part + ((tile * (kD / 8) + ch / 8) * a.tile_rows + row) * 8 + ch % 8;
}
__device__ __forceinline__ float2* part_ml(const WindowArgs& a, int slot, int t, int row) {
  float2* ml = reinterpret_cast<float2*>(a.part + static_cast<int64_t>(a.ctas) * 4 * a.tile_rows * kD);
  return ml + (static_cast<int64_t>(slot) * 2 + t) * a.tile_rows + row;
}
// Behind them what each CTA says of the item it cuts first (Walk::cut).
__device__ __forceinline__ int4* part_cut(const WindowArgs& a, int c) {
  return reinterpret_cast<int4*>(a.part + static_cast<int64_t>(a.ctas) * 4 * a.tile_rows * (kD + 2)) + c;
}

template <bool BF, bool LINE>
__global__ void __launch_bounds__(kWaThreads, 1)
    window_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap, const WindowArgs a) {
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
  if (LINE) pdl_trigger();   // the joining kernel may be placed; it waits for this one's end
  const uint32_t sq = tc::smem_base(smem), ring = sq + 2 * tc::kTileBytes;
  tc::Waits wait;
  Walk<LINE> walk(a);
  if (LINE && threadIdx.x == 0) *part_cut(a, blockIdx.x) = walk.cut;

  if (walk.idle) {
    // more CTAs than parts
  } else if (warp == kWaTmaWarp) {
    int slot = 0, par = 1, qs = 0;   // ring position; parity that an empty buffer shows; query loads
    for (int n = 0;; ++n) {
      const Place pl = walk.place(a);
      const int b = pl.b, hk = pl.hk;
      const Work w = work_of<LINE>(a, pl);
      if (w.nt > 0 && w.begin < w.end) {
        if (qs > 0) wait(smem_u32(&bar.qfree), (qs - 1) & 1);
        ++qs;
        if (lane == 0 && wait.ok) {
          tc::mbar_expect_tx(smem_u32(&bar.q), w.nt * a.qb.tb * a.hb * kD * 2);
          tma_queries(sq, &qmap, w.q0[0], w.group[0] * a.hb * a.qh, hk * a.qh, b * a.qbat, smem_u32(&bar.q));
          if (w.nt == 2)
            tma_queries(sq + tc::kTileBytes, &qmap, w.q0[1], w.group[1] * a.hb * a.qh, hk * a.qh, b * a.qbat, smem_u32(&bar.q));
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
      if (!LINE) {
        if (n >= 2) wait(smem_u32(&bar.heard[n & 1]), ((n >> 1) - 1) & 1);
        if (lane == 0 && wait.ok) ask_next(smem_u32(&answers[n & 1]), smem_u32(&bar.told[n & 1]));
      }
      if (!walk.next(a, bar, answers, n, wait)) break;
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
      const Work w = work_of<LINE>(a, walk.place(a));
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
      if (!walk.next(a, bar, answers, n, wait)) break;
    }
  } else {
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;   // the thread's TMEM lane is its row
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + kWaO + t * 128;
    const uint32_t ready[2] = {smem_u32(&bar.p[t][0]), smem_u32(&bar.p[t][1])};
    int s_par = 0, o_par = 0;
    for (int n = 0;; ++n) {
      const Place pl = walk.place(a);
      const int b = pl.b;
      const Work w = work_of<LINE>(a, pl);
      const Tile tile = tile_of(w, t);
      if (tile.live) {
        const int p = tile.pa + row % a.qb.tb;
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
        const int sub = row / a.qb.tb, q = tile.q0 + row - sub * a.qb.tb, h = tile.group * a.hb + sub;   // the row's query and head
        const bool write = sub < a.hb && h < a.rep && q < w.ql;
        const int head = pl.hk * a.rep + h;
        const int64_t at = (static_cast<int64_t>(b) * a.Hq + head) * a.Tq + q;
        const bool part = LINE && !pl.whole;
        const int slot = 2 * blockIdx.x + (n > 0);
        float inv = part ? 1.f : r.l == 0.f ? 0.f : 1.f / r.l;
        if (!wait.ok) inv = __int_as_float(0x7fffffff);
        uint8_t* dst = a.out.row(b, head, q);
        // A warp whose 32 rows follow one another, and count as far as there are any, hands them to the TMA
        // through a buffer of its own: written by the threads, 32 rows an instruction, they hold the warp up
        // (2 x 16384 rows of 4 heads under a window of 1024: 73 us, 69 this way).
        const int q_first = tile.q0 + (warp & 3) * 32;
        const bool whole_rows = !part && a.hb == 1 && h < a.rep && q_first < w.ql && (q_first + 32 <= w.ql || w.ql == a.Tq);
        if (__all_sync(0xffffffffu, whole_rows)) {
          const uint32_t stage = ring + kWaRing * tc::kTileBytes + warp * kWaOut;
#pragma unroll 1
          for (int c = 0; c < kD; c += 64) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");   // the buffer is free
            __syncwarp();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float o[32];
              if (tile.last >= 0) {
                ld32(to + c + half * 32, o);
                wait_ld();
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(stage + lane * 128 + (((half * 4 + k) ^ (lane & 7)) << 4)),
                             "r"(pack2<BF>(o[8 * k] * inv, o[8 * k + 1] * inv)), "r"(pack2<BF>(o[8 * k + 2] * inv, o[8 * k + 3] * inv)),
                             "r"(pack2<BF>(o[8 * k + 4] * inv, o[8 * k + 5] * inv)), "r"(pack2<BF>(o[8 * k + 6] * inv, o[8 * k + 7] * inv))
                             : "memory");
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];\n" ::"l"(&omap), "r"(c),
                           "r"(q_first), "r"(head), "r"(b), "r"(stage)
                           : "memory");
              asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
            }
          }
        } else {
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
              if (!part) {
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
                for (int e = 0; e < 32; e += 8) st_global32(part_sums(a, slot, t, row, c + e), u + e);
              }
            }
          }
        }
        if (part && write) {
          *part_ml(a, slot, t, row) = make_float2(r.m * a.scale, wait.ok ? r.l : inv);
        } else if (write && a.lse) {
          const float v = r.l == 0.f ? -INFINITY : (r.m * a.scale + (log2f(r.l) - Weights<BF>::shift)) * 0.6931471805599453f;
          a.lse[at] = wait.ok ? v : inv;
        }
        tc::fence_before_sync();   // the sums are read before the next item's products overwrite them
      }
      if (!walk.next(a, bar, answers, n, wait)) break;
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");   // the last rows are written before the CTA ends
  }
  if (!wait.ok) tc::report_giveup(tc::kGiveupWindow);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWaMmaWarp) tc::tmem_dealloc(tmem, kWaCols);
}

constexpr int kLineWords = (kNumSMs + 31) / 32;
// CTA (slice, k): joins ROWS rows of the k-th item of the line that is cut, in a fixed order.  A thread
// takes 8 channels of a row (a part's rows lie side by side); GROUPS sets of threads share the parts,
// BATCH of them requested together.
template <bool BF, int ROWS, int GROUPS, int BATCH>
__global__ void __launch_bounds__(ROWS * (kD / 8) * GROUPS) window_join_kernel(const WindowArgs a) {
  constexpr int kThreads = ROWS * (kD / 8);   // of a group
  __shared__ float s_o[GROUPS > 1 ? GROUPS - 1 : 1][8][kThreads];
  __shared__ float2 s_ml[GROUPS > 1 ? GROUPS - 1 : 1][kThreads];
  const int tid = threadIdx.x % kThreads, group = threadIdx.x / kThreads, lane = threadIdx.x & 31;
  pdl_wait();
  int c0 = -1;   // the first CTA of that item: the k-th that has begun one and not ended it
  if (a.share > 0) {
    c0 = blockIdx.y * a.share;
  } else {
    int k = blockIdx.y;
    uint32_t begun[kLineWords];
#pragma unroll
    for (int w = 0; w < kLineWords; ++w) begun[w] = __ballot_sync(0xffffffffu, w * 32 + lane < a.ctas && part_cut(a, w * 32 + lane)->z >= 0);
#pragma unroll
    for (int w = 0; w < kLineWords; ++w) {
      const uint32_t hit = __ballot_sync(0xffffffffu, (begun[w] >> lane & 1u) && __popc(begun[w] & ((1u << lane) - 1u)) == k);
      if (hit) c0 = w * 32 + __ffs(hit) - 1;
      k -= __popc(begun[w]);
    }
    if (c0 < 0) return;
  }
  const int4 cut = *part_cut(a, c0);
  const int c1 = cut.z;
  if (c1 < 0) return;
  const int b = cut.x / a.qb.blocks, blk = a.qb.blocks - 1 - cut.x % a.qb.blocks, hk = cut.y / a.per, u = cut.y % a.per;
  const int rows = a.tile_rows, ch = tid / ROWS * 8;
  const int i = blockIdx.x * ROWS + tid % ROWS, t = i >= rows, row = i - t * rows, sub = row / a.qb.tb;
  const int heads = a.qb.pair_heads ? 2 * u + t : u, h = heads * a.hb + sub;
  const int q = first_row(a.qb, blk) + (a.qb.pair_heads ? 0 : t * a.qb.tb) + row - sub * a.qb.tb;
  const bool live = i < 2 * rows && heads < a.groups && h < a.rep && q < q_len(a, b);
  float m = -INFINITY, l = 0.f, o[8] = {};
  const auto add = [&](float2 x, const float (&p)[8]) {
    const float mn = fmaxf(m, x.x), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ref), fx = ex2(x.x - ref);
    l = l * f + x.y * fx;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * f + p[e] * fx;
    m = mn;
  };
  if (live) {
    for (int p0 = c0 + group; p0 <= c1; p0 += BATCH * GROUPS) {
      float2 x[BATCH];
      float4 v[BATCH][2];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int p = p0 + e * GROUPS, slot = 2 * p + (p == c0 ? cut.w : 0);
        x[e] = make_float2(-INFINITY, 0.f);
        v[e][0] = v[e][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p <= c1) {
          const float4* sums = reinterpret_cast<const float4*>(part_sums(a, slot, t, row, ch));
          x[e] = *part_ml(a, slot, t, row);
          v[e][0] = sums[0];
          v[e][1] = sums[1];
        }
      }
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        // a sum of 0: nothing seen there, and no sums written
        const bool none = x[e].y == 0.f;
        const float w[8] = {none ? 0.f : v[e][0].x, none ? 0.f : v[e][0].y, none ? 0.f : v[e][0].z, none ? 0.f : v[e][0].w,
                            none ? 0.f : v[e][1].x, none ? 0.f : v[e][1].y, none ? 0.f : v[e][1].z, none ? 0.f : v[e][1].w};
        add(x[e], w);
      }
    }
  }
  if (GROUPS > 1) {
    if (group > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s_o[group - 1][e][tid] = o[e];
      s_ml[group - 1][tid] = make_float2(m, l);
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < GROUPS - 1; ++g) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = s_o[g][e][tid];
      add(s_ml[g][tid], w);
    }
  }
  if (!live) return;
  const int head = hk * a.rep + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint4*>(a.out.row(b, head, q) + ch * 2) =
      make_uint4(pack2<BF>(o[0] * inv, o[1] * inv), pack2<BF>(o[2] * inv, o[3] * inv), pack2<BF>(o[4] * inv, o[5] * inv),
                 pack2<BF>(o[6] * inv, o[7] * inv));
  if (ch == 0 && a.lse)
    a.lse[(static_cast<int64_t>(b) * a.Hq + head) * a.Tq + q] =
        l == 0.f ? -INFINITY : (m + (log2f(l) - Weights<BF>::shift)) * 0.6931471805599453f;
}

// The layout of a call: rows and heads of a tile, items, and whether their key tiles form a line.
struct Plan {
  QueryBlocks qb;
  int hb, groups, per, tile_rows, ctas, share;   // ctas: of the line; 0: a CTA an item
  int64_t per_head;            // items of one key head and batch row
};
// `pack`: heads of a group may share a tile (their rows are apart in memory).
Plan plan_of(int B, int Hq, int Hkv, int Tq, int Tk, int window, int sinks, bool pack) {
  Plan p;
  const int rep = Hq / Hkv;
  p.hb = pack ? std::min(rep, std::max(1, kWaRows / Tq)) : 1;
  p.qb.tb = p.hb > 1 ? Tq : kWaRows;
  p.tile_rows = std::min(p.qb.tb, Tq) * p.hb;
  p.qb.window = window;
  p.qb.sinks = sinks;
  p.groups = (rep + p.hb - 1) / p.hb;
  const int blocks = (Tq + p.qb.tb - 1) / p.qb.tb;
  p.qb.pair_heads = p.groups % 2 == 0 || blocks == 1;
  p.qb.blocks = p.qb.pair_heads ? blocks : (blocks + 1) / 2;
  p.per = p.qb.pair_heads ? (p.groups + 1) / 2 : p.groups;
  p.per_head = static_cast<int64_t>(p.qb.blocks) * p.per;
  p.ctas = p.share = 0;
  // How the call ends soonest, by estimates in key tiles of an item's two query tiles (1.4 us each; an
  // item costs 3 beside its own).
  //   a CTA an item: the longest item bounds the end, and items of about one length run in whole waves
  //   up to half as many items as SMs: `share` CTAs each (the sums of cut items go out to memory and come
  //     back: 2, and 0.7 for every 16 parts)
  //   more: equal parts of the line, 13 and 3 a wave for the cuts
  // Measured, a CTA an item / cut: 8192 causal rows of 4 heads, 128 items, 99 / 66 us; 4096 of 8 heads, 128
  // items, 54 / 46; 2048 of 32, 256 items, 46 / 49; 64 rows of 8 heads behind 16384 keys, 4 items, 184 / 17; one row
  // of 32 heads behind 700 keys, 8 items, 13 / 11, behind 300, 9 / 10; 2 x 256 rows of 16 heads behind 2744, 64
  // items, two CTAs each 22 us, as a line 25.
  const int64_t items = p.per_head * Hkv * B;
  const int64_t rows = static_cast<int64_t>(p.qb.pair_heads ? 1 : 2) * p.qb.tb;
  double longest = Tk, mean = Tk - 0.5 * std::min(Tq, Tk);
  if (window > 0) {
    longest = std::min<double>(longest, static_cast<double>(window) + sinks + rows);
    mean = std::min(mean, longest);
  }
  longest = std::max(1.0, longest / kWaRows);
  mean = std::max(1.0, mean / kWaRows);
  const double waves = static_cast<double>(items) / kNumSMs;
  double best = std::max(longest + 3, (mean > 0.75 * longest ? std::ceil(waves) : waves + 0.5) * (mean + 3));
  if (items <= kNumSMs / 2) {
    for (int s = 2; s <= kNumSMs / items && longest / s >= 1.0; ++s) {
      const double est = longest / s + 5 + 0.7 * ((s + 15) / 16);
      if (est < best - 1e-9) {
        best = est;
        p.share = s;
        p.ctas = static_cast<int>(items) * s;
      }
    }
  } else if (waves * (mean + 6) + 13 < best && items <= 8 * kNumSMs && static_cast<int64_t>(B) * p.qb.blocks <= 256 &&
             static_cast<double>(items) * (static_cast<double>(Tk) / kWaRows + 2 + kItemPlaces) < 2147483647.0) {
    // (a warp adds up the entries in a few steps, and places stay below 2^31)
    p.ctas = kNumSMs;
  }
  return p;
}
size_t part_bytes(const Plan& p) { return static_cast<size_t>(p.ctas) * 4 * p.tile_rows * (kD + 2) * 4 + p.ctas * 16; }
bool packs(const mikv_rows& q, int Hq) { return Hq == 1 || q.stride_h >= kD; }

// 4-D tensor map (channel, row, head, batch row) of a strided view, box 64 x 128 x 1 x 1 with
// 128-byte swizzle.  A dimension of stride 0 (a repeated head or batch row) has one entry in
// the map; *mb and *mh tell whether the coordinate counts.
int encode_view(CUtensorMap* map, const mikv_rows& r, int T, int H, int B, int rows, const char* name, int* mb, int* mh) {
  const auto enc = tc::tensor_map_encoder();
  if (!enc) return fail(MIKV_ECUDA, "window_attention: cuTensorMapEncodeTiled unavailable");
  *mh = H > 1 && r.stride_h != 0;
  *mb = B > 1 && r.stride_b != 0;
  const cuuint64_t row = T > 1 ? static_cast<cuuint64_t>(r.stride_t) * 2 : kD * 2;
  const cuuint64_t dims[4] = {kD, static_cast<cuuint64_t>(T), *mh ? static_cast<cuuint64_t>(H) : 1, *mb ? static_cast<cuuint64_t>(B) : 1};
  const cuuint64_t strides[3] = {row, *mh ? static_cast<cuuint64_t>(r.stride_h) * 2 : row, *mb ? static_cast<cuuint64_t>(r.stride_b) * 2 : row};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1}, estr[4] = {1, 1, 1, 1};
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
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(p.qb.tb), static_cast<cuuint32_t>(p.hb), 1, 1}, estr[5] = {1, 1, 1, 1, 1};
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
    most = std::max(most, part_bytes(plan_of(B, Hq, Hkv, Tq, Tk, window >= Tk ? 0 : window, std::min(sinks, Tk), pack)));
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
  CUtensorMap qm, km, vm, om;
  WindowArgs a;
  a.out = row_view(*out);
  a.lse = lse;
  a.q_lens = q_lens;
  a.k_lens = k_lens;
  a.Hq = Hq;
  a.rep = Hq / Hkv;
  a.Tq = Tq;
  a.Tk = Tk;
  a.B = B;
  a.Hkv = Hkv;
  a.wide_out = ((reinterpret_cast<uintptr_t>(out->data) | static_cast<uintptr_t>(a.out.sb | a.out.sh | a.out.st)) & 31u) == 0;
  a.scale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
  // a window that reaches every key is none
  const Plan p = plan_of(B, Hq, Hkv, Tq, Tk, window >= Tk ? 0 : window, std::min(sinks, Tk), packs(*q, Hq));
  a.qb = p.qb;
  a.hb = p.hb;
  a.groups = p.groups;
  a.per = p.per;
  a.tile_rows = p.tile_rows;
  a.ctas = p.ctas;
  a.share = p.share;
  if (p.per_head > 0x7fffffffLL) return fail(MIKV_ESHAPE, "window_attention: Tq=%d Hq=%d", Tq, Hq);
  const size_t need = mikv_window_attention_workspace_bytes(B, Hq, Hkv, Tq, Tk, window, sinks);   // whatever q's strides
  if (need > 0) {
    if (!ws) return fail(MIKV_EINVAL, "window_attention: null workspace");
    if (reinterpret_cast<uintptr_t>(ws) & 31u) return fail(MIKV_EALIGN, "window_attention: workspace must be 32-byte aligned");
    if (ws_bytes < need) return fail(MIKV_ESHAPE, "window_attention: workspace %zu < %zu", ws_bytes, need);
  }
  a.part = static_cast<float*>(ws);
  if (int e = encode_queries(&qm, *q, Tq, a.rep, Hkv, B, p, &a.qbat, &a.qh)) return e;
  if (int e = encode_view(&km, *k, Tk, Hkv, B, kWaRows, "k", &a.kb, &a.kh)) return e;
  if (int e = encode_view(&vm, *v, Tk, Hkv, B, kWaRows, "v", &a.vb, &a.vh)) return e;
  int ob, oh;   // rows of out are apart: both coordinates count where there is more than one
  if (int e = encode_view(&om, *out, Tq, Hq, B, 32, "out", &ob, &oh)) return e;
  const bool bf = type == MIKV_PAGES_BF16;
  const bool line = p.ctas > 0;
  const auto kern = bf ? line ? window_attention_kernel<true, true> : window_attention_kernel<true, false>
                       : line ? window_attention_kernel<false, true> : window_attention_kernel<false, false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kWaSmem);
  if (e != cudaSuccess) return check_launch_after(e, "window_attention_kernel");
  const cudaStream_t st = as_stream(stream);
  const dim3 grid = line ? dim3(p.ctas) : dim3(static_cast<unsigned>(p.per_head), Hkv, B);
  kern<<<grid, kWaThreads, kWaSmem, st>>>(qm, km, vm, om, a);
  if (int r = check_launch("window_attention_kernel")) return r;
  if (p.ctas < 2) return MIKV_OK;
  // With 12 parts an item and more, few rows a CTA and 32 parts requested together: five rows of 8 heads, 32
  // parts: 12.6 us in all, 15.9 with 16 rows a CTA and 16 parts; with few parts many rows a CTA (64 items of two
  // parts: 22 us, 33 with threads that find no part).
  const int64_t items = p.per_head * Hkv * B;
  const bool wide = p.ctas >= 12 * items;
  const auto join = wide ? bf ? window_join_kernel<true, 4, 8, 4> : window_join_kernel<false, 4, 8, 4>
                         : bf ? window_join_kernel<true, 16, 1, 4> : window_join_kernel<false, 16, 1, 4>;
  const int rows = wide ? 4 : 16;
  const dim3 joins((2 * a.tile_rows + rows - 1) / rows, static_cast<unsigned>(std::min<int64_t>(p.ctas - 1, items)));
  return check_launch_after(launch_after(join, joins, dim3(wide ? 512 : 256), 0, st, a),
                            "window_join_kernel");
}
