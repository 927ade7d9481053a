// Attention of the rows of a packed batch over the paged cache: chunks of prompts and single tokens side
// by side, under a sliding window with sinks (tcgen05).
//
// Mathematics: one pass over the visible keys, out = sum_j p_j v_j / sum_j p_j with p_j = exp2(l_j - m)
// and a reference m per row (attention_tile.cuh).  Bound by the tensor cores where a request has many
// rows (4 * 128 flop per visible query-key pair), by HBM where it has few (512 or 272 bytes a slot and
// key head).
//
// A CTA holds two tiles of 128 query rows over one key head (chunk_index.h), and walks key tiles of 128
// slots: per key tile i and query tile t
//   S_t = Q_t K_i^T     tcgen05, both operands in shared memory, 128 fp32 TMEM columns
//   P_t = exp2(...)     four warps, one query row a thread, written over S_t as 16-bit pairs
//   O_t += P_t V_i      tcgen05, P from TMEM, V as it lies (rows are the contraction)
// Lengths are known on the device alone and differ from request to request, so that all key tiles of a
// call form one line, of which each CTA takes an equal part; a CTA finds its part in sums over the
// requests, which all of its threads make before it begins.  Items that are cut are joined by the CTA that begins them,
// where the rest is there by then, or by a second kernel.
//
// Four warps bring keys and values from the pages to a ring of four 32 KB buffers (128-byte swizzle), each
// to a buffer of its own: by TMA where the pages' size is a multiple of 8 rows, a page or the largest power of
// two that divides it in a box; row by row (cp.async) otherwise, where a tile begins and ends inside pages.
// Rows that no query of the item sees may hold anything: values are cleared there behind the TMA, or never
// copied.  One more warp walks the line, and tells the others what each item is.
//
// Weights are rounded once to 16 bits, after their sum is taken; two parts of each, as paged attention has them, would be half
// as many products again for chunks, and for few rows a longer way from a tile's scores to its sums: with the rows twice in the
// tile, for either part, 64 single tokens take 187 us instead of 180, two chunks beside 198 tokens 199 instead of 148.
//
// INT8 pages: s * code + z is held as two fp16 numbers, the nearest one and what is left (22 bits): keys rounded
// to fp16 alone put 1e-4 into lse and half as much again into the outputs.  A key tile has 64 keys then, the
// two parts of each 64 rows apart in its buffer, so that all copies and products are as above: S_t has the two parts'
// scores side by side, and P_t meets both parts of the values.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <type_traits>

#include "attention_tile.cuh"
#include "chunk_index.h"

namespace mikv {

int chunk_attention_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

using namespace at;

constexpr int kCaRows = kKeyRows;           // query rows of a tile, and rows of a buffer
constexpr int kCaNarrow = 32;               // columns of a tile that holds the last few sinks
constexpr int kCaRing = 4;
// Warps: 2 x 4 for the softmax of a query tile each, the loading ones, 2 that issue products, the walking one, an idle one.
// INT8 takes eight loading warps: converting codes is most of the work beside the products (four of them
// bring 64 single tokens behind up to 8192 slots in 463 us, eight in 365).  Registers of a thread, by warpgroups, are shares of those at launch.
template <bool Q8>
struct Warps {
  static constexpr int load = 8, loaders = Q8 ? 8 : 4, mma = load + loaders, walk = mma + 2, threads = (mma + 4) * 32;
  static constexpr int launch_regs = Q8 ? 96 : 128, softmax_regs = Q8 ? 128 : 176, load_regs = Q8 ? 80 : 88, mma_regs = Q8 ? 64 : 72;
  static_assert(256 * softmax_regs + 32 * loaders * load_regs + 128 * mma_regs <= threads * launch_regs && threads * launch_regs <= 65536,
                "register split");
};
constexpr int kCaTold = 4;                  // items that the other warps may be behind
constexpr int kCaSmem = (2 + kCaRing) * tc::kTileBytes + 1024;
constexpr uint32_t kCaCols = 512;           // S_0, S_1, O_0, O_1: 128 columns each
constexpr uint32_t kCaO = 256;
constexpr int kMaxRequests = 4096;
constexpr int kMaxChunkRows = 1 << 20;      // of a call: the sums of its blocks fit the ring
template <int TYPE>
constexpr int kKeys = TYPE == MIKV_PAGES_INT8 ? 64 : kCaRows;   // of a tile

// fp16 weights reach 2^15.9, and may grow by 2^7.9 before the reference follows: every rescaling of the sums holds up a
// warp's 32 rows (with 2^13 and 2^2: four chunks of 512 behind 8192, 117 us instead of 109; chunk_window_int8's 158 instead of
// 146).  A weight below 2^-22 of the largest is a subnormal number then, which the products keep, in steps of 2^-32.
template <bool BF>
struct RowWeights {
  static constexpr float shift = BF ? 0.f : 8.f, grow = BF ? 8.f : 7.9375f;
};
struct Mask {
  int32_t window, sinks;
};
struct ChunkArgs {
  Pool p;
  RowView q, out;
  float* lse;
  float* part;                 // the line's cut items, see part_sums and part_ml
  const int32_t *seqs, *start, *row_start;
  int layer, n, rows, Hq, rep, ctas;
  int tile_rows;               // rows of a tile that can count
  Mask qb;
  int box;                     // rows of a TMA box: a power of two from 8 on that divides a page and a tile; 0: no TMA
  bool wide_out;               // rows of out begin at multiples of 32 bytes
  float scale;                 // log2(e) / sqrt(D)
  uint64_t tag;                // of this call, see part_ready
};

struct CaBars {
  uint64_t told[kCaTold], heard[kCaTold];   // the item is known; every warp is done with it
  uint64_t full[kCaRing], empty[kCaRing];   // buffer landed; the products that read it are done
  uint64_t boxes[kCaRing];                  // its boxes landed: rows of it have to be cleared yet
  uint64_t turn[2];                         // the tile's products may be issued
  uint64_t qfree;                           // the products that read the queries are done
  uint64_t q, s[2], p[2][2], o[2];          // queries landed; scores, half the weights, last sums written
  uint64_t one_s[2], one_p[2][2], one_o;    // of an item of one query tile: its scores and weights by key tiles in turn; sums
};

// A request as every warp reads it.
struct Request {
  int row0, seq;
  Rows r;
  RowTiles t;
};
__device__ __forceinline__ int request_row(const ChunkArgs& a, int i) { return min(max(a.row_start[i], 0), a.rows); }
__device__ __forceinline__ Request request_of(const ChunkArgs& a, int i) {
  Request q;
  q.row0 = request_row(a, i);
  const int rows = max(request_row(a, i + 1) - q.row0, 0);
  q.seq = a.seqs ? a.seqs[i] : i;
  const bool there = static_cast<uint32_t>(q.seq) < static_cast<uint32_t>(a.p.max_seqs);
  const int held = there ? a.p.len_of(q.seq) : 0;   // (asked for beside the rows that tell whether it counts)
  q.r = rows_of(rows, rows > 0 ? held : 0, a.start != nullptr, a.start ? a.start[i] : 0);
  q.t = row_tiles_of(rows, a.rep);
  return q;
}

// What of an item that is cut the joining kernel has to know; written by the CTA that begins it.
struct Cut {
  int last;          // the CTA that ends it; -1: none is cut
  int before;        // whether that CTA's part of the line has items before
  int row0, rows, q0[2], head[2], heads[2], tb;   // per tile: first row of the request, first head of q, heads (0: no tile)
  uint8_t done[2][4];   // 32 rows of a tile that the CTA has joined itself
};
static_assert(kNumSMs * sizeof(Cut) % sizeof(uint64_t) == 0, "tags lie behind");

// What one CTA works on, in shared memory: written by the walking warp, read by the others.
struct Work {
  int head[2], heads[2], q0[2];   // per tile: first head of q, heads of it that count; first row of the request
  int pa[2], pb[2];       // positions of its first and last row
  int from[2], last[2];   // query tile t sees the sinks' key tiles and tiles from .. last; last -1: none
  int begin, end;         // key tiles of this part: of ts of the sinks, then tw0, tw0 + 1, ...
  int ts, tw0;
  int ns;                 // key tiles that hold sinks, of either part of the list
  int nt;                 // query tiles; -1: there is no further item
  int whole;              // all of the item
  int two;                // the next CTA has the rest of it
  int rest;               // the end of an item that a CTA before begins, with more items behind
  int row0, rows, keys, tb, seq;   // of the request
  template <int KT>
  __device__ __forceinline__ int j0(int i) const { return (i < ts ? i : tw0 + i - ts) * KT; }
  __device__ __forceinline__ bool sees(int t, int i) const { return i <= last[t] && (i < ns || i >= from[t]); }
};
// Item `item` of block `blk`, key tiles t0 .. t1 of it.
template <int KT>
__device__ __forceinline__ Work work_of(const ChunkArgs& a, const Request& q, int blk, int item, int t0, int t1) {
  Work w;
  const int hk = item / q.t.per, u = item - hk * q.t.per;
  const int q0 = block_row(q.t, blk);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int group = q.t.pair_heads ? 2 * u + t : u;
    w.head[t] = hk * a.rep + group * q.t.hb;
    w.heads[t] = min(q.t.hb, a.rep - group * q.t.hb);
    w.q0[t] = q0 + (q.t.pair_heads ? 0 : t * q.t.tb);
    w.pa[t] = q.r.off + w.q0[t];
    w.pb[t] = q.r.off + min(w.q0[t] + q.t.tb, q.r.rows) - 1;
  }
  w.nt = w.q0[1] >= q.r.rows || w.heads[1] <= 0 ? 1 : 2;
  const KeyTiles k = chunk_tiles<KT>(q.t, q.r, a.qb.window, a.qb.sinks, blk);
  w.ts = k.ts;
  w.tw0 = k.tw0;
  w.ns = k.ns;
  w.begin = min(t0, k.tiles);
  w.end = min(t1, k.tiles);
  w.whole = t0 == 0 && t1 >= k.tiles;
  w.two = w.rest = 0;
  w.row0 = q.row0;
  w.rows = q.r.rows;
  w.keys = q.r.keys;
  w.tb = q.t.tb;
  w.seq = q.seq;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int e = min(w.pb[t], q.r.keys - 1) < 0 ? -1 : min(w.pb[t], q.r.keys - 1) / KT;
    w.from[t] = w.ts + (a.qb.window > 0 ? max(w.pa[t] - a.qb.window + 1, 0) / KT - w.tw0 : 0);
    int last = t >= w.nt || e < 0 ? -1 : e - w.tw0 + w.ts;   // the last one of this part
    last = min(last, w.end - 1);
    if (last < w.from[t]) last = min(last, w.ns - 1);
    if (last < w.begin) last = -1;
    w.last[t] = last;
  }
  return w;
}
// Whether all rows of query tile t see all of the key tile at j0.
template <int KT>
__device__ __forceinline__ bool tile_whole(const ChunkArgs& a, int pa, int pb, int keys, int j0) {
  return j0 + KT - 1 <= min(pa, keys - 1) && (a.qb.window == 0 || j0 > pb - a.qb.window || j0 + KT <= a.qb.sinks);
}
// Whether key tile i, at j0, counts with its first kCaNarrow columns alone: the sinks' last tile, mostly.
__device__ __forceinline__ bool tile_narrow(const ChunkArgs& a, int ts, int i, int j0) { return i < ts && a.qb.sinks - j0 <= kCaNarrow; }

// A CTA's part of the line, walked by one warp of it.
template <int KT>
struct Walk {
  int req, blk, item;    // the item
  int places, weight;    // its places, and those of a key tile
  int t0, t1;            // its key tiles of this part
  int left;              // items of the block behind it
  int64_t to_go;         // places of this CTA's part from the item's begin on
  bool two;              // the item that this CTA begins and does not end is ended by the next one
  Request q;
  bool idle;

  __device__ __forceinline__ void open(const ChunkArgs& a) {   // places of block `blk`
    places = uniform(chunk_places<KT>(q.t, q.r, a.qb.window, a.qb.sinks, blk));
    weight = uniform(tile_weight<KT>(q.t));
  }
  __device__ __forceinline__ void load(const ChunkArgs& a) { load(request_of(a, req)); }
  __device__ __forceinline__ void load(const Request& r) {
    q = r;
    q.row0 = uniform(q.row0);
    q.seq = uniform(q.seq);
    q.r.rows = uniform(q.r.rows);
    q.r.off = uniform(q.r.off);
    q.r.keys = uniform(q.r.keys);
  }
  __device__ __forceinline__ Work work(const ChunkArgs& a) const {
    Work w = work_of<KT>(a, q, blk, item, t0, t1);
    w.two = two && t0 == 0 && !w.whole;
    w.rest = t0 > 0 && to_go > places;
    return w;
  }
  __device__ __forceinline__ void set_end() { t1 = uniform(chunk_tile(static_cast<int>(min(to_go, static_cast<int64_t>(places))), weight)); }
  // On to the next item, by the whole warp; false where there is none.
  __device__ __forceinline__ bool next(const ChunkArgs& a, bool ok) {
    to_go -= places;
    if (!__all_sync(0xffffffffu, to_go > 0 && ok)) return false;
    if (--left < 0) {
      if (++blk == q.t.blocks) {
        blk = 0;
        do {
          if (++req >= a.n) return false;   // never: the part would be longer than the line
          load(a);
        } while (__all_sync(0xffffffffu, q.r.rows == 0));
      }
      left = a.p.Hkv * q.t.per - 1;
      item = 0;
      open(a);
    } else {
      ++item;
    }
    t0 = 0;
    set_end();
    return true;
  }
};

// A CTA has two slots for parts of items that others hold too, for its first and its last.  A slot: the
// rows of two query tiles, 128 sums each, as [query tile][8 channels][row][8], so that the rows of a warp are written
// side by side; the rows' (maximum, sum) behind all slots, and behind them what each CTA cuts.
__device__ __forceinline__ float* part_sums(const ChunkArgs& a, int slot, int t, int row, int ch) {
  const int64_t tile = static_cast<int64_t>(slot) * 2 + t;
  return a.part + ((tile * (kD / 8) + ch / 8) * a.tile_rows + row) * 8 + ch % 8;
}
__device__ __forceinline__ float2* part_ml(const ChunkArgs& a, int slot, int t, int row) {
  float2* ml = reinterpret_cast<float2*>(a.part + static_cast<int64_t>(a.ctas) * 4 * a.tile_rows * kD);
  return ml + (static_cast<int64_t>(slot) * 2 + t) * a.tile_rows + row;
}
__device__ __forceinline__ Cut* part_cut(const ChunkArgs& a, int c) {
  return reinterpret_cast<Cut*>(a.part + static_cast<int64_t>(a.ctas) * 4 * a.tile_rows * (kD + 2)) + c;
}

// The tag of the call once the 32 rows that the warp holds of its first item's tile t lie in its slot; the joining kernel
// clears it.  (A tag is one of 2^64 that the host draws anew for every call, so that what a workspace held before, or
// what a call left that was captured with another tag, does not pass for it.)
__device__ __forceinline__ uint64_t* part_ready(const ChunkArgs& a, int c, int t, int warp) {
  return reinterpret_cast<uint64_t*>(part_cut(a, a.ctas)) + (c * 2 + t) * 4 + warp;
}
// Joins parts one after the other: the factors of what is there and of what comes.  Written out in single operations, so that
// it is the same to the bit wherever a part is joined.
struct Joined {
  float m = -INFINITY, l = 0.f;
  __device__ __forceinline__ float2 add(float2 x) {
    const float mn = fmaxf(m, x.x), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ref), fx = ex2(x.x - ref);
    l = __fmaf_rn(x.y, fx, __fmul_rn(l, f));
    m = mn;
    return make_float2(f, fx);
  }
};
__device__ __forceinline__ float joined(float o, float p, float2 f) { return __fadd_rn(__fmaf_rn(p, f.y, __fmul_rn(o, f.x)), 0.f); }   // (never -0)
template <bool BF>
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + (log2f(l) - RowWeights<BF>::shift)) * 0.6931471805599453f;
}

// Inclusive sum over the block; `sums` holds a value a warp.
template <int THREADS>
__device__ __forceinline__ int64_t scan_block(int64_t v, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();   // the last pass's sums have been read
  if (lane == 31) sums[w] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const int64_t s = sums[i];
    if (i < w) v += s;
    total += s;
  }
  return v;
}
// The entry e of `n` with base[e] <= x < base[e + 1].
template <typename T>
__device__ __forceinline__ int find_entry(const T* base, int n, int64_t x) {
  int lo = 0, hi = n;   // base[lo] <= x < base[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (base[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// This CTA's part of the line, by all threads of it, for its walking warp.  `scratch`: 16 bytes a request, (n + 1) * 4
// for the blocks before each, and 8 bytes a block for the places before it (180 KB at most).
template <int KT, class W>
__device__ __forceinline__ Walk<KT> find_part(const ChunkArgs& a, uint8_t* scratch, int64_t* sums) {
  const int tid = threadIdx.x;
  int4* reqs = reinterpret_cast<int4*>(scratch);   // first row, rows, first position, keys
  int64_t* place = reinterpret_cast<int64_t*>(reqs + a.n);
  const auto request = [&](int i) {
    const int4 x = reqs[i];
    return Request{x.x, a.seqs ? a.seqs[i] : i, {x.y, x.z, x.w}, row_tiles_of(x.y, a.rep)};
  };
  int32_t* blocks = reinterpret_cast<int32_t*>(place + a.rows / kCaRows + a.n + 2);   // a request has a block more than rows / 128 at most
  int64_t done = 0, total;
  for (int i0 = 0; i0 < a.n; i0 += W::threads) {
    const int i = i0 + tid;
    int64_t v = 0;
    if (i < a.n) {
      const Request q = request_of(a, i);
      reqs[i] = make_int4(q.row0, q.r.rows, q.r.off, q.r.keys);
      v = q.t.blocks;
    }
    v = scan_block<W::threads>(v, sums, total);
    if (i < a.n) blocks[i + 1] = static_cast<int32_t>(done + v);
    done += total;
  }
  if (tid == 0) blocks[0] = 0;
  __syncthreads();
  // requests whose rows overlap (row_start does not ascend) could have more blocks than there is room for
  const int entries = static_cast<int>(min(done, static_cast<int64_t>(a.rows / kCaRows + a.n + 1)));
  done = 0;
  for (int e0 = 0; e0 < entries; e0 += W::threads) {
    const int e = e0 + tid;
    int64_t v = 0;
    if (e < entries) {
      const int i = find_entry(blocks, a.n, e);
      const Request q = request(i);
      v = static_cast<int64_t>(chunk_places<KT>(q.t, q.r, a.qb.window, a.qb.sinks, e - blocks[i])) * a.p.Hkv * q.t.per;
    }
    v = scan_block<W::threads>(v, sums, total);
    if (e < entries) place[e + 1] = done + v;
    done += total;
  }
  if (tid == 0) place[0] = 0;
  __syncthreads();
  Walk<KT> w;
  w.idle = true;
  if (tid / 32 != W::walk) return w;
  const int workers = chunk_workers(done, a.ctas), c = blockIdx.x;
  Cut cut = {};
  cut.last = -1;
  if (c < workers && done > 0) {
    int64_t x = split_begin(done, workers, c), y = split_begin(done, workers, c + 1);
    const int e = find_entry(place, entries, x);
    w.req = uniform(find_entry(blocks, a.n, e));
    w.blk = uniform(e - blocks[w.req]);
    w.load(request(w.req));
    w.open(a);
    const int in = static_cast<int>((x - place[e]) % w.places);
    w.item = uniform(static_cast<int>((x - place[e]) / w.places));
    w.left = a.p.Hkv * w.q.t.per - 1 - w.item;
    w.t0 = uniform(chunk_tile(in, w.weight));
    if (w.t0 == 0) x -= in;            // a boundary among an item's first places is its begin
    const int64_t begin = x - (w.t0 == 0 ? 0 : in);
    if (y < done) {
      const int f = find_entry(place, entries, y), i = find_entry(blocks, a.n, f);
      const Request q = request(i);
      const int blk = f - blocks[i], places = chunk_places<KT>(q.t, q.r, a.qb.window, a.qb.sinks, blk);
      const int item = static_cast<int>((y - place[f]) / places);
      const int64_t b = place[f] + static_cast<int64_t>(item) * places;
      if (chunk_tile(static_cast<int>(y - b), tile_weight<KT>(q.t)) == 0) {
        y = b;
      } else if (b >= x) {   // begun here, and goes on in later CTAs
        const Work k = work_of<KT>(a, q, blk, item, 0, places);
        cut.last = split_owner(done, workers, b + places - 1);
        cut.before = b > x;
        cut.row0 = q.row0;
        cut.rows = q.r.rows;
        cut.tb = q.t.tb;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          cut.q0[t] = k.q0[t];
          cut.head[t] = k.head[t];
          cut.heads[t] = t < k.nt ? k.heads[t] : 0;
        }
      }
    }
    w.idle = x >= y;
    w.two = cut.last == c + 1;
    w.to_go = y - begin;
    w.set_end();
  }
  if ((tid & 31) == 0) *part_cut(a, c) = cut;
  return w;
}

// A tile of 128 rows into shared memory by one warp, two rows an instruction; lane l holds the pool rows of rows l, 32 + l,
// 64 + l and 96 + l (kNoRow: zeros).
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint8_t* rows, const uint32_t (&at)[4]) {
  const int lane = threadIdx.x & 31, piece = lane & 15, odd = lane >> 4;
  rows += piece * 16;
  dst += (piece >> 3) * tc::kKBlock + odd * 128;
  uint32_t swz[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) swz[e] = dst + (((piece & 7) ^ (2 * e + odd)) << 4);
#pragma unroll
  for (int j = 0; j < kCaRows / 2; ++j) {
    const uint32_t row = __shfl_sync(0xffffffffu, at[j >> 4], 2 * (j & 15) + odd);
    const bool ok = row != kNoRow;
    cp_async16(swz[j & 3] + j * 256, rows + static_cast<size_t>(ok ? row : 0u) * (kD * 2), ok);
  }
}
// ROWS rows of a query tile from row r0 on by one warp, lane l holding the address of row r0 + l (null: zeros).
template <int ROWS>
__device__ __forceinline__ void copy_queries(uint32_t dst, int r0, const uint8_t* src, const uint8_t* any) {
  const int lane = threadIdx.x & 31, piece = lane & 15;
#pragma unroll
  for (int j = 0; j < ROWS / 2; ++j) {
    const int e = 2 * j + (lane >> 4), r = r0 + e;
    const uint64_t x = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), e);
    cp_async16(dst + (piece >> 3) * tc::kKBlock + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
               x ? reinterpret_cast<const uint8_t*>(x) + piece * 16 : any, x != 0);
  }
}
// This warp's copies and stores so far are in shared memory, for the tensor core too: an arrival at `bar`.
__device__ __forceinline__ void land(uint32_t bar) {
  tc::fence_proxy_async();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}
// A box of pool rows, both halves of the channels, by one lane.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t row, uint32_t bar) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
            dst + j * tc::kKBlock),
        "l"(map), "r"(j * 64), "r"(row), "r"(bar)
        : "memory");
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(REGS)); }

// The value s * code + z of 16 codes as two fp16 numbers each: the first rounded towards zero, so that none passes
// fp16's largest number, and what is left.
__device__ __forceinline__ void split16(const uint4& c, __half2 m, uint32_t (&hi)[8], uint32_t (&lo)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const float s = __low2float(m), z = __high2float(m);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // a code as the last bits of 2^23 + code; s * code is exact
    const float2 x = make_float2(__uint_as_float(__byte_perm(w[e >> 1], 0x4B000000u, 0x7440u + 2 * (e & 1))),
                                 __uint_as_float(__byte_perm(w[e >> 1], 0x4B000000u, 0x7441u + 2 * (e & 1))));
    const float2 f = __ffma2_rn(__fadd2_rn(x, make_float2(-8388608.f, -8388608.f)), make_float2(s, s), make_float2(z, z));
    // (cut to fp16's 11 bits by a mask: a conversion back costs more)
    const float2 h = make_float2(__uint_as_float(__float_as_uint(f.x) & 0xffffe000u), __uint_as_float(__float_as_uint(f.y) & 0xffffe000u));
    asm("cvt.rz.f16x2.f32 %0, %1, %2;\n" : "=r"(hi[e]) : "f"(h.y), "f"(h.x));
    const float2 r = __fadd2_rn(f, make_float2(-h.x, -h.y));
    lo[e] = pack2<false>(r.x, r.y);
  }
}
// 16 keys of an INT8 tile: the codes and scales that a lane takes of them, four keys an instruction, 16 channels of each.
struct CodeRows {
  uint4 c[4];
  __half2 m[4];
};
__device__ __forceinline__ void load_codes(CodeRows& x, const uint8_t* codes, const uint8_t* meta, uint32_t at) {   // lane l < 16: the pool row of key l
  const int lane = threadIdx.x & 31, piece = lane & 7;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t row = __shfl_sync(0xffffffffu, at, 4 * j + (lane >> 3));
    x.c[j] = make_uint4(0, 0, 0, 0);
    x.m[j] = __float2half2_rn(0.f);
    if (row != kNoRow) {
      x.c[j] = *reinterpret_cast<const uint4*>(codes + static_cast<size_t>(row) * kD + piece * 16);
      x.m[j] = reinterpret_cast<const __half2*>(meta + static_cast<size_t>(row) * kMetaBytes)[piece >> 2];
    }
  }
}
// Keys r0 .. r0 + 15 of a tile into its buffer: the numbers' first parts in rows 0 .. 63, the second ones behind.
__device__ __forceinline__ void store_codes(const CodeRows& x, uint32_t dst, int r0) {
  const int lane = threadIdx.x & 31, piece = lane & 7;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + 4 * j + (lane >> 3);
    uint32_t v[2][8];
    split16(x.c[j], x.m[j], v[0], v[1]);
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int half = 0; half < 2; ++half) {   // channels 16 piece + 8 half ..
        const int ch = (piece & 3) * 2 + half;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(dst + (piece >> 2) * tc::kKBlock + (part * kKeys<MIKV_PAGES_INT8> + r) * 128 +
                                                                        ((ch ^ (r & 7)) << 4)),
                     "r"(v[part][4 * half]), "r"(v[part][4 * half + 1]), "r"(v[part][4 * half + 2]), "r"(v[part][4 * half + 3])
                     : "memory");
      }
  }
}

template <int TYPE>
__global__ void __launch_bounds__(Warps<TYPE == MIKV_PAGES_INT8>::threads, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const ChunkArgs a) {
  constexpr bool BF = TYPE == MIKV_PAGES_BF16, Q8 = TYPE == MIKV_PAGES_INT8;
  constexpr int KT = kKeys<TYPE>;
  using W = Warps<Q8>;
  extern __shared__ uint8_t smem[];
  __shared__ CaBars bar;
  __shared__ Work works[kCaTold];
  __shared__ int64_t sums[W::threads / 32];
  __shared__ uint32_t tslot;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kCaRing; ++i) {
      tc::mbar_init(smem_u32(&bar.full[i]), Q8 ? W::loaders / 2 : 1);
      tc::mbar_init(smem_u32(&bar.empty[i]), 2);
      tc::mbar_init(smem_u32(&bar.boxes[i]), 1);
    }
    for (int i = 0; i < kCaTold; ++i) {
      tc::mbar_init(smem_u32(&bar.told[i]), 1);
      tc::mbar_init(smem_u32(&bar.heard[i]), W::walk);   // all but the last two warps
    }
    tc::mbar_init(smem_u32(&bar.q), W::loaders);
    tc::mbar_init(smem_u32(&bar.qfree), 2);
    tc::mbar_init(smem_u32(&bar.one_o), 1);
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(smem_u32(&bar.turn[t]), 1);
      tc::mbar_init(smem_u32(&bar.s[t]), 1);
      tc::mbar_init(smem_u32(&bar.p[t][0]), 4);
      tc::mbar_init(smem_u32(&bar.p[t][1]), 4);
      tc::mbar_init(smem_u32(&bar.o[t]), 1);
      tc::mbar_init(smem_u32(&bar.one_s[t]), 1);
      tc::mbar_init(smem_u32(&bar.one_p[t][0]), 4);
      tc::mbar_init(smem_u32(&bar.one_p[t][1]), 4);
    }
    tc::mbar_init_fence();
  }
  if (warp == W::mma) tc::tmem_alloc(smem_u32(&tslot), kCaCols);
  const uint32_t sq = tc::smem_base(smem), ring = sq + 2 * tc::kTileBytes;
  Walk<KT> walk = find_part<KT, W>(a, smem + (sq - smem_u32(smem)), sums);
  tc::fence_before_sync();
  __syncthreads();     // the sums have been read: the tiles may be written over them
  tc::fence_proxy_async();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(tslot);
  pdl_trigger();       // the joining kernel may be placed; it waits for this one's end
  tc::Waits wait;
  // Item n, as the walking warp tells it; null behind the last one, or where a wait gave up.
  const auto hear = [&](int n) -> const Work* {
    wait(smem_u32(&bar.told[n % kCaTold]), (n / kCaTold) & 1);
    const Work* w = &works[n % kCaTold];
    return __all_sync(0xffffffffu, wait.ok) && uniform(w->nt) >= 0 ? w : nullptr;
  };
  const auto heard = [&](int n) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(smem_u32(&bar.heard[n % kCaTold]));
  };

  if (warp >= W::mma) fewer_registers<W::mma_regs>();   // (one instruction for all of a warpgroup)
  if (warp >= W::walk) {
    bool some = !walk.idle;
    for (int n = 0; warp == W::walk; ++n) {
      if (n >= kCaTold) wait(smem_u32(&bar.heard[n % kCaTold]), (n / kCaTold - 1) & 1);
      Work next;
      if (some) next = walk.work(a);
      if (lane == 0) {
        if (some)
          works[n % kCaTold] = next;
        else
          works[n % kCaTold].nt = -1;
        tc::mbar_arrive(smem_u32(&bar.told[n % kCaTold]));
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, some && wait.ok)) break;
      some = walk.next(a, wait.ok);
    }
  } else if (warp >= W::mma) {
    // One warp per query tile, so that neither waits in the other's place.  The whole warp walks
    // the steps, so that addresses and descriptors stay uniform; one elected lane issues.
    const int t = warp - W::mma;
    bool lead = elect_one();
    constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;
    constexpr uint32_t kScores = tc::idesc_f16(kCaRows, kCaRows) | kType, kFew = tc::idesc_f16(kCaRows, kCaNarrow) | kType;
    constexpr uint32_t kValues = tc::idesc_f16(kCaRows, kD) | kType | (1u << 16);   // B: rows along the contraction
    const uint32_t ts = tmem + t * 128, to = tmem + kCaO + t * 128;
    const uint64_t qd = tc::smem_desc(sq + t * tc::kTileBytes), k0 = tc::smem_desc(ring), v0 = value_desc(ring);
    int p_par = 0, q_par = 0;        // parity of the next weights, and queries
    uint32_t one_par = 0;            // of an item of one tile: of the next weights, by key tiles in turn
    // Tile 1's scores and those of one tile's odd key tiles lie in the same columns, and two warps issue the products
    // that read them: whoever comes next there waits until the other's last sums are made.
    int sums[2] = {0, 0};            // items whose sums of tile 0, and of tile 1, have been announced
    bool was_one = false;
    int slot = 0, par = 0;           // ring position and parity
    // The two warps issue in turns, one step each: the tiles then stay half a step apart, and one's
    // weights are made while the tensor core works for the other.
    int turn = t;   // tile 0 begins without waiting
    const auto take_turn = [&] {
      if (turn > 0) wait(smem_u32(&bar.turn[t]), (turn - 1) & 1);
      ++turn;
    };
    for (int n = 0;; ++n) {
      const Work* told = hear(n);
      if (!told) break;
      const Work& w = *told;
      const int begin = uniform(w.begin), end = uniform(w.end);
      if (begin < end) {
        const int last = uniform(w.last[t]), from = uniform(w.from[t]), ns = uniform(w.ns), sinks = uniform(w.ts);
        const auto narrow = [&](int i) { return !Q8 && tile_narrow(a, sinks, i, i * KT); };
        bool more = false, before = false, few = false;
        int vslot = 0, vpar = 0;     // the last step's values
        wait(smem_u32(&bar.q), q_par);
        q_par ^= 1;
        const auto advance = [&] {   // the values of a tile follow its keys in the ring
          vslot = slot + 1 == kCaRing ? 0 : slot + 1;
          vpar = vslot == 0 ? par ^ 1 : par;
          slot = vslot + 1 == kCaRing ? 0 : vslot + 1;
          par = slot == 0 ? vpar ^ 1 : vpar;
        };
        if (uniform(w.nt) == 1) {
          // One query tile: its scores lie in turn where both tiles' would, and those of the next key tile are made before
          // this one's weights are there.
          if (t == 0 && sums[1] > 0) wait(smem_u32(&bar.o[1]), (sums[1] - 1) & 1);
          ++sums[0];
          was_one = true;
          for (int i = begin; i <= end; ++i) {
            const bool keys = i < end;
            if (keys) {
              wait(smem_u32(&bar.full[slot]), par);
              lead &= __all_sync(0xffffffffu, wait.ok) != 0;
              tc::fence_after_sync();
              if (lead && t == 0) {
                const uint64_t kd = k0 + slot * desc_step(tc::kTileBytes);
                const uint32_t scores = narrow(i) ? kFew : kScores;
#pragma unroll
                for (int c = 0; c < kD / 16; ++c) {
                  const uint64_t off = desc_step((c >> 2) * tc::kKBlock + (c & 3) * 32);
                  tc::mma_f16(tmem + (i & 1) * 128, qd + off, kd + off, scores, c > 0);
                }
                tc::commit(smem_u32(&bar.one_s[i & 1]));
              }
              if (lead) {
                tc::commit(smem_u32(&bar.empty[slot]));
                if (i == end - 1) tc::commit(smem_u32(&bar.qfree));
              }
            }
            if (i > begin) {
              wait(smem_u32(&bar.full[vslot]), vpar);
              if (t == 0) {
                const int b = (i - 1) & 1;
                wait(smem_u32(&bar.one_p[b][0]), (one_par >> b) & 1);
                wait(smem_u32(&bar.one_p[b][1]), (one_par >> b) & 1);
                one_par ^= 1u << b;
                lead &= __all_sync(0xffffffffu, wait.ok) != 0;
                tc::fence_after_sync();
                if (lead) {
                  const uint64_t vd = v0 + vslot * desc_step(tc::kTileBytes);
                  const int steps = few ? kCaNarrow / 16 : kCaRows / 16;
#pragma unroll
                  for (int c = 0; c < kCaRows / 16; ++c)
                    if (c < steps) mma_ts(to, tmem + b * 128 + (Q8 ? c & 3 : c) * 8, vd + desc_step(c * 2048), kValues, more || c > 0);
                  tc::commit(smem_u32(&bar.one_o));
                  if (i == end) tc::commit(smem_u32(&bar.o[0]));
                }
                more = true;
              }
              lead &= __all_sync(0xffffffffu, wait.ok) != 0;
              if (lead) tc::commit(smem_u32(&bar.empty[vslot]));
            }
            few = keys && narrow(i);
            if (keys) advance();
          }
          heard(n);
          continue;
        }
        if (t == 1 && was_one) wait(smem_u32(&bar.o[0]), (sums[0] - 1) & 1);
        was_one = false;
        sums[0] += uniform(w.last[0]) >= 0;
        sums[1] += uniform(w.last[1]) >= 0;
        // after a wait that gave up no lane leads, nothing more is issued, and the others' waits run out
        for (int i = begin; i <= end; ++i) {
          // this step's scores from key tile i, behind the last step's sums over value tile i - 1
          const bool keys = i < end, here = keys && i <= last && (i < ns || i >= from);
          const uint64_t kd = k0 + slot * desc_step(tc::kTileBytes), vd = v0 + vslot * desc_step(tc::kTileBytes);
          if (i > begin) wait(smem_u32(&bar.full[vslot]), vpar);
          if (keys) wait(smem_u32(&bar.full[slot]), par);
          if (before) wait(smem_u32(&bar.p[t][0]), p_par);
          take_turn();
          lead &= __all_sync(0xffffffffu, wait.ok) != 0;
          tc::fence_after_sync();
          if (before) {
            const auto sums = [&](int c0, int c1) {
#pragma unroll
              for (int c = c0; c < c1; ++c)   // (INT8: the same weights meet both parts)
                mma_ts(to, ts + (Q8 ? c & 3 : c) * 8, vd + desc_step(c * 2048), kValues, more || c > 0);
            };
            // the tensor core's queue holds about two products: a wait between them leaves it idle
            if (few) {
              wait(smem_u32(&bar.p[t][1]), p_par);
              lead &= __all_sync(0xffffffffu, wait.ok) != 0;
              if (lead) sums(0, kCaNarrow / 16);
            } else if (Q8) {
              wait(smem_u32(&bar.p[t][1]), p_par);
              lead &= __all_sync(0xffffffffu, wait.ok) != 0;
              tc::fence_after_sync();
              if (lead) sums(0, kCaRows / 16);
            } else if (__all_sync(0xffffffffu, tc::mbar_wait(smem_u32(&bar.p[t][1]), p_par, 1))) {
              tc::fence_after_sync();
              if (lead) sums(0, kCaRows / 16);
            } else {
              if (lead) sums(0, kCaRows / 32);
              wait(smem_u32(&bar.p[t][1]), p_par);
              lead &= __all_sync(0xffffffffu, wait.ok) != 0;
              tc::fence_after_sync();
              if (lead) sums(kCaRows / 32, kCaRows / 16);
            }
            p_par ^= 1;
            more = true;
          }
          const uint32_t scores = keys && narrow(i) ? kFew : kScores;
          if (lead) {
            if (before && i - 1 == last) tc::commit(smem_u32(&bar.o[t]));
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
          few = keys && narrow(i);
          if (lead) {
            if (i > begin) tc::commit(smem_u32(&bar.empty[vslot]));
            if (keys) tc::commit(smem_u32(&bar.empty[slot]));
            if (i == end - 1) tc::commit(smem_u32(&bar.qfree));   // the last scores
          }
          if (keys) advance();
        }
      }
      heard(n);
    }
  } else if (warp >= W::load) {
    fewer_registers<W::load_regs>();
    const int me = warp - W::load;
    const size_t layer0 = a.p.layer_rows() * a.layer;
    const uint8_t* k0 = a.p.k + layer0 * (Q8 ? kD : kD * 2);
    const uint8_t* v0 = a.p.v + layer0 * (Q8 ? kD : kD * 2);
    int used = 0, qs = 0;   // uses of this warp's buffer (INT8: tiles so far); items whose queries were loaded
    int ahead = 0;          // buffers of all items before, modulo the ring
    int cleared = 0;        // of this warp's tiles so far, those with rows to clear
    int boxed = 0;          // and those whose boxes were asked for
    for (int n = 0;; ++n) {
      const Work* told = hear(n);
      if (!told) break;
      const Work& w = *told;
      const int begin = uniform(w.begin), end = uniform(w.end);
      if (begin < end) {
        const int32_t* table = a.p.table + static_cast<size_t>(uniform(w.seq)) * a.p.max_pages;
        const int hk = uniform(w.head[0] / a.rep), keys = uniform(w.keys);
        // the pool row of slot j, kNoRow for one that no row of the item sees
        const int first = uniform(a.qb.window > 0 ? max(w.pa[0] - a.qb.window + 1, 0) : 0);
        const auto place = [&](int i, int r) {
          const int j = w.j0<KT>(i) + r;
          uint32_t row = kNoRow;
          if (i < end && j < keys && (j >= first || j < a.qb.sinks)) {
            const uint32_t pg = div_of(static_cast<uint32_t>(j), a.p.ps);
            row = pool_row(__ldg(table + pg), a.p.n_pages, a.p.Hkv, hk, a.p.ps.d, j - pg * a.p.ps.d);
            if (row == kNoRow) tc::report_giveup(tc::kBadPage);
          }
          return row;
        };
        // this warp's share of the queries; the last item's products still read theirs
        const auto queries = [&] {
          if (qs > 0) wait(smem_u32(&bar.qfree), (qs - 1) & 1);
          ++qs;
          if (!__all_sync(0xffffffffu, wait.ok)) return;
          constexpr int kRows = kCaRows / W::loaders;
          const int r = me * kRows + lane % kRows, sub = r / w.tb;
          for (int t = 0; t < w.nt; ++t) {
            const int q = w.q0[t] + r - sub * w.tb;
            copy_queries<kRows>(sq + t * tc::kTileBytes, me * kRows,
                         sub < w.heads[t] && q < w.rows ? a.q.row(0, w.head[t] + sub, w.row0 + q) : nullptr, a.q.p);
          }
          cp_async_commit();
          cp_async_wait<0>();
          land(smem_u32(&bar.q));
        };
        if constexpr (Q8) {
          // four warps for the keys and four for the values, 16 of each tile; the next one's codes are under way meanwhile
          const int kv = me >> 2, r0 = (me & 3) * 16;
          const uint8_t* codes = kv ? v0 : k0;
          const uint8_t* meta = (kv ? a.p.vm : a.p.km) + layer0 * kMetaBytes;
          const auto at = [&](int i) { return lane < 16 ? place(i, r0 + lane) : kNoRow; };
          CodeRows x;
          load_codes(x, codes, meta, at(begin));
          uint32_t next = at(begin + 1);
          for (int i = begin; i < end; ++i) {
            const int slot = (2 * used + kv) & (kCaRing - 1);
            wait(smem_u32(&bar.empty[slot]), (used / 2 & 1) ^ 1);
            ++used;
            if (__all_sync(0xffffffffu, wait.ok)) {
              store_codes(x, ring + slot * tc::kTileBytes, r0);
              land(smem_u32(&bar.full[slot]));
            }
            if (i + 1 < end) load_codes(x, codes, meta, next);
            next = at(i + 2);
            if (i == begin) queries();
          }
        } else {
          // this warp has every fourth buffer: keys (c even) or values of tile begin + c / 2
          int c = (me - ahead) & (kCaRing - 1);
          const int count = 2 * (end - begin);
          uint32_t at[4];   // pool rows of the tile's rows 32 e + lane; with TMA, of box `lane`
          const auto look = [&](int i) {
            if (a.box > 0) {
              at[0] = at[1] = kNoRow;
              const int r = lane * a.box, j = i < end ? w.j0<KT>(i) + r : 0;
              // boxes with a row that is seen; at[1] tells one whose page lies outside the pool
              if (i < end && r < kCaRows && j < keys && (j + a.box > first || j < a.qb.sinks)) {
                const uint32_t pg = div_of(static_cast<uint32_t>(j), a.p.ps);
                at[0] = pool_row(__ldg(table + pg), a.p.n_pages, a.p.Hkv, hk, a.p.ps.d, j - pg * a.p.ps.d);
                if (at[0] == kNoRow) {
                  tc::report_giveup(tc::kBadPage);
                  at[1] = 0;
                }
              }
              return;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) at[e] = place(i, e * 32 + lane);
          };
          // the boxes of tile i to this warp's buffer
          const auto fetch = [&](int i, bool values) {
            const uint32_t dst = ring + me * tc::kTileBytes;
            const uint32_t boxes = __ballot_sync(0xffffffffu, at[0] != kNoRow), bad = __ballot_sync(0xffffffffu, at[1] != kNoRow);
            const int j0 = w.j0<KT>(i);
            const int z0 = min(max(a.qb.sinks - j0, 0), kCaRows), z1 = min(first - j0, kCaRows), z2 = min(keys - j0, kCaRows);
            const bool clear = bad != 0 || (values && (z0 < z1 || z2 < kCaRows));
            const uint32_t on = smem_u32(clear ? &bar.boxes[me] : &bar.full[me]);
            ++boxed;
            if (lane == 0) tc::mbar_expect_tx(on, __popc(boxes) * a.box * kD * 2);
            __syncwarp();
            if (at[0] != kNoRow) tma_box(dst + lane * a.box * 128, values ? &vmap : &kmap, at[0], on);
            __syncwarp();
            if (!clear) return;
            const int shift = 31 - __clz(a.box);
            wait(on, cleared++ & 1);
            for (int e = lane; e < kCaRows * 16; e += 32) {   // 16-byte pieces, both channel blocks
              const int r = e >> 4, piece = e & 15;
              if ((r >= z0 && r < z1) || r >= z2 || (bad >> (r >> shift) & 1u))
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(dst + (piece >> 3) * tc::kKBlock + r * 128 + (piece & 7) * 16),
                             "r"(0)
                             : "memory");
            }
            land(smem_u32(&bar.full[me]));
          };
          look(begin + (c >> 1));
          // The item's queries, behind this warp's first buffer of it; before, where that one (the second values') is free only
          // when the last item's products are all done, and its scores' are done before.
          bool one = true;
          if (c == kCaRing - 1) {
            queries();
            one = false;
          }
          for (; c < count || one; c += kCaRing) {
            if (c < count) {
              wait(smem_u32(&bar.empty[me]), (used & 1) ^ 1);
              ++used;
              if (a.box > 0) {
                if (__all_sync(0xffffffffu, wait.ok)) fetch(begin + (c >> 1), c & 1);
                look(begin + (c >> 1) + 2);
              } else if (__all_sync(0xffffffffu, wait.ok)) {
                copy_tile(ring + me * tc::kTileBytes, c & 1 ? v0 : k0, at);
                cp_async_commit();
                look(begin + (c >> 1) + 2);   // the next one's places are looked up meanwhile
                cp_async_wait<0>();
                land(smem_u32(&bar.full[me]));
              }
            }
            if (one) queries();
            one = false;
          }
          ahead = (ahead + count) & (kCaRing - 1);
        }
      }
      heard(n);
    }
    // every release of this warp's buffer has arrived before the CTA ends
    for (int c = Q8 ? me >> 2 : me; c < kCaRing; c += Q8 ? 2 : kCaRing)   // INT8: tile u's keys or values were in buffer (2 u + kv) % 4
      wait(smem_u32(&bar.empty[c]), ((Q8 ? (used + 1 - (c >> 1)) / 2 : used) & 1) ^ 1);
    if (qs > 0) wait(smem_u32(&bar.qfree), (qs - 1) & 1);
    // after a wait that gave up nobody may have waited for the last boxes: they land before the CTA ends
    if (!wait.ok && boxed > 0) wait(smem_u32(&bar.full[me]), (boxed - 1) & 1);
  } else {
    more_registers<W::softmax_regs>();
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;   // the thread's TMEM lane is its row
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + kCaO + t * 128;
    uint32_t pars = 0;        // parities of the next scores: of a tile of two; of one tile's key tiles in turn
    int done = 0, o_par = 0;  // key tiles of single tiles so far
    for (int n = 0;; ++n) {
      const Work* told = hear(n);
      if (!told) break;
      const Work& w = *told;
      if (t < w.nt) {
        Row r;
        const bool one = w.nt == 1;   // (sees every key tile of its list)
        // (one loop that asks for every tile which it is took 382 us where this takes 361: 8192 causal rows of 32 heads)
        const auto tiles = [&](auto alone) {
          constexpr bool kOne = decltype(alone)::value;
          const int p = w.pa[t] + row % w.tb, last = min(p, w.keys - 1);
          for (int i = w.begin; i < w.end; ++i) {
            if (!kOne && !w.sees(t, i)) continue;
            const int j0 = w.j0<KT>(i);
            const bool whole = tile_whole<KT>(a, w.pa[t], w.pb[t], w.keys, j0), few = !Q8 && tile_narrow(a, w.ts, i, j0);
            const int b = kOne ? i & 1 : t, which = kOne ? 1 + b : 0;
            const uint32_t ts = tmem + lanes + b * 128;
            const uint32_t first_half = smem_u32(kOne ? &bar.one_p[b][0] : &bar.p[t][0]), ready[2] = {first_half, first_half + 8};
            const auto settle = [&] {   // one tile: the last sums were issued behind these scores
              if (kOne) {
                wait(smem_u32(&bar.one_o), (done - 1) & 1);
                tc::fence_after_sync();
              }
            };
            wait(smem_u32(kOne ? &bar.one_s[b] : &bar.s[t]), (pars >> which) & 1);
            pars ^= 1u << which;
            tc::fence_after_sync();
            if (few)
              softmax_tile<BF, kCaNarrow, 1, RowWeights<BF>>(a, ts, to, false, p, last, j0, r, ready, settle);
            else
              softmax_tile<BF, KT, Q8 ? 2 : 1, RowWeights<BF>>(a, ts, to, whole, p, last, j0, r, ready, settle);
            done += kOne;
          }
        };
        if (one)
          tiles(std::true_type{});
        else
          tiles(std::false_type{});
        const bool any = one ? w.begin < w.end : w.last[t] >= 0;
        if (any) {
          wait(smem_u32(&bar.o[t]), o_par);
          o_par ^= 1;
        }
        tc::fence_after_sync();
        const int sub = row / w.tb, q = w.q0[t] + row - sub * w.tb, head = w.head[t] + sub;   // the row's query and head
        const bool write = sub < w.heads[t] && q < w.rows;
        // An item of two parts is joined here if the next CTA, which begins with its end, is done with it: most are, as this
        // CTA ends with the item's begin.  (All left to the second kernel: three chunks of 1500 rows of 20 heads under a window
        // of 2048, 88 us instead of 84; chunk_window_int8 145 instead of 141.)  Whoever has that item alone does not look: both end at once.
        bool join = false;
        if (w.two && n > 0 && __all_sync(0xffffffffu, wait.ok)) {
          uint64_t tag;
          asm volatile("ld.acquire.gpu.global.b64 %0, [%1];\n" : "=l"(tag) : "l"(part_ready(a, blockIdx.x + 1, t, warp & 3)) : "memory");
          join = __all_sync(0xffffffffu, tag == a.tag);
        }
        const bool part = !w.whole && !join;
        const int slot = 2 * blockIdx.x + (n > 0), at = w.row0 + q;
        Joined sum;
        float2 own = make_float2(1.f, 1.f), other = make_float2(1.f, 0.f);
        float rest = 0.f;   // the other part's sum of weights
        if (join) {
          own = sum.add(make_float2(r.m * a.scale, r.l));
          if (write) {
            const float2 x = __ldcg(part_ml(a, 2 * (blockIdx.x + 1), t, row));
            other = sum.add(x);
            rest = x.y;
          }
          if (lane == 0) part_cut(a, blockIdx.x)->done[t][warp & 3] = 1;
        }
        const float l = join ? sum.l : r.l;
        float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
        if (!wait.ok) inv = __int_as_float(0x7fffffff);
        uint8_t* dst = a.out.row(0, head, at);
#pragma unroll 1
        for (int c = 0; c < kD; c += 32) {
          float o[32];
          if (any) {
            ld32(to + c, o);
            wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (join && write) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float4 p[2] = {};
              if (rest != 0.f) {
                const float4* from = reinterpret_cast<const float4*>(part_sums(a, 2 * (blockIdx.x + 1), t, row, c + e));
                p[0] = __ldcg(from);
                p[1] = __ldcg(from + 1);
              }
              const float x[8] = {p[0].x, p[0].y, p[0].z, p[0].w, p[1].x, p[1].y, p[1].z, p[1].w};
#pragma unroll
              for (int k = 0; k < 8; ++k) o[e + k] = joined(joined(0.f, r.l == 0.f ? 0.f : o[e + k], own), x[k], other);
            }
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
            } else if (any) {   // a part without a visible key is told by its sum of 0
#pragma unroll
              for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * inv);
#pragma unroll
              for (int e = 0; e < 32; e += 8) st_global32(part_sums(a, slot, t, row, c + e), u + e);
            }
          }
        }
        if (part && write) {
          *part_ml(a, slot, t, row) = make_float2(r.m * a.scale, wait.ok ? r.l : inv);
        } else if (write && a.lse) {
          const float v = join ? lse_of<BF>(sum.m, sum.l) : lse_of<BF>(r.m * a.scale, r.l);
          a.lse[static_cast<int64_t>(at) * a.Hq + head] = wait.ok ? v : inv;
        }
        if (w.rest) {
          __syncwarp();   // (the release covers what the other lanes have written before)
          if (lane == 0)
            asm volatile("st.release.gpu.global.b64 [%0], %1;\n" ::"l"(part_ready(a, blockIdx.x, t, warp & 3)), "l"(a.tag) : "memory");
        }
        tc::fence_before_sync();   // the sums are read before the next item's products overwrite them
      }
      heard(n);
    }
  }
  if (!wait.ok) tc::report_giveup(tc::kGiveupChunk);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == W::mma) tc::tmem_dealloc(tmem, kCaCols);
}

// CTA (slice, c): joins ROWS rows of the item that CTA c has begun and not ended, in a fixed order.  A thread takes 8
// channels of a row (a part's rows lie side by side); GROUPS sets of threads share the parts, BATCH of them
// requested together.
constexpr int kJoinThreads = 256;
template <bool BF, int GROUPS, int BATCH>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const ChunkArgs a) {
  constexpr int kThreads = kJoinThreads / GROUPS, kRows = kThreads / (kD / 8);   // of a group
  __shared__ float s_o[GROUPS > 1 ? GROUPS - 1 : 1][8][kThreads];
  __shared__ float2 s_ml[GROUPS > 1 ? GROUPS - 1 : 1][kThreads];
  const int tid = threadIdx.x % kThreads, group = threadIdx.x / kThreads, c0 = blockIdx.y;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x < 8) *part_ready(a, c0, threadIdx.x >> 2, threadIdx.x & 3) = 0;
  const Cut cut = *part_cut(a, c0);
  const int c1 = cut.last;
  if (c1 < 0) return;
  const int ch = tid / kRows * 8, i = blockIdx.x * kRows + tid % kRows, t = i >= a.tile_rows, row = i - t * a.tile_rows;
  const int sub = row / cut.tb, q = (t ? cut.q0[1] : cut.q0[0]) + row - sub * cut.tb;
  const bool live = i < 2 * a.tile_rows && sub < (t ? cut.heads[1] : cut.heads[0]) && q < cut.rows &&
                    !part_cut(a, c0)->done[t & 1][row >> 5 & 3];
  Joined sum;
  float o[8] = {};
  const auto add = [&](float2 x, const float (&p)[8]) {
    const float2 f = sum.add(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = joined(o[e], p[e], f);
  };
  if (live) {
    for (int p0 = c0 + group; p0 <= c1; p0 += BATCH * GROUPS) {
      float2 x[BATCH];
      float4 v[BATCH][2];
#pragma unroll
      for (int e = 0; e < BATCH; ++e) {
        const int p = p0 + e * GROUPS, slot = 2 * p + (p == c0 ? cut.before : 0);
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
      s_ml[group - 1][tid] = make_float2(sum.m, sum.l);
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
  const int head = (t ? cut.head[1] : cut.head[0]) + sub, at = cut.row0 + q;
  const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
  *reinterpret_cast<uint4*>(a.out.row(0, head, at) + ch * 2) =
      make_uint4(pack2<BF>(o[0] * inv, o[1] * inv), pack2<BF>(o[2] * inv, o[3] * inv), pack2<BF>(o[4] * inv, o[5] * inv),
                 pack2<BF>(o[6] * inv, o[7] * inv));
  if (ch == 0 && a.lse)
    a.lse[static_cast<int64_t>(at) * a.Hq + head] = lse_of<BF>(sum.m, sum.l);
}

int tile_rows_of(int rows, int rep) { return static_cast<int>(std::min<int64_t>(kCaRows, static_cast<int64_t>(rows) * rep)); }
size_t part_bytes(int rows, int rep) {
  return static_cast<size_t>(kNumSMs) * (static_cast<size_t>(4) * tile_rows_of(rows, rep) * (kD + 2) * 4 + sizeof(Cut) + 8 * sizeof(uint64_t));
}
uint64_t new_tag() {
  static std::atomic<uint64_t> calls{static_cast<uint64_t>(std::chrono::system_clock::now().time_since_epoch().count())};
  uint64_t x = calls += 0x9E3779B97F4A7C15ull;   // splitmix64 (Steele, Lea and Flood), a permutation of the counter
  x = (x ^ x >> 30) * 0xBF58476D1CE4E5B9ull;
  x = (x ^ x >> 27) * 0x94D049BB133111EBull;
  return x ^ x >> 31;
}
bool sizes_ok(const mikv_pages* p, int n, int rows, int Hq) {
  return n >= 0 && n <= kMaxRequests && rows >= 0 && rows <= kMaxChunkRows && Hq >= 1 && Hq % p->Hkv == 0 && Hq / p->Hkv <= 1024 &&
         static_cast<int64_t>(p->max_pages) * p->page_size <= kMaxPos;
}

// Rows of one layer of the pool as [rows][D], boxes of a.box rows and 64 channels.
int encode_pool(CUtensorMap* map, const uint8_t* base, const ChunkArgs& a, const char* name) {
  const auto enc = tc::tensor_map_encoder();
  if (!enc) return fail(MIKV_ECUDA, "chunk_attention: cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[2] = {kD, static_cast<cuuint64_t>(a.p.layer_rows())}, strides[1] = {kD * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(a.box)}, estr[2] = {1, 1};
  const CUresult e = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<uint8_t*>(base + a.p.layer_rows() * a.layer * (kD * 2)), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (e != CUDA_SUCCESS) return fail(MIKV_ECUDA, "chunk_attention: tensor map of %s (error %d)", name, static_cast<int>(e));
  return MIKV_OK;
}

template <int TYPE>
int launch(const ChunkArgs& a, cudaStream_t st) {
  CUtensorMap km{}, vm{};
  if (a.box > 0) {
    if (int e = encode_pool(&km, a.p.k, a, "keys")) return e;
    if (int e = encode_pool(&vm, a.p.v, a, "values")) return e;
  }
  using W = Warps<TYPE == MIKV_PAGES_INT8>;
  const auto kern = chunk_attention_kernel<TYPE>;
  // the warps share out what the block has at launch: with less of it they would wait for ever
  static std::atomic<bool> known{false};
  if (!known.load(std::memory_order_relaxed)) {
    cudaFuncAttributes f;
    cudaError_t e = cudaFuncGetAttributes(&f, kern);
    if (e == cudaSuccess && f.numRegs != W::launch_regs) e = cudaErrorLaunchOutOfResources;
    if (e != cudaSuccess) return check_launch_after(e, "chunk_attention_kernel");
    known.store(true, std::memory_order_relaxed);
  }
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCaSmem);
  if (e != cudaSuccess) return check_launch_after(e, "chunk_attention_kernel");
  kern<<<a.ctas, W::threads, kCaSmem, st>>>(km, vm, a);
  if (int r = check_launch("chunk_attention_kernel")) return r;
  // Few rows an item: many parts, perhaps, and threads that share them (one token behind 65536 slots, one key head,
  // 152 parts: 31.5 us in all with four sets, 27 with eight); else 16 rows a CTA, whose few registers leave room for five an
  // SM (2048 causal rows of 32 heads: 58 us in all with 64 rows a CTA, one an SM, 55 this way).
  constexpr bool BF = TYPE == MIKV_PAGES_BF16;
  const bool few = a.tile_rows <= 32, fewest = a.tile_rows <= 8;
  const auto join = fewest ? chunk_join_kernel<BF, 8, 8> : few ? chunk_join_kernel<BF, 4, 4> : chunk_join_kernel<BF, 1, 2>;
  const int rows = fewest ? 2 : few ? 4 : 16;
  return check_launch_after(launch_after(join, dim3((2 * a.tile_rows + rows - 1) / rows, a.ctas), dim3(kJoinThreads), 0, st, a),
                            "chunk_join_kernel");
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_chunk_attention_workspace_bytes(const mikv_pages* p, int n, int rows, int Hq) {
  Pool pool;
  if (check_pages(p, "chunk_attention", &pool) || n < 1 || rows < 1 || !sizes_ok(p, n, rows, Hq)) return 0;
  return part_bytes(rows, Hq / p->Hkv);
}

extern "C" int mikv_chunk_attention(const mikv_rows* q, const mikv_pages* pages, int layer, const int32_t* seqs, const int32_t* start,
                                    const int32_t* row_start, int n, int rows, int Hq, int window, int sinks, const mikv_rows* out,
                                    float* lse, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  ChunkArgs a;
  if (int e = check_pages(pages, "chunk_attention", &a.p)) return e;
  if (layer < 0 || layer >= a.p.layers) return fail(MIKV_ESHAPE, "chunk_attention: layer=%d of %d", layer, a.p.layers);
  if (!sizes_ok(pages, n, rows, Hq) || (!seqs && n > a.p.max_seqs))
    return fail(MIKV_ESHAPE, "chunk_attention: n=%d rows=%d Hq=%d Hkv=%d max_pages=%d page_size=%d", n, rows, Hq, a.p.Hkv, a.p.max_pages,
                pages->page_size);
  if (window < 0 || sinks < 0) return fail(MIKV_EINVAL, "chunk_attention: window=%d sinks=%d", window, sinks);
  if (n == 0 || rows == 0) return MIKV_OK;
  if (int e = check_rows(q, "chunk_attention", "q")) return e;
  if (int e = check_rows(out, "chunk_attention", "out")) return e;
  const int64_t st = out->stride_t, sh = out->stride_h;   // apart: the heads of a row side by side, or the rows of a head
  const bool heads_in = (Hq == 1 || sh >= kD) && (rows == 1 || st >= (Hq - 1) * sh + kD);
  const bool rows_in = (rows == 1 || st >= kD) && (Hq == 1 || sh >= (rows - 1) * st + kD);
  if (!heads_in && !rows_in) return fail(MIKV_EINVAL, "chunk_attention: rows of out overlap");
  if (!row_start || !ws) return fail(MIKV_EINVAL, "chunk_attention: null pointer");
  if (reinterpret_cast<uintptr_t>(ws) & 31u) return fail(MIKV_EALIGN, "chunk_attention: workspace must be 32-byte aligned");
  a.rep = Hq / a.p.Hkv;
  const size_t need = part_bytes(rows, a.rep);
  if (ws_bytes < need) return fail(MIKV_ESHAPE, "chunk_attention: workspace %zu < %zu", ws_bytes, need);
  a.q = row_view(*q);
  a.out = row_view(*out);
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.seqs = seqs;
  a.start = start;
  a.row_start = row_start;
  a.layer = layer;
  a.n = n;
  a.rows = rows;
  a.Hq = Hq;
  a.ctas = kNumSMs;
  a.tile_rows = tile_rows_of(rows, a.rep);
  a.tag = new_tag();
  a.qb.window = window > kMaxPos ? 0 : window;   // one that reaches every key is none
  a.qb.sinks = std::min(sinks, kMaxPos);
  a.box = std::min(kCaRows, pages->page_size & -pages->page_size);
  // (coordinates are signed)
  if (a.p.type == MIKV_PAGES_INT8 || a.box < 8 || a.p.layer_rows() > 0x7fffffffULL) a.box = 0;
  a.wide_out = ((reinterpret_cast<uintptr_t>(out->data) | static_cast<uintptr_t>(a.out.sh | a.out.st)) & 31u) == 0;
  a.scale = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
  switch (a.p.type) {
    case MIKV_PAGES_FP16: return launch<MIKV_PAGES_FP16>(a, as_stream(stream));
    case MIKV_PAGES_BF16: return launch<MIKV_PAGES_BF16>(a, as_stream(stream));
    default: return launch<MIKV_PAGES_INT8>(a, as_stream(stream));
  }
}
