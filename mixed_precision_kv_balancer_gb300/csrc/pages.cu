// Page bookkeeping of the paged cache: reserve, fork, free, copy and compact.
//
// The state is one reference count per page (0 = free), one table row and one length per
// sequence.  New pages are the free pages of lowest number, given out in request order, so the
// same calls always give the same tables; references only ever change by additions, whose
// order does not show.  A page is shared by forked sequences only while all its slots are
// filled: a fork copies a parent's last, partly filled page, so a sequence's next tokens never
// land in a page that another sequence reads.
//
// reserve, fork and compact begin with one CTA that checks the requests, adds up the pages
// they need and collects that many free pages (page_plan_kernel); what moves data follows in
// launches over all SMs, chained with programmatic dependent launch.
#include <algorithm>

#include "paged.cuh"

namespace mikv {

int check_pages(const mikv_pages* p, const char* what, Pool* out) {
  if (!p) return fail(MIKV_EINVAL, "%s: null pages", what);
  if (p->type != MIKV_PAGES_FP16 && p->type != MIKV_PAGES_BF16 && p->type != MIKV_PAGES_INT8)
    return fail(MIKV_EINVAL, "%s: type=%d", what, p->type);
  if (p->D != kD) return fail(MIKV_EUNSUPPORTED, "%s: D=%d (only %d)", what, p->D, kD);
  if (p->layers < 1 || p->n_pages < 1 || p->page_size < 1 || p->page_size > 4096 || p->Hkv < 1 || p->Hkv > 1024 ||
      p->max_seqs < 1 || p->max_pages < 1)
    return fail(MIKV_ESHAPE, "%s: layers=%d n_pages=%d page_size=%d Hkv=%d max_seqs=%d max_pages=%d", what, p->layers,
                p->n_pages, p->page_size, p->Hkv, p->max_seqs, p->max_pages);
  if (static_cast<int64_t>(p->max_pages) * p->page_size > 0x7fffffffLL - 4096)
    return fail(MIKV_ESHAPE, "%s: max_pages * page_size=%lld slots a sequence", what,
                static_cast<long long>(p->max_pages) * p->page_size);
  if (static_cast<double>(p->n_pages) * p->Hkv * p->page_size >= 4294967295.0)
    return fail(MIKV_ESHAPE, "%s: n_pages * Hkv * page_size above 2^32", what);
  const bool q8 = p->type == MIKV_PAGES_INT8;
  if (!p->k || !p->v || !p->table || !p->lens || !p->refs || (q8 && (!p->k_meta || !p->v_meta)))
    return fail(MIKV_EINVAL, "%s: null buffer in pages", what);
  if (!aligned16(p->k) || !aligned16(p->v) || (q8 && (!aligned16(p->k_meta) || !aligned16(p->v_meta))))
    return fail(MIKV_EALIGN, "%s: page buffers must be 16-byte aligned", what);
  out->k = static_cast<uint8_t*>(p->k);
  out->v = static_cast<uint8_t*>(p->v);
  out->km = q8 ? static_cast<uint8_t*>(p->k_meta) : nullptr;
  out->vm = q8 ? static_cast<uint8_t*>(p->v_meta) : nullptr;
  out->table = p->table;
  out->lens = p->lens;
  out->refs = p->refs;
  out->layers = p->layers;
  out->n_pages = p->n_pages;
  out->Hkv = p->Hkv;
  out->max_seqs = p->max_seqs;
  out->max_pages = p->max_pages;
  out->cap = p->max_pages * p->page_size;
  out->row_bytes = q8 ? kD : kD * 2;
  out->type = p->type;
  out->ps = make_fast_div(static_cast<uint32_t>(p->page_size));
  return MIKV_OK;
}

int check_rows(const mikv_rows* r, const char* what, const char* name) {
  if (!r || !r->data) return fail(MIKV_EINVAL, "%s: null %s", what, name);
  if (!aligned16(r->data) || r->stride_b % 8 || r->stride_h % 8 || r->stride_t % 8)
    return fail(MIKV_EALIGN, "%s: %s and its strides must be multiples of 16 bytes", what, name);
  if (r->stride_b < 0 || r->stride_h < 0 || r->stride_t < 0)
    return fail(MIKV_EINVAL, "%s: negative stride of %s", what, name);
  return MIKV_OK;
}

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMaxRequests = 4096;      // of one reserve, fork or compact call
constexpr int kScanInts = 16;           // references a thread reads per pass of the free-page search

enum class Op { kReserve, kFork, kCompact };

struct PlanArgs {
  const int32_t* seq;     // reserve, compact: the sequence (or null: 0, 1, ...); fork: the parent
  const int32_t* other;   // reserve: tokens to add; fork: the child; compact: tokens to keep
  int n, most;            // requests; compact: the longest keep list
  int32_t* flag;          // reserve: start; fork, compact: ok
  int32_t* fresh;         // workspace: the free pages, in request order
  int32_t* first;         // workspace: request i's first entry of `fresh`
};

// Inclusive sum over the block of `v`; `total` receives the block's sum.  `warp_sums` holds 32 values.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // the previous call's sums have been read
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  T s = lane < (blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  total = __shfl_sync(0xffffffffu, s, (blockDim.x >> 5) - 1);
  const T before = __shfl_sync(0xffffffffu, s, (w + 31) & 31);
  return w ? v + before : v;
}

// Whether `x` is among a[0 .. n).
__device__ __forceinline__ bool among(const int32_t* a, int n, int32_t x) {
  bool hit = false;
#pragma unroll 8
  for (int j = 0; j < n; ++j) hit |= a[j] == x;
  return hit;
}

// One CTA: validates the requests, gives each its pages of `fresh`, and (reserve) carries them
// out.  A request that is not valid needs nothing and is refused; of the valid ones, in order,
// those are served that need no page, or whose pages, together with all earlier valid requests',
// do not exceed the free ones.  (A compaction's positions are not looked at here: one that
// page_check_kernel refuses for them has counted.)  Bound by latency: the references are read kScanInts a thread at a time until enough
// free pages are found (65,536 pages: four passes).
template <Op OP>
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const Pool p, const PlanArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* s_seq = sm;            // [n]
  int32_t* s_other = sm + a.n;    // [n]
  int32_t* s_need = sm + 2 * a.n; // [n]: new pages, -1 where the request is not valid
  __shared__ int warp_sums[32];
  __shared__ int64_t warp_sums64[32];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i < a.n; i += kPlanThreads) {
    s_seq[i] = a.seq ? a.seq[i] : i;
    s_other[i] = a.other[i];
  }
  __syncthreads();
  int64_t base = 0;   // of all requests: past 32 bits where they ask for more than any pool has
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int need = 0, ok = 0;
    if (i < a.n) {
      const int32_t s = s_seq[i], o = s_other[i];
      ok = static_cast<uint32_t>(s) < static_cast<uint32_t>(p.max_seqs);
      if (OP == Op::kFork) {
        ok = ok && static_cast<uint32_t>(o) < static_cast<uint32_t>(p.max_seqs);
        ok = ok && !among(s_seq, a.n, o) && !among(s_other, i, o) && p.lens[o] == 0;
        if (ok) need = p.len_of(s) % static_cast<int>(p.ps.d) ? 1 : 0;
      } else {
        ok = ok && !(a.seq && among(s_seq, i, s));
        if (ok) {
          const int len = p.len_of(s);
          if (OP == Op::kReserve) {
            ok = o >= 0 && o <= p.cap - len;
            need = ok ? pages_of(len + o, p.ps) - pages_of(len, p.ps) : 0;
          } else {
            ok = o >= 0 && o <= a.most && o <= len;
            need = ok ? pages_of(o, p.ps) : 0;
          }
        }
      }
    }
    int64_t sum;
    const int64_t incl = block_scan<int64_t>(need, warp_sums64, sum);
    if (i < a.n) {
      s_need[i] = ok ? need : -1;
      a.first[i] = static_cast<int32_t>(min(base + incl - need, static_cast<int64_t>(0x7fffffff)));
    }
    base += sum;
  }
  // the lowest `base` free pages
  int found = 0;
  for (int64_t r0 = 0; found < base && r0 < p.n_pages; r0 += kPlanThreads * kScanInts) {
    const int64_t at = r0 + static_cast<int64_t>(tid) * kScanInts;
    uint32_t free_mask = 0;
    if (at + kScanInts <= p.n_pages && (reinterpret_cast<uintptr_t>(p.refs) & 15u) == 0) {
      int4 x[kScanInts / 4];
#pragma unroll
      for (int j = 0; j < kScanInts / 4; ++j) x[j] = reinterpret_cast<const int4*>(p.refs + at)[j];
#pragma unroll
      for (int j = 0; j < kScanInts / 4; ++j)
        free_mask |= ((x[j].x == 0) | (x[j].y == 0) << 1 | (x[j].z == 0) << 2 | (x[j].w == 0) << 3) << (4 * j);
    } else {
      for (int j = 0; j < kScanInts; ++j)
        if (at + j < p.n_pages && p.refs[at + j] == 0) free_mask |= 1u << j;
    }
    int sum;
    int rank = found + block_scan(__popc(free_mask), warp_sums, sum) - __popc(free_mask);
    for (; free_mask && rank < base; free_mask &= free_mask - 1, ++rank)
      a.fresh[rank] = static_cast<int32_t>(at) + __ffs(free_mask) - 1;
    found += sum;
  }
  __syncthreads();  // `fresh` and `first` are read below (and by the next launch)
  const int64_t avail = min(static_cast<int64_t>(found), base);
  const auto served = [&](int i) {
    const int need = s_need[i];
    return need == 0 || (need > 0 && static_cast<int64_t>(a.first[i]) + need <= avail);
  };
  if (OP == Op::kReserve) {
    const int w = tid >> 5, lane = tid & 31;
    for (int i = w; i < a.n; i += kPlanThreads / 32) {
      const int need = s_need[i], f = a.first[i];
      const bool ok = served(i);
      const int32_t s = s_seq[i];
      const int len = ok ? p.len_of(s) : 0;
      __syncwarp();
      if (ok) {
        int32_t* row = p.table + static_cast<size_t>(s) * p.max_pages + pages_of(len, p.ps);
        for (int j = lane; j < need; j += 32) {
          const int32_t page = a.fresh[f + j];
          row[j] = page;
          p.refs[page] = 1;
        }
        if (lane == 0) p.lens[s] = len + s_other[i];
      }
      if (lane == 0) a.flag[i] = ok ? len : -1;
    }
  } else {
    for (int i = tid; i < a.n; i += kPlanThreads) a.flag[i] = served(i);
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;   // rows of one CTA's move

// CTA (piece, i): refuses request i (ok -> -1, which page_commit_kernel turns into 0) where one
// of its positions, or the page of one, is outside.  A pass of its own, before any row moves: a
// refused request changes nothing.
__global__ void __launch_bounds__(kMoveThreads) page_check_kernel(const Pool p, const int32_t* seq, const int32_t* keep_pos,
                                                                  const int32_t* keep_n, int n, int most, int32_t* ok) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.y;
  if (ok[i] == 0) return;
  const int32_t s = seq ? seq[i] : i;
  const int keep = keep_n[i], len = p.len_of(s);
  const int32_t* table = p.table + static_cast<size_t>(s) * p.max_pages;
  const int64_t total = static_cast<int64_t>(p.layers) * p.Hkv * keep;
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; c < total;
       c += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
    const int64_t unit = c / keep;   // (layer, head)
    const int64_t at = ((unit / p.Hkv * n + i) * p.Hkv + unit % p.Hkv) * most + c % keep;
    const int32_t pos = keep_pos[at];
    if (pos < 0 || pos >= len || !p.has(table[div_of(pos, p.ps)])) ok[i] = -1;  // every writer writes the same value
  }
}

// CTA (layer, request, head, chunk of 64 kept slots): row keep_pos[j] of the old pages to row j
// of the new ones, keys and values (and INT8 scales).  Bound by HBM: each kept row is read and
// written once, 8 loads of 16 bytes in flight a thread.
__global__ void __launch_bounds__(kMoveThreads) page_compact_kernel(const Pool p, const int32_t* seq, const int32_t* keep_pos,
                                                                    const int32_t* keep_n, int n, int most, int chunks,
                                                                    const int32_t* ok, const int32_t* fresh,
                                                                    const int32_t* first) {
  __shared__ uint32_t src[kMoveRows], dst[kMoveRows];
  pdl_wait();
  pdl_trigger();
  int64_t id = blockIdx.x;
  const int chunk = static_cast<int>(id % chunks);
  id /= chunks;
  const int h = static_cast<int>(id % p.Hkv);
  id /= p.Hkv;
  const int i = static_cast<int>(id % n);
  const int layer = static_cast<int>(id / n);
  if (ok[i] <= 0) return;
  const int32_t s = seq ? seq[i] : i;
  const int keep = keep_n[i], j0 = chunk * kMoveRows;
  if (j0 >= keep) return;
  const int rows = min(kMoveRows, keep - j0);
  if (threadIdx.x < kMoveRows) {
    uint32_t from = kNoRow, to = kNoRow;
    if (static_cast<int>(threadIdx.x) < rows) {
      const int j = j0 + threadIdx.x;
      const int32_t pos = keep_pos[((static_cast<int64_t>(layer) * n + i) * p.Hkv + h) * most + j];
      uint32_t q = div_of(pos, p.ps);
      from = pool_row(p.table[static_cast<size_t>(s) * p.max_pages + q], p.n_pages, p.Hkv, h, p.ps.d, pos - q * p.ps.d);
      q = div_of(j, p.ps);
      to = pool_row(fresh[first[i] + q], p.n_pages, p.Hkv, h, p.ps.d, j - q * p.ps.d);
    }
    src[threadIdx.x] = from;
    dst[threadIdx.x] = to;
  }
  __syncthreads();
  const size_t lrow = p.layer_rows() * layer;
  const int per_row = p.row_bytes / 16;                 // 16-byte pieces: 16 or 8
  const int pieces = rows * per_row;
#pragma unroll 1
  for (int c0 = threadIdx.x; c0 < pieces; c0 += kMoveThreads * 4) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * kMoveThreads;
      if (c < pieces) {
        const size_t off = (lrow + src[c / per_row]) * p.row_bytes + (c % per_row) * 16;
        a[u] = *reinterpret_cast<const uint4*>(p.k + off);
        b[u] = *reinterpret_cast<const uint4*>(p.v + off);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * kMoveThreads;
      if (c < pieces) {
        const size_t off = (lrow + dst[c / per_row]) * p.row_bytes + (c % per_row) * 16;
        *reinterpret_cast<uint4*>(p.k + off) = a[u];
        *reinterpret_cast<uint4*>(p.v + off) = b[u];
      }
    }
  }
  if (p.km && static_cast<int>(threadIdx.x) < rows) {
    reinterpret_cast<uint2*>(p.km)[lrow + dst[threadIdx.x]] = reinterpret_cast<const uint2*>(p.km)[lrow + src[threadIdx.x]];
    reinterpret_cast<uint2*>(p.vm)[lrow + dst[threadIdx.x]] = reinterpret_cast<const uint2*>(p.vm)[lrow + src[threadIdx.x]];
  }
}

// CTA i: the compacted sequence takes its new pages and gives back its old ones.
__global__ void __launch_bounds__(kMoveThreads) page_commit_kernel(const Pool p, const int32_t* seq, const int32_t* keep_n,
                                                                   int32_t* ok, const int32_t* fresh, const int32_t* first) {
  pdl_wait();
  const int i = blockIdx.x;
  const int state = ok[i];
  __syncthreads();  // all have read it before thread 0 rewrites it
  if (state == 0) return;
  if (state < 0) {
    if (threadIdx.x == 0) ok[i] = 0;
    return;
  }
  const int32_t s = seq ? seq[i] : i;
  const int old = pages_of(p.len_of(s), p.ps), now = pages_of(keep_n[i], p.ps);
  __syncthreads();
  int32_t* row = p.table + static_cast<size_t>(s) * p.max_pages;
  for (int j = threadIdx.x; j < max(old, now); j += kMoveThreads) {
    const int32_t was = row[j];
    if (j < old && p.has(was)) atomicSub(p.refs + was, 1);
    row[j] = -1;
    if (j < now) {
      const int32_t page = fresh[first[i] + j];
      row[j] = page;
      p.refs[page] = 1;  // it was free: no other sequence counts it
    }
  }
  if (threadIdx.x == 0) p.lens[s] = keep_n[i];
}

// CTA (piece, i): fork i.  Piece 0 gives the child its table row and counts the shared pages;
// every piece copies its share (layers and heads) of the parent's partly filled last page.
__global__ void __launch_bounds__(kMoveThreads) page_fork_kernel(const Pool p, const int32_t* parent, const int32_t* child,
                                                                 const int32_t* ok, const int32_t* fresh, const int32_t* first) {
  pdl_wait();
  const int i = blockIdx.y;
  if (!ok[i]) return;
  const int32_t s = parent[i], c = child[i];
  const int len = p.len_of(s);
  const int full = static_cast<int>(div_of(len, p.ps)), rest = len - full * static_cast<int>(p.ps.d);
  const int32_t* from = p.table + static_cast<size_t>(s) * p.max_pages;
  const int32_t page = rest ? fresh[first[i]] : -1;
  if (blockIdx.x == 0) {
    int32_t* to = p.table + static_cast<size_t>(c) * p.max_pages;
    for (int j = threadIdx.x; j < full; j += kMoveThreads) {
      const int32_t q = from[j];
      to[j] = q;
      if (p.has(q)) atomicAdd(p.refs + q, 1);
    }
    if (threadIdx.x == 0) {
      if (rest) {
        to[full] = page;
        p.refs[page] = 1;
      }
      p.lens[c] = len;
    }
  }
  if (!rest || !p.has(from[full])) return;
  // units of one (layer, head): `rest` consecutive rows
  const int per = rest * p.row_bytes / 16, units = p.layers * p.Hkv;
  const int64_t total = static_cast<int64_t>(units) * per;
  const uint32_t src0 = static_cast<uint32_t>(from[full]) * p.Hkv, dst0 = static_cast<uint32_t>(page) * p.Hkv;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMoveThreads;
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; c0 < total; c0 += step) {
    const int u = static_cast<int>(c0 / per), piece = static_cast<int>(c0 % per);
    const int layer = u / p.Hkv, h = u % p.Hkv;
    const size_t lrow = p.layer_rows() * layer;
    const size_t so = (lrow + static_cast<size_t>(src0 + h) * p.ps.d) * p.row_bytes + piece * 16;
    const size_t to = (lrow + static_cast<size_t>(dst0 + h) * p.ps.d) * p.row_bytes + piece * 16;
    const uint4 a = *reinterpret_cast<const uint4*>(p.k + so);
    const uint4 b = *reinterpret_cast<const uint4*>(p.v + so);
    *reinterpret_cast<uint4*>(p.k + to) = a;
    *reinterpret_cast<uint4*>(p.v + to) = b;
    if (p.km && piece % (kD / 16) == 0) {
      const int r = piece / (kD / 16);
      const size_t sm = lrow + static_cast<size_t>(src0 + h) * p.ps.d + r, tm = lrow + static_cast<size_t>(dst0 + h) * p.ps.d + r;
      reinterpret_cast<uint2*>(p.km)[tm] = reinterpret_cast<const uint2*>(p.km)[sm];
      reinterpret_cast<uint2*>(p.vm)[tm] = reinterpret_cast<const uint2*>(p.vm)[sm];
    }
  }
}

// CTA i: gives back every page of sequence i.  A sequence named twice is released once.
__global__ void __launch_bounds__(kMoveThreads) page_free_kernel(const Pool p, const int32_t* seq, int32_t* ok) {
  __shared__ int twice;
  const int i = blockIdx.x;
  const int32_t s = seq ? seq[i] : i;
  if (threadIdx.x == 0) twice = 0;
  __syncthreads();
  if (seq)
    for (int j = threadIdx.x; j < i; j += kMoveThreads)
      if (seq[j] == s) twice = 1;
  __syncthreads();
  const bool valid = static_cast<uint32_t>(s) < static_cast<uint32_t>(p.max_seqs) && !twice;
  if (threadIdx.x == 0) ok[i] = valid;
  if (!valid) return;
  const int used = pages_of(p.len_of(s), p.ps);
  __syncthreads();
  int32_t* row = p.table + static_cast<size_t>(s) * p.max_pages;
  for (int j = threadIdx.x; j < used; j += kMoveThreads) {
    const int32_t page = row[j];
    if (p.has(page)) atomicSub(p.refs + page, 1);
    row[j] = -1;
  }
  if (threadIdx.x == 0) p.lens[s] = 0;
}

// CTA (piece, i): its share of page src[i] of every layer to page dst[i].  A pair is refused
// whose pages are outside the pool, whose destination an earlier pair writes, or whose
// destination another pair reads: what is left reads nothing that the launch writes.
__global__ void __launch_bounds__(kMoveThreads) page_copy_kernel(const Pool p, const int32_t* src, const int32_t* dst, int n,
                                                                 int32_t* ok) {
  __shared__ int refused;
  const int i = blockIdx.y;
  const int32_t s = src[i], d = dst[i];
  if (threadIdx.x == 0) refused = !(p.has(s) && p.has(d));
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += kMoveThreads)
    if (j != i && (src[j] == d || (j < i && dst[j] == d))) refused = 1;
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) ok[i] = !refused;
  if (refused || s == d) return;
  const size_t page_rows = static_cast<size_t>(p.Hkv) * p.ps.d;
  const int per = static_cast<int>(page_rows * p.row_bytes / 16);   // 16-byte pieces of one layer's page
  const int meta = p.km ? static_cast<int>(page_rows) : 0;          // 8-byte pieces
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMoveThreads;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x;
  const int64_t total = static_cast<int64_t>(p.layers) * per;
  for (int64_t c0 = t0; c0 < total; c0 += 4 * step) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t c = c0 + u * step;
      if (c < total) {
        const size_t off = (p.layer_rows() * (c / per) + s * page_rows) * p.row_bytes + (c % per) * 16;
        a[u] = *reinterpret_cast<const uint4*>(p.k + off);
        b[u] = *reinterpret_cast<const uint4*>(p.v + off);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t c = c0 + u * step;
      if (c < total) {
        const size_t off = (p.layer_rows() * (c / per) + d * page_rows) * p.row_bytes + (c % per) * 16;
        *reinterpret_cast<uint4*>(p.k + off) = a[u];
        *reinterpret_cast<uint4*>(p.v + off) = b[u];
      }
    }
  }
  for (int64_t c = t0; c < static_cast<int64_t>(p.layers) * meta; c += step) {
    const size_t lrow = p.layer_rows() * (c / meta);
    const size_t from = lrow + s * page_rows + c % meta, to = lrow + d * page_rows + c % meta;
    reinterpret_cast<uint2*>(p.km)[to] = reinterpret_cast<const uint2*>(p.km)[from];
    reinterpret_cast<uint2*>(p.vm)[to] = reinterpret_cast<const uint2*>(p.vm)[from];
  }
}

struct PageWs {
  int32_t *fresh, *first;
};
size_t ws_bytes_of(const mikv_pages* p, int n) {
  return align_up(static_cast<size_t>(p->n_pages) * 4, 16) + align_up(static_cast<size_t>(n) * 4, 16);
}
int check_ws(const mikv_pages* p, int n, void* ws, size_t ws_bytes, const char* what, PageWs* out) {
  if (!ws) return fail(MIKV_EINVAL, "%s: null workspace", what);
  if (!aligned16(ws)) return fail(MIKV_EALIGN, "%s: workspace must be 16-byte aligned", what);
  if (ws_bytes < ws_bytes_of(p, n)) return fail(MIKV_ESHAPE, "%s: workspace %zu < %zu", what, ws_bytes, ws_bytes_of(p, n));
  out->fresh = static_cast<int32_t*>(ws);
  out->first = out->fresh + align_up(static_cast<size_t>(p->n_pages) * 4, 16) / 4;
  return MIKV_OK;
}

template <Op OP>
int launch_plan(const Pool& p, const PlanArgs& a, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(a.n) * 12;
  if (smem > 40 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(page_plan_kernel<OP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRequests * 12);
    if (e != cudaSuccess) return check_launch_after(e, "page_plan_kernel");
  }
  page_plan_kernel<OP><<<1, kPlanThreads, smem, st>>>(p, a);
  return check_launch("page_plan_kernel");
}

// CTAs per request for a copy of `pieces` 16-byte pieces: as many as give each thread a few,
// at most what fills the SMs a few times over.
int move_ctas(int64_t pieces, int requests) {
  const int64_t want = (pieces + kMoveThreads * 4 - 1) / (kMoveThreads * 4);
  const int64_t fill = std::max<int64_t>(1, 8LL * kNumSMs / std::max(1, requests));
  return static_cast<int>(std::max<int64_t>(1, std::min(want, fill)));
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" size_t mikv_page_workspace_bytes(const mikv_pages* p, int n) {
  if (!p || p->n_pages < 1 || n < 1 || n > kMaxRequests) return 0;
  return ws_bytes_of(p, n);
}

extern "C" int mikv_page_reserve(const mikv_pages* pages, const int32_t* seqs, const int32_t* add, int n, int32_t* start,
                                 void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  Pool p;
  if (int e = check_pages(pages, "page_reserve", &p)) return e;
  if (n < 0 || n > kMaxRequests || (!seqs && n > p.max_seqs)) return fail(MIKV_ESHAPE, "page_reserve: n=%d", n);
  if (n == 0) return MIKV_OK;
  if (!add || !start) return fail(MIKV_EINVAL, "page_reserve: null pointer");
  PageWs w;
  if (int e = check_ws(pages, n, ws, ws_bytes, "page_reserve", &w)) return e;
  return launch_plan<Op::kReserve>(p, {seqs, add, n, 0, start, w.fresh, w.first}, as_stream(stream));
}

extern "C" int mikv_page_fork(const mikv_pages* pages, const int32_t* parent, const int32_t* child, int n, int32_t* ok,
                              void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  Pool p;
  if (int e = check_pages(pages, "page_fork", &p)) return e;
  if (n < 0 || n > kMaxRequests) return fail(MIKV_ESHAPE, "page_fork: n=%d", n);
  if (n == 0) return MIKV_OK;
  if (!parent || !child || !ok) return fail(MIKV_EINVAL, "page_fork: null pointer");
  PageWs w;
  if (int e = check_ws(pages, n, ws, ws_bytes, "page_fork", &w)) return e;
  const cudaStream_t st = as_stream(stream);
  if (int e = launch_plan<Op::kFork>(p, {parent, child, n, 0, ok, w.fresh, w.first}, st)) return e;
  const int64_t pieces = static_cast<int64_t>(p.layers) * p.Hkv * p.ps.d * p.row_bytes / 16;
  return check_launch_after(launch_after(page_fork_kernel, dim3(move_ctas(pieces, n), n), dim3(kMoveThreads), 0, st, p, parent,
                                         child, static_cast<const int32_t*>(ok), static_cast<const int32_t*>(w.fresh),
                                         static_cast<const int32_t*>(w.first)),
                            "page_fork_kernel");
}

extern "C" int mikv_page_free(const mikv_pages* pages, const int32_t* seqs, int n, int32_t* ok, void* stream) {
  clear_error();
  Pool p;
  if (int e = check_pages(pages, "page_free", &p)) return e;
  if (n < 0 || n > 65535 || (!seqs && n > p.max_seqs)) return fail(MIKV_ESHAPE, "page_free: n=%d", n);
  if (n == 0) return MIKV_OK;
  if (!ok) return fail(MIKV_EINVAL, "page_free: null ok");
  page_free_kernel<<<n, kMoveThreads, 0, as_stream(stream)>>>(p, seqs, ok);
  return check_launch("page_free_kernel");
}

extern "C" int mikv_page_copy(const mikv_pages* pages, const int32_t* src, const int32_t* dst, int n, int32_t* ok,
                              void* stream) {
  clear_error();
  Pool p;
  if (int e = check_pages(pages, "page_copy", &p)) return e;
  if (n < 0 || n > 65535) return fail(MIKV_ESHAPE, "page_copy: n=%d", n);
  if (n == 0) return MIKV_OK;
  if (!src || !dst || !ok) return fail(MIKV_EINVAL, "page_copy: null pointer");
  const int64_t pieces = static_cast<int64_t>(p.layers) * p.Hkv * p.ps.d * p.row_bytes / 16;
  page_copy_kernel<<<dim3(move_ctas(pieces, n), n), kMoveThreads, 0, as_stream(stream)>>>(p, src, dst, n, ok);
  return check_launch("page_copy_kernel");
}

extern "C" int mikv_page_compact(const mikv_pages* pages, const int32_t* seqs, const int32_t* keep_pos, const int32_t* keep_n,
                                 int n, int max_keep, int32_t* ok, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  Pool p;
  if (int e = check_pages(pages, "page_compact", &p)) return e;
  if (n < 0 || n > kMaxRequests || (!seqs && n > p.max_seqs)) return fail(MIKV_ESHAPE, "page_compact: n=%d", n);
  if (max_keep < 0 || max_keep > p.cap) return fail(MIKV_ESHAPE, "page_compact: max_keep=%d", max_keep);
  if (n == 0) return MIKV_OK;
  if ((!keep_pos && max_keep > 0) || !keep_n || !ok) return fail(MIKV_EINVAL, "page_compact: null pointer");
  PageWs w;
  if (int e = check_ws(pages, n, ws, ws_bytes, "page_compact", &w)) return e;
  const int chunks = std::max(1, (max_keep + kMoveRows - 1) / kMoveRows);
  const int64_t ctas = static_cast<int64_t>(p.layers) * n * p.Hkv * chunks;
  if (ctas > 0x7fffffffLL) return fail(MIKV_ESHAPE, "page_compact: layers * n * Hkv * max_keep too large for one call");
  const cudaStream_t st = as_stream(stream);
  if (int e = launch_plan<Op::kCompact>(p, {seqs, keep_n, n, max_keep, ok, w.fresh, w.first}, st)) return e;
  const int32_t *fresh = w.fresh, *first = w.first;
  const int64_t checks = (static_cast<int64_t>(p.layers) * p.Hkv * max_keep + kMoveThreads * 4 - 1) / (kMoveThreads * 4);
  const int per = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(checks, std::max(1, 8 * kNumSMs / n))));
  if (int e = check_launch_after(launch_after(page_check_kernel, dim3(per, n), dim3(kMoveThreads), 0, st, p, seqs, keep_pos, keep_n, n,
                                              max_keep, ok),
                                 "page_check_kernel"))
    return e;
  const int32_t* checked = ok;
  if (int e = check_launch_after(launch_after(page_compact_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kMoveThreads), 0, st, p,
                                              seqs, keep_pos, keep_n, n, max_keep, chunks, checked, fresh, first),
                                 "page_compact_kernel"))
    return e;
  return check_launch_after(launch_after(page_commit_kernel, dim3(n), dim3(kMoveThreads), 0, st, p, seqs, keep_n, ok, fresh, first),
                            "page_commit_kernel");
}
