// Which sequence, position and slot every row of a packed batch has.
//
// Request i has counts[i] rows, one request after the other.  A CTA adds up all counts (they are
// few, and an L2 read away), and each of its threads finds the requests of four rows by a binary
// search in the sums.  One launch, bound by latency: counts, then lengths and starts, then the
// table are three dependent reads.  A sequence that two requests name belongs to the first: a
// hash table in shared memory keeps the lowest request of each (one insertion a request; comparing
// all pairs would be n^2 / 2 reads).
#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int batch_rows_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kMapThreads = 256;
constexpr int kMapRows = 4 * kMapThreads;   // of a CTA
constexpr int kMaxBatch = 4096;             // requests of a call
constexpr int kMaxMapRows = 1 << 30;        // and its rows: numbers of a CTA behind the last one fit 32 bits too
constexpr int kMapSmem = (kMaxBatch + 1 + 2 * 2 * kMaxBatch) * 4;   // the most that a call needs: sums, and a table of two words a slot

struct MapArgs {
  Pool p;
  const int32_t *seqs, *start, *counts;
  int n, rows, slots;        // slots of the hash table: a power of two, twice the requests at least
  int32_t *row_start, *row_seq, *row_pos, *row_slot;
};

__device__ __forceinline__ uint32_t hash_of(int32_t s, int slots) {
  return (static_cast<uint32_t>(s) * 2654435761u) >> 7 & static_cast<uint32_t>(slots - 1);   // Knuth's multiplier
}

__global__ void __launch_bounds__(kMapThreads) batch_rows_kernel(const MapArgs a) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t warp_sums[kMapThreads / 32];
  int32_t* first = smem;                 // [n + 1] rows before each request, held at `rows`
  int32_t* key = first + a.n + 1;        // [slots] sequence, -1 free
  int32_t* who = key + a.slots;          // [slots] its first request
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (a.seqs)
    for (int i = tid; i < a.slots; i += kMapThreads) {
      key[i] = -1;
      who[i] = a.n;
    }
  int64_t before = 0;
  for (int i0 = 0; i0 < a.n; i0 += kMapThreads) {
    const int i = i0 + tid;
    const int64_t c = i < a.n ? max(a.counts[i], 0) : 0;
    int64_t v = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();   // the last pass's sums have been read; the table is clear
    if (lane == 31) warp_sums[w] = v;
    __syncthreads();
    int64_t sum = 0;
#pragma unroll
    for (int k = 0; k < kMapThreads / 32; ++k) {
      if (k < w) v += warp_sums[k];
      sum += warp_sums[k];
    }
    if (i < a.n) first[i + 1] = static_cast<int32_t>(min(before + v, static_cast<int64_t>(a.rows)));
    before += sum;
    if (a.seqs && i < a.n) {
      const int32_t s = a.seqs[i];
      if (s >= 0)
        for (uint32_t h = hash_of(s, a.slots);; h = (h + 1) & (a.slots - 1)) {
          const int32_t old = atomicCAS(&key[h], -1, s);
          if (old == -1 || old == s) {
            atomicMin(&who[h], i);
            break;
          }
        }
    }
  }
  if (tid == 0) first[0] = 0;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = tid; i <= a.n; i += kMapThreads) a.row_start[i] = first[i];
#pragma unroll
  for (int e = 0; e < kMapRows / kMapThreads; ++e) {
    const int r = blockIdx.x * kMapRows + e * kMapThreads + tid;
    if (r >= a.rows) return;
    int lo = 0, hi = a.n;   // the first request that ends behind r; n: none
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (first[mid + 1] > r)
        hi = mid;
      else
        lo = mid + 1;
    }
    int32_t seq = -1, pos = -1, slot = -1;
    if (lo < a.n) {
      const int32_t s = a.seqs ? a.seqs[lo] : lo;
      bool mine = static_cast<uint32_t>(s) < static_cast<uint32_t>(a.p.max_seqs);
      if (mine && a.seqs) {
        uint32_t h = hash_of(s, a.slots);
        while (key[h] != s) h = (h + 1) & (a.slots - 1);
        mine = who[h] == lo;
      }
      if (mine) {
        const int32_t len = a.p.len_of(s);
        const int32_t from = a.start ? a.start[lo] : len - (first[lo + 1] - first[lo]);   // the rows that the arrays hold
        if (from >= 0) {   // else refused, or more rows than slots
          const int64_t at = static_cast<int64_t>(from) + (r - first[lo]);
          seq = s;
          pos = static_cast<int32_t>(min(at, static_cast<int64_t>(0x7fffffff)));
          if (at < len) {
            const uint32_t q = div_of(static_cast<uint32_t>(at), a.p.ps);
            const int32_t page = a.p.table[static_cast<size_t>(s) * a.p.max_pages + q];
            if (a.p.has(page))
              slot = page * static_cast<int32_t>(a.p.ps.d) + static_cast<int32_t>(static_cast<uint32_t>(at) - q * a.p.ps.d);
            else
              tc::report_giveup(tc::kBadPage);
          }
        }
      }
    }
    a.row_seq[r] = seq;
    a.row_pos[r] = pos;
    a.row_slot[r] = slot;
  }
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" int mikv_batch_rows(const mikv_pages* pages, const int32_t* seqs, const int32_t* start, const int32_t* counts, int n,
                               int rows, int32_t* row_start, int32_t* row_seq, int32_t* row_pos, int32_t* row_slot, void* stream) {
  clear_error();
  MapArgs a;
  if (int e = check_pages(pages, "batch_rows", &a.p)) return e;
  if (static_cast<int64_t>(a.p.n_pages) * a.p.ps.d > 0x7fffffffLL)
    return fail(MIKV_ESHAPE, "batch_rows: n_pages * page_size above 2^31");
  if (n < 0 || n > kMaxBatch || rows < 0 || rows > kMaxMapRows || (!seqs && n > a.p.max_seqs)) return fail(MIKV_ESHAPE, "batch_rows: n=%d rows=%d", n, rows);
  if (n == 0 && rows == 0) return MIKV_OK;
  if (!row_start || (n && !counts) || (rows && (!row_seq || !row_pos || !row_slot))) return fail(MIKV_EINVAL, "batch_rows: null pointer");
  a.seqs = seqs;
  a.start = start;
  a.counts = counts;
  a.n = n;
  a.rows = rows;
  a.row_start = row_start;
  a.row_seq = row_seq;
  a.row_pos = row_pos;
  a.row_slot = row_slot;
  a.slots = 0;
  if (seqs)
    for (a.slots = 64; a.slots < 2 * n;) a.slots *= 2;
  const size_t smem = (static_cast<size_t>(n) + 1 + 2 * a.slots) * 4;
  // The limit belongs to the kernel, not to the launch: all that set it set the same one, which holds for what other threads launch.
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(batch_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMapSmem);
    if (e != cudaSuccess) return check_launch_after(e, "batch_rows_kernel");
  }
  const int ctas = rows ? (rows - 1) / kMapRows + 1 : 1;
  batch_rows_kernel<<<ctas, kMapThreads, smem, as_stream(stream)>>>(a);
  return check_launch("batch_rows_kernel");
}
