// Attention of a prompt, or of a chunk of one, under a sliding window with sinks.
//
// Mathematics: one pass over the visible keys with a running maximum and sum per query row,
// out = sum_j exp(l_j - m) v_j / sum_j exp(l_j - m).  A CTA holds 64 query rows of one head;
// tiles of 64 keys that none of its rows sees are not read.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {

int window_attention_status(unsigned* out, bool clear) { return tc::wait_giveups(out, clear); }

namespace {

constexpr int kWaThreads = 128, kWaQ = 64, kWaK = 64;
constexpr int kWaTile = kWaK * kD * 2;

struct WindowArgs {
  RowView q, k, v, out;
  float* lse;
  const int32_t *q_lens, *k_lens;
  int B, Hq, Hkv, Tq, Tk, window, sinks;
  float scale;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma16816(d, a[0], a[1], a[2], a[3], b0, b1);
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

template <bool BF>
__global__ void __launch_bounds__(kWaThreads) window_attention_kernel(const WindowArgs a) {
  constexpr float kShift = BF ? 0.f : 15.f;  // fp16 weights carry 2^15: no subnormals down to 2^-29 of the largest
  extern __shared__ __align__(128) uint8_t smem[];
  const int b = blockIdx.z, h = blockIdx.y, q0 = blockIdx.x * kWaQ, tid = threadIdx.x;
  const int w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int ql = a.q_lens ? min(max(a.q_lens[b], 0), a.Tq) : a.Tq, kl = a.k_lens ? min(max(a.k_lens[b], 0), a.Tk) : a.Tk;
  if (q0 >= ql) return;
  const int hk = h / (a.Hq / a.Hkv), p0 = kl - ql + q0, p1 = min(p0 + kWaQ - 1, kl - 1);  // positions of the rows
  // key tiles: the sinks', then from the first row's window to the last row
  const int lo = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
  const int tw0 = lo / kWaK, tw1 = p1 < 0 ? 0 : p1 / kWaK + 1;
  const int ts = a.window > 0 ? min((min(a.sinks, kl) + kWaK - 1) / kWaK, min(tw0, tw1)) : 0;
  const int tiles = ts + max(tw1 - tw0, 0);
  const uint32_t s0 = smem_u32(smem);
  const auto load = [&](int i) {
    const int j0 = (i < ts ? i : tw0 + i - ts) * kWaK;
    const uint32_t st = s0 + (i & 1) * 2 * kWaTile;
#pragma unroll
    for (int u = 0; u < kWaK * 16 / kWaThreads; ++u) {
      const int c = tid + u * kWaThreads, r = c >> 4, p = c & 15;
      const bool ok = j0 + r < kl;
      const uint32_t off = r * (kD * 2) + ((p ^ (r & 7)) << 4);
      cp_async16(st + off, ok ? a.k.row(b, hk, j0 + r) + p * 16 : a.k.p, ok);
      cp_async16(st + kWaTile + off, ok ? a.v.row(b, hk, j0 + r) + p * 16 : a.v.p, ok);
    }
  };
  uint32_t qf[kD / 16][4];
  const int r0 = q0 + w * 16 + g;
#pragma unroll
  for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = r0 + 8 * (j & 1);
      qf[ks][j] = row < ql ? *reinterpret_cast<const uint32_t*>(a.q.row(b, h, row) + (16 * ks + 8 * (j >> 1) + 2 * t) * 2) : 0u;
    }
  float o[kD / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  if (tiles > 0) load(0);
  cp_async_commit();
  for (int i = 0; i < tiles; ++i) {
    if (i + 1 < tiles) load(i + 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const uint32_t st = s0 + (i & 1) * 2 * kWaTile;
    const int j0 = (i < ts ? i : tw0 + i - ts) * kWaK;
    float s[kWaK / 8][4];
#pragma unroll
    for (int nt = 0; nt < kWaK / 8; ++nt) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k2 = 0; k2 < kD / 32; ++k2) {
        const int r = nt * 8 + (lane & 7), c = k2 * 4 + (lane >> 3);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(st + r * (kD * 2) + ((c ^ (r & 7)) << 4), b0, b1, b2, b3);
        mma<BF>(d, qf[2 * k2], b0, b1);
        mma<BF>(d, qf[2 * k2 + 1], b2, b3);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = kl - ql + r0 + 8 * (j >> 1), key = j0 + nt * 8 + 2 * t + (j & 1);
        const bool see = key <= p && (a.window == 0 || key > p - a.window || key < a.sinks);
        s[nt][j] = see ? d[j] * a.scale : -INFINITY;
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = m[r];
#pragma unroll
      for (int nt = 0; nt < kWaK / 8; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * r], s[nt][2 * r + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float sub = mx == -INFINITY ? 0.f : mx - kShift, alpha = mx == -INFINITY ? 0.f : ex2(m[r] - mx);
      m[r] = mx;
      l[r] *= alpha;
#pragma unroll
      for (int c = 0; c < kD / 8; ++c) {
        o[c][2 * r] *= alpha;
        o[c][2 * r + 1] *= alpha;
      }
#pragma unroll
      for (int nt = 0; nt < kWaK / 8; ++nt)
#pragma unroll
        for (int j = 2 * r; j < 2 * r + 2; ++j) {
          s[nt][j] = ex2(s[nt][j] - sub);
          l[r] += s[nt][j];
        }
    }
#pragma unroll
    for (int kt = 0; kt < kWaK / 16; ++kt) {
      const uint32_t pf[4] = {pack2<BF>(s[2 * kt][0], s[2 * kt][1]), pack2<BF>(s[2 * kt][2], s[2 * kt][3]),
                              pack2<BF>(s[2 * kt + 1][0], s[2 * kt + 1][1]), pack2<BF>(s[2 * kt + 1][2], s[2 * kt + 1][3])};
#pragma unroll
      for (int c = 0; c < kD / 8; c += 2) {
        const int r = kt * 16 + (lane & 15), cc = c + (lane >> 4);
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(st + kWaTile + r * (kD * 2) + ((cc ^ (r & 7)) << 4), b0, b1, b2, b3);
        mma<BF>(o[c], pf, b0, b1);
        mma<BF>(o[c + 1], pf, b2, b3);
      }
    }
    __syncthreads();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = r0 + 8 * r;
    if (row >= ql) continue;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
    for (int c = 0; c < kD / 8; ++c)
      *reinterpret_cast<uint32_t*>(a.out.row(b, h, row) + (c * 8 + 2 * t) * 2) = pack2<BF>(o[c][2 * r] * inv, o[c][2 * r + 1] * inv);
    if (t == 0 && a.lse) a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Tq + row] = (m[r] + (log2f(l[r]) - kShift)) * 0.6931471805599453f;
  }
}

}  // namespace
}  // namespace mikv

using namespace mikv;

extern "C" int mikv_window_attention(const mikv_rows* q, const mikv_rows* k, const mikv_rows* v, int B, int Hq, int Hkv, int Tq,
                                     int Tk, int D, int type, const int32_t* q_lens, const int32_t* k_lens, int window, int sinks,
                                     const mikv_rows* out, float* lse, void* stream) {
  clear_error();
  if (type != MIKV_PAGES_FP16 && type != MIKV_PAGES_BF16) return fail(MIKV_EINVAL, "window_attention: type=%d", type);
  if (D != kD) return fail(MIKV_EUNSUPPORTED, "window_attention: D=%d (only %d)", D, kD);
  if (window < 0 || sinks < 0) return fail(MIKV_EINVAL, "window_attention: window=%d sinks=%d", window, sinks);
  if (B < 0 || B > 65535 || Hkv < 1 || Hq < 1 || Hq > 65535 || Hq % Hkv || Tq < 1 || Tk < 1)
    return fail(MIKV_ESHAPE, "window_attention: B=%d Hq=%d Hkv=%d Tq=%d Tk=%d", B, Hq, Hkv, Tq, Tk);
  if (B == 0) return MIKV_OK;
  if (int e = check_rows(q, "window_attention", "q")) return e;
  if (int e = check_rows(k, "window_attention", "k")) return e;
  if (int e = check_rows(v, "window_attention", "v")) return e;
  if (int e = check_rows(out, "window_attention", "out")) return e;
  const WindowArgs a = {row_view(*q), row_view(*k), row_view(*v), row_view(*out), lse, q_lens, k_lens,
                        B, Hq, Hkv, Tq, Tk, window, sinks, 1.4426950408889634f * 0.08838834764831845f};
  const auto kern = type == MIKV_PAGES_BF16 ? window_attention_kernel<true> : window_attention_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kWaTile);
  if (e != cudaSuccess) return check_launch_after(e, "window_attention_kernel");
  kern<<<dim3((Tq + kWaQ - 1) / kWaQ, Hq, B), kWaThreads, 4 * kWaTile, as_stream(stream)>>>(a);
  return check_launch("window_attention_kernel");
}
