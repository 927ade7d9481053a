// What the tcgen05 attention kernels share: a query tile's softmax over a tile of scores in TMEM, and the
// tensor-memory and matrix primitives around it (internal; not part of the C ABI).
//
// A query row is one TMEM lane and one thread.  Its weights are exp2(l - m) with a reference m that follows the running
// maximum: it is moved, and the accumulated sums rescaled, only where the maximum has outgrown it by 2^grow.
#pragma once

#include <cuda_bf16.h>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace mikv {
namespace at {

template <bool BF>
struct Weights {
  static constexpr float shift = BF ? 0.f : 13.f;  // log2 of the weights' factor
  static constexpr float grow = BF ? 8.f : 2.f;    // log2 of the growth that moves the reference
};

// The same value in every lane, told to the compiler: what depends on it stays in uniform
// registers, which the matrix instructions read.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

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
// `last`: the last key that the row may see, its position p or less.  Args: qb.window, qb.sinks and scale.
// PARTS 2: the scores are the sum of two products, the second COLS columns behind the first.
// W: the weights' factor, and how far the reference may lag.
// A weight is rounded once to 16 bits, half a step of its own, as the products take it; why, the kernels say.
// `settle` returns once all products into the accumulator that were issued are done; it is called before a rescaling.
template <bool BF, int COLS, int PARTS, class W = Weights<BF>, class Args, class Settle>
__device__ __forceinline__ void softmax_tile(const Args& a, uint32_t ts, uint32_t to, bool whole, int p, int last, int j0, Row& r,
                                             const uint32_t (&ready)[2], const Settle& settle) {
  float s[COLS];
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) ld32(ts + c * 32, s + c * 32);
  wait_ld();
  if (PARTS == 2) {
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      float x[32];
      ld32(ts + COLS + c, x);
      wait_ld();
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 y = __fadd2_rn(make_float2(s[c + i], s[c + i + 1]), make_float2(x[i], x[i + 1]));
        s[c + i] = y.x;
        s[c + i + 1] = y.y;
      }
    }
  }
  if (!whole) {
    // the row sees columns lo .. hi and those below sk; 32 columns whole to the warp's rows are left alone
    const int hi = last - j0, lo = a.qb.window > 0 ? p - j0 - a.qb.window + 1 : 0, sk = a.qb.sinks - j0;
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
  const bool grew = (top - r.m) * a.scale > W::grow;   // from -inf too; never by NaN
  if (__any_sync(0xffffffffu, grew)) {
    // a row whose own maximum has not outgrown its reference keeps it: its result does not hang on
    // the other rows of the warp, which may be rows that do not count
    const float alpha = grew ? ex2((r.m - top) * a.scale) : 1.f;
    if (grew) r.m = top;
    r.l *= alpha;
    if (!r.first) {
      settle();
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
  const float neg = r.m == -INFINITY ? 0.f : W::shift - r.m * a.scale;
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
        if (COLS <= 64) tc::mbar_arrive(ready[1]);
      }
    }
  }
  r.l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

}  // namespace at
}  // namespace mikv
