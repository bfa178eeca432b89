// diff_sm100.cuh -- device helpers shared by the differential-attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "diff.h"
#include "sm100.cuh"

namespace skl {

// 4-D tiled load of one box [1][1][rows][64 features]; c0 (features) is 0, 64,
// 128 or 192 elements, so it starts on a 16-byte boundary.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// kind::f16 instruction descriptor; A and B are both bf16 or both fp16.
template <bool F16>
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, int a_mn = 0, int b_mn = 0) {
  return F16 ? (idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10)))
             : idesc_bf16(M, N, a_mn, b_mn);
}

// A descriptor as this point of the program computes it: keeps the compiler from
// holding every product's descriptor of a loop in registers (and spilling them).
__device__ __forceinline__ uint64_t here(uint64_t desc) {
  asm volatile("" : "+l"(desc));
  return desc;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<__half2*>(&w));
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
}

__device__ __forceinline__ float load_lam(const Lambda& l, long long b, long long h, long long n,
                                          bool f16) {
  const long long i = b * l.b + h * l.h + n * l.n;
  if (l.f32) return static_cast<const float*>(l.ptr)[i];
  if (f16) return __half2float(static_cast<const __half*>(l.ptr)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(l.ptr)[i]);
}

// The reference m of a row's weights 2^(x - m), x in log2: what a row's largest x
// sets it to, and how far x may rise above it before it is set anew.  Weights go
// into the value product in 16 bits.  bf16 has fp32's range: the largest weight is
// between 1 and 2^8.  fp16 ends at 2^16 and loses bits under 2^-14, so its largest
// is between 2^11 and 2^15: weights keep 11 bits down to 2^-25 of the largest, and
// half its smallest step is 2^-36 of it.  (With references as for bf16 the step
// would be 2^-25 of it: keys 18 nats under the largest would not count.)  The
// smaller slack costs rescales where scores are wide: B1 H16 N4096 d64/128 causal,
// scores of standard deviation 4: 131 us against 128; of 1: 117 both ways.  The
// roundings up and down hold the upper end for scores of any size (a score of 2^28
// has steps of 32).
template <bool F16>
struct WeightRef {
  static constexpr float kHead = F16 ? 11.f : 0.f, kSlack = F16 ? 4.f : 8.f;
  // a score's x, no less than what the exponential will see
  static __device__ __forceinline__ float top(float score, float c) {
    return F16 ? __fmul_ru(score, c) : score * c;
  }
  static __device__ __forceinline__ float at(float top) { return F16 ? __fsub_ru(top, kHead) : top; }
  // the largest x that m still serves
  static __device__ __forceinline__ float limit(float m) {
    return F16 ? __fadd_rd(m, kHead + kSlack) : m + kSlack;
  }
};

// Lengths of batch b, clamped to the tensors.
struct Lens {
  int q, k;
};
__device__ __forceinline__ Lens diff_lens(const DiffShape& s, int b) {
  Lens l;
  l.q = s.q_lens ? min(max(s.q_lens[b], 0), s.NQ) : s.NQ;
  l.k = s.k_lens ? min(max(s.k_lens[b], 0), s.NK) : s.NK;
  return l;
}

// Rows [r0, r1) of a 128-byte-swizzled tile (64-feature chunks of `rows` x 128
// bytes) set to zero by one warp.  The swizzle permutes 16-byte pieces within
// a row, so whole rows need no address arithmetic.
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int chunks, int rows, int r0, int r1,
                                               int lane) {
  const int n = (r1 - r0) * 8;
  for (int c = 0; c < chunks; ++c) {
    uint4* dst = reinterpret_cast<uint4*>(tile + c * rows * 128 + r0 * 128);
    for (int i = lane; i < n; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Waits for something that may come any time until the kernel's end (a ragged
// tile some units ahead): ends with the phase, with an abort that another role
// raised when one of its own bounded waits ran out, or after 1024 wait limits.
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity, const WaitCtl& c) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait(a, parity)) return true;
    if (*c.abort) return false;
    if (globaltimer_ns() - t0 > 1024 * c.limit_ns) {
      raise_abort(c, kStatusTimeout);
      return false;
    }
    __nanosleep(200);
  }
}

// Transposes NP 16-byte pieces among each NP neighbouring lanes: lane i of such
// a group starts with pieces 0..NP-1 of its own row and ends with piece i of the
// group's rows 0..NP-1, so that one store of the group covers a row's NP pieces.
// (Each lane storing its own row touches 32 lines with every instruction.)
template <int NP>
__device__ __forceinline__ void transpose_pieces(uint4 (&p)[NP], int lane) {
#pragma unroll
  for (int s = 1; s < NP; s <<= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      if (j & s) continue;
      uint4 give = up ? p[j] : p[j | s];
      give.x = __shfl_xor_sync(0xffffffffu, give.x, s);
      give.y = __shfl_xor_sync(0xffffffffu, give.y, s);
      give.z = __shfl_xor_sync(0xffffffffu, give.z, s);
      give.w = __shfl_xor_sync(0xffffffffu, give.w, s);
      if (up) p[j] = give;
      else p[j | s] = give;
    }
  }
}

// Units dealt to a persistent grid in a snake order (longest first).
struct SnakeSched {
  int total, G, cta, round;
  __device__ SnakeSched(int t)
      : total(t), G(static_cast<int>(gridDim.x)), cta(static_cast<int>(blockIdx.x)), round(0) {}
  __device__ __forceinline__ bool next(int& u) {
    for (;;) {
      const int base = round * G;  // at most total + G: the host keeps units below 2^30
      if (base >= total) return false;
      const int uu = base + ((round & 1) ? (G - 1 - cta) : cta);
      ++round;
      if (uu < total) {
        u = uu;
        return true;
      }
    }
  }
};

}  // namespace skl
