// diff_bwd_sm100.cu -- backward of differential attention for sm_100a.
//
// With G = dO V^T, P_t = 2^(c_t x_t - LSE_t log2e) regenerated from the saved
// LSEs and D_t[i] = <dO[i], O_t[i]>,
//
//   A   = P1 - lam P2              dV   = A^T dO
//   X1  = P1 (G - D1)              dQ1  = s1 X1 K1    dK1 = s1 X1^T Q1
//   X2  = lam P2 (D2 - G)          dQ2  = s2 X2 K2    dK2 = s2 X2^T Q2
//   dlam[i] = -sum_j P2 G, summed over what lam is broadcast over (D2 again, but from
//             the unrounded P2: as a sum of few large terms it would show the
//             rounding of O2)
//
// Two kinds of pass of one kernel template, each with a resident 128-row tile R
// and streamed 64-row tiles C, so that every gradient is accumulated in TMEM by one
// CTA in a fixed order: no atomics, and results that repeat bit for bit.
//
//   kDiffKV  R = K1, K2, V   C = Q1, Q2, dO of every query head that shares
//            the key head: its gradients are one sum over the group
//   kDiffQ   R = Q1, Q2, dO  C = K1, K2, V
//
// Per step: S1, S2 and G (M = 128 resident rows, N = 64 streamed rows) by
// tcgen05 from shared memory; the compute warps turn them into X1, X2 and A in
// 16 bits and store those to TMEM, where they are the A operands of the output
// products OUT += X C (C read with its features contiguous).
// TMEM: S1 [0,64) S2 [64,128) G [128,192) X1 [192,224) X2 [224,256) OUT [256,..)
// With X1 and X2 both there, A goes through shared memory (K-major, 128-byte
// swizzle); in the dV-only pass it takes X1's place.
//
// Two threads issue.  One gives out S(t+1) as soon as the warps have read S(t),
// and G(t+1) as soon as they have read G(t); the other the output products of
// step t once X(t) is written.  S, its exponentials and G are then under way
// while the step before is contracted, the next unit's begin during this one's
// end, and one thread's waits are filled with the other's products.
//
// TMEM holds 256 output columns beside the 256 above, shared memory the
// resident tiles and two stages. That decides the passes:
//   d = 64            two passes: kDiffKV gives dK1, dK2 and dV at once
//   d = 128           three: dV has a pass of its own (S1, S2 only; 128 value columns)
//   d = 128, dv = 256 three, with twice the units: one of kDiffKV or kDiffQ has one
//                     map (SEL 1, either map), as V, dO and both maps' tiles do not
//                     fit at once, and one of the dV pass a half of the values
//
// The passes read the same records and write different outputs, so each starts
// while the one before still runs (programmatic launch) and takes the
// multiprocessors as they become free (B1 H16 N4096 d64/128 causal: 347 us against
// 356).
//
// What bounds it: S and G are M128 N64 products, which hold the tensor pipe for as
// long as N128 ones.  Over all passes a product is given out every 109 clocks (B1
// H16 N4096 causal: 353 us at 1845 MHz for d64/128, 593 us at 1762 MHz for
// d128/128), of which the pipe is busy for 65 to 83.  Beside them every visible
// pair takes 4 exponentials at d = 64, 6 at d = 128 and 8 at dv = 256.
//
// X1, X2 and A are rounded to 16 bits for their products, as any 16-bit tensor-core
// product needs, after their arithmetic in fp32; D1 and D2 are formed from O and O2
// as the forward stored them, in 16 bits (dlam, which would show that rounding, is
// not).  Every sum is in fp32.
#include "diff_sm100.cuh"

#include <type_traits>

namespace skl {
namespace {

constexpr int R = kDiffRows;
constexpr int CB = kDiffStep;
constexpr int NWG = 4;             // compute warpgroups
constexpr int CPW = CB / NWG;      // streamed rows per compute warpgroup
constexpr int NTHREADS = (3 + 1 + 4 * NWG) * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kColS2 = 64, kColG = 128, kColX1 = 192, kColX2 = 224, kColOut = 256;
constexpr int kNever = 1 << 30;

template <int PASS, int D, int DV, int SEL>
struct BwdLay {
  static constexpr bool KV = PASS == kDiffKV;
  static constexpr bool S1 = (SEL & 5) != 0, S2 = (SEL & 6) != 0;  // maps whose P is formed
  static constexpr bool X1 = (SEL & 1) != 0, X2 = (SEL & 2) != 0;
  static constexpr bool ONE = SEL == 1;            // one map, chosen per unit
  static constexpr bool WG = (SEL & 3) != 0, WV = (SEL & 4) != 0;
  static constexpr int r1 = S1 ? R * D * 2 : 0;
  static constexpr int r2 = S2 ? R * D * 2 : 0;
  static constexpr int r3 = WG ? R * DV * 2 : 0;   // the dV-only pass needs no V
  static constexpr int c1 = S1 ? CB * D * 2 : 0;
  static constexpr int c2 = S2 ? CB * D * 2 : 0;
  static constexpr int c3 = CB * DV * 2;
  static constexpr int rec = KV ? CB * kDiffRec * 4 : 0;
  // dO (kKV) or V (kQ) rides in the ring with the other streamed tiles where the
  // output products read it too (dV); where only G does, it has a ring of its
  // own and is freed a step earlier, which at d = 128 makes room for a third stage.
  static constexpr bool CR3 = WV;
  static constexpr bool AS = WV && WG;             // A through shared memory
  static constexpr int budget = 232448 - 1024 - 512;
  static constexpr int a_off = r1 + r2 + r3;
  static constexpr int v_off = a_off + (AS ? 2 * R * CB * 2 : 0);
  static constexpr int stage = c1 + c2 + (CR3 ? c3 : 0);
  static constexpr int load_bytes = stage + rec;
  static constexpr int NSV = CR3 ? 0 : (v_off + 2 * c3 + 3 * (stage + rec) <= budget ? 2 : 1);
  static constexpr int c_off = v_off + NSV * c3;
  static constexpr int fit = (budget - c_off) / (stage + rec);
  static constexpr int NST = fit > 4 ? 4 : fit;
  static constexpr int rec_off = c_off + NST * stage;
  static constexpr int bar_off = rec_off + NST * rec;
  // cfull cempty craw [NST], vfull vempty vraw [NSV], rfull rempty sfull sempty
  // gfull xfull xempty ofull oempty drain[2]
  static constexpr int nbar = 3 * NST + 3 * NSV + 11;
  static constexpr int misc_off = bar_off + nbar * 8;
  static constexpr int alloc = misc_off + 16 + 1024;
  static constexpr int o1 = kColOut;
  static constexpr int o2 = o1 + (X1 ? D : 0);
  static constexpr int o3 = o2 + (X2 ? D : 0);
  static_assert(o3 + (WV ? DV : 0) <= 512, "TMEM budget exceeded");
  static_assert(NST >= 3, "streamed ring too shallow");
  static_assert(alloc <= 232448, "shared memory budget exceeded");
  static_assert(!(PASS == kDiffQ && WV), "dV belongs to the key pass");
};

// A unit: 128 resident rows, and the streamed tiles [c_first, c_first + tiles)
// of each of `heads` query heads (kQ: of one key head).  `half`: the value half,
// or with one map per unit (SEL 1) that map.
struct BwdUnit {
  int b, h, hk, half, r0, c_first, tiles, heads, lo, hi;
  Lens l;
  // Streamed rows [lo, hi) are in the problem; a tile that reaches past either
  // end, yet not beyond the tensor, is ragged and cleaned before use.
  __device__ __forceinline__ bool ragged(int tile, int n) const {
    const int c0 = (c_first + tile) * CB;
    return c0 < lo || (c0 + CB > hi && hi < n);
  }
};

template <int PASS>
__device__ __forceinline__ BwdUnit decode(const DiffBwdParams& p, int u) {
  BwdUnit w;
  w.half = u & (p.nhalf - 1);
  u >>= p.nhalf - 1;
  const int tile = p.by_heads(u);
  if (PASS == kDiffKV) {
    // key tiles that the most rows see first, heads innermost
    const int bh = u - tile * (p.s.B * p.s.HK);
    w.r0 = tile * R;
    w.b = p.s.by_HK(bh);
    w.hk = bh - w.b * p.s.HK;
    w.heads = p.s.by_HK(p.s.H);
    w.h = w.hk * w.heads;
    w.l = diff_lens(p.s, w.b);
    const int off = w.l.k - w.l.q;
    w.lo = p.s.causal ? max(0, -off) : 0;  // rows before see no key at all
    w.hi = w.l.q;
    int first = w.lo;
    if (p.s.causal) first = max(first, w.r0 - off);  // first row that sees key r0
    w.c_first = first / CB;
    w.tiles = (w.r0 < w.l.k && first < w.hi) ? (w.hi + CB - 1) / CB - w.c_first : 0;
  } else {
    const int bh = u - tile * (p.s.B * p.s.H);
    w.r0 = ((p.s.NQ + R - 1) / R - 1 - tile) * R;
    w.b = p.s.by_H(bh);
    w.h = bh - w.b * p.s.H;
    w.hk = p.s.by_share(w.h);
    w.heads = 1;
    w.l = diff_lens(p.s, w.b);
    w.lo = 0;
    w.hi = w.l.k;
    int keys = w.l.k;
    if (p.s.causal) keys = min(keys, min(w.r0 + R, w.l.q) + w.l.k - w.l.q);
    if (w.r0 >= w.l.q) keys = 0;
    w.c_first = 0;
    w.tiles = keys > 0 ? (keys + CB - 1) / CB : 0;
  }
  return w;
}

// The power of two by which A = P1 - lam P2 of a key unit goes into its product in
// fp16: the largest that keeps |A| <= 1 + |lam| below 2^15.  A row that spreads over
// n keys has entries of 1 / n, which no scale of dO changes: without this they
// would lose bits from n = 2^14 on and vanish at 2^25.  lam of the unit's rows is
// read from their records by the whole warp: two values a step of the unit, or one
// a head where a head's rows share it.
__device__ __forceinline__ float key_scale(const DiffBwdParams& p, const BwdUnit& w, int lane) {
  float most = 0.f;
  if (w.tiles > 0) {
    const float* r = p.rec + static_cast<size_t>(w.b * p.s.H + w.h) * p.NQpad * kDiffRec + 4 * CB;
    const size_t head = static_cast<size_t>(p.NQpad) * kDiffRec;
    if (p.lam_rows) {
      for (int g = 0; g < w.heads; ++g)
        for (int t = w.c_first; t < w.c_first + w.tiles; ++t) {
          const float* at = r + g * head + static_cast<size_t>(t) * (CB * kDiffRec) + lane;
          most = fmaxf(most, fmaxf(fabsf(at[0]), fabsf(at[32])));
        }
    } else {
      const int i = w.hi - 1;  // a row that sees a key, as all of a unit that streams any
      for (int g = lane; g < w.heads; g += 32)
        most = fmaxf(most, fabsf(r[g * head + static_cast<size_t>(i / CB) * (CB * kDiffRec) + i % CB]));
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, k));
  }
  // 2^e <= 1 + most < 2^(e + 1); the result is 2^(14 - e), but no less than 2^-6:
  // past |lam| = 2^20 entries overflow rather than that other rows' vanish
  const int e = min(static_cast<int>(__float_as_uint(1.f + most) >> 23) - 127, 20);
  return __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
}

// X1, X2 and A of one resident row and CPW streamed rows.  Per streamed row
// (KV) or for the thread's own row: rec = -LSE1 log2e, -LSE2 log2e, D1, D2, lam.
// Streamed rows i in [lo, hi] are visible (MASK only).
template <class Lay, bool MASK>
__device__ __forceinline__ void form_p(uint32_t (&s1)[CPW], uint32_t (&s2)[CPW], const float* rr,
                                       const float (&rec)[kDiffRec], float c1, float c2, int lo,
                                       int hi, int map) {
  // P1 over s1 and P2 over s2; resident keys: lam P2, and one map alone P1 or -lam P2
  const float2 C1 = make_float2(c1, c1), C2 = make_float2(c2, c2);
#pragma unroll
  for (int q = 0; q < CPW; q += 4) {
    float4 b1 = make_float4(rec[0], rec[0], rec[0], rec[0]);
    float4 b2 = make_float4(rec[1], rec[1], rec[1], rec[1]);
    float4 lm = make_float4(0.f, 0.f, 0.f, 0.f);
    if (Lay::KV) {
      if (Lay::S1) b1 = ld_shared_f4(rr + map * CB + q);
      if (Lay::S2) b2 = ld_shared_f4(rr + 1 * CB + q);
      if (Lay::S2 || (Lay::ONE && map)) lm = ld_shared_f4(rr + 4 * CB + q);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = q + 2 * e;
      const bool vx = !MASK || (i >= lo && i <= hi), vy = !MASK || (i + 1 >= lo && i + 1 <= hi);
      if (Lay::S1) {
        const float2 x = make_float2(__uint_as_float(s1[i]), __uint_as_float(s1[i + 1]));
        const float2 u = __ffma2_rn(x, C1, e ? make_float2(b1.z, b1.w) : make_float2(b1.x, b1.y));
        s1[i] = vx ? __float_as_uint(ex2(u.x)) : 0u;
        s1[i + 1] = vy ? __float_as_uint(ex2(u.y)) : 0u;
        if (Lay::KV && Lay::ONE && map) {
          s1[i] = __float_as_uint(-__uint_as_float(s1[i]) * (e ? lm.z : lm.x));
          s1[i + 1] = __float_as_uint(-__uint_as_float(s1[i + 1]) * (e ? lm.w : lm.y));
        }
      }
      if (Lay::S2) {
        const float2 x = make_float2(__uint_as_float(s2[i]), __uint_as_float(s2[i + 1]));
        const float2 u = __ffma2_rn(x, C2, e ? make_float2(b2.z, b2.w) : make_float2(b2.x, b2.y));
        float2 r = make_float2(vx ? ex2(u.x) : 0.f, vy ? ex2(u.y) : 0.f);
        if (Lay::KV) r = __fmul2_rn(r, e ? make_float2(lm.z, lm.w) : make_float2(lm.x, lm.y));
        s2[i] = __float_as_uint(r.x);
        s2[i + 1] = __float_as_uint(r.y);
      }
    }
  }
}

template <int PASS, int D, int DV, int SEL, bool F16>
__global__ void __launch_bounds__(NTHREADS, 1)
    streamkl_diff_bwd_kernel(const __grid_constant__ DiffBwdParams p) {
  using Lay = BwdLay<PASS, D, DV, SEL>;
  constexpr int NST = Lay::NST, NSV = Lay::NSV;
  constexpr bool KV = Lay::KV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* cfull = reinterpret_cast<uint64_t*>(smem + Lay::bar_off);
  uint64_t* cempty = cfull + NST;
  uint64_t* craw = cempty + NST;  // a ragged tile has landed, to be cleaned
  uint64_t* vfull = craw + NST;   // the same for the ring of G's own tiles
  uint64_t* vempty = vfull + NSV;
  uint64_t* vraw = vempty + NSV;
  uint64_t* rfull = vraw + NSV;
  uint64_t* rempty = rfull + 1;
  uint64_t* sfull = rempty + 1;  // S1, S2 of a step are in TMEM
  uint64_t* sempty = sfull + 1;  // ... and have been read
  uint64_t* gfull = sempty + 1;  // G is in TMEM
  uint64_t* xfull = gfull + 1;   // X1, X2, A are written (and G has been read)
  uint64_t* xempty = xfull + 1;  // ... and have been contracted
  uint64_t* ofull = xempty + 1;
  uint64_t* oempty = ofull + 1;
  uint64_t* drain = oempty + 1;  // [2]: the issuers' own products are done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::misc_off + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
  // The next pass may start on multiprocessors that this one leaves idle.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < NST; ++s) {
      mbar_init(&cfull[s], 1);
      mbar_init(&cempty[s], 1);
      mbar_init(&craw[s], 1);
    }
    for (int s = 0; s < NSV; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
      mbar_init(&vraw[s], 1);
    }
    mbar_init(rfull, 1);
    mbar_init(rempty, 1);
    mbar_init(sfull, 1);
    mbar_init(sempty, 4 * NWG);
    mbar_init(gfull, 1);
    mbar_init(xfull, 4 * NWG);
    mbar_init(xempty, 1);
    mbar_init(ofull, 1);
    mbar_init(oempty, 4 * NWG);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    fence_mbar_init();
    if (Lay::S1) tma_prefetch_desc(&p.tmR1);
    if (Lay::S2 || Lay::ONE) tma_prefetch_desc(&p.tmR2);
    if (Lay::WG) tma_prefetch_desc(&p.tmR3);
    if (Lay::S1) tma_prefetch_desc(&p.tmC1);
    if (Lay::S2 || Lay::ONE) tma_prefetch_desc(&p.tmC2);
    tma_prefetch_desc(&p.tmC3);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  uint8_t* r1_s = smem;
  uint8_t* r2_s = r1_s + Lay::r1;
  uint8_t* r3_s = r2_s + Lay::r2;
  uint8_t* a_s = smem + Lay::a_off;
  auto c1_s = [&](int s) { return smem + Lay::c_off + s * Lay::stage; };
  auto c2_s = [&](int s) { return c1_s(s) + Lay::c1; };
  auto c3_s = [&](int s) {  // s counts the ring that holds it
    return Lay::CR3 ? c1_s(s) + Lay::c1 + Lay::c2 : smem + Lay::v_off + s * Lay::c3;
  };
  auto rec_s = [&](int s) { return reinterpret_cast<float*>(smem + Lay::rec_off + s * Lay::rec); };
  const int nrows = KV ? p.s.NK : p.s.NQ;    // resident extent
  const int nstream = KV ? p.s.NQ : p.s.NK;  // streamed extent
  SnakeSched sched(p.s.B * (KV ? p.s.HK : p.s.H) * ((nrows + R - 1) / R) * p.nhalf);
  int u;

  // Of the launch's 96 registers x 640 threads the first warpgroup hands over
  // what it does not need (128 x 64 + 512 x 104 = 640 x 96).
  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ------------------------------------------------------------ compute
    const int part = (warp - 4) >> 2;  // streamed rows [part*CPW, part*CPW + CPW) of each step
    const int quarter = warp & 3;
    const int j = quarter * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int cs = 0, gt = 0;  // gt: steps so far
    uint32_t cph = 0, sph = 0, gph = 0, xph = 0, oph = 0;
    bool ok = true;
    while (ok && sched.next(u)) {
      const BwdUnit w = decode<PASS>(p, u);
      const int mine = w.r0 + j;  // key (kKV) or query (kQ)
      const int map = Lay::ONE ? p.map0 + w.half : 0;
      const int off = w.l.k - w.l.q;
      float rec[kDiffRec] = {-INFINITY, -INFINITY, 0.f, 0.f, 0.f};
      if (!KV && mine < w.l.q && w.tiles) {
        const float* r = p.rec + (static_cast<size_t>(w.b * p.s.H + w.h) * p.NQpad + (mine / CB) * CB) *
                                     kDiffRec + (mine % CB);
#pragma unroll
        for (int f = 0; f < kDiffRec; ++f) rec[f] = r[f * CB];
        if (Lay::ONE && map) {
          rec[0] = rec[1];
          rec[2] = rec[3];
        }
      }
      // kQ: X_t = P_t (f_t G + fd_t), f_1 = 1 and f_2 = -lam, fd_t = -f_t D_t
      const float f1 = Lay::ONE && map ? -rec[4] : 1.f, fd1 = -f1 * rec[2];
      const float f2 = -rec[4], fd2 = -f2 * rec[3];
      const float ascale = Lay::WV && F16 ? key_scale(p, w, lane) : 1.f;
      float2 d2sum = make_float2(0.f, 0.f);
      const int steps = w.heads * w.tiles;
      int tile = 0;
      for (int t = 0; t < steps; ++t) {
        const int c0 = (w.c_first + tile) * CB;
        const int cc = c0 + part * CPW;
        if (++tile == w.tiles) tile = 0;
        if (KV && !(ok = mbar_wait(&cfull[cs], cph, ctl))) break;  // the step's records
        if (!(ok = mbar_wait(sfull, sph, ctl))) break;
        sph ^= 1;
        tc_fence_after();
        uint32_t a[CPW], b[CPW], g[CPW];
        if (Lay::S1) tmem_ld_32x32b_x16(tl + part * CPW, a);
        if (Lay::S2) tmem_ld_32x32b_x16(tl + kColS2 + part * CPW, b);
        tmem_ld_wait();
        if (Lay::S1) reg_fence(a);
        if (Lay::S2) reg_fence(b);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty);
        // visible streamed rows lo..hi; rows that see nothing have P = 0 from their record
        int lo = -kNever, hi = kNever;
        bool masked;
        if (KV) {
          masked = p.s.causal && c0 + off < w.r0 + R - 1;
          if (p.s.causal) lo = mine - off - cc;
        } else {
          masked = c0 + CB > w.l.k || (p.s.causal && c0 + CB - 1 > w.r0 + off);
          hi = w.l.k - 1 - cc;
          if (p.s.causal) hi = min(hi, mine + off - cc);
        }
        const float* rr = KV ? rec_s(cs) + part * CPW : nullptr;
        if (masked)
          form_p<Lay, true>(a, b, rr, rec, map ? p.c2 : p.c1, p.c2, lo, hi, map);
        else
          form_p<Lay, false>(a, b, rr, rec, map ? p.c2 : p.c1, p.c2, lo, hi, map);
        const float2 NEG = make_float2(-1.f, -1.f);
        uint32_t w1[CPW / 2], w2[CPW / 2], w3[CPW / 2];
        auto pair = [](const uint32_t (&v)[CPW], int i) {
          return make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
        };
        if (Lay::WV) {
#pragma unroll
          for (int i = 0; i < CPW; i += 2) {
            float2 x = __ffma2_rn(pair(b, i), NEG, pair(a, i));
            if (F16) x = __fmul2_rn(x, make_float2(ascale, ascale));
            w3[i / 2] = pack2<F16>(x.x, x.y);
          }
        }
        if (Lay::AS) {
          // Row j, 16-byte pieces 2 part and 2 part + 1 of its 128 bytes.  The buffer
          // was contracted two steps ago, which the last wait on xempty covered.
          uint4* arow = reinterpret_cast<uint4*>(a_s + (gt & 1) * (R * CB * 2) + j * 128);
          arow[(2 * part) ^ (j & 7)] = make_uint4(w3[0], w3[1], w3[2], w3[3]);
          arow[(2 * part + 1) ^ (j & 7)] = make_uint4(w3[4], w3[5], w3[6], w3[7]);
          fence_proxy_async_smem();
        }
        if (Lay::WG) {
          if (!(ok = mbar_wait(gfull, gph, ctl))) break;
          gph ^= 1;
          tc_fence_after();
          tmem_ld_32x32b_x16(tl + kColG + part * CPW, g);
          tmem_ld_wait();
          reg_fence(g);
        }
#pragma unroll
        for (int q = 0; q < CPW; q += 4) {
          float4 d1 = make_float4(rec[2], rec[2], rec[2], rec[2]);
          float4 d2 = make_float4(rec[3], rec[3], rec[3], rec[3]);
          if (KV && Lay::X1) d1 = ld_shared_f4(rr + (2 + map) * CB + q);
          if (KV && Lay::X2) d2 = ld_shared_f4(rr + 3 * CB + q);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = q + 2 * e;
            if (Lay::X1) {
              const float2 d = e ? make_float2(d1.z, d1.w) : make_float2(d1.x, d1.y);
              const float2 y = KV ? __ffma2_rn(d, NEG, pair(g, i))
                                  : __ffma2_rn(pair(g, i), make_float2(f1, f1), make_float2(fd1, fd1));
              const float2 x = __fmul2_rn(pair(a, i), y);
              w1[i / 2] = pack2<F16>(x.x, x.y);
              if (!KV && Lay::ONE) d2sum = __ffma2_rn(pair(a, i), pair(g, i), d2sum);
            }
            if (Lay::X2) {
              const float2 d = e ? make_float2(d2.z, d2.w) : make_float2(d2.x, d2.y);
              const float2 y = KV ? __ffma2_rn(pair(g, i), NEG, d)
                                  : __ffma2_rn(pair(g, i), make_float2(f2, f2), make_float2(fd2, fd2));
              const float2 x = __fmul2_rn(pair(b, i), y);
              w2[i / 2] = pack2<F16>(x.x, x.y);
              if (!KV) d2sum = __ffma2_rn(pair(b, i), pair(g, i), d2sum);
            }
          }
        }
        if (!(ok = mbar_wait(xempty, xph ^ 1, ctl))) break;
        xph ^= 1;
        tc_fence_after();
        if (Lay::X1) tmem_st_32x32b_x8(tl + kColX1 + part * (CPW / 2), w1);
        if (Lay::X2) tmem_st_32x32b_x8(tl + kColX2 + part * (CPW / 2), w2);
        if (Lay::WV && !Lay::AS) tmem_st_32x32b_x8(tl + kColX1 + part * (CPW / 2), w3);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(xfull);
        ++gt;
        if (++cs == NST) {
          cs = 0;
          cph ^= 1;
        }
      }
      if (!ok) break;
      // Unit epilogue: this warpgroup writes a quarter of each output's columns.
      if (steps > 0) {
        if (!(ok = mbar_wait(ofull, oph, ctl))) break;
        oph ^= 1;
        tc_fence_after();
      }
      // Decoded again, from values that the compiler takes as new: what only the
      // epilogue needs is then not held in registers through the steps.
      int eu = u, ej = j, ep = part;
      asm volatile("" : "+r"(eu), "+r"(ej), "+r"(ep));
      const BwdUnit e = decode<PASS>(p, eu);
      const int row = e.r0 + ej;
      const bool in_tensor = row < nrows;
      // rows behind their sequence, and rows that see nothing, get exact zeros
      const bool live = steps > 0 && row < (KV ? e.l.k : e.l.q) &&
                        (KV || !p.s.causal || row + e.l.k - e.l.q >= 0);
      if (!KV && p.d2 && (!Lay::ONE || p.map0 + e.half == 1)) {
        float v = live ? d2sum.x + d2sum.y : 0.f;
        const int nrt = (p.s.NQ + R - 1) / R, rt = e.r0 / R;
        const size_t bh = static_cast<size_t>(e.b) * p.s.H + e.h;
        if (p.d2_rows) {
          p.d2[(static_cast<size_t>(ep) * p.s.B * p.s.H + bh) * (nrt * static_cast<size_t>(R)) + row] = v;
        } else {
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
          if (lane == 0) p.d2[(bh * nrt + rt) * 16 + ep * 4 + quarter] = v;
        }
      }
      const int h = KV ? e.hk : e.h;
      // one output after the other, 16 columns at a time: a loop, so that its
      // values do not take registers from the steps
#pragma unroll 1
      for (int o = 0; o < 3; ++o) {
        const bool made = Lay::ONE ? o == p.map0 + e.half : o == 0 ? Lay::X1 : o == 1 ? Lay::X2 : Lay::WV;
        void* base = o == 0 ? p.out1 : o == 1 ? p.out2 : p.out3;
        if (!made || !base) continue;
        const Strides& st = o == 0 ? p.so1 : o == 1 ? p.so2 : p.so3;
        const int cols = (o < 2 ? D : DV) / NWG, first = (o < 2 ? 0 : e.half * DV) + ep * cols;
        const uint32_t col = (Lay::ONE || o == 0 ? Lay::o1 : o == 1 ? Lay::o2 : Lay::o3) + ep * cols;
        const float f = o == 0 ? p.s1 : o == 1 ? p.s2 : 1.f / ascale;
        uint16_t* dst = static_cast<uint16_t*>(base) + e.b * st.b + h * st.h + row * st.n + first;
#pragma unroll 1
        for (int c = 0; c < cols; c += 16) {
          uint32_t v[16] = {};
          if (steps > 0) {
            tmem_ld_32x32b_x16(tl + col + c, v);
            tmem_ld_wait();
            reg_fence(v);
          }
          uint32_t x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            x[k] = live ? pack2<F16>(__uint_as_float(v[2 * k]) * f, __uint_as_float(v[2 * k + 1]) * f) : 0u;
          if (in_tensor) {
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(x[4], x[5], x[6], x[7]);
          }
        }
      }
      if (steps > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(oempty);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        int cs = 0, vs = 0;
        uint32_t rph = 0, cph = 0, vph = 0, rawph = 0, vrawph = 0;  // bit s of rawph: parity of craw[s]
        uint32_t armed_r = 0, armed_c[NST] = {}, armed_v[NSV + 1] = {};  // last armed phase + 1; + 2 on raw
        bool ok = true;
        while (ok && sched.next(u)) {
          const BwdUnit w = decode<PASS>(p, u);
          if (w.tiles == 0) continue;
          if (!(ok = mbar_wait(rempty, rph ^ 1, ctl))) break;
          mbar_arrive_expect_tx(rfull, Lay::r1 + Lay::r2 + Lay::r3);
          const int rh = KV ? w.hk : w.h;
          const int map = Lay::ONE ? p.map0 + w.half : 0;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            if (Lay::S1)
              tma_load_4d(r1_s + c * (R * 128), map ? &p.tmR2 : &p.tmR1, rfull, c * 64, w.r0, rh, w.b);
            if (Lay::S2) tma_load_4d(r2_s + c * (R * 128), &p.tmR2, rfull, c * 64, w.r0, rh, w.b);
          }
          if (Lay::WG) {
            // V is read per key head, dO per query head
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
              tma_load_4d(r3_s + c * (R * 128), &p.tmR3, rfull, c * 64, w.r0, rh, w.b);
          }
          armed_r = rph + 1;
          rph ^= 1;
          for (int g = 0; g < w.heads && ok; ++g) {
            const int ch = KV ? w.h + g : w.hk;
            for (int t = 0; t < w.tiles; ++t) {
              const int c0 = (w.c_first + t) * CB;
              if (!(ok = mbar_wait(&cempty[cs], cph ^ 1, ctl))) break;
              // a ragged tile lands on craw; warp 2 cleans it and completes cfull
              const bool ragged = w.ragged(t, nstream);
              uint64_t* bar = ragged ? &craw[cs] : &cfull[cs];
              mbar_arrive_expect_tx(bar, Lay::load_bytes);
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                if (Lay::S1)
                  tma_load_4d(c1_s(cs) + c * (CB * 128), map ? &p.tmC2 : &p.tmC1, bar, c * 64, c0, ch, w.b);
                if (Lay::S2) tma_load_4d(c2_s(cs) + c * (CB * 128), &p.tmC2, bar, c * 64, c0, ch, w.b);
              }
              auto load3 = [&](int slot, uint64_t* on) {
#pragma unroll
                for (int c = 0; c < DV / 64; ++c)
                  tma_load_4d(c3_s(slot) + c * (CB * 128), &p.tmC3, on, (Lay::ONE ? 0 : w.half) * DV + c * 64, c0, ch,
                              w.b);
              };
              if (Lay::CR3) load3(cs, bar);
              if (KV)
                bulk_load(rec_s(cs),
                          p.rec + (static_cast<size_t>(w.b * p.s.H + ch) * p.NQpad + c0) * kDiffRec,
                          Lay::rec, bar);
              armed_c[cs] = ragged ? 3 + ((rawph >> cs) & 1u) : cph + 1;
              if (ragged) rawph ^= 1u << cs;
              if (++cs == NST) {
                cs = 0;
                cph ^= 1;
              }
              if (!Lay::CR3) {
                if (!(ok = mbar_wait(&vempty[vs], vph ^ 1, ctl))) break;
                uint64_t* von = ragged ? &vraw[vs] : &vfull[vs];
                mbar_arrive_expect_tx(von, Lay::c3);
                load3(vs, von);
                armed_v[vs] = ragged ? 3 + ((vrawph >> vs) & 1u) : vph + 1;
                if (ragged) vrawph ^= 1u << vs;
                if (++vs == NSV) {
                  vs = 0;
                  vph ^= 1;
                }
              }
            }
          }
        }
        if (!ok) {
          // Aborting: let the copies already in flight land before the CTA exits.
          volatile int zero = 0;
          WaitCtl dctl{&zero, p.status, p.wait_limit_ns};
          if (armed_r) mbar_wait(rfull, armed_r - 1, dctl);
          for (int s = 0; s < NST; ++s)
            if (armed_c[s])
              mbar_wait(armed_c[s] > 2 ? &craw[s] : &cfull[s], (armed_c[s] - 1) & 1u, dctl);
          for (int s = 0; s < NSV; ++s)
            if (armed_v[s])
              mbar_wait(armed_v[s] > 2 ? &vraw[s] : &vfull[s], (armed_v[s] - 1) & 1u, dctl);
        }
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------ issuer of S and G
      if (lane == 0) {
        constexpr uint32_t idS = idesc_16<F16>(R, CB);
        const uint64_t r1d = sdesc_sw128(smem_u32(r1_s), 16, 1024);
        const uint64_t r2d = sdesc_sw128(smem_u32(r2_s), 16, 1024);
        const uint64_t r3d = sdesc_sw128(smem_u32(r3_s), 16, 1024);
        int cn = 0, cg = 0;  // stages of the next S, and of the next G's streamed tile
        uint32_t rph = 0, cph = 0, vph = 0, seph = 0, xph = 0;
        bool ok = true, first_s = true, first_g = true;  // of the whole run: nothing was read before
        auto product = [&](uint32_t col, uint64_t resident, uint8_t* tile, int width) {
          const uint64_t rd = here(resident);
          const uint64_t cd = sdesc_sw128(smem_u32(tile), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < width / 16; ++kk)
            umma_bf16_ss(tmem + col, sdesc_advance(rd, (kk >> 2) * (R * 128) + (kk & 3) * 32),
                         sdesc_advance(cd, (kk >> 2) * (CB * 128) + (kk & 3) * 32), idS, kk > 0);
        };
        // S, once its tiles are there and the warps have read the S before
        auto issue_s = [&]() -> bool {
          if (!mbar_wait(&cfull[cn], cph, ctl)) return false;
          if (!first_s) {
            if (!mbar_wait(sempty, seph, ctl)) return false;
            seph ^= 1;
          }
          first_s = false;
          tc_fence_after();
          if (Lay::S1) product(0, r1d, c1_s(cn), D);
          if (Lay::S2) product(kColS2, r2d, c2_s(cn), D);
          umma_commit(sfull);
          if (++cn == NST) {
            cn = 0;
            cph ^= 1;
          }
          return true;
        };
        // G, once the warps have read the G before (xfull says that too)
        auto issue_g = [&]() -> bool {
          if (!first_g) {
            if (!mbar_wait(xfull, xph, ctl)) return false;
            xph ^= 1;
          }
          first_g = false;
          if (!Lay::CR3 && !mbar_wait(&vfull[cg], vph, ctl)) return false;
          tc_fence_after();
          product(kColG, r3d, c3_s(cg), DV);
          umma_commit(gfull);
          if (!Lay::CR3) umma_commit(&vempty[cg]);
          if (++cg == (Lay::CR3 ? NST : NSV)) {
            cg = 0;
            vph ^= 1;
          }
          return true;
        };
        while (ok && sched.next(u)) {
          const BwdUnit w = decode<PASS>(p, u);
          if (w.tiles == 0) continue;
          if (!(ok = mbar_wait(rfull, rph, ctl))) break;
          rph ^= 1;
          const int steps = w.heads * w.tiles;
          if (!(ok = issue_s())) break;
          for (int t = 0; t < steps; ++t) {
            if (Lay::WG) {
              ok = issue_g();
              if (!ok) break;
            }
            if (t + 1 < steps) {
              ok = issue_s();
              if (!ok) break;
            }
          }
          if (!ok) break;
          umma_commit(rempty);
        }
        umma_commit(&drain[1]);
        volatile int zero = 0;
        WaitCtl dctl{&zero, p.status, p.wait_limit_ns};
        mbar_wait(&drain[1], 0, dctl);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ issuer of the output products
      if (lane == 0) {
        constexpr uint32_t idD = idesc_16<F16>(R, D, 0, 1);  // B = C, features contiguous
        constexpr uint32_t idV = idesc_16<F16>(R, DV, 0, 1);
        const uint64_t ad = sdesc_sw128(smem_u32(a_s), 16, 1024);
        int cs = 0, gt = 0;  // stage, and steps so far: A alternates between two buffers
        uint32_t xph = 0, oph = 0;
        bool ok = true;
        while (ok && sched.next(u)) {
          const BwdUnit w = decode<PASS>(p, u);
          if (w.tiles == 0) continue;
          const int steps = w.heads * w.tiles;
          for (int t = 0; t < steps; ++t) {
            if (!(ok = mbar_wait(xfull, xph, ctl))) break;
            xph ^= 1;
            if (t == 0) {
              if (!(ok = mbar_wait(oempty, oph ^ 1, ctl))) break;
              oph ^= 1;
            }
            tc_fence_after();
            const uint64_t c1m = sdesc_sw128(smem_u32(c1_s(cs)), CB * 128, 1024);
            const uint64_t c2m = sdesc_sw128(smem_u32(c2_s(cs)), CB * 128, 1024);
            const uint64_t c3m = sdesc_sw128(smem_u32(c3_s(Lay::CR3 ? cs : 0)), CB * 128, 1024);
            const uint64_t a_d = sdesc_advance(here(ad), (gt & 1) * (R * CB * 2));
#pragma unroll
            for (int kk = 0; kk < CB / 16; ++kk) {
              const uint32_t acc = t > 0 || kk > 0;
              if (Lay::X1)
                umma_bf16_ts(tmem + Lay::o1, tmem + kColX1 + kk * 8, sdesc_advance(c1m, kk * 2048), idD, acc);
              if (Lay::X2)
                umma_bf16_ts(tmem + Lay::o2, tmem + kColX2 + kk * 8, sdesc_advance(c2m, kk * 2048), idD, acc);
              if (Lay::AS)
                umma_bf16_ss(tmem + Lay::o3, sdesc_advance(a_d, kk * 32), sdesc_advance(c3m, kk * 2048), idV, acc);
              else if (Lay::WV)
                umma_bf16_ts(tmem + Lay::o3, tmem + kColX1 + kk * 8, sdesc_advance(c3m, kk * 2048), idV, acc);
            }
            // S and G of this step were complete before X was formed from them, so
            // this commit also says that nothing reads the stage any more
            umma_commit(&cempty[cs]);
            umma_commit(xempty);
            ++gt;
            if (++cs == NST) cs = 0;
          }
          if (!ok) break;
          umma_commit(ofull);
        }
        umma_commit(&drain[0]);
        volatile int zero = 0;
        WaitCtl dctl{&zero, p.status, p.wait_limit_ns};
        mbar_wait(&drain[0], 0, dctl);
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ ragged tiles
      int item = 0;  // ring items before this head of this unit
      uint32_t rawph = 0, vrawph = 0;
      bool ok = true;
      while (ok && sched.next(u)) {
        const BwdUnit w = decode<PASS>(p, u);
        for (int g = 0; g < (w.tiles ? w.heads : 0) && ok; ++g, item += w.tiles) {
          // only the first and the last tile can be ragged
          for (int e = 0; e < (w.tiles > 1 ? 2 : 1); ++e) {
            const int t = e ? w.tiles - 1 : 0;
            if (!w.ragged(t, nstream)) continue;
            const int s = static_cast<int>((static_cast<unsigned>(item) + t) % NST), c0 = (w.c_first + t) * CB;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait_long(&craw[s], (rawph >> s) & 1u, ctl)))) break;
            rawph ^= 1u << s;
            const int lo = max(0, w.lo - c0), hi = min(CB, max(0, w.hi - c0));
            auto clean = [&](uint8_t* tile, int chunks) {
              if (lo > 0) zero_tile_rows(tile, chunks, CB, 0, lo, lane);
              if (hi < CB) zero_tile_rows(tile, chunks, CB, hi, CB, lane);
            };
            if (Lay::S1) clean(c1_s(s), D / 64);
            if (Lay::S2) clean(c2_s(s), D / 64);
            if (Lay::CR3) clean(c3_s(s), DV / 64);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cfull[s]);
            if (!Lay::CR3) {
              const int v = static_cast<int>((static_cast<unsigned>(item) + t) % (NSV + Lay::CR3));
              if (!(ok = __all_sync(0xffffffffu, mbar_wait_long(&vraw[v], (vrawph >> v) & 1u, ctl)))) break;
              vrawph ^= 1u << v;
              clean(c3_s(v), DV / 64);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&vfull[v]);
            }
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // A pass that started early ends only when the one before has ended, so that
  // what follows on the stream finds them all done.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int PASS, int D, int DV, int SEL, bool F16>
cudaError_t launch_t(const DiffBwdParams& p, int num_sms, cudaStream_t stream) {
  using Lay = BwdLay<PASS, D, DV, SEL>;
  auto kern = streamkl_diff_bwd_kernel<PASS, D, DV, SEL, F16>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, Lay::alloc, ready);
  if (e != cudaSuccess) return e;
  const int nrows = PASS == kDiffKV ? p.s.NK : p.s.NQ;
  const int units = p.s.B * (PASS == kDiffKV ? p.s.HK : p.s.H) * ((nrows + R - 1) / R) * p.nhalf;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units < num_sms ? units : num_sms);
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = Lay::alloc;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = p.after_pass ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool F16>
cudaError_t launch_type(const DiffBwdParams& p, DiffPass pass, int d, int dv, int sel, int num_sms,
                        cudaStream_t stream) {
  if (pass == kDiffKV) {
    if (d == 64 && dv == 64 && sel == 7) return launch_t<kDiffKV, 64, 64, 7, F16>(p, num_sms, stream);
    if (d == 64 && dv == 128 && sel == 7) return launch_t<kDiffKV, 64, 128, 7, F16>(p, num_sms, stream);
    if (d == 128 && dv == 128 && sel == 3) return launch_t<kDiffKV, 128, 128, 3, F16>(p, num_sms, stream);
    if (d == 128 && dv == 256 && sel == 1) return launch_t<kDiffKV, 128, 256, 1, F16>(p, num_sms, stream);
    if (d == 128 && sel == 4) return launch_t<kDiffKV, 128, 128, 4, F16>(p, num_sms, stream);
  } else {
    if (d == 64 && dv == 64 && sel == 3) return launch_t<kDiffQ, 64, 64, 3, F16>(p, num_sms, stream);
    if (d == 64 && dv == 128 && sel == 3) return launch_t<kDiffQ, 64, 128, 3, F16>(p, num_sms, stream);
    if (d == 128 && dv == 128 && sel == 3) return launch_t<kDiffQ, 128, 128, 3, F16>(p, num_sms, stream);
    if (d == 128 && dv == 256 && sel == 1) return launch_t<kDiffQ, 128, 256, 1, F16>(p, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

// Row records: D2 = <dO, O2>, D1 = <dO, O> + lam D2 (O = O1 - lam O2).  A block
// takes 64 rows, DV / 8 lanes a row; bound by HBM (or L2, behind the forward).
template <int DV, bool F16>
__global__ void __launch_bounds__(256, 4) streamkl_diff_prep_kernel(const DiffPrepParams p) {
  constexpr int L = DV / 8, RPT = CB * L / 256;  // lanes a row, rows a thread
  __shared__ float out[4][CB];  // [2] <dO, O>, [3] <dO, O2>
  const int steps = p.NQpad / CB, u = blockIdx.x;
  const int bh = u / steps, i0 = (u - bh * steps) * CB;
  const int b = bh / p.s.H, h = bh - b * p.s.H;
  const Lens l = diff_lens(p.s, b);
  auto sees = [&](int i) { return i < l.q && l.k > 0 && (!p.s.causal || i + l.k - l.q >= 0); };
  // what needs one thread a row is on its way first
  float n1 = -INFINITY, n2 = -INFINITY, lam = 0.f;
  if (threadIdx.x < CB && sees(i0 + threadIdx.x)) {
    const long long v = static_cast<long long>(bh) * p.s.NQ + i0 + threadIdx.x;
    // LSE = -inf: all visible scores are, and the map has no weights (as in the forward)
    const float l1 = p.LSE1[v], l2 = p.LSE2[v];
    n1 = l1 == -INFINITY ? l1 : -l1 * kLog2e;
    n2 = l2 == -INFINITY ? l2 : -l2 * kLog2e;
    lam = load_lam(p.lam, b, h, i0 + threadIdx.x, F16);
  }
  const int sub = threadIdx.x % L, r0 = threadIdx.x / L;
#pragma unroll
  for (int k = 0; k < RPT; ++k) {
    const int row = r0 + k * (256 / L), i = i0 + row;
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x, z = x;
    if (sees(i)) {
      const long long oo = b * p.so.b + h * p.so.h + i * p.so.n + sub * 8;
      x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dO) + b * p.sdo.b + h * p.sdo.h +
                                          i * p.sdo.n + sub * 8);
      y = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.O) + oo);
      z = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.O2) + oo);
    }
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
    float d = 0.f, d2 = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = unpack2<F16>(xs[e]), o = unpack2<F16>(ys[e]), o2 = unpack2<F16>(zs[e]);
      d = fmaf(a.x, o.x, fmaf(a.y, o.y, d));
      d2 = fmaf(a.x, o2.x, fmaf(a.y, o2.y, d2));
    }
#pragma unroll
    for (int s = L / 2; s > 0; s >>= 1) {
      d += __shfl_xor_sync(0xffffffffu, d, s);
      d2 += __shfl_xor_sync(0xffffffffu, d2, s);
    }
    if (sub == 0) {
      out[2][row] = d;
      out[3][row] = d2;
    }
  }
  __syncthreads();
  if (threadIdx.x < CB) {
    const int row = threadIdx.x;
    float* dst = p.rec + static_cast<long long>(u) * (CB * kDiffRec) + row;
    dst[0 * CB] = n1;
    dst[1 * CB] = n2;
    dst[2 * CB] = fmaf(lam, out[3][row], out[2][row]);
    dst[3 * CB] = out[3][row];
    dst[4 * CB] = lam;
  }
}

template <class P>
__device__ __forceinline__ void store_lam(const P& p, long long e, float v) {
  if (p.f32) static_cast<float*>(p.out)[e] = v;
  else if (p.f16) static_cast<__half*>(p.out)[e] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p.out)[e] = __float2bfloat16_rn(v);
}

// One block per element of dlam that sums whole rows' axes (en = 1): each thread a
// strided share in order, then a tree: the same sum every time.
__global__ void __launch_bounds__(256) streamkl_diff_lam_kernel(const DiffLamParams p) {
  __shared__ float part[8];
  const int e = blockIdx.x;
  const int h0 = e % p.eh, b0 = e / p.eh;
  const int nb = p.eb == 1 ? p.B : 1, nh = p.eh == 1 ? p.H : 1;
  const int n = (p.NQ + R - 1) / R * 16;
  float s = 0.f;
  for (int q = 0; q < nb * nh; ++q) {
    const float* d = p.d2 + (static_cast<size_t>(b0 + q / nh) * p.H + h0 + q % nh) * n;
    for (int k = threadIdx.x; k < n; k += blockDim.x) s += d[k];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
    for (int k = 0; k < 8; ++k) s += part[k];
    store_lam(p, e, -s);
  }
}

// dlam with an element per row (en = NQ), one thread each.
__global__ void __launch_bounds__(256) streamkl_diff_lam_rows_kernel(const DiffLamParams p) {
  const long long total = static_cast<long long>(p.eb) * p.eh * p.NQ;
  const size_t pad = static_cast<size_t>((p.NQ + R - 1) / R) * R, BH = static_cast<size_t>(p.B) * p.H;
  const int nb = p.eb == 1 ? p.B : 1, nh = p.eh == 1 ? p.H : 1;
  for (long long e = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; e < total;
       e += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int i = static_cast<int>(e % p.NQ), h0 = static_cast<int>(e / p.NQ % p.eh),
              b0 = static_cast<int>(e / p.NQ / p.eh);
    float s = 0.f;
    for (int q = 0; q < nb * nh; ++q) {
      const float* d = p.d2 + (static_cast<size_t>(b0 + q / nh) * p.H + h0 + q % nh) * pad + i;
      s += (d[0] + d[BH * pad]) + (d[2 * BH * pad] + d[3 * BH * pad]);
    }
    store_lam(p, e, -s);
  }
}

}  // namespace

cudaError_t launch_diff_bwd(const DiffBwdParams& p, DiffPass pass, int d, int dv, int sel, bool f16,
                            int num_sms, cudaStream_t stream) {
  return f16 ? launch_type<true>(p, pass, d, dv, sel, num_sms, stream)
             : launch_type<false>(p, pass, d, dv, sel, num_sms, stream);
}

cudaError_t launch_diff_prep(const DiffPrepParams& p, cudaStream_t stream) {
  const int grid = p.s.B * p.s.H * (p.NQpad / CB);
  auto run = [&](auto f16) {
    constexpr bool F16 = decltype(f16)::value;
    if (p.dv == 64) streamkl_diff_prep_kernel<64, F16><<<grid, 256, 0, stream>>>(p);
    else if (p.dv == 128) streamkl_diff_prep_kernel<128, F16><<<grid, 256, 0, stream>>>(p);
    else streamkl_diff_prep_kernel<256, F16><<<grid, 256, 0, stream>>>(p);
  };
  if (p.f16) run(std::true_type{});
  else run(std::false_type{});
  return cudaGetLastError();
}

cudaError_t launch_diff_lam(const DiffLamParams& p, cudaStream_t stream) {
  const long long n = static_cast<long long>(p.eb) * p.eh * p.en;
  if (p.en > 1 || p.NQ == 1) {
    const long long blocks = (n + 255) / 256;
    streamkl_diff_lam_rows_kernel<<<static_cast<int>(blocks < 2048 ? blocks : 2048), 256, 0, stream>>>(p);
  } else {
    streamkl_diff_lam_kernel<<<static_cast<unsigned>(n), 256, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace skl
