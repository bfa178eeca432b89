// diff_fwd_sm100.cu -- differential attention forward for sm_100a.
//
//   O = (softmax(s1 Q1 K1^T) - lam softmax(s2 Q2 K2^T)) V
//
// over the visible keys of each row, in one pass over the keys: each map keeps
// a running reference m_t, a sum l_t and its own output O_t = sum_j p_tj V_j
// with p_tj = 2^(c_t x_tj - m_t); the end forms O_1/l_1 - lam O_2/l_2.  The two
// outputs stay apart because their references move independently.
//
// What bounds it: per visible pair 2 exponentials and 4d + 4dv FLOP.  At 16
// exponentials and 8192 FLOP per clock and SM, d = 64 with dv = 128 is bound by
// the exponentials (0.125 against 0.094 clocks a pair), d = dv = 128 by both
// alike (0.125 against 0.125).
//
// One CTA per SM, persistent; a unit is (batch, head, 128 query rows, 128 value
// columns):
//   warp 0       TMA producer: Q1/Q2 once a unit, keys and values through a
//                ring of 32 KB slots (d = 64: K1 and K2 share a slot)
//   warp 1       TMEM owner and UMMA issuer
//   warp 2       sets value rows behind a sequence's end to zero, so that what
//                the padding holds (NaN too) meets a weight of 0 as 0
//   warps 4..11  two softmax warpgroups, one per map, thread = row = TMEM lane
// TMEM: S1 [0,128) S2 [128,256) O1 [256,384) O2 [384,512).  P_t replaces S_t
// in 16 bits (columns [0,64) of the slot) and is the A operand of the value
// product.  The issuer's order is PV_1(j) S_1(j+1) PV_2(j) S_2(j+1): while one
// map's warps take exponentials, the tensor pipe works for the other map.
// P is rounded to 16 bits for the product, as any 16-bit tensor-core product
// needs; l_t sums the unrounded values.
//
// O_t is rescaled only when a row's largest score has risen by more than the
// slack of its type (see WeightRef): p then stays inside the type, and most tiles
// skip the round trip of O through registers.
#include "diff_sm100.cuh"

#include <type_traits>

namespace skl {
namespace {

constexpr int R = kDiffRows;
constexpr int BK = 128;
constexpr int NTHREADS = 12 * 32;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kColO = 256;

template <int D>
struct FwdLay {
  static constexpr int q_bytes = R * D * 2;
  static constexpr int slot_bytes = 32768;
  static constexpr int NS = D == 64 ? 6 : 5;
  static constexpr int KITEMS = D == 64 ? 1 : 2;  // ring items holding a tile's keys
  static constexpr int ITEMS = KITEMS + 1;
  static constexpr int q_off = 0;
  static constexpr int ring_off = 2 * q_bytes;
  static constexpr int inv_off = ring_off + NS * slot_bytes;  // [2][R] fp32
  static constexpr int bar_off = inv_off + 2 * R * 4;
  // full[NS] empty[NS] raw[NS] qfull qempty sfull[2] pfull[2][2] ofull oempty ifull drain
  static constexpr int nbar = 3 * NS + 12;
  static constexpr int misc_off = bar_off + nbar * 8;
  static constexpr int alloc = misc_off + 16 + 1024;
  static_assert(alloc <= 232448, "shared memory budget exceeded");
};

struct FwdUnit {
  int b, h, hk, half, q0, nkt, qlen, klen;
  bool ragged;  // the last tile reaches rows behind klen that are not beyond the tensor
};

__device__ __forceinline__ FwdUnit decode(const DiffFwdParams& p, int u) {
  FwdUnit w;
  const int nqt = (p.s.NQ + R - 1) / R;
  // Heads in groups: within a group the query tiles that see the most keys
  // first, heads innermost, the value halves of a tile next to each other.
  const int gs = p.head_group;
  const int g = p.by_group_units(u);
  int r = u - g * (gs * nqt * p.nhalf);
  w.half = r & (p.nhalf - 1);
  r >>= p.nhalf - 1;
  const int tile = p.by_group(r), bh = g * gs + r - tile * gs;
  w.q0 = (nqt - 1 - tile) * R;
  w.b = p.s.by_H(bh);
  w.h = bh - w.b * p.s.H;
  w.hk = p.s.by_share(w.h);
  const Lens l = diff_lens(p.s, w.b);
  w.qlen = l.q;
  w.klen = l.k;
  int keys = l.k;
  if (p.s.causal) keys = min(keys, min(w.q0 + R, l.q) + l.k - l.q);
  if (w.q0 >= l.q) keys = 0;
  w.nkt = keys > 0 ? (keys + BK - 1) / BK : 0;
  w.ragged = w.nkt > 0 && w.nkt * BK > l.k && l.k < p.s.NK;
  return w;
}

// Scales a thread's row of O_t (NC columns from `col`) by f.
template <int NC>
__device__ __forceinline__ void rescale(uint32_t col, float f) {
#pragma unroll
  for (int c = 0; c < NC; c += 32) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(col + c, v);
    tmem_ld_wait();
    reg_fence(v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
    tmem_st_32x32b_x32(col + c, v);
  }
  tmem_st_wait();
}

template <int D, int DVH, bool F16>
__global__ void __launch_bounds__(NTHREADS, 1)
    streamkl_diff_fwd_kernel(const __grid_constant__ DiffFwdParams p) {
  using Lay = FwdLay<D>;
  using Ref = WeightRef<F16>;
  constexpr int NS = Lay::NS;
  // d = 64: the first 64 keys' value products start while the others' weights are
  // formed (B1 H16 N8192 d64/128: 767 against 850 us).  At d = 128 the issuer has
  // more products of the other map to give out and waiting twice costs more than
  // it brings (B1 H16/4 N8192: 1012 against 938 us).
  constexpr bool HALVES = D == 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::bar_off);
  uint64_t* empty = full + NS;
  uint64_t* raw = empty + NS;  // a ragged value tile has landed, to be cleaned
  uint64_t* qfull = raw + NS;
  uint64_t* qempty = qfull + 1;
  uint64_t* sfull = qempty + 1;  // [2] S_t of a tile is in TMEM (and PV_t of the one before is done)
  uint64_t* pfull = sfull + 2;   // [map][half] 64 keys of P_t are in its place
  uint64_t* ofull = pfull + 4;
  uint64_t* oempty = ofull + 1;
  uint64_t* ifull = oempty + 1;  // both maps' 1/l are in shared memory
  uint64_t* drain = ifull + 1;
  float* inv_s = reinterpret_cast<float*>(smem + Lay::inv_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::misc_off + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&raw[s], 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pfull[2 * t], 4);
      mbar_init(&pfull[2 * t + 1], 4);
    }
    mbar_init(ofull, 1);
    mbar_init(oempty, 8);
    mbar_init(ifull, 8);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&p.tmQ1);
    tma_prefetch_desc(&p.tmQ2);
    tma_prefetch_desc(&p.tmK1);
    tma_prefetch_desc(&p.tmK2);
    tma_prefetch_desc(&p.tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  uint8_t* q1_s = smem + Lay::q_off;
  uint8_t* q2_s = q1_s + Lay::q_bytes;
  auto slot_s = [&](int s) { return smem + Lay::ring_off + s * Lay::slot_bytes; };
  SnakeSched sched(p.s.B * p.s.H * ((p.s.NQ + R - 1) / R) * p.nhalf);
  int u;

  // A softmax thread holds a row's 128 products at once: of the launch's 168
  // registers x 384 threads the first warpgroup hands over what it does not need
  // (128 x 88 + 256 x 208 = 384 x 168).
  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;  // map
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t scol = tl + t * BK, ocol = tl + kColO + t * 128;
    const float c = t ? p.c2 : p.c1;
    const float2 C = make_float2(c, c);
    uint32_t sph = 0, oph = 0, iph = 0;
    bool ok = true;
    while (ok && sched.next(u)) {
      const FwdUnit w = decode(p, u);
      const int i = w.q0 + row;
      int lim = i < w.qlen ? w.klen : 0;  // visible keys [0, lim)
      if (p.s.causal) lim = min(lim, i + w.klen - w.qlen + 1);
      float m = -INFINITY, l = 0.f;
      for (int kt = 0; kt < w.nkt; ++kt) {
        if (!(ok = mbar_wait(&sfull[t], sph, ctl))) break;
        sph ^= 1;
        tc_fence_after();
        uint32_t v[BK];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tmem_ld_32x32b_x32(scol + q * 32, reinterpret_cast<uint32_t(&)[32]>(v[q * 32]));
        tmem_ld_wait();
        reg_fence(v);
        const int nv = lim - kt * BK;
        if (nv < BK) {
#pragma unroll
          for (int j = 0; j < BK; ++j)
            if (j >= nv) v[j] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < BK; j += 2)
          mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
        const float most = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        const float top = Ref::top(most, c);
        if (kt == 0) {
          m = Ref::at(top);  // no output yet: the value product overwrites O_t
        } else {
          const bool grow = top > Ref::limit(m);
          if (__any_sync(0xffffffffu, grow)) {
            // sfull was committed behind PV_t of the tile before, so O_t is complete
            const float to = grow ? Ref::at(top) : m;
            const float f = grow ? ex2(m - to) : 1.f;
            l *= f;
            m = to;
            rescale<DVH>(ocol, f);
          }
        }
        // a row that has seen no key keeps m = -inf; its values are all -inf
        const float mu = m == -INFINITY ? 0.f : m;
        const float2 M = make_float2(-mu, -mu);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w16[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 x = make_float2(__uint_as_float(v[q * 32 + j]), __uint_as_float(v[q * 32 + j + 1]));
            const float2 y = __ffma2_rn(x, C, M);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], e);
            w16[j >> 1] = pack2<F16>(e.x, e.y);
          }
          tmem_st_32x32b_x16(scol + q * 16, w16);
          if (q == 3 || (HALVES && q == 1)) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[2 * t + (HALVES ? q >> 1 : 0)]);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      // Epilogue: the maps exchange 1/l_t, then each warpgroup forms half the columns.
      // A row counts by its mask, so that NaN and infinities of what it sees come out.
      const bool sees = lim > 0;
      if (w.half == 0 && i < p.s.NQ) {
        float* L = t ? p.LSE2 : p.LSE1;
        if (L)
          L[(static_cast<long long>(w.b) * p.s.H + w.h) * p.s.NQ + i] =
              sees ? kLn2 * (m + lg2(l)) : -INFINITY;
      }
      // Rows are stored NP lanes together (see transpose_pieces): this lane has one
      // 16-byte piece of each of the NP rows from g0 on.
      constexpr int CW = DVH / 2, NP = CW / 8;
      const bool row_ok = i < p.s.NQ;
      const int g0 = w.q0 + quarter * 32 + lane / NP * NP;
      const long long o0 = w.b * p.o.b + w.h * p.o.h + g0 * p.o.n + w.half * DVH + t * CW + lane % NP * 8;
      if (w.nkt == 0) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          if (g0 + k < p.s.NQ) {
            const long long o = o0 + k * p.o.n;
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + o) = make_uint4(0u, 0u, 0u, 0u);
            if (p.O2) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O2) + o) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        continue;
      }
      const float lam = row_ok ? load_lam(p.lam, w.b, w.h, i, F16) : 0.f;
      if (!(ok = mbar_wait(ofull, oph, ctl))) break;
      oph ^= 1;
      // The value products behind ofull waited until every warp had left the
      // epilogue before, so no one still reads the old 1/l.
      // A map whose visible scores are all -inf has no weights (l = 0) and gives 0.
      inv_s[t * R + row] = l != 0.f ? 1.f / l : 0.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(ifull);
      if (!(ok = mbar_wait(ifull, iph, ctl))) break;
      iph ^= 1;
      tc_fence_after();
      const float i1 = inv_s[row], i2 = inv_s[R + row];
      // all of this thread's columns at once: the row's products are no longer held
      const uint32_t c1 = tl + kColO + t * CW, c2 = c1 + 128;
      uint32_t a[CW], b[CW];
#pragma unroll
      for (int e = 0; e < CW; e += 32) {
        tmem_ld_32x32b_x32(c1 + e, reinterpret_cast<uint32_t(&)[32]>(a[e]));
        tmem_ld_32x32b_x32(c2 + e, reinterpret_cast<uint32_t(&)[32]>(b[e]));
      }
      tmem_ld_wait();
      reg_fence(a);
      reg_fence(b);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(oempty);  // the next unit's value products may begin
      // rows without a visible key are 0 whatever the accumulators hold
      const float2 I1 = make_float2(i1, i1), I2 = make_float2(i2, i2), NL = make_float2(-lam, -lam);
      auto pair = [](const uint32_t* v) { return make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])); };
      auto pieces = [&](auto second, void* out) {
        uint4 x[NP];
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // both maps' outputs are rounded alike, so that equal maps cancel exactly
            float2 r = __fmul2_rn(pair(&b[8 * e + 2 * k]), I2);
            if (!decltype(second)::value) r = __ffma2_rn(r, NL, __fmul2_rn(pair(&a[8 * e + 2 * k]), I1));
            v[k] = sees ? pack2<F16>(r.x, r.y) : 0u;
          }
          x[e] = make_uint4(v[0], v[1], v[2], v[3]);
        }
        transpose_pieces<NP>(x, lane);
        uint16_t* dst = static_cast<uint16_t*>(out) + o0;
#pragma unroll
        for (int k = 0; k < NP; ++k)
          if (g0 + k < p.s.NQ) *reinterpret_cast<uint4*>(dst + k * p.o.n) = x[k];
      };
      pieces(std::false_type{}, p.O);
      if (p.O2) pieces(std::true_type{}, p.O2);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        int s = 0;
        uint32_t ph = 0, qph = 0, rawph = 0;  // bit s of rawph: parity of raw[s]
        uint32_t armed[NS] = {}, armed_q = 0;  // last armed phase + 1; + 2 on raw
        bool ok = true;
        uint64_t* bar = full;
        auto claim = [&](uint32_t bytes, bool ragged) -> bool {
          if (!mbar_wait(&empty[s], ph ^ 1, ctl)) return false;
          // a ragged tile lands on raw; warp 2 cleans it and completes full
          bar = ragged ? &raw[s] : &full[s];
          mbar_arrive_expect_tx(bar, bytes);
          armed[s] = ragged ? 3 + ((rawph >> s) & 1u) : ph + 1;
          if (ragged) rawph ^= 1u << s;
          return true;
        };
        auto step = [&]() {
          if (++s == NS) {
            s = 0;
            ph ^= 1;
          }
        };
        while (ok && sched.next(u)) {
          const FwdUnit w = decode(p, u);
          if (w.nkt == 0) continue;
          if (!(ok = mbar_wait(qempty, qph ^ 1, ctl))) break;
          mbar_arrive_expect_tx(qfull, 2 * Lay::q_bytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            tma_load_4d(q1_s + c * (R * 128), &p.tmQ1, qfull, c * 64, w.q0, w.h, w.b);
            tma_load_4d(q2_s + c * (R * 128), &p.tmQ2, qfull, c * 64, w.q0, w.h, w.b);
          }
          armed_q = qph + 1;
          qph ^= 1;
          for (int kt = 0; kt < w.nkt; ++kt) {
            const int k0 = kt * BK;
            if constexpr (D == 64) {
              if (!(ok = claim(2 * BK * 128, false))) break;
              tma_load_4d(slot_s(s), &p.tmK1, bar, 0, k0, w.hk, w.b);
              tma_load_4d(slot_s(s) + BK * 128, &p.tmK2, bar, 0, k0, w.hk, w.b);
              step();
            } else {
              if (!(ok = claim(BK * D * 2, false))) break;
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(slot_s(s) + c * (BK * 128), &p.tmK1, bar, c * 64, k0, w.hk, w.b);
              step();
              if (!(ok = claim(BK * D * 2, false))) break;
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(slot_s(s) + c * (BK * 128), &p.tmK2, bar, c * 64, k0, w.hk, w.b);
              step();
            }
            if (!(ok = claim(BK * DVH * 2, w.ragged && kt + 1 == w.nkt))) break;
#pragma unroll
            for (int c = 0; c < DVH / 64; ++c)
              tma_load_4d(slot_s(s) + c * (BK * 128), &p.tmV, bar, w.half * DVH + c * 64, k0,
                          w.hk, w.b);
            step();
          }
        }
        if (!ok) {
          // Aborting: let the copies already in flight land before the CTA exits.
          volatile int zero = 0;
          WaitCtl dctl{&zero, p.status, p.wait_limit_ns};
          for (int i = 0; i < NS; ++i)
            if (armed[i]) mbar_wait(armed[i] > 2 ? &raw[i] : &full[i], (armed[i] - 1) & 1u, dctl);
          if (armed_q) mbar_wait(qfull, armed_q - 1, dctl);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ UMMA issuer
      if (lane == 0) {
        constexpr uint32_t idS = idesc_16<F16>(R, BK);
        constexpr uint32_t idO = idesc_16<F16>(R, DVH, 0, 1);  // B = V, features contiguous
        const uint64_t q1d = sdesc_sw128(smem_u32(q1_s), 16, 1024);
        const uint64_t q2d = sdesc_sw128(smem_u32(q2_s), 16, 1024);
        int s = 0;
        uint32_t ph = 0, qph = 0, oph = 0, pph = 0;
        bool ok = true;
        auto step = [&]() {
          if (++s == NS) {
            s = 0;
            ph ^= 1;
          }
        };
        // S_t of the keys at `tile`
        auto issue_s = [&](int t, uint8_t* tile) {
          const uint64_t kd = sdesc_sw128(smem_u32(tile), 16, 1024);
          const uint64_t qd = here(t ? q2d : q1d);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * (BK * 128) + (kk & 3) * 32;
            umma_bf16_ss(tmem + t * BK, sdesc_advance(qd, o), sdesc_advance(kd, o), idS, kk > 0);
          }
          umma_commit(&sfull[t]);
        };
        // PV_t, each half of the keys as soon as its weights are there
        auto issue_pv = [&](int t, uint8_t* tile, bool first) -> bool {
          const uint64_t vd = sdesc_sw128(smem_u32(tile), BK * 128, 1024);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            if (kk == 0 || (HALVES && kk == 4)) {
              if (!mbar_wait(&pfull[2 * t + kk / 4], pph, ctl)) return false;
              tc_fence_after();
            }
            umma_bf16_ts(tmem + kColO + t * 128, tmem + t * BK + kk * 8, sdesc_advance(vd, kk * 2048),
                         idO, !first || kk > 0);
          }
          return true;
        };
        while (ok && sched.next(u)) {
          const FwdUnit w = decode(p, u);
          if (w.nkt == 0) continue;
          if (!(ok = mbar_wait(qfull, qph, ctl))) break;
          qph ^= 1;
          // the first tile's S
          if (!(ok = mbar_wait(&full[s], ph, ctl))) break;
          tc_fence_after();
          issue_s(0, slot_s(s));
          if constexpr (D == 64) {
            issue_s(1, slot_s(s) + BK * 128);
            umma_commit(&empty[s]);
            step();
          } else {
            umma_commit(&empty[s]);
            step();
            if (!(ok = mbar_wait(&full[s], ph, ctl))) break;
            tc_fence_after();
            issue_s(1, slot_s(s));
            umma_commit(&empty[s]);
            step();
          }
          if (w.nkt == 1) umma_commit(qempty);
          for (int kt = 0; kt < w.nkt; ++kt) {
            const int sv = s;  // this tile's values
            const bool more = kt + 1 < w.nkt;
            if (!(ok = mbar_wait(&full[sv], ph, ctl))) break;
            step();
            if (kt == 0) {
              if (!(ok = mbar_wait(oempty, oph ^ 1, ctl))) break;
              oph ^= 1;
            }
            if (!(ok = issue_pv(0, slot_s(sv), kt == 0))) break;
            if (more) {
              if (!(ok = mbar_wait(&full[s], ph, ctl))) break;
              tc_fence_after();
              issue_s(0, slot_s(s));
              if constexpr (D != 64) {
                umma_commit(&empty[s]);
                step();
              }
            }
            if (!(ok = issue_pv(1, slot_s(sv), kt == 0))) break;
            pph ^= 1;
            umma_commit(&empty[sv]);
            if (more) {
              if constexpr (D == 64) {
                issue_s(1, slot_s(s) + BK * 128);
              } else {
                if (!(ok = mbar_wait(&full[s], ph, ctl))) break;
                tc_fence_after();
                issue_s(1, slot_s(s));
              }
              umma_commit(&empty[s]);
              step();
              if (kt + 2 == w.nkt) umma_commit(qempty);  // the unit's last S products
            }
          }
          if (!ok) break;
          umma_commit(ofull);
        }
        // Every UMMA issued by this thread completes before TMEM is released.
        umma_commit(drain);
        volatile int zero = 0;
        WaitCtl dctl{&zero, p.status, p.wait_limit_ns};
        mbar_wait(drain, 0, dctl);
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ ragged value tiles
      unsigned item = 0;  // ring items up to this unit's end
      uint32_t rawph = 0;
      while (sched.next(u)) {
        const FwdUnit w = decode(p, u);
        if (w.nkt == 0) continue;
        item += w.nkt * Lay::ITEMS;
        if (!w.ragged) continue;
        const int s = static_cast<int>((item - 1) % NS);
        if (!__all_sync(0xffffffffu, mbar_wait_long(&raw[s], (rawph >> s) & 1u, ctl))) break;
        rawph ^= 1u << s;
        zero_tile_rows(slot_s(s), DVH / 64, BK, w.klen - (w.nkt - 1) * BK, BK, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
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
}

template <int D, int DVH, bool F16>
cudaError_t launch_t(const DiffFwdParams& p, int num_sms, cudaStream_t stream) {
  constexpr int smem = FwdLay<D>::alloc;
  auto kern = streamkl_diff_fwd_kernel<D, DVH, F16>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, smem, ready);
  if (e != cudaSuccess) return e;
  const int units = p.s.B * p.s.H * ((p.s.NQ + R - 1) / R) * p.nhalf;
  const int grid = units < num_sms ? units : num_sms;
  kern<<<grid, NTHREADS, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_fwd(const DiffFwdParams& p, int d, int dv, bool f16, int num_sms,
                            cudaStream_t stream) {
  if (d == 64 && dv == 64)
    return f16 ? launch_t<64, 64, true>(p, num_sms, stream) : launch_t<64, 64, false>(p, num_sms, stream);
  if (d == 64 && dv == 128)
    return f16 ? launch_t<64, 128, true>(p, num_sms, stream) : launch_t<64, 128, false>(p, num_sms, stream);
  if (d == 128 && (dv == 128 || dv == 256))
    return f16 ? launch_t<128, 128, true>(p, num_sms, stream) : launch_t<128, 128, false>(p, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace skl
