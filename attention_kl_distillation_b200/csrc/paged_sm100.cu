// paged_sm100.cu -- single-token attention over a paged cache, through one
// softmax map or the difference of two, and the write of new rows into pages.
//
//   O[b,h] = softmax(s1 Q1 K1^T) V  [ - lam softmax(s2 Q2 K2^T) V ]
//
// over the first lens[b] tokens of sequence b; token t lives in row t mod
// page_size of page table[b][t / page_size].
//
// What bounds it: every cached row is read once, 2 (maps d + dv) bytes, for the
// 2 maps g (d + 2 dv) FLOP of the products that the g query heads sharing it issue
// (a value product per map and factor of the weights): 12 to 20 FLOP a byte at g = 8,
// where a full tensor pipe would do 250.  That is HBM, so the products
// use warp-level mma with the keys on M and up to 8 query heads on N (no
// padding of 8 heads to 128 rows) and each warp streams its own keys through
// cp.async without a barrier among warps.
//
// Work split: a team (a warp; dv = 256: two, each with 128 value columns) takes
// 16 keys of one work item at a time, an item being a key head and up to 8 of
// the query heads that share it.  The teams of a CTA take neighbouring items of
// a sequence (HW of them, as many as divide the items) at the same tokens:
// together they read whole rows of the cache, [token][head][feature], where one
// head's 128 or 256 bytes at a time would use a fraction of each DRAM page
// (B32 H16 d64/128, 410 to 4096 tokens: 102 us against 127 with HW = 1).  Where HW is less than
// the teams, they also split the tokens, and are joined at an item's end.
// The tiles of all sequences and groups of items form one line, cut into equal
// stretches, one per CTA: lengths may differ by any factor and every CTA still
// reads the same number of rows.  The cut is computed on the device from lens,
// so a captured graph stays right when lengths change.  A stretch may hold
// several whole sequences (written at once) and a part of one at either end
// (state to the workspace, joined by a second kernel in a fixed order).
#include "diff_sm100.cuh"

namespace skl {
namespace {

constexpr int KT = 16;       // keys per team and tile
constexpr int NW = 8;        // warps per CTA
constexpr int HB = 8;        // query heads per work item (mma N)
constexpr int kMaxBatch = 2048;
constexpr int kJoinThreads = 512;
constexpr int kBehind = -2147483647 - 1;

template <int D, int DV, int MAPS>
struct PagedLay {
  static constexpr int WPT = DV > 128 ? 2 : 1;  // warps per team: each owns <= 128 value columns
  static constexpr int TEAMS = NW / WPT;
  static constexpr int DVW = DV / WPT;
  static constexpr int MT = DVW / 16;           // value m-tiles per warp
  static constexpr int k_bytes = KT * D * 2;
  static constexpr int v_bytes = KT * DV * 2;
  static constexpr int stage = MAPS * k_bytes + v_bytes;
  static constexpr int fit = 196608 / (stage * TEAMS);
  static constexpr int NST = fit > 6 ? 6 : fit;
  static constexpr int NREG = MAPS * MT * 4;    // output registers per lane
  static constexpr int ring = NST * stage * TEAMS;
  static constexpr int frag = 32 * (NREG + 4 * MAPS);      // floats of one warp's state
  static constexpr int buf = 2 * frag * 4;                 // two warps' states at a time
  static constexpr int buf_off = ring;
  static constexpr int mask_off = buf_off + buf;
  static constexpr int cum_off = mask_off + NST * TEAMS * 4;
  static constexpr int alloc(int B) { return cum_off + (B + 1) * 4; }
  static_assert(NST >= 2, "ring too shallow");
  static_assert(alloc(kMaxBatch) + 1024 <= 232448,  // 1 KB: the statically sized part
                "shared memory budget exceeded");
  // Workspace of one stretch end and team: outputs and (m, l) per map and head, in
  // the fragment order of its warps.
  static constexpr int image = 32 * NREG + 2 * MAPS * HB;  // floats of one warp's part, 8 heads
  static constexpr int slot_floats = WPT * image;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// How a problem's work items are dealt to `grid` CTAs: `groups` groups of `hw`
// items a sequence, `tile` tokens per tile of the line.  Every cut through a
// group costs a state of each of its items, so a group is no wider than leaves
// about half as many groups as CTAs.
struct Deal {
  int g, blocks, hw, groups, tile;
  __host__ __device__ __forceinline__ Deal(const PagedParams& p, int teams, int grid) {
    g = p.H / p.HK;
    blocks = (g + HB - 1) / HB;
    const int items = p.HK * blocks;
    hw = teams;
    while (hw > 1 && (items % hw != 0 || 2 * p.B * (items / hw) < grid)) hw >>= 1;
    groups = items / hw;
    tile = KT * teams / hw;
  }
};

// Tokens of sequence b that are attended to: lens[b] within the table.
__device__ __forceinline__ int paged_len(const PagedParams& p, int b) {
  const long long most = static_cast<long long>(p.max_pages) * p.page_size;
  const int n = max(p.lens[b], 0);
  if (n > most) {
    atomicCAS(p.status, 0, static_cast<int>(STREAMKL_EDEVICE));
    return static_cast<int>(most);
  }
  return n;
}

__device__ __forceinline__ long long stretch_start(long long total, int c, int n) {
  return total * c / n;
}

// cum[b] = tiles of the sequences before b; cum[B] the total.
__device__ void tile_line(const PagedParams& p, const Deal& d, int* cum, int* scratch) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const int per = (p.B + nt - 1) / nt;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int s = 0;
  for (int b = b0; b < b1; ++b) {
    const int t = (paged_len(p, b) + d.tile - 1) / d.tile * d.groups;
    cum[b + 1] = t;
    s += t;
  }
  const int lane = tid & 31, warp = tid >> 5;
  int x = s;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, k);
    if (lane >= k) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int base = x - s;
  for (int w = 0; w < warp; ++w) base += scratch[w];
  for (int b = b0; b < b1; ++b) {
    base += cum[b + 1];
    cum[b + 1] = base;
  }
  if (tid == 0) cum[0] = 0;
  __syncthreads();
}

// A position on the line of tiles, for one team: its item within the group is
// team % hw, its tokens of a tile are those from 16 (team / hw) on.
struct Cursor {
  int b, group, tile, ntiles, len;  // ntiles of one group
  int hk, first;                    // the item's key head, and first query head of its block
  __device__ __forceinline__ void head(const Deal& d, int team) {
    const int item = group * d.hw + (team & (d.hw - 1));
    hk = item / d.blocks;
    first = (item - hk * d.blocks) * HB;
  }
  __device__ __forceinline__ void seek(const PagedParams& p, const int* cum, const Deal& d, int team, int t) {
    int lo = 0, hi = p.B - 1;  // the sequence with cum[b] <= t < cum[b + 1]
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    ntiles = (cum[b + 1] - cum[b]) / d.groups;
    group = (t - cum[b]) / ntiles;
    tile = (t - cum[b]) % ntiles;
    len = paged_len(p, b);
    head(d, team);
  }
  __device__ __forceinline__ void advance(const PagedParams& p, const int* cum, const Deal& d, int team) {
    if (++tile < ntiles) return;
    tile = 0;
    if (++group < d.groups) {
      head(d, team);
      return;
    }
    group = 0;
    head(d, team);
    do ++b;
    while (b < p.B && cum[b + 1] == cum[b]);
    if (b < p.B) {
      ntiles = (cum[b + 1] - cum[b]) / d.groups;
      len = paged_len(p, b);
    }
  }
};

// The state of one warp: outputs O^T (value row lane/4 (+8), heads 2c, 2c+1 of
// c = lane mod 4) and per map and head the reference and the sum.
template <int MAPS, int MT>
struct State {
  float o[MAPS][MT][4];
  float m[MAPS][2], l[MAPS][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < MAPS; ++t) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][k][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = -INFINITY;
        l[t][e] = 0.f;
      }
    }
  }
  // Image in fragment order, for another warp of this CTA: one float per lane at
  // a stride of 32.
  __device__ __forceinline__ void put(float* dst, int lane) const {
    int k = 0;
#pragma unroll
    for (int t = 0; t < MAPS; ++t)
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[32 * k++ + lane] = o[t][q][e];
#pragma unroll
    for (int t = 0; t < MAPS; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        dst[32 * k++ + lane] = m[t][e];
        dst[32 * k++ + lane] = l[t][e];
      }
  }
  // joins another warp's image: both sides rescaled to the larger reference
  __device__ __forceinline__ void join(const float* src, int lane) {
    const float* ml = src + 32 * (MAPS * MT * 4);
#pragma unroll
    for (int t = 0; t < MAPS; ++t) {
      float fa[2], fb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float om = ml[32 * ((t * 2 + e) * 2) + lane], ol = ml[32 * ((t * 2 + e) * 2 + 1) + lane];
        const float n = fmaxf(m[t][e], om);
        // a side that saw nothing has m = -inf and weight 0
        fa[e] = m[t][e] == -INFINITY ? 0.f : ex2(m[t][e] - n);
        fb[e] = om == -INFINITY ? 0.f : ex2(om - n);
        l[t][e] = fmaf(l[t][e], fa[e], ol * fb[e]);
        m[t][e] = n;
      }
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[t][q][e] = fmaf(o[t][q][e], fa[e & 1], src[32 * ((t * MT + q) * 4 + e) + lane] * fb[e & 1]);
    }
  }
  // Part of the first `heads` heads for the second kernel: per map, value row and
  // head as they lie in the outputs' order [8 rows][head][8], then (m, l) per map
  // and head.
  __device__ __forceinline__ void put_part(float* dst, int heads, int lane) const {
    float* ml = dst + MAPS * MT * 16 * heads;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = (lane & 3) * 2 + e;
      if (h >= heads) continue;
#pragma unroll
      for (int t = 0; t < MAPS; ++t) {
#pragma unroll
        for (int q = 0; q < MT; ++q) {
          dst[((t * MT + q) * 2 * heads + h) * 8 + (lane >> 2)] = o[t][q][e];
          dst[(((t * MT + q) * 2 + 1) * heads + h) * 8 + (lane >> 2)] = o[t][q][e + 2];
        }
        if (lane < 4) {
          ml[(t * heads + h) * 2] = m[t][e];
          ml[(t * heads + h) * 2 + 1] = l[t][e];
        }
      }
    }
  }
  // O_1/l_1 - lam O_2/l_2 of the heads first..first+HB-1 below `heads`
  template <bool F16>
  __device__ __forceinline__ void finish(const PagedParams& p, int b, int head0, int heads, int col0,
                                         int lane) const {
    float inv[MAPS][2];
#pragma unroll
    for (int t = 0; t < MAPS; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) inv[t][e] = l[t][e] > 0.f ? 1.f / l[t][e] : 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = (lane & 3) * 2 + e;
      if (k >= heads) continue;
      const int h = head0 + k;
      const float f1 = inv[0][e];
      float f2 = 0.f;
      if (MAPS == 2) f2 = -inv[MAPS - 1][e] * load_lam(p.lam, b, h, 0, F16);
      uint16_t* dst = static_cast<uint16_t*>(p.O) + b * p.o_b + h * p.o_h + col0 + (lane >> 2);
#pragma unroll
      for (int q = 0; q < MT; ++q) {
        float x = o[0][q][e] * f1, y = o[0][q][e + 2] * f1;
        if (MAPS == 2) {
          x = fmaf(o[MAPS - 1][q][e], f2, x);
          y = fmaf(o[MAPS - 1][q][e + 2], f2, y);
        }
        const uint32_t w = pack2<F16>(x, y);
        dst[q * 16] = static_cast<uint16_t>(w);
        dst[q * 16 + 8] = static_cast<uint16_t>(w >> 16);
      }
    }
  }
};

// Joins the states of teams that differ by a multiple of `hw` into those of the
// first hw teams, in a fixed order, through a buffer of two warps' states.
template <class Lay, class S>
__device__ __forceinline__ void join_teams(S& st, float* buf, int warp, int lane, int hw) {
  auto hand = [&](int from, int to, int count) {  // warps [from, from + count) to [to, ..)
    __syncthreads();
    if (warp >= from && warp < from + count) st.put(buf + (warp - from) * Lay::frag, lane);
    __syncthreads();
    if (warp >= to && warp < to + count) st.join(buf + (warp - to) * Lay::frag, lane);
  };
  const int keep = hw * Lay::WPT;  // warps that end up with an item's state
  if (keep <= 4) {
    hand(4, 0, 2);
    hand(6, 2, 2);
  }
  if (keep <= 2) hand(2, 0, 2);
  if (keep <= 1) hand(1, 0, 1);
}

template <int D, int DV, int MAPS, bool F16>
__global__ void __launch_bounds__(NW * 32, 1)
    streamkl_paged_kernel(const __grid_constant__ PagedParams p) {
  using Lay = PagedLay<D, DV, MAPS>;
  using Ref = WeightRef<F16>;
  constexpr int NST = Lay::NST, WPT = Lay::WPT, MT = Lay::MT;
  constexpr int VP = DV / 8;       // 16-byte pieces of a row
  constexpr int CHUNK = KT * 128;  // bytes of 64 features of a tile
  extern __shared__ __align__(1024) uint8_t smem_paged[];
  __shared__ int scratch[NW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / WPT, member = warp % WPT;
  uint8_t* ring = smem_paged + team * (NST * Lay::stage);
  float* buf = reinterpret_cast<float*>(smem_paged + Lay::buf_off);
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem_paged + Lay::mask_off) + team * NST;
  int* cum = reinterpret_cast<int*>(smem_paged + Lay::cum_off);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Deal deal(p, Lay::TEAMS, gridDim.x);
  tile_line(p, deal, cum, scratch);
  const long long total = cum[p.B];
  const int n = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  const int c = blockIdx.x;

  // sequences without a token: zeros
  for (int b = c; b < p.B; b += gridDim.x) {
    if (cum[b + 1] != cum[b]) continue;
    for (int k = threadIdx.x; k < p.H * (DV / 8); k += blockDim.x)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + b * p.o_b + (k / VP) * p.o_h +
                                (k % VP) * 8) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (c >= n) {
    if (threadIdx.x == 0) p.cuts[c] = make_int4(0, 0, 0, 0);
    return;
  }
  const int t0 = static_cast<int>(stretch_start(total, c, n));
  const int t1 = static_cast<int>(stretch_start(total, c + 1, n));

  const uint32_t ring_a = smem_u32(ring);
  const int g = deal.g, kw = team / deal.hw, mine = team & (deal.hw - 1);  // item of the group
  // Page and row of token tok; page sizes are mostly powers of two.
  auto page_index = [&](int tok) { return p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size; };
  auto page_row = [&](int tok) { return p.page_shift >= 0 ? tok & (p.page_size - 1) : tok % p.page_size; };
  auto token = [&](const Cursor& cur) { return cur.tile * deal.tile + kw * KT + (lane & 15); };
  // Lane r (and r + 16) reads the table entry of row r a tile ahead of its use;
  // what it holds is looked at only then.  kBehind: no such token.
  auto page_of = [&](const Cursor& cur) -> int {
    const int tok = token(cur);
    return tok < cur.len ? p.table[cur.b * p.table_stride + page_index(tok)] : kBehind;
  };
  // Issues the copies of tile `cur` into stage s.
  auto issue = [&](const Cursor& cur, int page, int s) {
    if (page != kBehind && (page < 0 || page >= p.pages)) {  // not a page: left out, and reported
      atomicCAS(p.status, 0, static_cast<int>(STREAMKL_EDEVICE));
      page = -1;
    }
    const int slot = page_row(token(cur));
    const uint32_t seen = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
    if (member == 0 && lane == 0) masks[s] = seen;
    // Eight lanes copy 128 bytes of a row at a time, four rows in turn.  The
    // layout: chunks of 64 features, 16 rows of 128 bytes each, 16-byte pieces
    // exchanged by the row's low three bits (ldmatrix then meets no bank twice).
    const uint16_t* k1 = static_cast<const uint16_t*>(p.K1.ptr) + cur.hk * p.K1.head + (lane & 7) * 8;
    const uint16_t* k2 = static_cast<const uint16_t*>(p.K2.ptr) + cur.hk * p.K2.head + (lane & 7) * 8;
    const uint16_t* v = static_cast<const uint16_t*>(p.V.ptr) + cur.hk * p.V.head + (lane & 7) * 8;
    const uint32_t a = ring_a + s * Lay::stage;
#pragma unroll
    for (int i = 0; i < KT / 4; ++i) {
      if (WPT == 2 && (i & 1) != member) continue;  // the team's warps take turns
      const int r = i * 4 + (lane >> 3);
      const int pg = __shfl_sync(0xffffffffu, page, r), sl = __shfl_sync(0xffffffffu, slot, r);
      const bool ok = pg >= 0;
      const long long pgl = ok ? pg : 0, sll = ok ? sl : 0;  // what is not read still has an address
      const int bytes = ok ? 16 : 0;
      const uint32_t dst = a + r * 128 + (((lane & 7) ^ (r & 7)) * 16);
      const uint16_t* src = k1 + pgl * p.K1.page + sll * p.K1.row;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) cp_async16(dst + c * CHUNK, src + c * 64, bytes);
      if (MAPS == 2) {
        src = k2 + pgl * p.K2.page + sll * p.K2.row;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) cp_async16(dst + Lay::k_bytes + c * CHUNK, src + c * 64, bytes);
      }
      src = v + pgl * p.V.page + sll * p.V.row;
#pragma unroll
      for (int c = 0; c < DV / 64; ++c)
        cp_async16(dst + MAPS * Lay::k_bytes + c * CHUNK, src + c * 64, bytes);
    }
  };
  auto team_sync = [&]() {
    if (WPT == 1) __syncwarp();
    else asm volatile("bar.sync %0, 64;" ::"r"(1 + team) : "memory");
  };

  Cursor ld, cur;
  ld.seek(p, cum, deal, team, t0);
  cur = ld;
  // For the second kernel: the group of items that the cut in front of this
  // stretch goes through, if it is the first cut through it, and its parts.
  if (c > 0 && threadIdx.x == 0) {
    const int start = t0 - cur.tile, end = start + cur.ntiles;
    int parts = 0;
    if (cur.tile > 0 && start >= static_cast<int>(stretch_start(total, c - 1, n)))
      for (parts = 2; c - 1 + parts < n && stretch_start(total, c - 1 + parts, n) < end;) ++parts;
    p.cuts[c] = make_int4(cur.b, cur.group, parts, 0);
  }
  int tl = t0;  // next tile to be issued
  int page = page_of(ld);
  auto issue_next = [&](int s) {
    if (tl < t1) {
      issue(ld, page, s);
      ++tl;
      if (tl < t1) {
        ld.advance(p, cum, deal, team);
        page = page_of(ld);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) issue_next(s);

  State<MAPS, MT> st;
  uint32_t qf[MAPS][D / 16][2];
  auto load_q = [&]() {
    const int hk = cur.hk, k = cur.first + (lane >> 2);
#pragma unroll
    for (int t = 0; t < MAPS; ++t) {
      const uint16_t* q = t ? static_cast<const uint16_t*>(p.Q2) + cur.b * p.q2_b + (hk * g + k) * p.q2_h
                            : static_cast<const uint16_t*>(p.Q1) + cur.b * p.q1_b + (hk * g + k) * p.q1_h;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[t][kk][e] = k < g ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + e * 8 + (lane & 3) * 2) : 0u;
    }
  };
  int item_start = t0 - cur.tile;  // line position of the current item's first tile
  st.clear();
  load_q();

  // This lane's row and piece of an ldmatrix: keys as they lie (rows lane % 16,
  // features 8 (lane / 16) on), values transposed (rows lane % 8 + 8 (lane / 16),
  // features 8 (lane / 8 % 2) on).  Further features are an exclusive or away.
  const uint32_t k_lane = (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);
  const uint32_t v_lane = ((lane & 7) + ((lane >> 4) << 3)) * 128 + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
  int s = 0;
  for (int t = t0; t < t1; ++t) {
    cp_async_wait<NST - 2>();
    team_sync();
    issue_next(s == 0 ? NST - 1 : s - 1);  // the stage read in the last round
    const uint32_t a = ring_a + s * Lay::stage;
    const uint32_t seen = masks[s];
    if (seen) {
      // S^T of both maps: keys lane/4 (+8), heads 2c, 2c+1
      float x[MAPS][4];
#pragma unroll
      for (int m = 0; m < MAPS; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[m][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t af[4];
          ldsm4(((a + k_lane) ^ ((kk & 3) * 32)) + m * Lay::k_bytes + (kk >> 2) * CHUNK, af);
          mma16816<F16>(x[m], af, qf[m][kk][0], qf[m][kk][1]);
        }
      }
      if (seen != 0xffffu) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool ok = (seen >> ((lane >> 2) + (e >> 1) * 8)) & 1u;
#pragma unroll
          for (int m = 0; m < MAPS; ++m) x[m][e] = ok ? x[m][e] : -INFINITY;
        }
      }
      bool grow = false;
      float mx[MAPS][2];
#pragma unroll
      for (int m = 0; m < MAPS; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[m][e] = Ref::top(fmaxf(x[m][e], x[m][e + 2]), m ? p.c2 : p.c1);
          grow = grow || mx[m][e] > Ref::limit(st.m[m][e]);
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int m = 0; m < MAPS; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
              mx[m][e] = fmaxf(mx[m][e], __shfl_xor_sync(0xffffffffu, mx[m][e], d));
            const bool up = mx[m][e] > Ref::limit(st.m[m][e]);
            const float to = Ref::at(mx[m][e]);
            const float f = up ? ex2(st.m[m][e] - to) : 1.f;
            if (up) st.m[m][e] = to;
            st.l[m][e] *= f;
#pragma unroll
            for (int q = 0; q < MT; ++q) {
              st.o[m][q][e] *= f;
              st.o[m][q][e + 2] *= f;
            }
          }
      }
      uint32_t pf[MAPS][2], pr[MAPS][2];
#pragma unroll
      for (int m = 0; m < MAPS; ++m) {
        const float cm = m ? p.c2 : p.c1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = st.m[m][e & 1] == -INFINITY ? 0.f : st.m[m][e & 1];
          x[m][e] = ex2(fmaf(x[m][e], cm, -ref));
          st.l[m][e & 1] += x[m][e];
        }
        // P^T as the B operand: heads on rows after the transposition.  P goes in as
        // two 16-bit factors, its rounded value and what the rounding left, so that
        // the outputs are nearly as exact as fp32 weights would make them: a weight is
        // off by 2^-16 of itself (bf16), or by 2^-22 of itself or 2^-36 of the row's
        // largest (fp16, see WeightRef).  The kernel is bound by HBM and pays 0 to 2%
        // for the second product (B32 H16 d64/128: 101 -> 103 us).
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = pack2<F16>(x[m][2 * e], x[m][2 * e + 1]);
          const float2 back = unpack2<F16>(w);
          pf[m][e] = transpose8x8(w);
          pr[m][e] = transpose8x8(pack2<F16>(x[m][2 * e] - back.x, x[m][2 * e + 1] - back.y));
        }
      }
#pragma unroll
      for (int q = 0; q < MT; ++q) {
        uint32_t vf[4];
        ldsm4_t(((a + v_lane) ^ ((q & 3) * 32)) + MAPS * Lay::k_bytes +
                    (member * (Lay::DVW / 64) + (q >> 2)) * CHUNK,
                vf);
#pragma unroll
        for (int m = 0; m < MAPS; ++m) {
          mma16816<F16>(st.o[m][q], vf, pf[m][0], pf[m][1]);
          mma16816<F16>(st.o[m][q], vf, pr[m][0], pr[m][1]);
        }
      }
    }
    if (++s == NST) s = 0;

    const bool item_ends = cur.tile + 1 == cur.ntiles;
    if (item_ends || t + 1 == t1) {
      // This stretch's part of the group's items.
#pragma unroll
      for (int m = 0; m < MAPS; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) st.l[m][e] += __shfl_xor_sync(0xffffffffu, st.l[m][e], d);
      const Cursor at = cur;
      const bool begun_here = item_start >= t0;
      const int heads = min(HB, g - at.first);
      if (t + 1 < t1) {  // the next item's queries are on their way while this one is joined
        cur.advance(p, cum, deal, team);
        item_start = t + 1;
        load_q();
      }
      if (deal.hw < Lay::TEAMS) join_teams<Lay>(st, buf, warp, lane, deal.hw);
      if (kw == 0) {
        if (begun_here && item_ends) {
          st.template finish<F16>(p, at.b, at.hk * g + at.first, heads, member * Lay::DVW, lane);
        } else {
          // begun before this stretch: slot 2c; going on behind it: slot 2c + 1
          const long long slot = (2ll * c + (begun_here ? 1 : 0)) * Lay::TEAMS + mine;
          st.put_part(p.part + slot * Lay::slot_floats + member * Lay::image, heads, lane);
        }
      }
      st.clear();
    } else {
      ++cur.tile;
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of every item that stretches over several CTAs: block (c, k)
// has item k of the group through which the cut in front of stretch c is the
// first.  The parts' weights 2^(m_p - max m) come first, then every thread sums
// its outputs over the parts: independent loads, in the parts' order.
template <int D, int DV, int MAPS, bool F16>
__global__ void __launch_bounds__(kJoinThreads)
    streamkl_paged_join_kernel(const __grid_constant__ PagedParams p, int grid) {
  using Lay = PagedLay<D, DV, MAPS>;
  extern __shared__ float weight[];  // [parts][MAPS * heads] references, then weights; the same of sums
  __shared__ float inv[MAPS * HB];
  const Deal deal(p, Lay::TEAMS, grid);
  // Every block waits for the first kernel, so that this one does not end before it.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x + 1, mine = blockIdx.y;
  const int4 cut = p.cuts[c];  // sequence, group, parts
  const int parts = cut.z;
  if (parts == 0) return;
  Cursor cur;
  cur.group = cut.y;
  cur.head(deal, mine);
  const int heads = min(HB, deal.g - cur.first), n = MAPS * heads, vals = Lay::MT * 16 * heads;
  // part 0 ends stretch c - 1, part j > 0 begins stretch c - 1 + j
  auto part = [&](int j) {
    return p.part + ((2ll * (c - 1 + j) + (j == 0 ? 1 : 0)) * Lay::TEAMS + mine) * Lay::slot_floats;
  };
  float* sums = weight + parts * n;
  for (int k = threadIdx.x; k < parts * n; k += blockDim.x) {
    const float2 ml = *reinterpret_cast<const float2*>(part(k / n) + MAPS * vals + (k % n) * 2);
    weight[k] = ml.x;
    sums[k] = ml.y;
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < n) {
    float top = -INFINITY, sum = 0.f;
    for (int k = threadIdx.x; k < parts * n; k += n) top = fmaxf(top, weight[k]);
    for (int k = threadIdx.x; k < parts * n; k += n) {
      const float w = weight[k] == -INFINITY ? 0.f : ex2(weight[k] - top);  // a part that saw nothing
      weight[k] = w;
      sum = fmaf(sums[k], w, sum);
    }
    inv[threadIdx.x] = sum > 0.f ? 1.f / sum : 0.f;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < Lay::WPT * vals; k += blockDim.x) {
    const int member = k / vals, e = k - member * vals;
    const int h = e / 8 % heads, col = member * Lay::DVW + e / (8 * heads) * 8 + e % 8;
    float acc[MAPS] = {};
#pragma unroll 8
    for (int j = 0; j < parts; ++j) {
      const float* src = part(j) + member * Lay::image + e;
#pragma unroll
      for (int t = 0; t < MAPS; ++t) acc[t] = fmaf(src[t * vals], weight[j * n + t * heads + h], acc[t]);
    }
    const int head = cur.hk * deal.g + cur.first + h;
    float x = acc[0] * inv[h];
    if (MAPS == 2)
      x = fmaf(-load_lam(p.lam, cut.x, head, 0, F16), acc[MAPS - 1] * inv[(MAPS - 1) * heads + h], x);
    static_cast<uint16_t*>(p.O)[cut.x * p.o_b + head * p.o_h + col] =
        static_cast<uint16_t>(pack2<F16>(x, 0.f));
  }
}

template <int D, int DV, int MAPS, bool F16>
cudaError_t launch_t(const PagedParams& p, int num_sms, cudaStream_t stream) {
  using Lay = PagedLay<D, DV, MAPS>;
  auto kern = streamkl_paged_kernel<D, DV, MAPS, F16>;
  const int smem = Lay::alloc(p.B);
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, Lay::alloc(kMaxBatch), ready);
  if (e != cudaSuccess) return e;
  kern<<<num_sms, NW * 32, smem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // The join's blocks start while the first kernel still runs and wait for it.
  auto join = streamkl_paged_join_kernel<D, DV, MAPS, F16>;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms - 1, Deal(p, Lay::TEAMS, num_sms).hw);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 2 * static_cast<size_t>(num_sms) * MAPS * HB * sizeof(float);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join, p, num_sms);
}

template <int MAPS, bool F16>
cudaError_t launch_dims(const PagedParams& p, int d, int dv, int num_sms, cudaStream_t stream) {
  if (d == 64 && dv == 64) return launch_t<64, 64, MAPS, F16>(p, num_sms, stream);
  if (d == 64 && dv == 128) return launch_t<64, 128, MAPS, F16>(p, num_sms, stream);
  if (d == 128 && dv == 128) return launch_t<128, 128, MAPS, F16>(p, num_sms, stream);
  if (d == 128 && dv == 256) return launch_t<128, 256, MAPS, F16>(p, num_sms, stream);
  return cudaErrorInvalidValue;
}

// New rows into their slots, 16 bytes a thread and step, STEPS steps' loads in
// flight: four where that still fills the device (a batch of prompts, 8 heads, d128/256:
// 33 us against 35), one for a served batch's single tokens, which are bound by
// latency (64 rows of 16 heads, d64/128: 2.2 us against 3.4).  A negative slot is skipped (a padded row); one past the
// cache is skipped and reported.
template <int STEPS>
__global__ void __launch_bounds__(256) streamkl_paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
  const int w = blockIdx.y;
  const int vecs = p.vecs[w], per = p.HK * vecs;
  const long long total = static_cast<long long>(p.T) * per;
  const long long slots = static_cast<long long>(p.pages) * p.page_size;
  constexpr int kBlock = 256 * STEPS;
  for (long long base = static_cast<long long>(blockIdx.x) * kBlock; base < total;
       base += static_cast<long long>(gridDim.x) * kBlock) {
    // one wide division a block and step; the others by multiplication
    const int t0 = static_cast<int>(base / per);
    const unsigned r0 = static_cast<unsigned>(base - static_cast<long long>(t0) * per) + threadIdx.x;
    uint4 x[STEPS];
    uint8_t* dst[STEPS];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      dst[k] = nullptr;
      const unsigned i = r0 + k * 256;  // piece, counted from token t0
      const unsigned dt = p.by_token[w](i), r = i - dt * per, h = p.by_vecs[w](r), v = r - h * vecs;
      const long long t = static_cast<long long>(t0) + dt;
      if (t >= p.T) continue;
      const long long slot = p.slots64 ? static_cast<const long long*>(p.slots)[t]
                                       : static_cast<const int*>(p.slots)[t];
      if (slot < 0) continue;
      if (slot >= slots) {
        atomicCAS(p.status, 0, static_cast<int>(STREAMKL_EDEVICE));
        continue;
      }
      // slots of the cache fit in 31 bits: pages * page_size does
      const unsigned page = p.by_page(static_cast<unsigned>(slot));
      const unsigned row = static_cast<unsigned>(slot) - page * static_cast<unsigned>(p.page_size);
      x[k] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.rows[w]) +
                                             t * p.row_t[w] + h * p.row_h[w] + v * 16);
      dst[k] = static_cast<uint8_t*>(p.caches[w]) + page * p.page[w] + row * p.slot[w] + h * p.head[w] + v * 16;
    }
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
      if (dst[k]) *reinterpret_cast<uint4*>(dst[k]) = x[k];
  }
}

}  // namespace

size_t paged_workspace_bytes(int dv, int maps, int num_sms) {
  // the cuts, then two stretch ends per CTA, a state of every warp: HB heads'
  // outputs and (m, l)
  const int mt = (dv > 128 ? 128 : dv) / 16;
  return paged_cuts_bytes(num_sms) +
         static_cast<size_t>(2 * num_sms) * NW * (32 * maps * mt * 4 + 2 * maps * HB) * 4;
}

size_t paged_cuts_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * sizeof(int4) + 255) / 256 * 256; }

cudaError_t launch_paged(const PagedParams& p, int d, int dv, bool f16, int num_sms,
                         cudaStream_t stream) {
  if (p.B > kMaxBatch) return cudaErrorInvalidValue;
  if (p.Q2) return f16 ? launch_dims<2, true>(p, d, dv, num_sms, stream)
                       : launch_dims<2, false>(p, d, dv, num_sms, stream);
  return f16 ? launch_dims<1, true>(p, d, dv, num_sms, stream)
             : launch_dims<1, false>(p, d, dv, num_sms, stream);
}

cudaError_t launch_paged_write(const PagedWriteParams& p, int num_sms, cudaStream_t stream) {
  int most = 0;
  for (int i = 0; i < p.n; ++i) most = p.vecs[i] > most ? p.vecs[i] : most;
  const long long pieces = static_cast<long long>(p.T) * p.HK * most, cap = 8ll * num_sms;
  const int per = pieces >= 256 * 4 * cap ? 256 * 4 : 256;
  const long long blocks = (pieces + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap), static_cast<unsigned>(p.n));
  if (per == 256) streamkl_paged_write_kernel<1><<<grid, 256, 0, stream>>>(p);
  else streamkl_paged_write_kernel<4><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace skl
