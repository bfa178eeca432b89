// diff.h -- parameter blocks and launchers of the differential-attention and
// paged-cache kernels, and what their C-ABI layer (diff_api.cu) shares with
// streamkl_api.cu.  Internal to libstreamkl.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "streamkl.h"

namespace skl {

// ---------------------------------------------------------- host state (streamkl_api.cu)
// The current device: sm_100 check, SM count, device address of the status word.
streamkl_status api_device(int* num_sms, int** status);
unsigned long long api_wait_limit_ns();
void api_count_launches(int n);
// cuTensorMapEncodeTiled; valid once api_device has returned STREAMKL_OK.
using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                     const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                     const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncode api_encode();

// Sets a kernel's dynamic shared memory limit once per device.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

// Division of numbers below 2^31 by a divisor known on the host: with
// s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, n / d is
// (mulhi(n, m) + n) >> s (division by invariant integers using multiplication,
// Granlund and Montgomery 1994).
struct FastDiv {
  unsigned m = 0;
  int s = 0;
  FastDiv() = default;
  explicit FastDiv(unsigned d) {
    while ((1ull << s) < d) ++s;
    m = static_cast<unsigned>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ unsigned operator()(unsigned n) const { return (__umulhi(n, m) + n) >> s; }
#endif
};

// Element strides of a [B][H][N][d] tensor whose features are contiguous.
struct Strides {
  long long b, h, n;
};

// One weight lam[b][h][i] per query row, broadcast by zero strides; stored in
// fp32 or in the inputs' 16-bit type.
struct Lambda {
  const void* ptr;
  long long b, h, n;
  int f32;
};

// What every kernel of one differential-attention problem reads.  off = the
// last visible key of row 0 under the causal mask is klen - qlen.
struct DiffShape {
  int B, H, HK, NQ, NK, causal;
  const int* q_lens;  // [B] or null: NQ
  const int* k_lens;  // [B] or null: NK
  FastDiv by_H, by_HK, by_share;  // share = H / HK query heads per key head
};

constexpr int kDiffRows = 128;  // UMMA M: query rows (forward, dQ) or keys (dK, dV) per unit
constexpr int kDiffStep = 64;   // streamed rows per step of a backward pass
constexpr int kDiffRec = 5;     // fields of a row record

struct DiffFwdParams {
  CUtensorMap tmQ1, tmK1, tmQ2, tmK2, tmV;  // boxes of 64 features x 128 rows
  DiffShape s;
  Lambda lam;
  void* O;
  void* O2;     // map 2's own output, or null
  Strides o;    // of O and O2
  float* LSE1;  // [B][H][NQ] or null
  float* LSE2;
  float c1, c2;  // s_t * log2(e)
  int nhalf;     // value columns in groups of 128: 1, or 2 (dv = 256)
  int head_group;  // heads visited together; divides B * H
  FastDiv by_group, by_group_units;
  int* status;
  unsigned long long wait_limit_ns;
};
cudaError_t launch_diff_fwd(const DiffFwdParams& p, int d, int dv, bool f16, int num_sms,
                            cudaStream_t stream);

// Row records of the backward: per (b, h) and 64 query rows, field-major,
// -LSE1 log2e, -LSE2 log2e, D1, D2, lam.  Rows that see no key hold -inf, -inf, 0, 0, 0.
struct DiffPrepParams {
  DiffShape s;
  Lambda lam;
  const void* dO;
  const void* O;
  const void* O2;
  Strides sdo, so;  // O and O2 share so
  const float* LSE1;
  const float* LSE2;
  float* rec;  // [B*H][NQpad/64][kDiffRec][64]
  int NQpad, dv, f16;
};
cudaError_t launch_diff_prep(const DiffPrepParams& p, cudaStream_t stream);

// dlam from the sums of P2 G that the kQ pass leaves (dlam of a row is minus the
// row's), over what lam is broadcast over.
struct DiffLamParams {
  const float* d2;         // see DiffBwdParams
  void* out;               // contiguous [B or 1][H or 1][NQ or 1]
  int B, H, NQ;
  int eb, eh, en;          // extents of out
  int f32, f16;            // out's type: fp32, or fp16 / bf16
};
cudaError_t launch_diff_lam(const DiffLamParams& p, cudaStream_t stream);

// One backward pass: resident 128-row tiles against streamed 64-row tiles.
// kKV: resident keys, streamed queries, outputs dK1, dK2, dV.  kQ: resident
// queries, streamed keys, outputs dQ1, dQ2.
struct DiffBwdParams {
  CUtensorMap tmR1, tmR2, tmR3;  // 128-row boxes: K1, K2, V (kKV) or Q1, Q2, dO (kQ)
  CUtensorMap tmC1, tmC2, tmC3;  // 64-row boxes: Q1, Q2, dO (kKV) or K1, K2, V (kQ)
  DiffShape s;
  const float* rec;
  int NQpad;
  void* out1;  // dK1 or dQ1, or null
  void* out2;  // dK2 or dQ2, or null
  void* out3;  // dV (kKV), or null
  Strides so1, so2, so3;
  float c1, c2;  // s_t * log2(e)
  float s1, s2;
  int nhalf;     // dV-only pass: value columns in groups of 128; SEL 1: maps; 1 or 2
  FastDiv by_heads;  // B * HK (kKV) or B * H (kQ)
  int map0;      // SEL 1: the first map (0 or 1)
  int lam_rows;  // lam differs among the rows of a head
  // kQ, or null: sums over the keys of P2 G in fp32, a share per compute warpgroup.
  // d2_rows: of every row, [4][B*H][rows padded to 128]; else of the rows of a warp
  // together, [B*H][row tiles][4 warpgroups][4 warps].
  float* d2;
  int d2_rows;
  int after_pass;  // launched behind another pass, which it need not wait for
  int* status;
  unsigned long long wait_limit_ns;
};
enum DiffPass : int { kDiffKV = 0, kDiffQ = 1 };
// sel: 7 both maps and dV (d = 64), 3 both maps, 1 one map per unit (dv = 256),
// 4 dV alone (d = 128).
cudaError_t launch_diff_bwd(const DiffBwdParams& p, DiffPass pass, int d, int dv, int sel, bool f16,
                            int num_sms, cudaStream_t stream);

// ---------------------------------------------------------- paged caches
// A cache [pages][page_size][HK][width] read through table[b][pages of b].
struct PagedCache {
  const void* ptr;
  long long page, row, head;  // element strides
};

struct PagedParams {
  const void* Q1;
  const void* Q2;            // null: one map
  long long q1_b, q1_h, q2_b, q2_h;
  PagedCache K1, K2, V;
  const int* table;          // [B][table_stride]
  long long table_stride;
  const int* lens;           // [B]
  Lambda lam;                // [B][H] (n unused)
  void* O;                   // [B][H][dv]
  long long o_b, o_h;
  int B, H, HK, pages, page_size, max_pages;
  int page_shift;            // log2(page_size), or -1 when it is no power of two
  float c1, c2;
  int4* cuts;                // workspace: a record per CTA, then the partial states
  float* part;
  int* status;
};
size_t paged_cuts_bytes(int num_sms);
size_t paged_workspace_bytes(int dv, int maps, int num_sms);
cudaError_t launch_paged(const PagedParams& p, int d, int dv, bool f16, int num_sms,
                         cudaStream_t stream);

constexpr int kPagedWriteMax = 4;
struct PagedWriteParams {
  FastDiv by_vecs[kPagedWriteMax], by_token[kPagedWriteMax];  // pieces of a head's row, of a token
  FastDiv by_page;                                            // rows of a page
  const void* rows[kPagedWriteMax];
  void* caches[kPagedWriteMax];
  long long row_t[kPagedWriteMax], row_h[kPagedWriteMax];   // strides of the rows [T][HK][width], bytes
  long long page[kPagedWriteMax], slot[kPagedWriteMax], head[kPagedWriteMax];  // of the caches, bytes
  int vecs[kPagedWriteMax];  // 16-byte pieces of one head's row
  const void* slots;         // [T], int32 or int64
  int slots64;
  int n;                     // caches
  int T, HK, pages, page_size;
  int* status;
};
cudaError_t launch_paged_write(const PagedWriteParams& p, int num_sms, cudaStream_t stream);

}  // namespace skl
