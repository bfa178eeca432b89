// diff_api.cu -- C ABI of differential attention and the paged caches
// (declared in include/streamkl.h).  Host-side only: argument validation, TMA
// descriptors, launches on the caller's stream.
#include <cmath>
#include <cstdint>

#include "diff.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxUnits = 1 << 30;
constexpr int64_t kMaxStride = int64_t(1) << 38;  // bytes < 2^40 in a tensor map

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool widths_ok(int d, int dv) {
  return (d == 64 && (dv == 64 || dv == 128)) || (d == 128 && (dv == 128 || dv == 256));
}

// One axis of an outer layout: a positive multiple of 8 elements, unless its extent is 1.
bool axis_ok(int64_t stride, int64_t extent) {
  return extent == 1 || (stride > 0 && stride % 8 == 0 && stride <= kMaxStride);
}

bool tensor_ok(const streamkl_tensor* t, int64_t nb, int64_t nh, int64_t nn) {
  return t && t->ptr && aligned(t->ptr, 16) && axis_ok(t->b, nb) && axis_ok(t->h, nh) &&
         axis_ok(t->n, nn);
}

// A weight per (b, h, i): zero strides broadcast, others are any positive count.
bool lam_ok(const streamkl_tensor* t, bool fp32) {
  return t && t->ptr && aligned(t->ptr, fp32 ? 4 : 2) && t->b >= 0 && t->h >= 0 && t->n >= 0;
}

float scale_of(float s, int d) { return s > 0.f ? s : 1.0f / std::sqrt(static_cast<float>(d)); }

streamkl_status check_diff(const streamkl_diff_problem* pr) {
  if (!pr) return STREAMKL_EINVAL;
  if (pr->B < 1 || pr->H < 1 || pr->HK < 1 || pr->NQ < 1 || pr->NK < 1) return STREAMKL_EINVAL;
  if (pr->H % pr->HK != 0) return STREAMKL_EINVAL;
  if ((pr->causal | pr->lam_fp32) & ~1) return STREAMKL_EINVAL;
  if (!std::isfinite(pr->s1) || !std::isfinite(pr->s2)) return STREAMKL_EINVAL;
  const int64_t BH = static_cast<int64_t>(pr->B) * pr->H;
  if (BH > kMaxUnits || pr->NQ > (1 << 29) || pr->NK > (1 << 29)) return STREAMKL_EINVAL;
  // work units (two value halves at most), and steps of one backward unit, are counted in int
  if (BH * ((pr->NQ + 127) / 128) > kMaxUnits / 2 || BH * ((pr->NK + 127) / 128) > kMaxUnits / 2)
    return STREAMKL_EINVAL;
  if (pr->dtype != STREAMKL_BF16 && pr->dtype != STREAMKL_FP16) return STREAMKL_EUNSUPPORTED;
  if (!widths_ok(pr->d, pr->dv)) return STREAMKL_EUNSUPPORTED;
  return STREAMKL_OK;
}

// 4-D map [B][heads][n][width] with boxes of 64 features (128 bytes, the
// swizzle span) by `rows` rows.  Rows past n read as zero.
streamkl_status map_of(const streamkl_tensor& t, int64_t B, int64_t heads, int64_t n, int width,
                       int rows, int dtype, CUtensorMap* out) {
  // the stride of an axis of extent 1 is never used; any valid value will do
  auto bytes = [](int64_t stride, int64_t extent) {
    return static_cast<cuuint64_t>(extent == 1 ? 512 : stride * 2);
  };
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(n),
                        static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {bytes(t.n, n), bytes(t.h, heads), bytes(t.b, B)};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type =
      dtype == STREAMKL_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUresult r =
      skl::api_encode()(out, type, 4, const_cast<void*>(t.ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? STREAMKL_OK : STREAMKL_ECUDA;
}

skl::DiffShape shape_of(const streamkl_diff_problem& pr, const int* q_lens, const int* k_lens) {
  return skl::DiffShape{pr.B, pr.H, pr.HK, pr.NQ, pr.NK, pr.causal, q_lens, k_lens,
                        skl::FastDiv(pr.H), skl::FastDiv(pr.HK), skl::FastDiv(pr.H / pr.HK)};
}

skl::Lambda lambda_of(const streamkl_tensor& t, int fp32) {
  return skl::Lambda{t.ptr, t.b, t.h, t.n, fp32};
}

skl::Strides strides_of(const streamkl_tensor& t) { return skl::Strides{t.b, t.h, t.n}; }

bool same_strides(const streamkl_tensor& a, const streamkl_tensor& b, const streamkl_diff_problem& pr) {
  return (pr.B == 1 || a.b == b.b) && (pr.H == 1 || a.h == b.h) && (pr.NQ == 1 || a.n == b.n);
}

streamkl_status check_inputs(const streamkl_diff_problem& pr, const streamkl_tensor* Q1,
                             const streamkl_tensor* K1, const streamkl_tensor* Q2,
                             const streamkl_tensor* K2, const streamkl_tensor* V,
                             const streamkl_tensor* lam, const int* q_lens, const int* k_lens) {
  if (!tensor_ok(Q1, pr.B, pr.H, pr.NQ) || !tensor_ok(Q2, pr.B, pr.H, pr.NQ) ||
      !tensor_ok(K1, pr.B, pr.HK, pr.NK) || !tensor_ok(K2, pr.B, pr.HK, pr.NK) ||
      !tensor_ok(V, pr.B, pr.HK, pr.NK) || !lam_ok(lam, pr.lam_fp32))
    return STREAMKL_EINVAL;
  if (!aligned(q_lens, 4) || !aligned(k_lens, 4)) return STREAMKL_EINVAL;
  return STREAMKL_OK;
}

int padded_rows(const streamkl_diff_problem& pr) {
  return (pr.NQ + skl::kDiffStep - 1) / skl::kDiffStep * skl::kDiffStep;
}

// Row records, then the shares of P2 G (four a row), in floats.
struct DiffWorkspace {
  size_t rec, d2;
};
DiffWorkspace diff_workspace(const streamkl_diff_problem& pr) {
  const size_t BH = static_cast<size_t>(pr.B) * pr.H;
  const size_t tiles = (static_cast<size_t>(pr.NQ) + skl::kDiffRows - 1) / skl::kDiffRows;
  return {BH * padded_rows(pr) * skl::kDiffRec, BH * tiles * skl::kDiffRows * 4};
}

streamkl_status check_paged(const streamkl_paged_problem* pr) {
  if (!pr) return STREAMKL_EINVAL;
  if (pr->B < 1 || pr->H < 1 || pr->HK < 1 || pr->pages < 1 || pr->page_size < 1 ||
      pr->max_pages < 1 || pr->H % pr->HK != 0)
    return STREAMKL_EINVAL;
  if (pr->lam_fp32 & ~1) return STREAMKL_EINVAL;
  if (!std::isfinite(pr->s1) || !std::isfinite(pr->s2)) return STREAMKL_EINVAL;
  if (pr->B > 2048) return STREAMKL_EINVAL;
  const int64_t most = static_cast<int64_t>(pr->max_pages) * pr->page_size;
  if (most > (1 << 30)) return STREAMKL_EINVAL;
  // Tiles are counted in int.  One holds 64 tokens of a work item (a key head, 8 of its
  // query heads) or more, or a share of them of several items.
  const int64_t items = static_cast<int64_t>(pr->HK) * ((pr->H / pr->HK + 7) / 8);
  if (items > (1 << 20) || pr->B * items * (most / 64 + 1) > INT32_MAX) return STREAMKL_EINVAL;
  if (pr->dtype != STREAMKL_BF16 && pr->dtype != STREAMKL_FP16) return STREAMKL_EUNSUPPORTED;
  if (!widths_ok(pr->d, pr->dv)) return STREAMKL_EUNSUPPORTED;
  return STREAMKL_OK;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

#define SKL_TRY(expr)                                   \
  do {                                                  \
    const streamkl_status st_ = (expr);                 \
    if (st_ != STREAMKL_OK) return st_;                 \
  } while (0)

}  // namespace

extern "C" {

streamkl_status streamkl_diff_fwd(const streamkl_diff_problem* prob, const streamkl_tensor* Q1,
                                  const streamkl_tensor* K1, const streamkl_tensor* Q2,
                                  const streamkl_tensor* K2, const streamkl_tensor* V,
                                  const streamkl_tensor* lam, const int* q_lens,
                                  const int* k_lens, const streamkl_tensor* O,
                                  const streamkl_tensor* O2, float* LSE1, float* LSE2,
                                  streamkl_stream_t stream) {
  SKL_TRY(check_diff(prob));
  const streamkl_diff_problem& pr = *prob;
  SKL_TRY(check_inputs(pr, Q1, K1, Q2, K2, V, lam, q_lens, k_lens));
  if (!tensor_ok(O, pr.B, pr.H, pr.NQ)) return STREAMKL_EINVAL;
  if (O2 && (!tensor_ok(O2, pr.B, pr.H, pr.NQ) || !same_strides(*O, *O2, pr))) return STREAMKL_EINVAL;
  if ((LSE1 == nullptr) != (LSE2 == nullptr) || !aligned(LSE1, 4) || !aligned(LSE2, 4))
    return STREAMKL_EINVAL;
  skl::DiffFwdParams p;
  int sms = 0;
  SKL_TRY(skl::api_device(&sms, &p.status));
  SKL_TRY(map_of(*Q1, pr.B, pr.H, pr.NQ, pr.d, 128, pr.dtype, &p.tmQ1));
  SKL_TRY(map_of(*Q2, pr.B, pr.H, pr.NQ, pr.d, 128, pr.dtype, &p.tmQ2));
  SKL_TRY(map_of(*K1, pr.B, pr.HK, pr.NK, pr.d, 128, pr.dtype, &p.tmK1));
  SKL_TRY(map_of(*K2, pr.B, pr.HK, pr.NK, pr.d, 128, pr.dtype, &p.tmK2));
  SKL_TRY(map_of(*V, pr.B, pr.HK, pr.NK, pr.dv, 128, pr.dtype, &p.tmV));
  p.s = shape_of(pr, q_lens, k_lens);
  p.lam = lambda_of(*lam, pr.lam_fp32);
  p.O = const_cast<void*>(O->ptr);
  p.O2 = O2 ? const_cast<void*>(O2->ptr) : nullptr;
  p.o = strides_of(*O);
  p.LSE1 = LSE1;
  p.LSE2 = LSE2;
  p.c1 = scale_of(pr.s1, pr.d) * kLog2e;
  p.c2 = scale_of(pr.s2, pr.d) * kLog2e;
  p.nhalf = pr.dv > 128 ? pr.dv / 128 : 1;
  // Once a head has a query tile per SM, the query heads of one key head at a
  // time: the CTAs running together then share its keys and values in L2.
  // Smaller problems interleave all heads, which keeps the last wave short.
  // Measured, one key head at a time against interleaved: 4096 tokens, H16 d64/128
  // causal: 186 us against 120; 18944 tokens: 1.98 ms against 2.07; 32768 tokens, H32/8
  // d128/128 without a mask: 33.0 ms against 35.2.  (Causal at 24576 and more tokens
  // goes either way: H16/4 d128/128 8.7 ms against 8.4, H16 d64/128 6.8 against 6.9.)
  const int nqt = (pr.NQ + skl::kDiffRows - 1) / skl::kDiffRows;
  p.head_group = nqt >= sms ? pr.H / pr.HK : pr.B * pr.H;
  p.by_group = skl::FastDiv(p.head_group);
  p.by_group_units = skl::FastDiv(static_cast<unsigned>(p.head_group) * nqt * p.nhalf);
  p.wait_limit_ns = skl::api_wait_limit_ns();
  if (skl::launch_diff_fwd(p, pr.d, pr.dv, pr.dtype == STREAMKL_FP16, sms,
                           reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return STREAMKL_ECUDA;
  skl::api_count_launches(1);
  return STREAMKL_OK;
}

size_t streamkl_diff_bwd_workspace_size(const streamkl_diff_problem* prob) {
  if (check_diff(prob) != STREAMKL_OK) return 0;
  const DiffWorkspace w = diff_workspace(*prob);
  return round256((w.rec + w.d2) * sizeof(float));
}

streamkl_status streamkl_diff_bwd(const streamkl_diff_problem* prob, const streamkl_tensor* dO,
                                  const streamkl_tensor* Q1, const streamkl_tensor* K1,
                                  const streamkl_tensor* Q2, const streamkl_tensor* K2,
                                  const streamkl_tensor* V, const streamkl_tensor* lam,
                                  const streamkl_tensor* O, const streamkl_tensor* O2,
                                  const float* LSE1, const float* LSE2, const int* q_lens,
                                  const int* k_lens, const streamkl_tensor* dQ1,
                                  const streamkl_tensor* dK1, const streamkl_tensor* dQ2,
                                  const streamkl_tensor* dK2, const streamkl_tensor* dV,
                                  void* dlam, void* workspace, size_t ws_bytes,
                                  streamkl_stream_t stream) {
  SKL_TRY(check_diff(prob));
  const streamkl_diff_problem& pr = *prob;
  SKL_TRY(check_inputs(pr, Q1, K1, Q2, K2, V, lam, q_lens, k_lens));
  if (!tensor_ok(dO, pr.B, pr.H, pr.NQ) || !tensor_ok(O, pr.B, pr.H, pr.NQ) ||
      !tensor_ok(O2, pr.B, pr.H, pr.NQ) || !same_strides(*O, *O2, pr))
    return STREAMKL_EINVAL;
  if (!LSE1 || !LSE2 || !aligned(LSE1, 4) || !aligned(LSE2, 4)) return STREAMKL_EINVAL;
  if (!dQ1 && !dK1 && !dQ2 && !dK2 && !dV && !dlam) return STREAMKL_EINVAL;
  if ((dQ1 && !tensor_ok(dQ1, pr.B, pr.H, pr.NQ)) || (dQ2 && !tensor_ok(dQ2, pr.B, pr.H, pr.NQ)) ||
      (dK1 && !tensor_ok(dK1, pr.B, pr.HK, pr.NK)) || (dK2 && !tensor_ok(dK2, pr.B, pr.HK, pr.NK)) ||
      (dV && !tensor_ok(dV, pr.B, pr.HK, pr.NK)) || !aligned(dlam, pr.lam_fp32 ? 4 : 2))
    return STREAMKL_EINVAL;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < streamkl_diff_bwd_workspace_size(prob))
    return STREAMKL_EINVAL;
  int sms = 0, *status = nullptr;
  SKL_TRY(skl::api_device(&sms, &status));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f16 = pr.dtype == STREAMKL_FP16;
  const skl::DiffShape shape = shape_of(pr, q_lens, k_lens);
  float* rec = static_cast<float*>(workspace);

  skl::DiffPrepParams pp;
  pp.s = shape;
  pp.lam = lambda_of(*lam, pr.lam_fp32);
  pp.dO = dO->ptr;
  pp.O = O->ptr;
  pp.O2 = O2->ptr;
  pp.sdo = strides_of(*dO);
  pp.so = strides_of(*O);
  pp.LSE1 = LSE1;
  pp.LSE2 = LSE2;
  pp.rec = rec;
  pp.NQpad = padded_rows(pr);
  pp.dv = pr.dv;
  pp.f16 = f16;
  if (skl::launch_diff_prep(pp, s) != cudaSuccess) return STREAMKL_ECUDA;
  skl::api_count_launches(1);

  skl::DiffBwdParams p;
  p.s = shape;
  p.rec = rec;
  p.NQpad = pp.NQpad;
  p.s1 = scale_of(pr.s1, pr.d);
  p.s2 = scale_of(pr.s2, pr.d);
  p.c1 = p.s1 * kLog2e;
  p.c2 = p.s2 * kLog2e;
  p.status = status;
  p.wait_limit_ns = skl::api_wait_limit_ns();
  auto maps = [&](bool kv) -> streamkl_status {
    const int rk = kv ? 128 : 64, rq = kv ? 64 : 128;  // keys resident, queries streamed; or reversed
    SKL_TRY(map_of(*K1, pr.B, pr.HK, pr.NK, pr.d, rk, pr.dtype, kv ? &p.tmR1 : &p.tmC1));
    SKL_TRY(map_of(*K2, pr.B, pr.HK, pr.NK, pr.d, rk, pr.dtype, kv ? &p.tmR2 : &p.tmC2));
    SKL_TRY(map_of(*V, pr.B, pr.HK, pr.NK, pr.dv, rk, pr.dtype, kv ? &p.tmR3 : &p.tmC3));
    SKL_TRY(map_of(*Q1, pr.B, pr.H, pr.NQ, pr.d, rq, pr.dtype, kv ? &p.tmC1 : &p.tmR1));
    SKL_TRY(map_of(*Q2, pr.B, pr.H, pr.NQ, pr.d, rq, pr.dtype, kv ? &p.tmC2 : &p.tmR2));
    SKL_TRY(map_of(*dO, pr.B, pr.H, pr.NQ, pr.dv, rq, pr.dtype, kv ? &p.tmC3 : &p.tmR3));
    return STREAMKL_OK;
  };
  p.after_pass = 0;
  p.d2 = nullptr;
  p.lam_rows = lam->n != 0;
  p.d2_rows = p.lam_rows || pr.NQ == 1;
  auto run = [&](skl::DiffPass pass, int sel, int nhalf, int map0 = 0) -> streamkl_status {
    p.nhalf = nhalf;
    p.by_heads = skl::FastDiv(static_cast<unsigned>(pr.B) * (pass == skl::kDiffKV ? pr.HK : pr.H));
    p.map0 = map0;
    if (skl::launch_diff_bwd(p, pass, pr.d, pr.dv, sel, f16, sms, s) != cudaSuccess)
      return STREAMKL_ECUDA;
    skl::api_count_launches(1);
    p.after_pass = 1;  // the passes share the records and nothing else
    return STREAMKL_OK;
  };
  auto put = [](const streamkl_tensor* t, void** out, skl::Strides* st) {
    *out = t ? const_cast<void*>(t->ptr) : nullptr;
    *st = t ? strides_of(*t) : skl::Strides{0, 0, 0};
  };
  if (dK1 || dK2 || dV) {
    SKL_TRY(maps(true));
    put(dK1, &p.out1, &p.so1);
    put(dK2, &p.out2, &p.so2);
    put(dV, &p.out3, &p.so3);
    if (pr.d == 64) {
      SKL_TRY(run(skl::kDiffKV, 7, 1));
    } else {
      if (pr.dv == 128) {
        if (dK1 || dK2) SKL_TRY(run(skl::kDiffKV, 3, 1));
      } else {
        if (dK1 || dK2) SKL_TRY(run(skl::kDiffKV, 1, dK1 && dK2 ? 2 : 1, dK1 ? 0 : 1));
      }
      if (dV) SKL_TRY(run(skl::kDiffKV, 4, pr.dv / 128));
    }
  }
  if (dQ1 || dQ2 || dlam) {
    SKL_TRY(maps(false));
    put(dQ1, &p.out1, &p.so1);
    put(dQ2, &p.out2, &p.so2);
    put(nullptr, &p.out3, &p.so3);
    if (dlam) p.d2 = rec + diff_workspace(pr).rec;
    const bool map1 = dQ1, map2 = dQ2 || dlam;
    if (pr.dv <= 128) {
      SKL_TRY(run(skl::kDiffQ, 3, 1));
    } else {
      SKL_TRY(run(skl::kDiffQ, 1, map1 && map2 ? 2 : 1, map1 ? 0 : 1));
    }
  }
  if (dlam) {
    skl::DiffLamParams lp;
    lp.d2 = p.d2;
    lp.out = dlam;
    lp.B = pr.B;
    lp.H = pr.H;
    lp.NQ = pr.NQ;
    lp.eb = lam->b ? pr.B : 1;
    lp.eh = lam->h ? pr.H : 1;
    lp.en = lam->n ? pr.NQ : 1;
    lp.f32 = pr.lam_fp32;
    lp.f16 = f16;
    if (skl::launch_diff_lam(lp, s) != cudaSuccess) return STREAMKL_ECUDA;
    skl::api_count_launches(1);
  }
  return STREAMKL_OK;
}

size_t streamkl_paged_workspace_size(const streamkl_paged_problem* prob, int maps) {
  if (check_paged(prob) != STREAMKL_OK || (maps != 1 && maps != 2)) return 0;
  int sms = 0, *status = nullptr;
  if (skl::api_device(&sms, &status) != STREAMKL_OK) return 0;
  return round256(skl::paged_workspace_bytes(prob->dv, maps, sms));
}

streamkl_status streamkl_paged_attn(const streamkl_paged_problem* prob, const streamkl_tensor* Q1,
                                    const streamkl_tensor* K1, const streamkl_tensor* Q2,
                                    const streamkl_tensor* K2, const streamkl_tensor* V,
                                    const streamkl_tensor* lam, const int* table,
                                    int64_t table_stride, const int* lens,
                                    const streamkl_tensor* O, void* workspace, size_t ws_bytes,
                                    streamkl_stream_t stream) {
  SKL_TRY(check_paged(prob));
  const streamkl_paged_problem& pr = *prob;
  const int maps = Q2 ? 2 : 1;
  if ((K2 != nullptr) != (Q2 != nullptr) || (lam != nullptr) != (Q2 != nullptr)) return STREAMKL_EINVAL;
  if (!tensor_ok(Q1, pr.B, pr.H, 1) || !tensor_ok(K1, pr.pages, pr.HK, pr.page_size) ||
      !tensor_ok(V, pr.pages, pr.HK, pr.page_size) || !tensor_ok(O, pr.B, pr.H, 1))
    return STREAMKL_EINVAL;
  if (Q2 && (!tensor_ok(Q2, pr.B, pr.H, 1) || !tensor_ok(K2, pr.pages, pr.HK, pr.page_size) ||
             !lam_ok(lam, pr.lam_fp32)))
    return STREAMKL_EINVAL;
  if (!table || !lens || !aligned(table, 4) || !aligned(lens, 4)) return STREAMKL_EINVAL;
  if (pr.B > 1 && table_stride < pr.max_pages) return STREAMKL_EINVAL;
  if (!workspace || !aligned(workspace, 256)) return STREAMKL_EINVAL;
  skl::PagedParams p;
  int sms = 0;
  SKL_TRY(skl::api_device(&sms, &p.status));
  if (ws_bytes < skl::paged_workspace_bytes(pr.dv, maps, sms)) return STREAMKL_EINVAL;
  auto cache = [](const streamkl_tensor& t) { return skl::PagedCache{t.ptr, t.b, t.n, t.h}; };
  p.Q1 = Q1->ptr;
  p.q1_b = Q1->b;
  p.q1_h = Q1->h;
  p.Q2 = Q2 ? Q2->ptr : nullptr;
  p.q2_b = Q2 ? Q2->b : 0;
  p.q2_h = Q2 ? Q2->h : 0;
  p.K1 = cache(*K1);
  p.K2 = K2 ? cache(*K2) : skl::PagedCache{nullptr, 0, 0, 0};
  p.V = cache(*V);
  p.table = table;
  p.table_stride = table_stride;
  p.lens = lens;
  p.lam = lam ? lambda_of(*lam, pr.lam_fp32) : skl::Lambda{nullptr, 0, 0, 0, 0};
  p.O = const_cast<void*>(O->ptr);
  p.o_b = O->b;
  p.o_h = O->h;
  p.B = pr.B;
  p.H = pr.H;
  p.HK = pr.HK;
  p.pages = pr.pages;
  p.page_size = pr.page_size;
  p.max_pages = pr.max_pages;
  p.page_shift = -1;
  for (int k = 0; k < 31; ++k)
    if (pr.page_size == 1 << k) p.page_shift = k;
  p.c1 = scale_of(pr.s1, pr.d) * kLog2e;
  p.c2 = scale_of(pr.s2, pr.d) * kLog2e;
  p.cuts = static_cast<int4*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + skl::paged_cuts_bytes(sms));
  if (skl::launch_paged(p, pr.d, pr.dv, pr.dtype == STREAMKL_FP16, sms,
                        reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return STREAMKL_ECUDA;
  skl::api_count_launches(2);
  return STREAMKL_OK;
}

streamkl_status streamkl_paged_write(int n, const streamkl_tensor* rows,
                                     const streamkl_tensor* caches, const int* widths,
                                     const void* slots, int slots_int64, int T, int HK, int pages,
                                     int page_size, streamkl_stream_t stream) {
  if (n < 1 || n > skl::kPagedWriteMax || !rows || !caches || !widths) return STREAMKL_EINVAL;
  if (T < 1 || HK < 1 || pages < 1 || page_size < 1 || (slots_int64 & ~1)) return STREAMKL_EINVAL;
  if (static_cast<int64_t>(pages) * page_size > INT32_MAX) return STREAMKL_EINVAL;
  if (!slots || !aligned(slots, slots_int64 ? 8 : 4)) return STREAMKL_EINVAL;
  skl::PagedWriteParams p;
  for (int k = 0; k < n; ++k) {
    if (widths[k] < 8 || widths[k] % 8 != 0 || static_cast<int64_t>(HK) * widths[k] > (1 << 30))
      return STREAMKL_EINVAL;
    if (!tensor_ok(&rows[k], 1, HK, T) || !tensor_ok(&caches[k], pages, HK, page_size))
      return STREAMKL_EINVAL;
    p.rows[k] = rows[k].ptr;
    p.caches[k] = const_cast<void*>(caches[k].ptr);
    p.row_t[k] = rows[k].n * 2;
    p.row_h[k] = rows[k].h * 2;
    p.page[k] = caches[k].b * 2;
    p.slot[k] = caches[k].n * 2;
    p.head[k] = caches[k].h * 2;
    p.vecs[k] = widths[k] / 8;
    p.by_vecs[k] = skl::FastDiv(static_cast<unsigned>(p.vecs[k]));
    p.by_token[k] = skl::FastDiv(static_cast<unsigned>(HK * p.vecs[k]));
  }
  p.slots = slots;
  p.slots64 = slots_int64;
  p.by_page = skl::FastDiv(static_cast<unsigned>(page_size));
  p.n = n;
  p.T = T;
  p.HK = HK;
  p.pages = pages;
  p.page_size = page_size;
  int sms = 0;
  SKL_TRY(skl::api_device(&sms, &p.status));
  if (skl::launch_paged_write(p, sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return STREAMKL_ECUDA;
  skl::api_count_launches(1);
  return STREAMKL_OK;
}

}  // extern "C"
