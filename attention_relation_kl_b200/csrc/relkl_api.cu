// Host side of the C ABI declared in include/relkl.h: argument validation,
// TMA descriptor encoding, kernel selection and launch.  No allocation and no
// state survives a call except two process-wide settings (the wait timeout
// and a per-device SM-count cache).
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/relkl.h"
#include "relkl_device.cuh"
#include "relkl_params.h"
#include "relkl_ranges.h"

namespace relkl {
cudaError_t tc_launch_fwd(const TcParams& p, int d, int grid, cudaStream_t stream);
cudaError_t tc_launch_bwd(const TcParams& p, int d, int grid, cudaStream_t stream);
cudaError_t simt_launch_fwd(const SimtParams& p, cudaStream_t stream);
cudaError_t simt_launch_bwd(const SimtParams& p, cudaStream_t stream);
cudaError_t launch_zero(float* ptr, int64_t n, int num_sms, cudaStream_t stream);
cudaError_t launch_cast_bf16(const float* src, void* dst, int64_t n, int num_sms,
                             cudaStream_t stream);
int schedule_check(const TcParams& p0, int d, bool bwd, int n_parts, const int* const* lens,
                   const int* const* offs, char* why, size_t why_len);
int tc_bwd_kind(const TcParams& p, int d, int sms);
cudaError_t launch_rope_bwd(const float* dx, void* out, int B, int H, int N, int d, bool bf16_out,
                            double base, double pos_scale, double pos_offset, int apply,
                            cudaStream_t stream);
cudaError_t launch_rotary(RotaryParams& p, bool x_bf16, bool y_bf16, bool interleaved,
                          int num_sms, cudaStream_t stream);
cudaError_t launch_adamw(const AdamwTensor* t, int n, const AdamwPlan& plan, bool bits8,
                         cudaStream_t stream);
int64_t norm_chunks(int64_t n, bool bf16);
cudaError_t launch_grad_norm(const NormTensor* t, int n, int64_t chunks, int grid, double* partial,
                             float* out, float max_norm, cudaStream_t stream);
cudaError_t launch_norm_finish(const double* partial, int n, float max_norm, float* out,
                               cudaStream_t stream);
cudaError_t launch_quantize_rows(const RowsParams& p, bool x_bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_gemv_i8(const GemvParams& p, bool x_bf16, bool y_bf16, int num_sms,
                           cudaStream_t stream);
cudaError_t launch_gemm_i8(I8Params& p, const I8Call& c, bool y_bf16, int num_sms, cudaStream_t stream);
using EncodeTiledFnG = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                    const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                    const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                    CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
int launch_wgrad(EncodeTiledFnG encode, long long rows, int D, int cols, const void* h,
                 const void* dx_pre, float* dw, int num_sms, DevStatus* status,
                 unsigned long long timeout_ns, cudaStream_t stream);
}  // namespace relkl

using namespace relkl;

namespace {

constexpr size_t kWorkspaceBytes = 256;
std::atomic<unsigned long long> g_timeout_ns{2000000000ull};
thread_local int32_t g_last_cuda = 0;

relkl_status cuda_fail(cudaError_t e) {
  g_last_cuda = static_cast<int32_t>(e);
  return RELKL_ERR_CUDA;
}

// NVTX range over the host side of one entry point (validation, descriptor
// encoding, launches), so that a profiler timeline shows which call queued
// which kernels.  NVTX3 is header-only: without an attached tool the push and
// pop are a load and a branch.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// cuTensorMapEncodeTiled, fetched from the driver through the runtime so the
// library needs no link-time dependency on libcuda.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;
std::once_flag g_encode_once;

EncodeTiledFn encode_fn() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  });
  return g_encode;
}

struct DevInfo {
  int sms = 0;
  int major = 0;
};
DevInfo g_dev[64];
std::mutex g_dev_mu;

relkl_status device_info(DevInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return RELKL_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (g_dev[dev].sms == 0) {
    int sms = 0, major = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e);
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) !=
        cudaSuccess)
      return cuda_fail(e);
    g_dev[dev].sms = sms;
    g_dev[dev].major = major;
  }
  *out = g_dev[dev];
  return RELKL_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Units of a desc: (b, h) of its [B, H, N, d] tensors, or (sequence, head)
// of packed sequences.
int64_t n_units(const relkl_desc& d) {
  return static_cast<int64_t>(d.cu_seqlens ? d.n_seq : d.B) * d.H;
}

relkl_status check_desc(const relkl_desc* d) {
  if (!d) return RELKL_ERR_INVALID;
  if (d->B < 0 || d->H < 0 || d->N < 0 || d->d < 1) return RELKL_ERR_INVALID;
  if (d->dtype != RELKL_BF16 && d->dtype != RELKL_FP32) return RELKL_ERR_INVALID;
  if (d->causal != 0 && d->causal != 1) return RELKL_ERR_INVALID;
  if (d->reserved != 0) return RELKL_ERR_INVALID;
  if (d->lengths && !aligned(d->lengths, 4)) return RELKL_ERR_INVALID;
  if (d->cu_seqlens) {
    if (!aligned(d->cu_seqlens, 4) || d->lengths || d->B != 1 || d->n_seq < 0 ||
        d->max_seqlen < 0 || d->max_seqlen > d->N)
      return RELKL_ERR_INVALID;
  } else if (d->n_seq != 0 || d->max_seqlen != 0) {
    return RELKL_ERR_INVALID;
  }
  if (!(d->scale >= 0.f) || !std::isfinite(d->scale)) return RELKL_ERR_INVALID;
  if (d->stride[3] != 1) return RELKL_ERR_INVALID;
  for (int i = 0; i < 3; ++i)
    if (d->stride[i] < 0) return RELKL_ERR_INVALID;
  if (d->d > 128) return RELKL_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->N) * d->d >= (int64_t(1) << 31)) return RELKL_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->B) * d->H * d->N >= (int64_t(1) << 40)) return RELKL_ERR_UNSUPPORTED;
  return RELKL_OK;
}

bool tc_shape(const relkl_desc& d) {
  return d.dtype == RELKL_BF16 && (d.d == 64 || d.d == 128);
}

// Tensor-core path needs 16-byte aligned bases and strides (TMA).
bool tc_layout_ok(const relkl_desc& d, const void* xt, const void* xs) {
  if (!aligned(xt, 16) || !aligned(xs, 16)) return false;
  for (int i = 0; i < 3; ++i)
    if ((d.stride[i] * 2) % 16 != 0) return false;
  return true;
}

float logit_scale(const relkl_desc& d) {
  return d.scale > 0.f ? d.scale : 1.0f / std::sqrt(static_cast<float>(d.d));
}

relkl_status encode_x(CUtensorMap* m, const relkl_desc& d, const void* x, cuuint32_t box_rows = 128) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return RELKL_ERR_CUDA;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d.d), static_cast<cuuint64_t>(d.N),
                              static_cast<cuuint64_t>(d.H), static_cast<cuuint64_t>(d.B)};
  // a dimension of extent 1 may carry any stride; give it a legal one
  auto stride_or = [&](int i, int64_t fallback) {
    return static_cast<cuuint64_t>((d.stride[i] > 0 ? d.stride[i] : fallback) * 2);
  };
  const int64_t row = d.stride[2] > 0 ? d.stride[2] : d.d;
  const cuuint64_t strides[3] = {stride_or(2, d.d), stride_or(1, row * d.N),
                                 stride_or(0, row * d.N * d.H)};
  const cuuint32_t box[4] = {64, box_rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? RELKL_OK : RELKL_ERR_UNSUPPORTED;
}

// dX [B,H,N,d] f32 contiguous: 4-D map, box 32 cols x 32 rows, 128B swizzle,
// the target of the backward's TMA reduce-adds.
relkl_status encode_dx(CUtensorMap* m, const relkl_desc& d, float* dx) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return RELKL_ERR_CUDA;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d.d), static_cast<cuuint64_t>(d.N),
                              static_cast<cuuint64_t>(d.H), static_cast<cuuint64_t>(d.B)};
  const cuuint64_t row = static_cast<cuuint64_t>(d.d) * 4;
  const cuuint64_t strides[3] = {row, row * d.N, row * d.N * d.H};
  const cuuint32_t box[4] = {32, 32, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, dx, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? RELKL_OK : RELKL_ERR_UNSUPPORTED;
}

relkl_status check_ws(const void* ws, size_t ws_bytes) {
  if (!ws || ws_bytes < kWorkspaceBytes || !aligned(ws, 256)) return RELKL_ERR_WORKSPACE;
  return RELKL_OK;
}

// Common validation of a multi-relation call.  Sets *empty when there is no
// work at all.
relkl_status check_multi(int32_t n_rel, const relkl_desc* descs, const void* const* xt,
                         const void* const* xs, bool* empty) {
  if (n_rel < 1 || n_rel > kMaxSeg || !descs || !xt || !xs) return RELKL_ERR_INVALID;
  int64_t units = 0;
  for (int r = 0; r < n_rel; ++r) {
    relkl_status s = check_desc(&descs[r]);
    if (s != RELKL_OK) return s;
    const relkl_desc& a = descs[0];
    const relkl_desc& b = descs[r];
    if (a.N != b.N || a.d != b.d || a.dtype != b.dtype || a.causal != b.causal ||
        a.scale != b.scale || (a.cu_seqlens == nullptr) != (b.cu_seqlens == nullptr) ||
        a.max_seqlen != b.max_seqlen)
      return RELKL_ERR_INVALID;
    units += n_units(b);
  }
  if (units >= (int64_t(1) << 30)) return RELKL_ERR_UNSUPPORTED;
  *empty = (units == 0 || descs[0].N == 0 || (descs[0].cu_seqlens && descs[0].max_seqlen == 0));
  if (*empty) return RELKL_OK;
  for (int r = 0; r < n_rel; ++r) {
    if (n_units(descs[r]) == 0) continue;
    if (!xt[r] || !xs[r]) return RELKL_ERR_INVALID;
    const size_t es = descs[r].dtype == RELKL_BF16 ? 2 : 4;
    if (!aligned(xt[r], es) || !aligned(xs[r], es)) return RELKL_ERR_INVALID;
  }
  return RELKL_OK;
}

bool use_tc(int32_t n_rel, const relkl_desc* descs, const void* const* xt, const void* const* xs) {
  if (!tc_shape(descs[0])) return false;
  for (int r = 0; r < n_rel; ++r)
    if (n_units(descs[r]) && !tc_layout_ok(descs[r], xt[r], xs[r])) return false;
  return true;
}

// The schedule fields of a tensor-core launch (everything but the tensor
// maps and pointers): shared by the launch and the host schedule check.
void fill_schedule(int32_t n_rel, const relkl_desc* descs, TcParams* p, int part, int n_parts) {
  std::memset(p, 0, sizeof(*p));
  const relkl_desc& d0 = descs[0];
  int seg = 0, ub = 0;
  for (int r = 0; r < n_rel; ++r) {
    if (n_units(descs[r]) == 0) continue;
    TcSeg& s = p->seg[seg];
    s.B = descs[r].cu_seqlens ? descs[r].n_seq : descs[r].B;
    s.H = descs[r].H;
    s.lengths = descs[r].lengths;
    s.cu_seqlens = descs[r].cu_seqlens;
    s.max_seqlen = descs[r].max_seqlen;
    s.unit_begin = ub;
    ub += static_cast<int>(n_units(descs[r]));
    ++seg;
  }
  p->n_seg = seg;
  p->N = d0.N;
  // rows a unit's work covers: every row, or at most max_seqlen of a packed sequence
  const int span = d0.cu_seqlens ? d0.max_seqlen : d0.N;
  p->nblk = (span + 127) / 128;
  p->n_pairs = (p->nblk + 1) / 2;
  p->n_units = ub;
  p->part = part;
  p->n_parts = n_parts;
  p->n_local = part < p->n_pairs ? (p->n_pairs - part + n_parts - 1) / n_parts : 0;
  p->n_items = ub * p->n_local;
  p->causal = d0.causal;
  p->scale = logit_scale(d0);
  p->sl2 = p->scale * 1.4426950408889634f;
}

relkl_status build_tc(int32_t n_rel, const relkl_desc* descs, const void* const* xt,
                      const void* const* xs, TcParams* p, void* ws, int part = 0,
                      int n_parts = 1) {
  fill_schedule(n_rel, descs, p, part, n_parts);
  for (int r = 0, seg = 0; r < n_rel; ++r) {
    if (n_units(descs[r]) == 0) continue;
    TcSeg& s = p->seg[seg++];
    relkl_status st = encode_x(&s.tm_t, descs[r], xt[r]);
    if (st != RELKL_OK) return st;
    if ((st = encode_x(&s.tm_s, descs[r], xs[r])) != RELKL_OK) return st;
  }
  p->status = reinterpret_cast<DevStatus*>(ws);
  p->timeout_ns = g_timeout_ns.load();
  return RELKL_OK;
}

relkl_status build_simt(int32_t n_rel, const relkl_desc* descs, const void* const* xt,
                        const void* const* xs, SimtParams* p, int part = 0, int n_parts = 1) {
  std::memset(p, 0, sizeof(*p));
  const relkl_desc& d0 = descs[0];
  int seg = 0, ub = 0;
  for (int r = 0; r < n_rel; ++r) {
    if (n_units(descs[r]) == 0) continue;
    SimtSeg& s = p->seg[seg];
    s.xt = xt[r];
    s.xs = xs[r];
    s.sb = descs[r].stride[0];
    s.sh = descs[r].stride[1];
    s.sn = descs[r].stride[2];
    s.B = descs[r].cu_seqlens ? descs[r].n_seq : descs[r].B;
    s.H = descs[r].H;
    s.lengths = descs[r].lengths;
    s.cu_seqlens = descs[r].cu_seqlens;
    s.max_seqlen = descs[r].max_seqlen;
    s.unit_begin = ub;
    ub += static_cast<int>(n_units(descs[r]));
    ++seg;
  }
  p->n_seg = seg;
  p->N = d0.N;
  p->d = d0.d;
  p->causal = d0.causal;
  p->is_bf16 = d0.dtype == RELKL_BF16;
  p->scale = logit_scale(d0);
  p->n_units = ub;
  p->part = part;
  p->n_parts = n_parts;
  const int nblk32 = ((d0.cu_seqlens ? d0.max_seqlen : d0.N) + 31) / 32;
  p->nblk_local = part < nblk32 ? (nblk32 - part + n_parts - 1) / n_parts : 0;
  return RELKL_OK;
}

// ---- rotary positions
// A difference of two rows' indices in one direction: lo..hi steps.
struct Steps {
  int64_t stride, lo, hi;
};

// Whether numbers of steps exist whose sum lies in [from, to].  Steps come by
// falling stride, so few numbers of one leave the rest in reach (one or two,
// where both tensors have the same strides); `left` bounds the search, and what
// it does not settle counts as found.
bool steps_reach(const Steps* s, int n, int64_t from, int64_t to, int& left) {
  if (n == 0) return from <= 0 && to >= 0;
  int64_t least = 0, most = 0;      // of the steps behind this one
  for (int k = 1; k < n; ++k) {
    least += s[k].lo * s[k].stride;
    most += s[k].hi * s[k].stride;
  }
  auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
  const int64_t first = std::max(s->lo, -floor_div(most - from, s->stride));
  const int64_t last = std::min(s->hi, floor_div(to - least, s->stride));
  for (int64_t m = first; m <= last; ++m) {
    if (--left < 0) return true;
    if (steps_reach(s + 1, n - 1, from - m * s->stride, to - m * s->stride, left)) return true;
  }
  return false;
}

// Whether two outputs of a call have an element in common; b begins `apart`
// elements behind a.
bool rows_meet(const RotaryTensor& a, const RotaryTensor& b, const relkl_rotary_plan& plan, int64_t apart) {
  Steps s[6];
  int n = 0;
  const int64_t ea[3] = {plan.B, a.H, plan.N}, eb[3] = {plan.B, b.H, plan.N};
  auto add = [&](int64_t stride, int64_t lo, int64_t hi) {
    if (stride == 0) return;        // one row only
    for (int k = 0; k < n; ++k)
      if (s[k].stride == stride) {
        s[k].lo += lo;
        s[k].hi += hi;
        return;
      }
    s[n++] = Steps{stride, lo, hi};
  };
  for (int i = 0; i < 3; ++i) {
    add(a.ys[i], 0, ea[i] - 1);
    add(b.ys[i], 1 - eb[i], 0);
  }
  std::sort(s, s + n, [](const Steps& x, const Steps& y) { return x.stride > y.stride; });
  int left = 20000;
  return steps_reach(s, n, apart - (plan.d - 1), apart + (plan.d - 1), left);
}

// ---- products in 8-bit integers
constexpr int64_t kMostStride = int64_t(1) << 48;   // keeps every offset far below 2^63

bool element_type(int32_t t) { return t == RELKL_BF16 || t == RELKL_FP32; }
size_t element_size(int32_t t) { return t == RELKL_BF16 ? 2 : 4; }

bool rows_ok(int64_t rows, int32_t K) {
  return rows >= 0 && rows <= (int64_t(1) << 31) && K > 0 && K < 131072;
}
bool codes_ok(const int8_t* q, int64_t stride, int32_t K) {
  return q && aligned(q, 16) && stride >= K && stride % 16 == 0 && stride <= (int64_t(1) << 39);
}
bool matrix_ok(const void* x, int32_t dtype, int64_t stride, int32_t K) {
  return x && element_type(dtype) && aligned(x, element_size(dtype)) && stride >= K &&
         stride <= kMostStride;
}
// rows of a matrix start at boundaries of 16 (or so many) bytes
bool wide_rows(const void* x, int32_t dtype, int64_t stride, int bytes = 16) {
  return aligned(x, bytes) && stride * static_cast<int64_t>(element_size(dtype)) % bytes == 0;
}
// rows of codes start at 128-byte lines, short ones at 16 bytes
int64_t code_pitch(int32_t K) {
  const int64_t line = K >= 128 ? 128 : 16;
  return (K + line - 1) / line * line;
}
bool few_rows(int64_t rows, int32_t K) {
  return rows <= kGemvRows && rows * code_pitch(K) <= kGemvBytes;
}

relkl_status matmul_i8(int64_t rows, int32_t cols, int32_t K, const int8_t* q, int64_t q_stride,
                       const float* q_scale, const int8_t* w, int64_t w_stride,
                       const float* w_scale, const float* bias, void* y, int32_t y_dtype,
                       int64_t y_stride, void* ws, bool after_rows, const DevInfo& dev,
                       cudaStream_t stream) {
  if (dev.major != 10) return RELKL_ERR_UNSUPPORTED;
  I8Call c = {q, w, q_stride, w_stride, K, after_rows, encode_fn()};
  if (!c.encode) return RELKL_ERR_CUDA;
  I8Params p;
  std::memset(&p, 0, sizeof(p));
  p.x_scale = q_scale;
  p.w_scale = w_scale;
  p.bias = bias;
  p.y = y;
  p.rows = rows;
  p.y_stride = y_stride;
  p.cols = cols;
  p.y_wide = wide_rows(y, y_dtype, y_stride, 32) ? 2 : wide_rows(y, y_dtype, y_stride);
  p.status = reinterpret_cast<DevStatus*>(ws);
  p.timeout_ns = g_timeout_ns.load();
  cudaError_t e = launch_gemm_i8(p, c, y_dtype == RELKL_BF16, dev.sms, stream);
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

relkl_status quantize_rows(int64_t rows, int32_t K, const void* x, int32_t x_dtype, int64_t x_stride,
                           int8_t* q, int64_t q_stride, float* scale, const DevInfo& dev,
                           cudaStream_t stream) {
  RowsParams p = {x, q, scale, rows, x_stride, q_stride, K, wide_rows(x, x_dtype, x_stride)};
  cudaError_t e = launch_quantize_rows(p, x_dtype == RELKL_BF16, dev.sms, stream);
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

// Index of relation r's segment (relations without units have none).
template <class P>
void set_seg_outputs(P* p, int32_t n_rel, const relkl_desc* descs, float* const* kl,
                     float* const* stats, const float* const* stats_in, const float* const* dkl,
                     float* const* dx) {
  int seg = 0;
  for (int r = 0; r < n_rel; ++r) {
    if (n_units(descs[r]) == 0) continue;
    auto& s = p->seg[seg++];
    if (kl) s.kl = kl[r];
    if (stats) s.stats = stats[r];
    if (stats_in) s.stats = const_cast<float*>(stats_in[r]);
    s.dkl = dkl ? dkl[r] : nullptr;
    if (dx) s.dx = dx[r];
  }
}

}  // namespace

extern "C" {

size_t relkl_workspace_bytes(void) { return kWorkspaceBytes; }

relkl_status relkl_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  relkl_status s = check_ws(ws, ws_bytes);
  if (s != RELKL_OK) return s;
  cudaError_t e = cudaMemsetAsync(ws, 0, kWorkspaceBytes, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

int32_t relkl_path_for(const relkl_desc* desc) {
  if (check_desc(desc) != RELKL_OK) return 0;
  return tc_shape(*desc) ? 1 : 2;
}

}  // extern "C"

namespace {

#ifdef RELKL_CHECKS
// Debug builds (-DRELKL_CHECKS): replay the launch's schedule on the host
// before enqueueing it (synchronous copies of lengths / packed offsets).
relkl_status debug_schedule_check(int32_t n_rel, const relkl_desc* descs, bool bwd, int part,
                                  int n_parts) {
  std::vector<std::vector<int32_t>> lens(n_rel), offs(n_rel);
  const int32_t* lp[kMaxSeg] = {nullptr, nullptr, nullptr};
  const int32_t* op[kMaxSeg] = {nullptr, nullptr, nullptr};
  for (int r = 0; r < n_rel; ++r) {
    if (descs[r].lengths) {
      lens[r].resize(descs[r].B);
      if (cudaMemcpy(lens[r].data(), descs[r].lengths, 4 * descs[r].B, cudaMemcpyDeviceToHost) !=
          cudaSuccess)
        return RELKL_ERR_CUDA;
      lp[r] = lens[r].data();
    }
    if (descs[r].cu_seqlens) {
      offs[r].resize(descs[r].n_seq + 1);
      if (cudaMemcpy(offs[r].data(), descs[r].cu_seqlens, 4 * (descs[r].n_seq + 1),
                     cudaMemcpyDeviceToHost) != cudaSuccess)
        return RELKL_ERR_CUDA;
      op[r] = offs[r].data();
    }
  }
  (void)part;
  char why[256];
  return relkl_check_schedule(n_rel, descs, bwd ? 1 : 0, n_parts, lp, op, why, sizeof why);
}
#endif

relkl_status fwd_impl(int32_t n_rel, const relkl_desc* descs, const void* const* x_t,
                      const void* const* x_s, float* const* kl, float* const* stats, int32_t part,
                      int32_t n_parts, void* ws, size_t ws_bytes, void* stream) {
  if (n_parts < 1 || part < 0 || part >= n_parts) return RELKL_ERR_INVALID;
  bool empty = false;
  relkl_status s = check_multi(n_rel, descs, x_t, x_s, &empty);
  if (s != RELKL_OK || empty) return s;
  if (!kl || !stats) return RELKL_ERR_INVALID;
  for (int r = 0; r < n_rel; ++r)
    if (n_units(descs[r]) && (!kl[r] || !stats[r] || !aligned(kl[r], 4) || !aligned(stats[r], 16)))
      return RELKL_ERR_INVALID;
  if ((s = check_ws(ws, ws_bytes)) != RELKL_OK) return s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  if (dev.major != 10) return RELKL_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (use_tc(n_rel, descs, x_t, x_s)) {
#ifdef RELKL_CHECKS
    if ((s = debug_schedule_check(n_rel, descs, false, part, n_parts)) != RELKL_OK) return s;
#endif
    TcParams p;
    if ((s = build_tc(n_rel, descs, x_t, x_s, &p, ws, part, n_parts)) != RELKL_OK) return s;
    set_seg_outputs(&p, n_rel, descs, kl, stats, nullptr, nullptr, nullptr);
    if (p.n_items == 0) return RELKL_OK;   // this part holds no work item
    const int grid = p.n_items < dev.sms ? p.n_items : dev.sms;
    e = tc_launch_fwd(p, descs[0].d, grid, st);
  } else {
    SimtParams p;
    build_simt(n_rel, descs, x_t, x_s, &p, part, n_parts);
    set_seg_outputs(&p, n_rel, descs, kl, stats, nullptr, nullptr, nullptr);
    e = simt_launch_fwd(p, st);
  }
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

relkl_status bwd_impl(int32_t n_rel, const relkl_desc* descs, const void* const* x_t,
                      const void* const* x_s, const float* const* stats, const float* const* dkl,
                      float* const* dx_s, int32_t part, int32_t n_parts, void* ws,
                      size_t ws_bytes, void* stream) {
  if (n_parts < 1 || part < 0 || part >= n_parts) return RELKL_ERR_INVALID;
  bool empty = false;
  relkl_status s = check_multi(n_rel, descs, x_t, x_s, &empty);
  if (s != RELKL_OK || empty) return s;
  if (!stats || !dx_s) return RELKL_ERR_INVALID;
  for (int r = 0; r < n_rel; ++r) {
    if (!n_units(descs[r])) continue;
    if (!stats[r] || !dx_s[r] || !aligned(stats[r], 16) || !aligned(dx_s[r], 16))
      return RELKL_ERR_INVALID;
    if (dkl && dkl[r] && !aligned(dkl[r], 4)) return RELKL_ERR_INVALID;
  }
  if ((s = check_ws(ws, ws_bytes)) != RELKL_OK) return s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  if (dev.major != 10) return RELKL_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool tc = use_tc(n_rel, descs, x_t, x_s);
  TcParams tp;
  SimtParams sp;
  if (tc) {
#ifdef RELKL_CHECKS
    if ((s = debug_schedule_check(n_rel, descs, true, part, n_parts)) != RELKL_OK) return s;
#endif
    if ((s = build_tc(n_rel, descs, x_t, x_s, &tp, ws, part, n_parts)) != RELKL_OK) return s;
    set_seg_outputs(&tp, n_rel, descs, nullptr, nullptr, stats, dkl, dx_s);
    for (int r = 0, seg = 0; r < n_rel; ++r) {
      if (!n_units(descs[r])) continue;
      TcSeg& sg = tp.seg[seg++];
      if ((s = encode_dx(&sg.tm_dx, descs[r], dx_s[r])) != RELKL_OK) return s;
      // 64-row boxes for the column tiles of the d = 128 backward
      if ((s = encode_x(&sg.tm_t64, descs[r], x_t[r], 64)) != RELKL_OK) return s;
      if ((s = encode_x(&sg.tm_s64, descs[r], x_s[r], 64)) != RELKL_OK) return s;
    }
  } else {
    build_simt(n_rel, descs, x_t, x_s, &sp, part, n_parts);
    set_seg_outputs(&sp, n_rel, descs, nullptr, nullptr, stats, dkl, dx_s);
  }
  // dX_s is accumulated by reduce-adds in L2: clear it first (same stream)
  for (int r = 0; r < n_rel; ++r) {
    if (!n_units(descs[r])) continue;
    // the whole [B, H, N, d] tensor (packed sequences: B = 1, every token)
    const int64_t n = static_cast<int64_t>(descs[r].B) * descs[r].H * descs[r].N * descs[r].d;
    if ((e = launch_zero(dx_s[r], n, dev.sms, st)) != cudaSuccess) return cuda_fail(e);
  }
  if (tc) {
    // the launcher sizes the grid (at most one CTA per SM) from the work items
    // of the kernel it picks; a part without items launches nothing
    e = tc_launch_bwd(tp, descs[0].d, dev.sms, st);
  } else {
    e = simt_launch_bwd(sp, st);
  }
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

relkl_status relkl_fwd_qkv(int32_t n_rel, const relkl_desc* descs, const void* const* x_t,
                           const void* const* x_s, float* const* kl, float* const* stats,
                           void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("relkl_fwd_qkv");
  return fwd_impl(n_rel, descs, x_t, x_s, kl, stats, 0, 1, ws, ws_bytes, stream);
}

relkl_status relkl_bwd_qkv(int32_t n_rel, const relkl_desc* descs, const void* const* x_t,
                           const void* const* x_s, const float* const* stats,
                           const float* const* dkl, float* const* dx_s, void* ws,
                           size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("relkl_bwd_qkv");
  return bwd_impl(n_rel, descs, x_t, x_s, stats, dkl, dx_s, 0, 1, ws, ws_bytes, stream);
}

relkl_status relkl_fwd_qkv_part(int32_t n_rel, const relkl_desc* descs, const void* const* x_t,
                                const void* const* x_s, float* const* kl, float* const* stats,
                                int32_t part, int32_t n_parts, void* ws, size_t ws_bytes,
                                void* stream) {
  NvtxRange nvtx_range("relkl_fwd_qkv_part");
  return fwd_impl(n_rel, descs, x_t, x_s, kl, stats, part, n_parts, ws, ws_bytes, stream);
}

relkl_status relkl_bwd_qkv_part(int32_t n_rel, const relkl_desc* descs, const void* const* x_t,
                                const void* const* x_s, const float* const* stats,
                                const float* const* dkl, float* const* dx_s, int32_t part,
                                int32_t n_parts, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("relkl_bwd_qkv_part");
  return bwd_impl(n_rel, descs, x_t, x_s, stats, dkl, dx_s, part, n_parts, ws, ws_bytes, stream);
}

relkl_status relkl_fwd(const relkl_desc* desc, const void* x_t, const void* x_s, float* kl,
                       float* stats, void* ws, size_t ws_bytes, void* stream) {
  const void* xt[1] = {x_t};
  const void* xs[1] = {x_s};
  float* k[1] = {kl};
  float* st[1] = {stats};
  return relkl_fwd_qkv(1, desc, xt, xs, k, st, ws, ws_bytes, stream);
}

relkl_status relkl_bwd(const relkl_desc* desc, const void* x_t, const void* x_s,
                       const float* stats, const float* dkl, float* dx_s, void* ws,
                       size_t ws_bytes, void* stream) {
  const void* xt[1] = {x_t};
  const void* xs[1] = {x_s};
  const float* st[1] = {stats};
  const float* g[1] = {dkl};
  float* dx[1] = {dx_s};
  return relkl_bwd_qkv(1, desc, xt, xs, st, g, dx, ws, ws_bytes, stream);
}

relkl_status relkl_get_device_error(const void* ws, void* stream, uint32_t* where) {
  if (where) *where = 0;
  relkl_status s = check_ws(ws, kWorkspaceBytes);
  if (s != RELKL_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e);
  DevStatus rec;
  e = cudaMemcpy(&rec, ws, sizeof(rec), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e);
  if (where) *where = rec.where;
  return rec.code == 0 ? RELKL_OK : RELKL_ERR_TIMEOUT;
}

uint64_t relkl_set_wait_timeout_ns(uint64_t ns) { return g_timeout_ns.exchange(ns); }

const char* relkl_status_string(relkl_status s) {
  switch (s) {
    case RELKL_OK: return "RELKL_OK";
    case RELKL_ERR_INVALID: return "RELKL_ERR_INVALID: invalid argument";
    case RELKL_ERR_UNSUPPORTED: return "RELKL_ERR_UNSUPPORTED: unsupported shape, layout or device";
    case RELKL_ERR_CUDA: return "RELKL_ERR_CUDA: a CUDA call failed";
    case RELKL_ERR_WORKSPACE: return "RELKL_ERR_WORKSPACE: workspace missing, misaligned or too small";
    case RELKL_ERR_TIMEOUT: return "RELKL_ERR_TIMEOUT: a bounded device wait ran out";
  }
  return "RELKL_ERR_UNKNOWN";
}

int32_t relkl_last_cuda_error(void) { return g_last_cuda; }

relkl_status relkl_check_schedule(int32_t n_rel, const relkl_desc* descs, int32_t is_bwd,
                                  int32_t n_parts, const int32_t* const* host_lengths,
                                  const int32_t* const* host_cu_seqlens, char* why,
                                  size_t why_len) {
  if (why && why_len) why[0] = 0;
  if (n_rel < 1 || n_rel > kMaxSeg || !descs || n_parts < 1) return RELKL_ERR_INVALID;
  int64_t units = 0;
  for (int r = 0; r < n_rel; ++r) {
    relkl_status s = check_desc(&descs[r]);
    if (s != RELKL_OK) return s;
    if (descs[r].N != descs[0].N || descs[r].causal != descs[0].causal ||
        (descs[r].cu_seqlens == nullptr) != (descs[0].cu_seqlens == nullptr) ||
        descs[r].max_seqlen != descs[0].max_seqlen || descs[r].d != descs[0].d)
      return RELKL_ERR_INVALID;
    if ((descs[r].lengths && (!host_lengths || !host_lengths[r])) ||
        (descs[r].cu_seqlens && (!host_cu_seqlens || !host_cu_seqlens[r])))
      return RELKL_ERR_INVALID;
    units += n_units(descs[r]);
  }
  if (!tc_shape(descs[0])) return RELKL_ERR_UNSUPPORTED;
  if (units == 0 || descs[0].N == 0) return RELKL_OK;
  TcParams p;
  fill_schedule(n_rel, descs, &p, 0, 1);
  // host copies in the launch's segment order (relations without units have none)
  const int* lens[kMaxSeg] = {nullptr, nullptr, nullptr};
  const int* offs[kMaxSeg] = {nullptr, nullptr, nullptr};
  for (int r = 0, seg = 0; r < n_rel; ++r) {
    if (n_units(descs[r]) == 0) continue;
    lens[seg] = host_lengths ? host_lengths[r] : nullptr;
    offs[seg] = host_cu_seqlens ? host_cu_seqlens[r] : nullptr;
    ++seg;
  }
  return schedule_check(p, descs[0].d, is_bwd != 0, n_parts, lens, offs, why, why_len) == 0
             ? RELKL_OK
             : RELKL_ERR_INVALID;
}

int32_t relkl_bwd_kernel_for(int32_t n_rel, const relkl_desc* descs, int32_t n_sms) {
  if (n_rel < 1 || n_rel > kMaxSeg || !descs || n_sms < 1) return 0;
  for (int r = 0; r < n_rel; ++r) {
    if (check_desc(&descs[r]) != RELKL_OK) return 0;
    if (descs[r].N != descs[0].N || descs[r].causal != descs[0].causal ||
        (descs[r].cu_seqlens == nullptr) != (descs[0].cu_seqlens == nullptr) ||
        descs[r].max_seqlen != descs[0].max_seqlen || descs[r].d != descs[0].d)
      return 0;
  }
  if (!tc_shape(descs[0])) return 1;
  TcParams p;
  fill_schedule(n_rel, descs, &p, 0, 1);
  return tc_bwd_kind(p, descs[0].d, n_sms);
}

relkl_status relkl_rope_bwd(int32_t B, int32_t H, int32_t N, int32_t d, const float* dx_post,
                            const relkl_rope* rope, int32_t out_dtype, void* dx_pre,
                            void* stream) {
  NvtxRange nvtx_range("relkl_rope_bwd");
  if (!rope || B < 0 || H < 0 || N < 0 || d < 2 || d > 512 || (d & 1)) return RELKL_ERR_INVALID;
  if (out_dtype != RELKL_BF16 && out_dtype != RELKL_FP32) return RELKL_ERR_INVALID;
  if (rope->reserved != 0 || (rope->apply != 0 && rope->apply != 1)) return RELKL_ERR_INVALID;
  if (!std::isfinite(rope->base) || !(rope->base > 1.0) || !std::isfinite(rope->pos_scale) ||
      !std::isfinite(rope->pos_offset))
    return RELKL_ERR_INVALID;
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens == 0 || H == 0) return RELKL_OK;
  if (tokens > 0x7fffffffLL) return RELKL_ERR_INVALID;
  if (!dx_post || !dx_pre || !aligned(dx_post, 4) || !aligned(dx_pre, out_dtype == RELKL_BF16 ? 2 : 4))
    return RELKL_ERR_INVALID;
  cudaError_t e = launch_rope_bwd(dx_post, dx_pre, B, H, N, d, out_dtype == RELKL_BF16, rope->base,
                                  rope->pos_scale, rope->pos_offset, rope->apply,
                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

relkl_status relkl_rotary(int32_t n_tensors, const relkl_rotary_tensor* tensors,
                          const relkl_rotary_plan* plan, void* stream) {
  NvtxRange nvtx_range("relkl_rotary");
  if (n_tensors < 1 || n_tensors > kMaxSeg || !tensors || !plan) return RELKL_ERR_INVALID;
  const relkl_rotary_plan& a = *plan;
  if (a.B < 0 || a.N < 0 || a.d < 1 || a.d > 512 || a.rot < 0 || a.rot > a.d || (a.rot & 1))
    return RELKL_ERR_INVALID;
  if ((a.x_dtype != RELKL_BF16 && a.x_dtype != RELKL_FP32) ||
      (a.y_dtype != RELKL_BF16 && a.y_dtype != RELKL_FP32))
    return RELKL_ERR_INVALID;
  if ((a.interleaved != 0 && a.interleaved != 1) || (a.inverse != 0 && a.inverse != 1))
    return RELKL_ERR_INVALID;
  if (!std::isfinite(a.pos_scale) || !std::isfinite(a.pos_offset) || !std::isfinite(a.mscale))
    return RELKL_ERR_INVALID;
  if (a.positions) {
    if ((a.pos_bytes != 4 && a.pos_bytes != 8) || !aligned(a.positions, a.pos_bytes) ||
        a.pos_stride[0] < 0 || a.pos_stride[1] < 0)
      return RELKL_ERR_INVALID;
  } else if (a.pos_bytes != 0) {
    return RELKL_ERR_INVALID;
  }
  const int64_t xs = a.x_dtype == RELKL_BF16 ? 2 : 4, ys = a.y_dtype == RELKL_BF16 ? 2 : 4;
  RotaryParams p;
  std::memset(&p, 0, sizeof(p));
  struct Range { const char *x0, *x1, *y0, *y1; bool in_place; } range[kMaxSeg];
  bool turns = false;
  for (int r = 0; r < n_tensors; ++r) {
    const relkl_rotary_tensor& t = tensors[r];
    if (t.H < 0 || (t.apply != 0 && t.apply != 1)) return RELKL_ERR_INVALID;
    if (t.H == 0 || a.B == 0 || a.N == 0) continue;
    if (!t.x || !t.y || !aligned(t.x, xs) || !aligned(t.y, ys)) return RELKL_ERR_INVALID;
    const int64_t extent[3] = {a.B, t.H, a.N};
    RotaryTensor& k = p.t[p.n];
    k.x = t.x;
    k.y = t.y;
    k.H = t.H;
    k.apply = t.apply && a.rot > 0;
    turns = turns || k.apply;
    bool same = t.x == t.y && a.x_dtype == a.y_dtype;
    int64_t x_span = a.d, y_span = a.d;   // elements from the first to behind the last
    for (int i = 0; i < 3; ++i) {
      // a dimension of extent 1 may carry any stride; the bound keeps every
      // offset below 2^62 bytes
      k.xs[i] = extent[i] > 1 ? t.x_stride[i] : 0;
      k.ys[i] = extent[i] > 1 ? t.y_stride[i] : 0;
      if (k.xs[i] < 0 || k.ys[i] < 0 || k.xs[i] > (int64_t(1) << 48) / extent[i] ||
          k.ys[i] > (int64_t(1) << 48) / extent[i])
        return RELKL_ERR_INVALID;
      same = same && k.xs[i] == k.ys[i];
      x_span += (extent[i] - 1) * k.xs[i];
      y_span += (extent[i] - 1) * k.ys[i];
    }
    // y's elements are distinct: by growing stride, each step passes all that
    // the smaller ones reach
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (k.ys[order[j]] > k.ys[order[j + 1]]) std::swap(order[j], order[j + 1]);
    int64_t reach = a.d;
    for (int i = 0; i < 3; ++i) {
      const int o = order[i];
      if (extent[o] == 1) continue;
      if (k.ys[o] < reach) return RELKL_ERR_INVALID;
      reach += (extent[o] - 1) * k.ys[o];
    }
    Range& g = range[p.n];
    g.x0 = static_cast<const char*>(t.x);
    g.x1 = g.x0 + x_span * xs;
    g.y0 = static_cast<const char*>(t.y);
    g.y1 = g.y0 + y_span * ys;
    g.in_place = same;
    ++p.n;
  }
  if (p.n == 0) return RELKL_OK;
  // Tensors that are parts of one buffer interleave their ranges, so where two
  // outputs' ranges meet their rows decide.  That settles two tensors rotated
  // in place too; elsewhere the range of an x may not meet that of a y.
  for (int i = 0; i < p.n; ++i)
    for (int j = 0; j < p.n; ++j) {
      if (j < i && range[i].y0 < range[j].y1 && range[j].y0 < range[i].y1 &&
          rows_meet(p.t[i], p.t[j], a, (range[j].y0 - range[i].y0) / ys))
        return RELKL_ERR_INVALID;
      if (range[i].in_place && range[j].in_place) continue;
      if (range[i].x0 < range[j].y1 && range[j].y0 < range[i].x1) return RELKL_ERR_INVALID;
    }
  if (turns && (!a.inv_freq || !aligned(a.inv_freq, 8))) return RELKL_ERR_INVALID;
  p.B = a.B;
  p.N = a.N;
  p.d = a.d;
  p.rot = a.rot;
  p.inv_freq = a.inv_freq;
  p.positions = a.positions;
  p.pos_stride[0] = a.pos_stride[0];
  p.pos_stride[1] = a.pos_stride[1];
  p.pos_bytes = a.pos_bytes;
  p.inverse = a.inverse;
  p.mscale = a.mscale;
  p.pos_scale = a.pos_scale;
  p.pos_offset = a.pos_offset;
  relkl_status s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  cudaError_t e = launch_rotary(p, a.x_dtype == RELKL_BF16, a.y_dtype == RELKL_BF16,
                                a.interleaved != 0, dev.sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

relkl_status relkl_adamw_check(int32_t n_tensors, const relkl_adamw_tensor* tensors,
                               const relkl_adamw_plan* plan) {
  if (n_tensors < 0 || !plan || (n_tensors > 0 && !tensors)) return RELKL_ERR_INVALID;
  const relkl_adamw_plan& a = *plan;
  if ((a.state_bits != 32 && a.state_bits != 8) || a.reserved != 0) return RELKL_ERR_INVALID;
  auto number = [](double x) { return std::isfinite(x) && x >= 0.0; };
  if (!(a.beta1 >= 0.0 && a.beta1 < 1.0 && a.beta2 >= 0.0 && a.beta2 < 1.0) || !number(a.eps))
    return RELKL_ERR_INVALID;
  if (a.lr_dev ? !aligned(a.lr_dev, 4) : !number(a.lr)) return RELKL_ERR_INVALID;
  if (a.step_dev ? !aligned(a.step_dev, 8) : a.step < 1) return RELKL_ERR_INVALID;
  if (!aligned(a.grad_scale, 4)) return RELKL_ERR_INVALID;
  const bool bits8 = a.state_bits == 8;
  // an eps that float32 does not hold would be 0, and 0 / 0 where m and v are 0;
  // the reciprocal of the 8-bit kernel takes a subnormal number for 0 as well
  const float eps = static_cast<float>(a.eps);
  if (a.eps > 0.0 && (eps == 0.0f || (bits8 && eps < FLT_MIN))) return RELKL_ERR_INVALID;
  for (int32_t k = 0; k < n_tensors; ++k) {
    const relkl_adamw_tensor& t = tensors[k];
    if (t.n < 0 || t.n > (int64_t(1) << 40) || t.reserved != 0 || !number(t.weight_decay))
      return RELKL_ERR_INVALID;
    if ((t.grad_dtype != RELKL_BF16 && t.grad_dtype != RELKL_FP32) ||
        (t.param_dtype != RELKL_BF16 && t.param_dtype != RELKL_FP32))
      return RELKL_ERR_INVALID;
    if (t.n == 0) continue;
    const size_t gs = t.grad_dtype == RELKL_BF16 ? 2 : 4, ps = t.param_dtype == RELKL_BF16 ? 2 : 4;
    const size_t ss = bits8 ? 1 : 4;
    if (!t.grad || !t.param || !t.m || !t.v || !aligned(t.grad, gs) || !aligned(t.param, ps) ||
        !aligned(t.copy, 2) || !aligned(t.m, ss) || !aligned(t.v, ss))
      return RELKL_ERR_INVALID;
    if (bits8 ? (!t.m_scale || !t.v_scale || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
              : (t.m_scale || t.v_scale))
      return RELKL_ERR_INVALID;
  }
  for (int32_t k = 0; k < n_tensors;) {   // by launches
    Range range[kAdamwRanges * kAdamwMost];
    int n = 0, nr = 0;
    for (; k < n_tensors && n < kAdamwMost; ++k) {
      if (tensors[k].n == 0) continue;
      nr += adamw_ranges(tensors[k], bits8, range + nr);
      ++n;
    }
    if (overlaps(range, nr)) return RELKL_ERR_INVALID;
  }
  return RELKL_OK;
}

relkl_status relkl_adamw(int32_t n_tensors, const relkl_adamw_tensor* tensors,
                         const relkl_adamw_plan* plan, void* stream) {
  NvtxRange nvtx_range("relkl_adamw");
  const relkl_status refused = relkl_adamw_check(n_tensors, tensors, plan);
  if (refused != RELKL_OK) return refused;
  const relkl_adamw_plan& a = *plan;
  const bool bits8 = a.state_bits == 8;
  AdamwPlan p;
  p.lr = a.lr;
  p.bc1 = 1.0 - std::pow(a.beta1, static_cast<double>(a.step));
  p.bc2 = 1.0 - std::pow(a.beta2, static_cast<double>(a.step));
  p.log_b1 = std::log(a.beta1);
  p.log_b2 = std::log(a.beta2);
  p.b1 = static_cast<float>(a.beta1);
  p.c1 = static_cast<float>(1.0 - a.beta1);
  p.b2 = static_cast<float>(a.beta2);
  p.c2 = static_cast<float>(1.0 - a.beta2);
  p.eps = static_cast<float>(a.eps);
  p.rbc2 = static_cast<float>(1.0 / std::sqrt(p.bc2));
  p.step_size = static_cast<float>(a.lr / p.bc1);
  p.lr_dev = a.lr_dev;
  p.step_dev = reinterpret_cast<const long long*>(a.step_dev);
  p.grad_scale = a.grad_scale;
  for (int32_t k = 0; k < n_tensors;) {
    AdamwTensor group[kAdamwMost];
    int n = 0;
    for (; k < n_tensors && n < kAdamwMost; ++k) {
      const relkl_adamw_tensor& t = tensors[k];
      if (t.n == 0) continue;
      const bool gb = t.grad_dtype == RELKL_BF16, pb = t.param_dtype == RELKL_BF16;
      AdamwTensor& g = group[n++];
      g.grad = t.grad;
      g.param = t.param;
      g.copy = t.copy;
      g.m = t.m;
      g.v = t.v;
      g.m_scale = t.m_scale;
      g.v_scale = t.v_scale;
      g.n = t.n;
      g.weight_decay = t.weight_decay;
      g.decay = static_cast<float>(1.0 - a.lr * static_cast<double>(t.weight_decay));
      g.grad_bf16 = gb;
      g.param_bf16 = pb;
      g.wide = aligned(t.grad, gb ? 8 : 16) && aligned(t.param, pb ? 8 : 16) &&
               aligned(t.copy, 8) && aligned(t.m, bits8 ? 8 : 16) && aligned(t.v, bits8 ? 8 : 16);
    }
    if (n > 0) {
      cudaError_t e = launch_adamw(group, n, p, bits8, static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_fail(e);
    }
  }
  return RELKL_OK;
}

size_t relkl_grad_norm_bytes(int32_t n_tensors) {
  const int64_t groups = n_tensors > 0 ? (static_cast<int64_t>(n_tensors) + kAdamwMost - 1) / kAdamwMost : 1;
  return static_cast<size_t>(groups) * kNormGrid * sizeof(double);
}

relkl_status relkl_grad_norm(int32_t n_tensors, const relkl_norm_tensor* tensors, float max_norm,
                             float* out, void* scratch, size_t scratch_bytes, void* stream) {
  NvtxRange nvtx_range("relkl_grad_norm");
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !(max_norm > 0.0f)) return RELKL_ERR_INVALID;
  if (!out || !aligned(out, 4)) return RELKL_ERR_INVALID;
  if (!scratch || !aligned(scratch, 8) || scratch_bytes < relkl_grad_norm_bytes(n_tensors))
    return RELKL_ERR_WORKSPACE;
  int32_t used = 0;
  int64_t all = 0;
  for (int32_t k = 0; k < n_tensors; ++k) {
    const relkl_norm_tensor& t = tensors[k];
    if (t.n < 0 || t.n > (int64_t(1) << 40) || t.reserved != 0 ||
        (t.dtype != RELKL_BF16 && t.dtype != RELKL_FP32))
      return RELKL_ERR_INVALID;
    if (t.n == 0) continue;
    if (!t.grad || !aligned(t.grad, t.dtype == RELKL_BF16 ? 2 : 4)) return RELKL_ERR_INVALID;
    ++used;
    all += norm_chunks(t.n, t.dtype == RELKL_BF16);
    if (all > 0x7fffffffLL) return RELKL_ERR_UNSUPPORTED;
  }
  relkl_status s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(scratch);
  const int most = dev.sms * 3 < kNormGrid ? dev.sms * 3 : kNormGrid;
  cudaError_t e = cudaSuccess;
  int sums = 0;
  for (int32_t k = 0; k < n_tensors;) {
    NormTensor group[kAdamwMost];
    int n = 0;
    int64_t chunks = 0;
    for (; k < n_tensors && n < kAdamwMost; ++k) {
      const relkl_norm_tensor& t = tensors[k];
      if (t.n == 0) continue;
      NormTensor& g = group[n++];
      g.grad = t.grad;
      g.n = t.n;
      g.bf16 = t.dtype == RELKL_BF16;
      g.wide = aligned(t.grad, 16);
      chunks += norm_chunks(t.n, g.bf16);
    }
    if (n == 0) break;
    // a few chunks are summed and finished by one CTA in one launch
    const bool one = all <= kNormOneCta;
    const int grid = one ? 1 : static_cast<int>(chunks < most ? chunks : most);
    e = launch_grad_norm(group, n, chunks, grid, partial + sums, one && used <= kAdamwMost ? out : nullptr,
                         max_norm, st);
    if (e != cudaSuccess) return cuda_fail(e);
    if (one && used <= kAdamwMost) return RELKL_OK;
    sums += grid;
  }
  e = launch_norm_finish(partial, sums, max_norm, out, st);
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

relkl_status relkl_quantize_rows(int64_t rows, int32_t K, const void* x, int32_t x_dtype,
                                 int64_t x_stride, int8_t* q, int64_t q_stride, float* scale,
                                 void* stream) {
  NvtxRange nvtx_range("relkl_quantize_rows");
  if (!rows_ok(rows, K)) return RELKL_ERR_INVALID;
  if (rows == 0) return RELKL_OK;
  if (!matrix_ok(x, x_dtype, x_stride, K) || !codes_ok(q, q_stride, K) || !scale || !aligned(scale, 4))
    return RELKL_ERR_INVALID;
  relkl_status s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  return quantize_rows(rows, K, x, x_dtype, x_stride, q, q_stride, scale, dev,
                       static_cast<cudaStream_t>(stream));
}

relkl_status relkl_matmul_i8(int64_t rows, int32_t cols, int32_t K, const int8_t* q,
                             int64_t q_stride, const float* q_scale, const int8_t* w,
                             int64_t w_stride, const float* w_scale, const float* bias, void* y,
                             int32_t y_dtype, int64_t y_stride, void* ws, size_t ws_bytes,
                             void* stream) {
  NvtxRange nvtx_range("relkl_matmul_i8");
  if (!rows_ok(rows, K) || cols < 0 || cols > (1 << 30)) return RELKL_ERR_INVALID;
  if (rows == 0 || cols == 0) return RELKL_OK;
  if (!codes_ok(q, q_stride, K) || !codes_ok(w, w_stride, K) || !matrix_ok(y, y_dtype, y_stride, cols) ||
      !q_scale || !w_scale || !aligned(q_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4))
    return RELKL_ERR_INVALID;
  relkl_status s = check_ws(ws, ws_bytes);
  if (s != RELKL_OK) return s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  return matmul_i8(rows, cols, K, q, q_stride, q_scale, w, w_stride, w_scale, bias, y, y_dtype,
                   y_stride, ws, false, dev, static_cast<cudaStream_t>(stream));
}

size_t relkl_linear_i8_bytes(int64_t rows, int32_t K) {
  if (!rows_ok(rows, K) || few_rows(rows, K)) return 0;
  return static_cast<size_t>(rows * code_pitch(K) + rows * 4);
}

relkl_status relkl_linear_i8(int64_t rows, int32_t cols, int32_t K, const void* x,
                             int32_t x_dtype, int64_t x_stride, const int8_t* w, int64_t w_stride,
                             const float* w_scale, const float* bias, void* y, int32_t y_dtype,
                             int64_t y_stride, void* scratch, size_t scratch_bytes, void* ws,
                             size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("relkl_linear_i8");
  if (!rows_ok(rows, K) || cols < 0 || cols > (1 << 30)) return RELKL_ERR_INVALID;
  if (rows == 0 || cols == 0) return RELKL_OK;
  if (!matrix_ok(x, x_dtype, x_stride, K) || !codes_ok(w, w_stride, K) ||
      !matrix_ok(y, y_dtype, y_stride, cols) || !w_scale || !aligned(w_scale, 4) || !aligned(bias, 4))
    return RELKL_ERR_INVALID;
  relkl_status s = check_ws(ws, ws_bytes);
  if (s != RELKL_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool few = few_rows(rows, K);
  if (!few && (!scratch || !aligned(scratch, 16) || scratch_bytes < relkl_linear_i8_bytes(rows, K)))
    return RELKL_ERR_WORKSPACE;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  if (few) {
    GemvParams p = {x, w, w_scale, bias, y, x_stride, w_stride, y_stride, static_cast<int>(rows),
                    cols, K, wide_rows(x, x_dtype, x_stride)};
    cudaError_t e = launch_gemv_i8(p, x_dtype == RELKL_BF16, y_dtype == RELKL_BF16, dev.sms, st);
    return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
  }
  int8_t* q = static_cast<int8_t*>(scratch);
  const int64_t pitch = code_pitch(K);
  float* scale = reinterpret_cast<float*>(q + rows * pitch);
  if ((s = quantize_rows(rows, K, x, x_dtype, x_stride, q, pitch, scale, dev, st)) != RELKL_OK) return s;
  return matmul_i8(rows, cols, K, q, pitch, scale, w, w_stride, w_scale, bias, y, y_dtype, y_stride,
                   ws, true, dev, st);
}

relkl_status relkl_cast_bf16(const float* src, void* dst, int64_t n, void* stream) {
  NvtxRange nvtx_range("relkl_cast_bf16");
  if (n < 0) return RELKL_ERR_INVALID;
  if (n == 0) return RELKL_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 2)) return RELKL_ERR_INVALID;
  // the two ranges may not overlap
  const char* a = reinterpret_cast<const char*>(src);
  const char* b = static_cast<const char*>(dst);
  if (a < b + 2 * n && b < a + 4 * n) return RELKL_ERR_INVALID;
  relkl_status s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  cudaError_t e = launch_cast_bf16(src, dst, n, dev.sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}

relkl_status relkl_weight_grad(int64_t rows, int32_t D, int32_t cols, const void* h,
                               const void* dx_pre, float* dw, void* ws, size_t ws_bytes,
                               void* stream) {
  NvtxRange nvtx_range("relkl_weight_grad");
  if (rows < 1 || rows > 0x7fffffffLL || D < 1 || cols < 1 || (D % 8) || (cols % 8))
    return RELKL_ERR_INVALID;
  if (!h || !dx_pre || !dw || !aligned(h, 16) || !aligned(dx_pre, 16) || !aligned(dw, 16))
    return RELKL_ERR_INVALID;
  relkl_status s = check_ws(ws, ws_bytes);
  if (s != RELKL_OK) return s;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  if (dev.major != 10) return RELKL_ERR_UNSUPPORTED;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return RELKL_ERR_CUDA;
  const int r = launch_wgrad(enc, rows, D, cols, h, dx_pre, dw, dev.sms,
                             reinterpret_cast<DevStatus*>(ws), g_timeout_ns.load(),
                             static_cast<cudaStream_t>(stream));
  if (r == 1) return RELKL_ERR_UNSUPPORTED;
  if (r != 0) return cuda_fail(static_cast<cudaError_t>(r - 2));
  return RELKL_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// relkl_fwd_noalloc: the tensor-core forward with its scratch (the device
// status record) in a static device array instead of a caller workspace.
// Host code must not hand the array's name to a kernel: on the host it is a
// stand-in, not a device address.  The address comes from
// cudaGetSymbolAddress, looked up once per device with that device current.
static __device__ __align__(256) unsigned char g_noalloc_scratch[RELKL_NOALLOC_SCRATCH_BYTES];

namespace {
// One slot per device index: the array's device address and the context it
// was looked up in.  A context torn down and created again (cudaDeviceReset,
// or a reset after a sticky error) loads the module again, possibly at another
// address, so a slot is only reused while the device's current context is the
// one recorded in it.
struct NoallocSlot {
  CUcontext ctx;
  void* addr;
};
NoallocSlot g_noalloc[64];
std::mutex g_noalloc_mu;

using CtxGetCurrentFn = CUresult (*)(CUcontext*);
CtxGetCurrentFn g_ctx_current = nullptr;
std::once_flag g_ctx_once;

CUcontext current_context() {
  std::call_once(g_ctx_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_ctx_current = reinterpret_cast<CtxGetCurrentFn>(fn);
  });
  CUcontext c = nullptr;
  if (g_ctx_current && g_ctx_current(&c) != CUDA_SUCCESS) c = nullptr;
  return c;
}

relkl_status noalloc_scratch(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return RELKL_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  NoallocSlot& slot = g_noalloc[dev];
  const CUcontext ctx = current_context();
  if (!slot.addr || ctx != slot.ctx) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess || !p) return cuda_fail(e != cudaSuccess ? e : cudaErrorInvalidSymbol);
    slot.addr = p;
    slot.ctx = current_context();   // the lookup made the device's context current
  }
  *out = slot.addr;
  return RELKL_OK;
}
}  // namespace

extern "C" relkl_status relkl_fwd_noalloc(const relkl_desc* desc, const void* x_t,
                                          const void* x_s, float* kl, float* stats,
                                          void* stream) {
  NvtxRange nvtx_range("relkl_fwd_noalloc");
  const void* xt[1] = {x_t};
  const void* xs[1] = {x_s};
  bool empty = false;
  relkl_status s = check_multi(1, desc, xt, xs, &empty);
  if (s != RELKL_OK || empty) return s;
  if (!kl || !stats || !aligned(kl, 4) || !aligned(stats, 16)) return RELKL_ERR_INVALID;
  if (!use_tc(1, desc, xt, xs)) return RELKL_ERR_UNSUPPORTED;
  if (kWorkspaceBytes > sizeof(g_noalloc_scratch)) return RELKL_ERR_WORKSPACE;
  DevInfo dev;
  if ((s = device_info(&dev)) != RELKL_OK) return s;
  if (dev.major != 10) return RELKL_ERR_UNSUPPORTED;
  void* scratch = nullptr;
  if ((s = noalloc_scratch(&scratch)) != RELKL_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the record keeps the previous call's contents: clear it on this stream first
  cudaError_t e = cudaMemsetAsync(scratch, 0, sizeof(DevStatus), st);
  if (e != cudaSuccess) return cuda_fail(e);
  TcParams p;
  if ((s = build_tc(1, desc, xt, xs, &p, scratch)) != RELKL_OK) return s;
  float* k[1] = {kl};
  float* sts[1] = {stats};
  set_seg_outputs(&p, 1, desc, k, sts, nullptr, nullptr, nullptr);
  const int grid = p.n_items < dev.sms ? p.n_items : dev.sms;
  e = tc_launch_fwd(p, desc->d, grid, st);
  return e == cudaSuccess ? RELKL_OK : cuda_fail(e);
}
