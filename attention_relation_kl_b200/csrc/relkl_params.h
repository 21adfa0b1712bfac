// Kernel parameter blocks shared by the launch code and the kernels.
#pragma once

#include <cstdint>
#include <cuda.h>

namespace relkl {

struct DevStatus;

constexpr int kMaxSeg = 3;   // relations per launch (Q, K, V)

// One relation inside a launch.  Units of relation r are numbered
// unit_begin .. unit_begin + B*H - 1, batch-major then head.
struct TcSeg {
  CUtensorMap tm_t;          // teacher [B,H,N,d] bf16, box 64 cols x 128 rows, 128B swizzle
  CUtensorMap tm_s;          // student, same geometry
  CUtensorMap tm_dx;         // dX [B,H,N,d] f32, box 32 cols x 32 rows, 128B swizzle (bwd)
  CUtensorMap tm_t64;        // teacher, box 64 cols x 64 rows (bwd column tiles, d = 128)
  CUtensorMap tm_s64;        // student, same geometry
  float* kl;                 // [B,H,N]
  float* stats;              // [B,H,N,4]
  const float* dkl;          // [B,H,N] or null (1/N)
  float* dx;                 // [B,H,N,d] float32
  const int* lengths;        // [B] valid lengths (device) or null (all N)
  const int* cu_seqlens;     // packed sequences: [n_seq + 1] token offsets (device), or null
  int B, H;                  // packed sequences: B = n_seq (units are (sequence, head))
  int unit_begin;
  int max_seqlen;            // packed sequences: bound on every sequence's length
};

struct TcParams {
  TcSeg seg[kMaxSeg];
  int n_seg;
  int N;
  int nblk;       // ceil(N / 128)
  int n_pairs;    // work items per unit (forward: ceil(nblk / 2), row blocks p and nblk-1-p)
  int n_units;
  // A call may cover one part of every unit's work items: items
  // part, part + n_parts, ... (rows of the other parts are not touched).
  int part, n_parts;
  int n_local;    // items per unit in this part: ceil((n_pairs - part) / n_parts)
  int n_items;    // n_units * n_local
  int causal;
  float scale;    // logit scale
  float sl2;      // scale * log2(e)
  DevStatus* status;
  unsigned long long timeout_ns;
};

// CUDA-core float32 path: plain pointers with element strides.
struct SimtSeg {
  const void* xt;
  const void* xs;
  int64_t sb, sh, sn;        // element strides of B, H, N (d is contiguous)
  float* kl;
  float* stats;
  const float* dkl;
  float* dx;
  const int* lengths;        // [B] valid lengths (device) or null (all N)
  const int* cu_seqlens;     // packed sequences: [n_seq + 1] token offsets, or null
  int B, H;                  // packed sequences: B = n_seq
  int unit_begin;
  int max_seqlen;
};

struct SimtParams {
  SimtSeg seg[kMaxSeg];
  int n_seg;
  int N, d;
  int causal;
  int is_bf16;
  float scale;
  int n_units;
  int part, n_parts;   // 32-row blocks part, part + n_parts, ... of every unit
  int nblk_local;      // ceil((ceil(N / 32) - part) / n_parts)
};

// One tensor of a rotary call: element (b, h, n, k) of x at
// x + b*xs[0] + h*xs[1] + n*xs[2] + k, of y likewise.
struct RotaryTensor {
  const void* x;
  void* y;
  int64_t xs[3], ys[3];      // element strides of B, H, N
  int H;
  int apply;                 // 0: moved and converted only
  // set by the launch: head groups; a thread's parts of a head, the first
  // rot_chunks of them rotated, the others `width` entries each
  int groups, chunks, rot_chunks, width;
};

struct RotaryParams {
  RotaryTensor t[kMaxSeg];
  int n;
  int B, N, d, rot;
  const double* inv_freq;    // [rot / 2] (device)
  const void* positions;     // int32 or int64 (device), or null (0, 1, ..., N - 1)
  int64_t pos_stride[2];
  int pos_bytes;
  int inverse;
  float mscale;
  double pos_scale, pos_offset;
  // set by the launch
  int heads_per_group;
  int64_t tokens;
};

// AdamW: tables of tensors travel in the kernel's parameters (32,764 bytes at
// most); a call with few of them copies a small table: with 3 tensors a launch
// takes 7.0, 8.0 and 9.1 us of the host with tables of 16, 96 and 384.
constexpr int kAdamwFew = 16;
constexpr int kAdamwSome = 96;
constexpr int kAdamwMost = 384;

struct AdamwTensor {
  const void* grad;
  void *param, *copy;        // copy: bf16 or null
  void *m, *v;               // float32, or e4m3 codes (v: of its root)
  float *m_scale, *v_scale;  // 8-bit states: one per 256 elements
  int64_t n;
  float weight_decay;
  float decay;               // 1 - lr weight_decay, of the plan's lr
  uint8_t grad_bf16, param_bf16;
  uint8_t wide;              // every pointer allows accesses of four (eight) elements
};

struct AdamwPlan {
  double lr, bc1, bc2, log_b1, log_b2;
  float b1, c1, b2, c2, eps;   // c = 1 - b
  float rbc2, step_size;       // 1 / sqrt(bc2), lr / bc1
  const float* lr_dev;         // device, or null: lr
  const long long* step_dev;   // device, or null: bc1, bc2
  const float* grad_scale;     // device, or null: 1
};

template <int CAP>
struct AdamwParams {
  AdamwPlan plan;
  int n;
  int first[CAP];            // a tensor's first CTA
  AdamwTensor t[CAP];
};

constexpr int kNormGrid = 1024;     // partial sums of one launch, at most
// Chunks of 32 KB that one CTA sums and finishes alone: one takes 6.1 us and two
// 7.5 (bf16) and 8.2 us (float32), a replayed graph's start and end included,
// where sums and a second launch take 8.2 us.
constexpr int kNormOneCta = 2;

struct NormTensor {
  const void* grad;
  int64_t n;
  uint8_t bf16, wide;
};

template <int CAP>
struct NormParams {
  int n, chunks;
  double* partial;
  float* out;                // null: write partial sums
  float max_norm;
  int first[CAP];            // a tensor's first chunk
  NormTensor t[CAP];
};

// Products in 8-bit integers: row codes, few rows, and the tensor-core product.
// Most rows of the kernel for few rows.  Against the tensor cores (coding and
// product, the second started early), us with 1, 2, 3 and 4 rows, weights from HBM:
//   K x channels   here                     there
//   1024 x 1024    2.5, 3.3, 4.2, 4.9       7.0
//   4096 x 1024    6.0, 6.9, 7.8, 9.0       7.9
//   4096 x 4096    7.6, 8.7, 10.2, 11.5     11.5
//   8192 x 8192    21.7, 24.1, 26.6, 29.2   20.6
//   4096 x 16384   18.9, 20.8, 22.6, 24.5   17.1
//   16384 x 4096   23.0, 26.2, 29.6, 33.2   23.5
// Five and six rows take longer than there from 4096 x 1024 on (10.1 and 11.1).
// Above 16 M weights it is behind by up to 45 % where these come from HBM; from L2 it
// is ahead up to two rows there too (8192 x 8192 10.3 and 13.2, there 17.9).  The
// limit does not look at the channels, as a caller asks for scratch by rows and K.
constexpr int kGemvRows = 4;
constexpr int kGemvBytes = 96 * 1024; // most bytes of their codes in shared memory

struct RowsParams {
  const void* x;
  int8_t* q;
  float* scale;
  int64_t rows, x_stride, q_stride;   // strides in elements
  int K;
  int wide;
};

struct GemvParams {
  const void* x;
  const int8_t* w;
  const float *w_scale, *bias;        // bias may be null
  void* y;
  int64_t x_stride, w_stride, y_stride;
  int rows, cols, K;
  int wide;                           // rows of x start at 16-byte boundaries
};

struct I8Params {
  CUtensorMap tm_a;                   // codes [rows, K]: box 128 bytes x up to 128 rows, 128B swizzle
  CUtensorMap tm_b;                   // weights [cols, K]: box 128 bytes x BN rows
  CUtensorMap tm_y;                   // y [rows, box_cols]: box 128 bytes x 32 rows, 128B swizzle (pairs, y_wide)
  const float *x_scale, *w_scale, *bias;
  void* y;
  int64_t rows, y_stride;
  int cols;
  int y_wide;                         // rows of y start at 16-byte (1) or 32-byte (2) boundaries
  int m_tiles, n_tiles, n_units, k_chunks, split;   // set by the launch
  int a_box;                          // rows of tm_a's box (one CTA for a tile)
  int box_cols;                       // columns of tm_y: cols, down to whole 16 bytes (pairs)
  DevStatus* status;
  unsigned long long timeout_ns;
};

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct I8Call {
  const int8_t *q, *w;
  int64_t q_stride, w_stride;
  int K;
  bool after_rows;   // the kernel before is the coding of q: start ahead of its end
  EncodeTiled encode;
};

static_assert(sizeof(AdamwParams<kAdamwMost>) <= 32764, "kernel parameters");
static_assert(sizeof(NormParams<kAdamwMost>) <= 32764, "kernel parameters");

}  // namespace relkl
