// Products in 8-bit integers with a scale for each token and each channel:
//
//   y[r, c] = sx[r] sw[c] sum_k qx[r, k] qw[c, k] + bias[c]
//
// with qx = rint(127 x / max|x_r|), sx = max|x_r| / 127 formed per call, and
// the frozen teacher's weights qw [cols, K], sw [cols] laid out once.  The sum
// is exact in int32, so neither the split of K nor any order changes a bit;
// it becomes float32 once, is scaled, and rounded once to the output's type.
//
// Four kernels:
//   * relkl_quantize_rows_kernel: one pass over the rows.  HBM: 32K x 4096 bf16
//     in 61 to 70 us, 6.6 to 5.7 TB/s.
//   * relkl_gemv_i8_kernel, up to kGemvRows rows: every CTA codes the rows for
//     itself in shared memory (they are small and in L2) while its warps'
//     weights are on the way, then one warp per channel sums with dp4a.  Bound
//     by the launch and the weights' bytes: 1 x 4096 x 4096 in 4.7 us where they are
//     in L2, 7.6 us from HBM.
//   * relkl_gemm_i8_kernel: tcgen05.mma kind::i8 (s8 x s8 -> s32) with both
//     operands K-major in 128-byte swizzled shared memory, fed by TMA; one tile
//     for a CTA, or K split over a cluster, for tens to hundreds of rows.
//   * relkl_gemm_i8_pair_kernel: the same by pairs of CTAs, persistent.  32K x
//     4096 x 4096 in 328 to 337 us, 3.35 to 3.27 POP/s, as long as the GPU is not
//     limited by its power (twice the measured bf16 burst rate is 3.31); after some
//     seconds 399 us.  A library product of the same codes to int32, without scales,
//     takes 336 and 390.  With the coding a call takes 387 us, after some seconds 456.
#include <algorithm>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "relkl_device.cuh"
#include "relkl_params.h"

namespace relkl {

namespace {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// The magnitude's bits order as the magnitudes do, with NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// rint(127 x / most), exactly, ties to even.
//
// Quick way: x times a number next to 127 / most, added to 1.5 * 2^23 in one
// fma, which rounds it to the nearest integer and leaves that, as a byte, in
// the sum's last bits.
//   * bf16: x = a 2^i and most = b 2^j with a, b < 256, so a quotient v that is
//     no half n + 1/2 is at least v / (254 a) = 1.5e-5 v away from every half,
//     and a factor off by 2^-23 of itself cannot carry it across.  Halves occur
//     where 254 a 2^(i - j) = (2n + 1) b: with b = 254 or 127, when 127 / most
//     is a power of two and the product exact, and at v = 63.5, where 64 is
//     right.  The factor rounded up gives all of these.
//   * float32: a factor just above and one just below.  Where they agree the
//     quotient between them has that code; they differ only within 2^-21 of
//     itself of a half, and then code() decides.
// code(): the nearest integers of x (127 / most), off by less than 127 * 2^-23
// = 1.6e-5, are told apart by the sign of 254 |x| - (2n + 1) most; both
// products have at most 32 bits, so each is held exactly as a float and its
// rest, and so is their difference.  Where 127 / most leaves float32's range
// the quotient is taken in double precision, which tells every half from its
// neighbours.
struct RowCoder {
  static constexpr float kNear = 0.5f - 2e-5f;
  float most, inv, above;
  bool easy;
  __device__ __forceinline__ explicit RowCoder(uint32_t bits) {
    most = __uint_as_float(bits);
    easy = most > 1e-30f && most < 1e30f;
    inv = easy ? 127.0f / most : 0.0f;
    above = easy ? __fdiv_ru(127.0f, most) : 0.0f;
  }
  // 0 for a row of zeros, NaN for a row that holds an infinity or a NaN: its
  // products are NaN
  __device__ __forceinline__ float scale() const {
    return isfinite(most) ? most / 127.0f : __int_as_float(0x7fc00000);
  }
  // the code of any x
  __device__ __forceinline__ int code(float x) const {
    if (!easy) {
      if (!(most > 0.0f) || !isfinite(most)) return 0;
      return static_cast<int>(rint(static_cast<double>(x) * 127.0 / static_cast<double>(most)));
    }
    const float q = x * inv, r = rintf(q);
    if (fabsf(q - r) < kNear) return static_cast<int>(r);
    const float ax = fabsf(x), n = floorf(ax * inv), odd = 2.0f * n + 1.0f;
    const float p = 254.0f * ax, t = odd * most;
    const float diff = (p - t) + (fmaf(254.0f, ax, -p) - fmaf(odd, most, -t));
    const int low = static_cast<int>(n);
    const int up = diff > 0.0f || (diff == 0.0f && (low & 1));
    return x < 0.0f ? -(low + up) : low + up;
  }
  // The codes of a group of eight, packed, from the quick way alone; `again`
  // where they have to be looked at by code().
  template <typename H>
  __device__ __forceinline__ uint2 codes(const H& held, bool& again) const {
    float x[8];
    held.get(x);
    uint32_t c[8];
    again = !easy;
    if constexpr (H::kBits == 16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = __float_as_uint(fmaf(x[k], above, 12582912.0f));
    } else {
      const float up = inv * (1.0f + 0x1p-22f), down = inv * (1.0f - 0x1p-22f);
      uint32_t differ = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[k] = __float_as_uint(fmaf(x[k], up, 12582912.0f));
        differ |= c[k] ^ __float_as_uint(fmaf(x[k], down, 12582912.0f));
      }
      again = again || differ != 0;
    }
    auto four = [&](int k) {
      return __byte_perm(__byte_perm(c[k], c[k + 1], 0x0040), __byte_perm(c[k + 2], c[k + 3], 0x0040), 0x5410);
    };
    return make_uint2(four(0), four(4));
  }
};

// Eight elements as they are held between two uses.
template <typename T>
struct Held;
template <>
struct Held<__nv_bfloat16> {
  static constexpr int kBits = 16;
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldcg(reinterpret_cast<const uint4*>(p)); }
  // from any element: words where they are aligned, else a half, three words
  // and a half
  __device__ __forceinline__ void load_any(const __nv_bfloat16* p) {
    if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
      w = make_uint4(__ldg(q), __ldg(q + 1), __ldg(q + 2), __ldg(q + 3));
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(h + 1);
      const uint32_t a = __ldg(h), b = __ldg(q), c = __ldg(q + 1), d = __ldg(q + 2), e = __ldg(h + 7);
      w = make_uint4(a | (b << 16), __funnelshift_l(b, c, 16), __funnelshift_l(c, d, 16), (d >> 16) | (e << 16));
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
};
template <>
struct Held<float> {
  static constexpr int kBits = 32;
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcg(reinterpret_cast<const float4*>(p));
    b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_any(const float* p) {
    a = make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
    b = make_float4(__ldg(p + 4), __ldg(p + 5), __ldg(p + 6), __ldg(p + 7));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// The largest magnitude so far, as the bits of a float or, for bf16, of two
// halves of which the larger counts.
__device__ __forceinline__ uint32_t largest(const Held<float>& h, uint32_t most) {
  most = max(most, max(max(magnitude(h.a.x), magnitude(h.a.y)), max(magnitude(h.a.z), magnitude(h.a.w))));
  return max(most, max(max(magnitude(h.b.x), magnitude(h.b.y)), max(magnitude(h.b.z), magnitude(h.b.w))));
}
__device__ __forceinline__ uint32_t largest(const Held<__nv_bfloat16>& h, uint32_t most) {
  constexpr uint32_t M = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(__vmaxu2(most, h.w.x & M), h.w.y & M), __vmaxu2(h.w.z & M, h.w.w & M));
}
__device__ __forceinline__ uint32_t largest(float x, uint32_t most) { return max(most, magnitude(x)); }
__device__ __forceinline__ uint32_t largest(__nv_bfloat16 x, uint32_t most) {
  return __vmaxu2(most, __bfloat16_as_ushort(x) & 0x7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t largest_bits(uint32_t most) {
  if constexpr (sizeof(T) == 4) return most;
  return max(most & 0xffff0000u, most << 16);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

template <typename U>
__device__ __forceinline__ U from_float(float v) {
  if constexpr (sizeof(U) == 4)
    return v;
  else
    return __float2bfloat16_rn(v);
}

}  // namespace

// groups of eight of a row that one thread holds
constexpr int kRowGroups = 4;
constexpr int GEMV_THREADS = 512;

// The largest magnitude among `warps` warps' (all of the block's threads call).
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* part) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int k = 1; k < static_cast<int>(blockDim.x >> 5); ++k) v = max(v, part[k]);
  return v;
}

// ------------------------------------------------------------ row codes
// A team of threads for each row, as many as give each kRowGroups groups of
// eight elements of it: a warp of eight (WARPS), or a block.  The groups stay
// in registers between the search for the largest and the coding; what a longer
// row has beyond them is read again (from L2).
// `wide`: rows of x start at 16-byte boundaries, so its groups can move at
// once.  32K rows of 4096 bf16: 64 us, 6.3 TB/s; with 2 or 8 groups
// to a thread 94 and 72 us.
template <typename T, bool WARPS>
__global__ void __launch_bounds__(512, 2) relkl_quantize_rows_kernel(const RowsParams p) {
  constexpr int HOLD = kRowGroups;
  __shared__ uint32_t part[16];
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t row = WARPS ? static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (WARPS && row >= p.rows) return;
  const int me = WARPS ? threadIdx.x & 31 : threadIdx.x, step = WARPS ? 32 : blockDim.x;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  int8_t* q = p.q + row * p.q_stride;
  const int groups = p.K / 8;
  Held<T> v[HOLD];
#pragma unroll
  for (int h = 0; h < HOLD; ++h)
    if (h * step + me < groups) p.wide ? v[h].load(x + 8 * (h * step + me)) : v[h].load_any(x + 8 * (h * step + me));
  uint32_t most = 0;
#pragma unroll
  for (int h = 0; h < HOLD; ++h)
    if (h * step + me < groups) most = largest(v[h], most);
  for (int g = HOLD * step + me; g < groups; g += step) {
    Held<T> h;
    p.wide ? h.load(x + 8 * g) : h.load_any(x + 8 * g);
    most = largest(h, most);
  }
#pragma unroll 4
  for (int i = 8 * groups + me; i < p.K; i += step) most = largest(x[i], most);
  const RowCoder coder(WARPS ? warp_max(largest_bits<T>(most)) : block_max(largest_bits<T>(most), part));
  // groups with a code near a half, in the order of this thread's groups: few,
  // so they are done once more behind the others, element by element
  uint32_t redo = 0;
#pragma unroll
  for (int h = 0; h < HOLD; ++h)
    if (h * step + me < groups) {
      bool again;
      __stcg(reinterpret_cast<uint2*>(q + 8 * (h * step + me)), coder.codes(v[h], again));
      redo |= static_cast<uint32_t>(again) << h;
    }
  while (redo) {
    const int g = (__ffs(redo) - 1) * step + me;
    redo &= redo - 1;
#pragma unroll 1
    for (int k = 8 * g; k < 8 * g + 8; ++k) q[k] = static_cast<int8_t>(coder.code(to_float(x[k])));
  }
  for (int g = HOLD * step + me; g < groups; g += step) {
    Held<T> h;
    p.wide ? h.load(x + 8 * g) : h.load_any(x + 8 * g);
    bool again;
    __stcg(reinterpret_cast<uint2*>(q + 8 * g), coder.codes(h, again));
    if (again)
#pragma unroll 1
      for (int k = 8 * g; k < 8 * g + 8; ++k) q[k] = static_cast<int8_t>(coder.code(to_float(x[k])));
  }
#pragma unroll 1
  for (int i = 8 * groups + me; i < p.K; i += step)
    q[i] = static_cast<int8_t>(coder.code(to_float(x[i])));
  if (me == 0) p.scale[row] = coder.scale();
}

// ------------------------------------------------------------ few rows
// Every CTA codes the rows for itself, all R of them side by side: a group of
// eight of each row to a thread, with three barriers whatever R is.  Shared
// memory: the rows' codes, each padded with zeros to 16 bytes.
template <typename T, typename U, int R>
__global__ void __launch_bounds__(GEMV_THREADS, 2) relkl_gemv_i8_kernel(const GemvParams p) {
  constexpr int WARPS = GEMV_THREADS / 32;
  extern __shared__ __align__(16) int8_t codes[];
  __shared__ uint32_t part[R][WARPS], largest_of[R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t c = static_cast<int64_t>(blockIdx.x) * WARPS + warp;
  const int pitch = (p.K + 15) / 16 * 16;
  const int vecs = p.K / 16, groups = p.K / 8;

  // the first of the weights are on their way while the rows are coded
  constexpr int AHEAD = 4;
  uint4 first[AHEAD];
  const int8_t* w = p.w + (c < p.cols ? c : 0) * p.w_stride;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (i * 32 + lane < vecs) first[i] = __ldcg(reinterpret_cast<const uint4*>(w) + i * 32 + lane);

  const T* x = static_cast<const T*>(p.x);
  auto load = [&](Held<T>& h, int r, int g) {
    const T* at = x + r * p.x_stride + 8 * g;
    p.wide ? h.load(at) : h.load_any(at);
  };
  Held<T> mine[R];
  const int me = threadIdx.x;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < p.rows && me < groups) load(mine[r], r, me);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= p.rows) break;
    uint32_t most = me < groups ? largest(mine[r], 0u) : 0u;
    for (int g = GEMV_THREADS + me; g < groups; g += GEMV_THREADS) {
      Held<T> h;
      load(h, r, g);
      most = largest(h, most);
    }
    if (8 * groups + me < p.K) most = largest(x[r * p.x_stride + 8 * groups + me], most);
    most = warp_max(largest_bits<T>(most));
    if (lane == 0) part[r][warp] = most;
  }
  __syncthreads();
  if (warp < R && warp < p.rows) {
    const uint32_t most = warp_max(lane < WARPS ? part[warp][lane] : 0u);
    if (lane == 0) largest_of[warp] = most;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= p.rows) break;
    const RowCoder coder(largest_of[r]);
    int8_t* q = codes + r * pitch;
    auto put = [&](const Held<T>& h, int g) {
      bool again;
      *reinterpret_cast<uint2*>(q + 8 * g) = coder.codes(h, again);
      if (again)
#pragma unroll 1
        for (int k = 8 * g; k < 8 * g + 8; ++k) q[k] = static_cast<int8_t>(coder.code(to_float(x[r * p.x_stride + k])));
    };
    if (me < groups) put(mine[r], me);
    for (int g = GEMV_THREADS + me; g < groups; g += GEMV_THREADS) {
      Held<T> h;
      load(h, r, g);
      put(h, g);
    }
    const int i = 8 * groups + me;       // the rest of the row, and its padding
    if (i < pitch) q[i] = i < p.K ? static_cast<int8_t>(coder.code(to_float(x[r * p.x_stride + i]))) : 0;
  }
  __syncthreads();

  for (; c < p.cols; c += static_cast<int64_t>(gridDim.x) * WARPS) {
    w = p.w + c * p.w_stride;
    int acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0;
    auto add = [&](const uint4& a, int at) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= p.rows) break;
        const uint4 b = *reinterpret_cast<const uint4*>(codes + r * pitch + at);
        acc[r] = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), acc[r]);
        acc[r] = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), acc[r]);
        acc[r] = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), acc[r]);
        acc[r] = __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), acc[r]);
      }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i * 32 + lane < vecs) add(first[i], 16 * (i * 32 + lane));
#pragma unroll 4
    for (int i = AHEAD * 32 + lane; i < vecs; i += 32)
      add(__ldcg(reinterpret_cast<const uint4*>(w) + i), 16 * i);
    // the bytes behind the last whole vector, one to a lane
    if (16 * vecs + lane < p.K) {
      const int b = w[16 * vecs + lane];
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < p.rows) acc[r] += b * codes[r * pitch + 16 * vecs + lane];
    }
    // the next channel's first weights
    const int64_t next = c + static_cast<int64_t>(gridDim.x) * WARPS;
    if (next < p.cols) {
      const uint4* n = reinterpret_cast<const uint4*>(p.w + next * p.w_stride);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i * 32 + lane < vecs) first[i] = __ldcg(n + i * 32 + lane);
    }
    int mine_of = 0;                     // lane r: row r's sum
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int sum = __reduce_add_sync(0xffffffffu, acc[r]);
      if (lane == r) mine_of = sum;
    }
    if (lane < R && lane < p.rows) {
      const float s = RowCoder(largest_of[lane]).scale() * p.w_scale[c];
      static_cast<U*>(p.y)[lane * p.y_stride + c] =
          from_float<U>(fmaf(static_cast<float>(mine_of), s, p.bias ? p.bias[c] : 0.0f));
    }
  }
}

// ------------------------------------------------------------ the product
namespace i8 {

constexpr int BM = 128, BK = 128;          // rows and K bytes of one stage
constexpr int THREADS = 192;               // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue
constexpr unsigned long long kDrainNs = 200000000ull;
constexpr int TURN_PITCH = 33;             // words of a turned row, against bank conflicts
constexpr int TURN_BYTES = 32 * TURN_PITCH * 4;

template <int BN>
struct Smem {
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int TURN = STAGES * STAGE;          // epilogue warps' blocks
  static constexpr int SCALES = TURN + 4 * TURN_BYTES;
  static constexpr int BARS = SCALES + 4 * 2 * BN * 4;   // full, empty, acc_full, drain
  static constexpr int MISC = BARS + (2 * STAGES + 2) * 8;
  static constexpr int ALLOC = MISC + 16 + 1024;
  // a CTA's share of a split sum: 128 rows, padded against bank conflicts
  static constexpr int PITCH = BN + 4;
  static_assert(BM * PITCH * 4 <= TURN, "partial sums take the stages' place");
  static_assert(ALLOC <= 232448, "shared memory exceeds 227 KB");
  static_assert(BN == 64 || BN == 128, "the accumulator takes a power of two of TMEM columns");
};

// s8 x s8 -> s32, dense, both operands K-major
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_lead(uint32_t leader, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                         uint32_t hi, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 e, %6, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::i8 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(id), "r"(accumulate), "r"(leader)
      : "memory");
}

// Waits for the kernel before this one where this one was started ahead of its
// end (the coding of the rows; elsewhere it returns at once).  What that kernel
// writes is read past the read-only cache, which takes its data as constant for
// a kernel's whole time.
__device__ __forceinline__ void rows_are_coded() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// an address of this CTA's shared memory in the CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ int4 ld_peer(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Eight consecutive sums of one row from column c0 on, scaled and stored.
template <typename U>
__device__ __forceinline__ void store_eight(const I8Params& p, int64_t row, int c0, float sx, const int (&acc)[8]) {
  U* y = static_cast<U*>(p.y) + row * p.y_stride + c0;
  const int left = p.cols - c0;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = min(c0 + k, p.cols - 1);
    v[k] = fmaf(static_cast<float>(acc[k]), sx * __ldg(p.w_scale + c), p.bias ? __ldg(p.bias + c) : 0.0f);
  }
  if (p.y_wide && left >= 8) {
    if constexpr (sizeof(U) == 4) {
      __stcs(reinterpret_cast<float4*>(y), make_float4(v[0], v[1], v[2], v[3]));
      __stcs(reinterpret_cast<float4*>(y) + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else {
      __stcs(reinterpret_cast<uint4*>(y), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                     pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) y[k] = from_float<U>(v[k]);
  }
}

// A warp keeps the scales and biases of its tile's N columns (a multiple of 32)
// in shared memory; they are fetched into registers ahead of their use.
template <int N>
struct Scales {
  float s[N / 32], b[N / 32];
  __device__ __forceinline__ void fetch(const I8Params& p, int c0) {
#pragma unroll
    for (int k = 0; k < N / 32; ++k) {
      const int c = c0 + 32 * k + (threadIdx.x & 31);
      const bool in = c < p.cols;
      s[k] = in ? __ldg(p.w_scale + c) : 0.0f;
      b[k] = in && p.bias ? __ldg(p.bias + c) : 0.0f;
    }
  }
  __device__ __forceinline__ void stage(float* scales) const {   // then N biases
    __syncwarp();                                    // the last tile's have been read
#pragma unroll
    for (int k = 0; k < N / 32; ++k) {
      scales[32 * k + (threadIdx.x & 31)] = s[k];
      scales[N + 32 * k + (threadIdx.x & 31)] = b[k];
    }
    __syncwarp();
  }
};

__device__ __forceinline__ void store32(void* y, const uint32_t* w) {   // 32 bytes, so aligned
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A lane's 32 sums of one row, scaled and rounded, as words of y.
template <typename U>
__device__ __forceinline__ void scaled_words(const float* scales, const float* biases, float sx,
                                             const float (&bits)[32], uint32_t (&w)[8 * sizeof(U)]) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float4 s = *reinterpret_cast<const float4*>(scales + k);
    const float4 b = *reinterpret_cast<const float4*>(biases + k);
    const float v0 = fmaf(static_cast<float>(__float_as_int(bits[k])), sx * s.x, b.x);
    const float v1 = fmaf(static_cast<float>(__float_as_int(bits[k + 1])), sx * s.y, b.y);
    const float v2 = fmaf(static_cast<float>(__float_as_int(bits[k + 2])), sx * s.z, b.z);
    const float v3 = fmaf(static_cast<float>(__float_as_int(bits[k + 3])), sx * s.w, b.w);
    if constexpr (sizeof(U) == 4) {
      w[k] = __float_as_uint(v0);
      w[k + 1] = __float_as_uint(v1);
      w[k + 2] = __float_as_uint(v2);
      w[k + 3] = __float_as_uint(v3);
    } else {
      w[k / 2] = pack_bf16x2(v0, v1);
      w[k / 2 + 1] = pack_bf16x2(v2, v3);
    }
  }
}

// Rows of y may start anywhere: then a warp turns its 32 rows through shared
// memory and stores along them, WORDS words of a row to as many lanes.  In
// bf16 a word is two columns; where a row starts in the middle of a word they
// are paired with one column's shift, and its first and last column go alone.
// Whole blocks, which is most of them, take the short loop: with the edges'
// conditions in it 30000 x 1024 x 3001 took 157 us.
template <typename U, int WORDS>
__device__ __forceinline__ void store_turned(const I8Params& p, const uint32_t* turn, int64_t row0, int c0) {
  const int lane = threadIdx.x & 31, l = lane % WORDS;
  constexpr int STEP = 32 / WORDS;                 // rows of one store
  const int left = p.cols - c0, first = lane / WORDS;
  __syncwarp();
  const uint32_t* from = turn + first * TURN_PITCH + l;
  U* y = static_cast<U*>(p.y) + (row0 + first) * p.y_stride + c0;
  if (row0 + 32 <= p.rows && left >= WORDS * static_cast<int>(4 / sizeof(U))) {
    char* at = reinterpret_cast<char*>(y) + 4 * l;
    const int64_t step = p.y_stride * STEP * static_cast<int64_t>(sizeof(U));
    if constexpr (sizeof(U) == 4) {
#pragma unroll 8
      for (int r = 0; r < 32; r += STEP, at += step)
        *reinterpret_cast<uint32_t*>(at) = from[r * TURN_PITCH];
    } else {
      uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(y) & 2);      // bytes
      const uint32_t odd = static_cast<uint32_t>(step & 2);
      const bool edge = l == 0 || l == WORDS - 1;
#pragma unroll 8
      for (int r = 0; r < 32; r += STEP, at += step, shift ^= odd) {
        const uint32_t a = from[r * TURN_PITCH], b = from[r * TURN_PITCH + (l < WORDS - 1)];
        const uint32_t pair = __byte_perm(a, b, shift ? 0x5432 : 0x3210);
        if (!shift || l < WORDS - 1) *reinterpret_cast<uint32_t*>(at + shift) = pair;
        if (shift && edge)
          *reinterpret_cast<unsigned short*>(at + (l ? 2 : 0)) = static_cast<unsigned short>(l ? a >> 16 : a);
      }
    }
  } else {
#pragma unroll 1
    for (int r = 0; r < 32 && row0 + first + r < p.rows; r += STEP, y += p.y_stride * STEP) {
      const uint32_t a = from[r * TURN_PITCH];
      if constexpr (sizeof(U) == 4) {
        if (l < left) y[l] = __uint_as_float(a);
      } else {
        unsigned short* h = reinterpret_cast<unsigned short*>(y) + 2 * l;
        if (2 * l < left) h[0] = static_cast<unsigned short>(a);
        if (2 * l + 1 < left) h[1] = static_cast<unsigned short>(a >> 16);
      }
    }
  }
  __syncwarp();     // read before the next block is written
}

// A warp's 32 rows x 32 columns, one row to a lane.  Where rows of y start at
// 32-byte boundaries (y_wide 2) each lane stores whole sectors of its row, at
// 16-byte boundaries (1) halves of them; else as above.
template <typename U>
__device__ __forceinline__ void store_block(const I8Params& p, uint32_t* turn, const float* scales,
                                            const float* biases, int64_t row, int c0, float sx,
                                            const float (&bits)[32]) {
  constexpr int W = 8 * sizeof(U);                   // words of the block's row
  uint32_t w[W];
  scaled_words<U>(scales, biases, sx, bits, w);
  if (!p.y_wide || c0 + 32 > p.cols) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < W; ++k) turn[lane * TURN_PITCH + k] = w[k];
    store_turned<U, W>(p, turn, row - lane, c0);
    return;
  }
  if (row >= p.rows) return;
  uint32_t* y = reinterpret_cast<uint32_t*>(static_cast<U*>(p.y) + row * p.y_stride + c0);
  if (p.y_wide == 2) {
#pragma unroll
    for (int k = 0; k < W; k += 8) store32(y + k, w + k);
  } else {
#pragma unroll
    for (int k = 0; k < W; k += 4)
      *reinterpret_cast<uint4*>(y + k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
  }
}

}  // namespace i8

// One output tile of 128 rows x BN channels for each cluster; its CTAs take
// equal shares of K (cluster dimension = split) and add their sums through
// distributed shared memory, each finishing BN / split of the columns.
template <int BN, typename U>
__global__ void __launch_bounds__(i8::THREADS, 1)
relkl_gemm_i8_kernel(const __grid_constant__ I8Params p) {
  using namespace i8;
  using S = Smem<BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + S::BARS;
  auto FULL = [&](int s) { return bars + 8u * s; };
  auto EMPTY = [&](int s) { return bars + 8u * (S::STAGES + s); };
  const uint32_t ACC = bars + 8u * (2 * S::STAGES), DRAIN = ACC + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + S::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + S::MISC + 4);
  WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  const int tile = blockIdx.x / p.split;
  const int rank = blockIdx.x % p.split;
  const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.k_chunks) * rank / p.split);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.k_chunks) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), 1);
    }
    mbar_init(ACC, 1);
    mbar_init(DRAIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t arms[S::STAGES] = {};
      // the weights of the first stages, which no kernel before this one
      // writes, are on their way while the rows are still being coded
      const uint32_t stage_bytes = p.a_box * BK + S::B_BYTES;
      const int early = min(k1 - k0, S::STAGES);
      for (int it = 0; it < early; ++it) {
        mbar_arrive_expect_tx(FULL(it), stage_bytes);
        tma_load_2d(base + it * S::STAGE + S::A_BYTES, &p.tm_b, FULL(it), (k0 + it) * BK, nt * BN);
        ++arms[it];
      }
      rows_are_coded();
      for (int it = 0; it < early; ++it)
        tma_load_2d(base + it * S::STAGE, &p.tm_a, FULL(it), (k0 + it) * BK, mt * BM);
      for (int kc = k0 + early, it = early; kc < k1; ++kc, ++it) {
        const int s = it % S::STAGES;
        if (!mbar_wait(EMPTY(s), ((it / S::STAGES) & 1) ^ 1, wc, W_TMA_EMPTY_J)) break;
        const uint32_t a = base + s * S::STAGE;
        mbar_arrive_expect_tx(FULL(s), stage_bytes);
        tma_load_2d(a, &p.tm_a, FULL(s), kc * BK, mt * BM);
        tma_load_2d(a + S::A_BYTES, &p.tm_b, FULL(s), kc * BK, nt * BN);
        ++arms[s];
      }
      for (int s = 0; s < S::STAGES; ++s)
        if (arms[s]) mbar_wait_drain(FULL(s), (arms[s] - 1) & 1, kDrainNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t lead = elect_leader();
    constexpr uint32_t ID = idesc(BM, BN);
    const uint32_t HI = sw128_desc_hi(1024);
    const uint32_t a0 = sw128_desc_lo(base, 16), b0 = sw128_desc_lo(base + S::A_BYTES, 16);
    bool issued = false;
    for (int kc = k0, it = 0; kc < k1; ++kc, ++it) {
      const int s = it % S::STAGES;
      if (!mbar_wait_warp(FULL(s), (it / S::STAGES) & 1, wc, W_MMA_FULL_J)) break;
      tc_fence_after();
      const uint32_t step = s * (S::STAGE >> 4);
#pragma unroll
      for (int k = 0; k < BK / 32; ++k)     // 32 K bytes an instruction
        mma_lead(lead, tmem, a0 + step + 2 * k, b0 + step + 2 * k, HI, ID, (it > 0 || k > 0) ? 1u : 0u);
      issued = true;
      umma_commit_lead(lead, EMPTY(s));
      if (kc == k1 - 1) umma_commit_lead(lead, ACC);
    }
    if (issued) {
      umma_commit_lead(lead, DRAIN);
      mbar_wait_drain(DRAIN, 0, kDrainNs);
    }
    __syncwarp();
  }
  const int q = warp & 3;      // TMEM lane quarter of an epilogue warp
  const int64_t row = static_cast<int64_t>(mt) * BM + q * 32 + lane;
  const bool live = warp >= 2 && row < p.rows;
  if (warp >= 2) rows_are_coded();
  const float sx = live ? __ldcg(p.x_scale + row) : 0.0f;
  uint32_t* turn = reinterpret_cast<uint32_t*>(gbase + S::TURN + (warp & 3) * TURN_BYTES);
  float* scales = reinterpret_cast<float*>(gbase + S::SCALES) + (warp & 3) * 2 * BN;
  if (warp >= 2) {
    if (p.split == 1) {
      Scales<BN> columns;
      columns.fetch(p, nt * BN);
      columns.stage(scales);
    }
    bool ok = mbar_wait(ACC, 0, wc, W_EPI_P_FULL);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const uint32_t addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        float bits[32];
        tmem_ld32(addr + c, bits);
        tmem_wait_ld();
        if (p.split == 1) {
          if (nt * BN + c < p.cols)
            store_block<U>(p, turn, scales + c, scales + BN + c, row, nt * BN + c, sx, bits);
        } else {
          const uint32_t dst = base + ((q * 32 + lane) * S::PITCH + c) * 4;
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            st_shared_v4(dst + 4 * k, __float_as_uint(bits[k]), __float_as_uint(bits[k + 1]),
                         __float_as_uint(bits[k + 2]), __float_as_uint(bits[k + 3]));
        }
      }
      tc_fence_before();
    }
  }
  if (p.split > 1) {
    cluster_sync();       // every CTA's sums are in its shared memory
    if (live) {
      const int width = BN / p.split;     // a multiple of 8
      const uint32_t src = base + ((q * 32 + lane) * S::PITCH + rank * width) * 4;
#pragma unroll 1
      for (int c = 0; c < width; c += 8) {
        const int col = nt * BN + rank * width + c;
        if (col >= p.cols) break;
        int acc[8] = {};
        for (int r = 0; r < p.split; ++r) {
          const uint32_t from = peer(src + 4 * c, r);
          const int4 u = ld_peer(from), v = ld_peer(from + 16);
          acc[0] += u.x; acc[1] += u.y; acc[2] += u.z; acc[3] += u.w;
          acc[4] += v.x; acc[5] += v.y; acc[6] += v.z; acc[7] += v.w;
        }
        store_eight<U>(p, row, col, sx, acc);
      }
    }
    __syncwarp();
    cluster_sync();       // nobody leaves while its memory is read
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, BN);
  }
}

// ------------------------------------------------- the product, CTA pairs
// A pair of CTAs (cta_group::2) computes 256 rows x BN channels: each holds its
// 128 rows of q and half of the channels' codes, so an SM reads (128 + BN / 2)
// x 32 bytes of shared memory for an instruction where one CTA by itself reads
// (128 + BN) x 32; at the int8 rate the latter needs more than the 128 bytes a
// clock that an SM has (32K x 4096 x 4096 with its coding: 936 us, then 437).
// Persistent; the sums of one tile are read from TMEM while the next one's are
// formed.  What the tiles fetch from L2, 15 TB/s, is next to bound it: results
// that left lane by lane (32 bytes of a row each) cost 372 us, as whole lines
// by TMA 337 at the same clock.
namespace i8 {

// warp 0 TMA, warp 1 MMA, warps 2-9 epilogue: two for each quarter of the
// TMEM lanes, one for each half of the columns
constexpr int PAIR_EPI = 8, PAIR_THREADS = 64 + 32 * PAIR_EPI;

template <int BN>
struct PairSmem {
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN / 2 * BK;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 5;
  static constexpr int OUT = STAGES * STAGE;           // epilogue warps' boxes of y, or turned blocks
  static constexpr int OUT_BYTES = 5120;
  static constexpr int SCALES = OUT + PAIR_EPI * OUT_BYTES;
  static constexpr int BARS = SCALES + PAIR_EPI * BN * 4;   // full, empty, acc_full[2], acc_empty[2], drain
  static constexpr int MISC = BARS + (2 * STAGES + 5) * 8;
  static constexpr int ALLOC = MISC + 16 + 1024;
  static_assert(ALLOC <= 232448, "shared memory exceeds 227 KB");
  static_assert(OUT % 1024 == 0 && OUT_BYTES % 1024 == 0 && OUT_BYTES >= TURN_BYTES, "swizzled boxes");
  static_assert(BN == 128 || BN == 256, "two accumulators take a power of two of TMEM columns");
};

// a load into this CTA's shared memory that signals the barrier `bar` of the
// pair's first CTA
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t leader, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                         uint32_t hi, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 e, %6, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::i8 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(id), "r"(accumulate), "r"(leader)
      : "memory");
}
// arrives at `bar` of both CTAs when the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 both;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "mov.b16 both, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], both;\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
// arrives at `bar` of this CTA when the MMAs issued so far are done
__device__ __forceinline__ void commit_own(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
// Without .release.cluster, which waits for the warp's stores to y (1.8 of 12.9
// stalled warps at K = 1024): what it hands over are TMEM columns, read to the
// end and ordered by tcgen05's own fences.
__device__ __forceinline__ void arrive_peer(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_wait_warp for arrivals from the other CTA
__device__ __forceinline__ bool wait_warp_cluster(uint32_t bar, uint32_t parity, const WaitCtl& c,
                                                  unsigned int where) {
  auto done = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  };
  bool ok = done();
  const unsigned long long t0 = globaltimer_ns();
  while (!ok) {
#pragma unroll 1
    for (int i = 0; i < 16 && !ok; ++i) ok = done();
    if (ok || *c.abort_flag) break;
    if (globaltimer_ns() - t0 > c.timeout_ns) {
      record_timeout(c, where);
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Tiles in bands of kBand rows of tiles, each band along all channels: the
// pairs that run together share a few rows' and a few channels' codes, which
// stay in L2 while the band lasts.
constexpr int kBand = 8;
__device__ __forceinline__ void pair_unit(const I8Params& p, int unit, int& mt, int& nt) {
  const int band = unit / (kBand * p.n_tiles), first = band * kBand;
  const int in = unit - band * kBand * p.n_tiles, high = min(kBand, p.m_tiles - first);
  mt = first + in % high;
  nt = in / high;
}

}  // namespace i8

template <int BN, typename U>
__global__ void __launch_bounds__(i8::PAIR_THREADS, 1)
relkl_gemm_i8_pair_kernel(const __grid_constant__ I8Params p) {
  using namespace i8;
  using S = PairSmem<BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;   // the same in both CTAs
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t bars = base + S::BARS;
  auto FULL = [&](int s) { return bars + 8u * s; };                       // the first CTA's are used
  auto EMPTY = [&](int s) { return bars + 8u * (S::STAGES + s); };        // each CTA's own
  auto ACC_FULL = [&](int b) { return bars + 8u * (2 * S::STAGES + b); };  // each CTA's own
  auto ACC_EMPTY = [&](int b) { return bars + 8u * (2 * S::STAGES + 2 + b); };   // the first CTA's
  const uint32_t DRAIN = bars + 8u * (2 * S::STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + S::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + S::MISC + 4);
  WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(ACC_FULL(b), 1);
      mbar_init(ACC_EMPTY(b), 2 * PAIR_EPI);   // the epilogue warps of both CTAs
    }
    mbar_init(DRAIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();       // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_a);
      tma_prefetch_desc(&p.tm_b);
      uint32_t it = 0;
      uint32_t arms[S::STAGES] = {};
      bool ok = true;
      int early = 0;
      for (int unit = first; ok && unit < p.n_units; unit += stride) {
        int mt, nt;
        pair_unit(p, unit, mt, nt);
        const int row = mt * 2 * BM + static_cast<int>(rank) * BM;
        const int col = nt * BN + static_cast<int>(rank) * (BN / 2);
        if (unit == first) {      // weights before the rows are coded, as above
          early = min(p.k_chunks, S::STAGES);
          for (int s = 0; s < early; ++s) {
            if (rank == 0) mbar_arrive_expect_tx(FULL(s), 2 * S::STAGE);
            load_pair(base + s * S::STAGE + S::A_BYTES, &p.tm_b, peer(FULL(s), 0), s * BK, col);
            ++arms[s];
          }
          rows_are_coded();
          for (int s = 0; s < early; ++s)
            load_pair(base + s * S::STAGE, &p.tm_a, peer(FULL(s), 0), s * BK, row);
          it = early;
        }
        for (int kc = unit == first ? early : 0; kc < p.k_chunks; ++kc, ++it) {
          const int s = it % S::STAGES;
          if (!(ok = mbar_wait(EMPTY(s), ((it / S::STAGES) & 1) ^ 1, wc, W_TMA_EMPTY_J))) break;
          const uint32_t a = base + s * S::STAGE;
          const uint32_t full = peer(FULL(s), 0);
          if (rank == 0) mbar_arrive_expect_tx(FULL(s), 2 * S::STAGE);   // both CTAs' bytes
          ++arms[s];
          load_pair(a, &p.tm_a, full, kc * BK, row);
          load_pair(a + S::A_BYTES, &p.tm_b, full, kc * BK, col);
        }
      }
      // the copies of both CTAs, and the first CTA's arrivals at these
      // barriers, before either leaves
      for (int s = 0; s < S::STAGES; ++s) {
        if (arms[s] == 0) continue;
        if (rank == 0) mbar_wait_drain(FULL(s), (arms[s] - 1) & 1, kDrainNs);
        mbar_wait_drain(EMPTY(s), (arms[s] - 1) & 1, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t lead = elect_leader();
      constexpr uint32_t ID = idesc(2 * BM, BN);
      const uint32_t HI = sw128_desc_hi(1024);
      const uint32_t a0 = sw128_desc_lo(base, 16), b0 = sw128_desc_lo(base + S::A_BYTES, 16);
      uint32_t it = 0, nacc = 0;
      bool ok = true, issued = false;
      for (int unit = first; ok && unit < p.n_units; unit += stride, ++nacc) {
        const int ab = nacc & 1;
        if (!(ok = wait_warp_cluster(ACC_EMPTY(ab), ((nacc >> 1) & 1) ^ 1, wc, W_MMA_P_EMPTY))) break;
        tc_fence_after();
        for (int kc = 0; kc < p.k_chunks; ++kc, ++it) {
          const int s = it % S::STAGES;
          if (!(ok = mbar_wait_warp(FULL(s), (it / S::STAGES) & 1, wc, W_MMA_FULL_J))) break;
          tc_fence_after();
          const uint32_t step = s * (S::STAGE >> 4);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            mma_pair(lead, tmem + ab * BN, a0 + step + 2 * k, b0 + step + 2 * k, HI, ID,
                     (kc > 0 || k > 0) ? 1u : 0u);
          issued = true;
          commit_pair(lead, EMPTY(s));
        }
        if (!ok) break;
        commit_pair(lead, ACC_FULL(ab));
      }
      if (issued) {
        commit_own(lead, DRAIN);
        mbar_wait_drain(DRAIN, 0, kDrainNs);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3, epi = warp - 2;
    const uint32_t box = base + S::OUT + epi * S::OUT_BYTES;
    uint32_t* turn = reinterpret_cast<uint32_t*>(gbase + S::OUT + epi * S::OUT_BYTES);
    float* scales = reinterpret_cast<float*>(gbase + S::SCALES) + epi * BN;   // and biases
    constexpr int COLS = BN / 2;
    const int half = (epi >> 2) * COLS;
    const uint32_t lane_addr = (static_cast<uint32_t>(q * 32) << 16) + half;
    uint32_t nacc = 0;
    rows_are_coded();
    // the next tile's place and scales are fetched while this one's sums are
    // still being formed
    int64_t row_next = 0;
    int col_next = 0;
    float sx_next = 0.0f;
    Scales<COLS> columns;
    auto fetch = [&](int unit) {
      int mt, nt;
      pair_unit(p, unit, mt, nt);
      row_next = static_cast<int64_t>(mt) * 2 * BM + rank * BM + q * 32 + lane;
      col_next = nt * BN + half;
      sx_next = row_next < p.rows ? __ldcg(p.x_scale + row_next) : 0.0f;
      columns.fetch(p, col_next);
    };
    if (first < p.n_units) fetch(first);
    for (int unit = first; unit < p.n_units; unit += stride, ++nacc) {
      const int ab = nacc & 1;
      const int64_t row = row_next;
      const int col = col_next;
      const float sx = sx_next;
      columns.stage(scales);
      if (unit + stride < p.n_units) fetch(unit + stride);
      if (!mbar_wait_warp(ACC_FULL(ab), (nacc >> 1) & 1, wc, W_EPI_P_FULL)) break;
      tc_fence_after();
      float bits[2][32];
      const uint32_t acc = tmem + lane_addr + ab * BN;
      tmem_ld32(acc, bits[0]);
#pragma unroll
      for (int k = 0; k < COLS / 32; ++k) {
        tmem_wait_ld();
        if (k + 1 < COLS / 32) {
          tmem_ld32(acc + 32 * (k + 1), bits[(k + 1) & 1]);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_peer(peer(ACC_EMPTY(ab), 0));
        }
        const int c = col + 32 * k;
        constexpr int W = 8 * sizeof(U), PER = 128 / (4 * W);   // words of a block's row; blocks of 128 bytes
        const int part = k % PER, c_box = c - 32 * part;
        uint32_t w[W];
        scaled_words<U>(scales + 32 * k, scales + COLS + 32 * k, sx, bits[k & 1], w);
        if (!p.y_wide) {
#pragma unroll
          for (int j = 0; j < W; ++j) turn[lane * TURN_PITCH + part * W + j] = w[j];
          if (part == PER - 1 && c_box < p.cols) store_turned<U, 32>(p, turn, row - lane, c_box);
          continue;
        }
        // boxes of 32 rows x 128 bytes, swizzled against bank conflicts, go to
        // y by TMA: whole lines, and what lies past the edges is left out, but
        // only in units of 16 bytes; the columns of a last, partial unit are
        // stored by themselves
        if (p.box_cols < p.cols && c + 32 > p.box_cols && row < p.rows) {
          U* y = static_cast<U*>(p.y) + row * p.y_stride + c;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j >= p.box_cols && c + j < p.cols) {
              if constexpr (sizeof(U) == 4)
                y[j] = __uint_as_float(w[j]);
              else
                reinterpret_cast<unsigned short*>(y)[j] = static_cast<unsigned short>(w[j / 2] >> (16 * (j & 1)));
            }
        }
        if (part == 0) {
          if (lane == 0) bulk_wait_read<0>();                   // the last box has been read
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < W / 4; ++j)
          st_shared_v4(box + lane * 128 + (((part * (W / 4) + j) ^ (lane & 7)) << 4), w[4 * j], w[4 * j + 1],
                       w[4 * j + 2], w[4 * j + 3]);
        if (part == PER - 1) {
          fence_proxy_async_smem();
          __syncwarp();
          const int64_t r_box = row - lane;
          if (lane == 0) {
            if (c_box < p.box_cols && r_box < p.rows) tma_store_2d(&p.tm_y, box, c_box, static_cast<int>(r_box));
            bulk_commit();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();       // no copy, product or arrival is under way in the pair
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN)
                 : "memory");
  }
}

// ------------------------------------------------------------- launches
namespace {

template <typename T>
cudaError_t quantize_rows(const RowsParams& p, int num_sms, cudaStream_t stream) {
  constexpr int one = 8 * kRowGroups * 32;   // a warp's elements
  int threads = (p.K + one - 1) / one * 32;
  threads = threads > 512 ? 512 : threads;
  if (threads == 32)
    relkl_quantize_rows_kernel<T, true><<<static_cast<unsigned>((p.rows + 7) / 8), 256, 0, stream>>>(p);
  else
    relkl_quantize_rows_kernel<T, false><<<static_cast<unsigned>(p.rows), threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(const RowsParams& p, bool x_bf16, int num_sms, cudaStream_t stream) {
  return x_bf16 ? quantize_rows<__nv_bfloat16>(p, num_sms, stream) : quantize_rows<float>(p, num_sms, stream);
}

namespace {

template <typename T, typename U, int R>
cudaError_t gemv(const GemvParams& p, int num_sms, cudaStream_t stream) {
  const int smem = p.rows * ((p.K + 15) / 16 * 16);
  cudaError_t e = cudaSuccess;
  // the most that any call takes, not this one's: the limit is the process's, and
  // another thread's launch may come between a smaller one and its own
  constexpr int fixed = R * (GEMV_THREADS / 32 + 1) * 4;   // the kernel's part[] and largest_of[]
  if (smem + fixed > 48 * 1024)
    e = cudaFuncSetAttribute(relkl_gemv_i8_kernel<T, U, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemvBytes);
  if (e != cudaSuccess) return e;
  // as many CTAs as the SMs hold at a time: more would code the rows once more
  const int need = (p.cols + GEMV_THREADS / 32 - 1) / (GEMV_THREADS / 32);
  const int most = num_sms * 2;
  relkl_gemv_i8_kernel<T, U, R><<<need < most ? need : most, GEMV_THREADS, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, typename U>
cudaError_t gemv_rows(const GemvParams& p, int num_sms, cudaStream_t stream) {
  if (p.rows == 1) return gemv<T, U, 1>(p, num_sms, stream);
  return gemv<T, U, kGemvRows>(p, num_sms, stream);
}

// K-major codes [rows, K] of `stride` bytes a row, as boxes of 128 bytes x `box` rows
bool encode_codes(CUtensorMap* m, const int8_t* q, int64_t rows, int K, int64_t stride, int box,
                  EncodeTiled encode) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t boxes[2] = {i8::BK, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(q), dims, strides, boxes, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y's first box_cols columns as boxes of 32 rows x 128 bytes
template <typename U>
bool encode_out(CUtensorMap* m, const I8Params& p, EncodeTiled encode) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.box_cols), static_cast<cuuint64_t>(p.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.y_stride) * sizeof(U)};
  const cuuint32_t boxes[2] = {128 / sizeof(U), 32}, ones[2] = {1, 1};
  return encode(m, sizeof(U) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.y,
                dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t launch_cluster(K kernel, const I8Params& p, unsigned grid, int threads, int cluster,
                           int smem, bool ahead, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ahead ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int BN, typename U>
cudaError_t gemm(I8Params& p, const I8Call& c, cudaStream_t stream) {
  using S = i8::Smem<BN>;
  p.m_tiles = static_cast<int>((p.rows + i8::BM - 1) / i8::BM);
  // A box of rows only as high as there are rows (in eights, the swizzle's
  // period): filling the rest of 128 with zeros costs more than reading them
  // would, 27 us instead of 18 for 9 x 8192 x 8192.  The rows behind the box
  // hold whatever the stage held; their sums are not stored.
  p.a_box = p.rows < i8::BM ? static_cast<int>((p.rows + 7) / 8 * 8) : i8::BM;
  if (!encode_codes(&p.tm_a, c.q, p.rows, c.K, c.q_stride, p.a_box, c.encode) ||
      !encode_codes(&p.tm_b, c.w, p.cols, c.K, c.w_stride, BN, c.encode))
    return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * ((p.cols + BN - 1) / BN);
  if (tiles * p.split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto* kernel = relkl_gemm_i8_kernel<BN, U>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::ALLOC);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, p, static_cast<unsigned>(tiles * p.split), i8::THREADS, p.split, S::ALLOC, c.after_rows, stream);
}

template <int BN, typename U>
cudaError_t gemm_pair(I8Params& p, const I8Call& c, int num_sms, cudaStream_t stream) {
  using S = i8::PairSmem<BN>;
  const int64_t m = (p.rows + 2 * i8::BM - 1) / (2 * i8::BM), n = (p.cols + BN - 1) / BN;
  constexpr int unit = 16 / sizeof(U);             // columns of 16 bytes
  p.box_cols = p.cols / unit * unit;
  if (p.box_cols == 0) p.y_wide = 0;
  if (!encode_codes(&p.tm_a, c.q, p.rows, c.K, c.q_stride, i8::BM, c.encode) ||
      !encode_codes(&p.tm_b, c.w, p.cols, c.K, c.w_stride, BN / 2, c.encode) ||
      (p.y_wide && !encode_out<U>(&p.tm_y, p, c.encode)))
    return cudaErrorInvalidValue;
  if (m * n + num_sms > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  p.m_tiles = static_cast<int>(m);
  p.n_tiles = static_cast<int>(n);
  p.n_units = static_cast<int>(m * n);
  auto* kernel = relkl_gemm_i8_pair_kernel<BN, U>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::ALLOC);
  if (e != cudaSuccess) return e;
  const int pairs = p.n_units < num_sms / 2 ? p.n_units : num_sms / 2;
  return launch_cluster(kernel, p, 2 * pairs, i8::PAIR_THREADS, 2, S::ALLOC, c.after_rows, stream);
}

// Four ways by the width of a tile, the one with the least estimated time:
// waves of tiles times the time of one wave, as measured (K = 4096, full
// waves: 9.3 us with one CTA and 64 columns, 11.0 with 128; pairs 8.5 with 128
// columns, 11.3 with 256; a single wave 10.9, 11.6, 11.6 and 15.0 us, so that
// pairs with 128 are counted as 9.5).  K = 4096, 4096 channels, weights from HBM:
// 128 and 256 rows take 64 columns a tile (12.4 and 11.9 us; the others 12.8 to
// 16.2), 500 rows pairs with 128 (13.5; one CTA with 128 13.1, with 64 21.6), 1000
// rows pairs with 256 (16.9; 39.7, 23.8 and 21.0).  The same weights for every K:
// at K of 256, 512 and 1024 (16 to 16384 rows, 1024 and 4096 channels) the choice
// was the fastest of the four or within 12 % of it (1000 x 512 x 4096 8.0 us,
// pairs with 128 7.2).
//
// Where tiles of 64 columns leave SMs idle, K is split over two or four of them.
// The shares' sums meet in shared memory, which costs as much as some chunks of K
// and one more for each 8 rows of a tile.  One share and four, 1024 channels,
// weights from HBM: 5 rows at K = 1280 5.0 and 5.1 us, 1536 5.4 and 5.2; 32 rows 1536
// 5.5 and 5.7, 1792 6.1 and 6.0; 77 rows 2304 7.4 and 7.7, 2560 8.1 and 7.9, 4096 10.8
// and 8.6; 128 rows 2560 8.3 and 9.0, 3584 10.0 and 9.7.  One and two, where four
// are more than the SMs (4096 channels): 5 rows at 3584 10.1 and 10.3, 4096 11.2 and
// 10.9; 32 rows 4096 11.2 and 11.1; 77 rows 4096 11.3 and 11.5, 8192 18.7 and 15.6.
template <typename U>
cudaError_t gemm_pick(I8Params& p, const I8Call& c, int num_sms, cudaStream_t stream) {
  p.k_chunks = (c.K + i8::BK - 1) / i8::BK;
  p.split = 1;
  auto tiles = [&](int bm, int bn) { return (p.rows + bm - 1) / bm * ((p.cols + bn - 1) / bn); };
  auto cost = [&](int64_t n, int at_once, int wave) { return (n + at_once - 1) / at_once * wave; };
  const int pairs = num_sms / 2;
  const int64_t t64 = tiles(i8::BM, 64);
  const int64_t one64 = cost(t64, num_sms, 93), one128 = cost(tiles(i8::BM, 128), num_sms, 110);
  const int64_t two128 = cost(tiles(2 * i8::BM, 128), pairs, 95);
  const int64_t two256 = cost(tiles(2 * i8::BM, 256), pairs, 115);
  const int64_t least = std::min(std::min(one64, one128), std::min(two128, two256));
  if (two256 == least) return gemm_pair<256, U>(p, c, num_sms, stream);
  if (one64 == least) {
    const int meet = static_cast<int>(std::min<int64_t>(p.rows, i8::BM)) / 8;
    if (t64 * 4 <= num_sms && p.k_chunks >= 12 + meet)
      p.split = 4;
    else if (t64 * 2 <= num_sms && p.k_chunks >= 28 + meet)
      p.split = 2;
    return gemm<64, U>(p, c, stream);
  }
  if (two128 == least) return gemm_pair<128, U>(p, c, num_sms, stream);
  return gemm<128, U>(p, c, stream);
}

}  // namespace

cudaError_t launch_gemv_i8(const GemvParams& p, bool x_bf16, bool y_bf16, int num_sms, cudaStream_t stream) {
  using H = __nv_bfloat16;
  if (x_bf16) return y_bf16 ? gemv_rows<H, H>(p, num_sms, stream) : gemv_rows<H, float>(p, num_sms, stream);
  return y_bf16 ? gemv_rows<float, H>(p, num_sms, stream) : gemv_rows<float, float>(p, num_sms, stream);
}

cudaError_t launch_gemm_i8(I8Params& p, const I8Call& c, bool y_bf16, int num_sms, cudaStream_t stream) {
  return y_bf16 ? gemm_pick<__nv_bfloat16>(p, c, num_sms, stream) : gemm_pick<float>(p, c, num_sms, stream);
}

}  // namespace relkl
