// One AdamW step over many tensors, and the norm of all their gradients:
//
//   g = coef * grad
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// The states m and v are float32, or 8-bit: each block of 256 consecutive
// elements holds m and r = sqrt(v) as e4m3 numbers times one float32 scale,
// its largest magnitude / 448.  The root is held and not v because an e4m3
// block spans 2^18: of v that would leave gradients 2^9 apart, of r it leaves
// 2^18.  A positive r below the smallest code is held as the smallest code,
// never as zero, so that no element's step is divided by eps alone.  p is
// updated from the new m and v before they are rounded to codes.
//
// What bounds it: HBM.  Every byte is read once and written once (26 to 30 B
// an element with float32 states and weights, by the gradient's type and the
// copies, and 14 to 18 with 8-bit states; bf16 weights and gradients 22 and 10),
// all tensors of a call go in one launch (their table travels in the kernel's
// parameters, so a captured graph needs no memory of its own for it), and the
// statistics of an 8-bit block stay in the registers of its warp.
//
// Measured (B200, copy bandwidth 6.56 TB/s), 201 M float32 weights with bf16
// copies and gradients: float32 states 824 us, 6.8 TB/s; 8-bit states 492 us, 6.6
// TB/s.  The 8-bit step is close to the issue rate too: with correctly rounded
// roots and quotients (99 instructions an element) it took 693 us in an earlier
// form, with one block for a warp 536 us, and with a lane's eight elements next to
// one another, so that each access touched half of its sectors, 569 us.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "relkl_params.h"

namespace relkl {

namespace {

constexpr int THREADS = 128;
// elements of one CTA: with 8-bit states a block for each warp, or two
constexpr int CHUNK = 1024;
constexpr int BLOCK8 = 256;
constexpr float E4M3_MAX = 448.0f;
constexpr float E4M3_MIN = 0.001953125f;   // 2^-9, the smallest positive code
constexpr float TINY = 1.1754943508222875e-38f;

struct Hyper {
  float coef, b1, c1, b2, c2, eps;
  float rbc2, step, decay;   // 1 / sqrt(1 - b2^t), lr / (1 - b1^t), 1 - lr wd
  bool skip;
};

// The step's scalars.  lr and the step number may live on the device, so that
// a replayed graph takes their values at the time; then one thread of a block
// forms what depends on them, in double precision as the host does otherwise.
__device__ __forceinline__ Hyper hyper(const AdamwPlan& a, const AdamwTensor& t) {
  Hyper h;
  h.coef = a.grad_scale ? *a.grad_scale : 1.0f;
  h.skip = !isfinite(h.coef);
  h.b1 = a.b1;
  h.c1 = a.c1;
  h.b2 = a.b2;
  h.c2 = a.c2;
  h.eps = a.eps;
  h.rbc2 = a.rbc2;
  h.step = a.step_size;
  h.decay = t.decay;
  if (a.lr_dev || a.step_dev) {
    __shared__ float formed[3];
    if (threadIdx.x == 0) {
      const double lr = a.lr_dev ? static_cast<double>(*a.lr_dev) : a.lr;
      double bc1 = a.bc1, bc2 = a.bc2;
      if (a.step_dev) {
        const double n = static_cast<double>(*a.step_dev);
        bc1 = -expm1(n * a.log_b1);
        bc2 = -expm1(n * a.log_b2);
      }
      formed[0] = static_cast<float>(1.0 / sqrt(bc2));
      formed[1] = static_cast<float>(lr / bc1);
      formed[2] = static_cast<float>(1.0 - lr * t.weight_decay);
    }
    __syncthreads();
    h.rbc2 = formed[0];
    h.step = formed[1];
    h.decay = formed[2];
  }
  return h;
}

__device__ __forceinline__ float moved(const Hyper& h, float p, float m, float root) {
  return fmaf(p, h.decay, -h.step * (m / fmaf(root, h.rbc2, h.eps)));
}

__device__ __forceinline__ float next_m(const Hyper& h, float m, float g) {
  return fmaf(h.c1, g, h.b1 * m);
}
__device__ __forceinline__ float next_v(const Hyper& h, float v, float g) {
  return fmaf(h.c2, g * g, h.b2 * v);
}
__device__ __forceinline__ void update(const Hyper& h, float g, float& p, float& m, float& v) {
  g *= h.coef;
  m = next_m(h, m, g);
  v = next_v(h, v, g);
  p = moved(h, p, m, sqrtf(v));
}

// --------------------------------------------------------- accesses
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4) return __ldcg(p);
  return __uint_as_float(
      static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short*>(p))) << 16);
}
template <typename T>
__device__ __forceinline__ void store1(T* p, float v) {
  if constexpr (sizeof(T) == 4)
    __stcg(p, v);
  else
    __stcg(reinterpret_cast<unsigned short*>(p), __bfloat16_as_ushort(__float2bfloat16_rn(v)));
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
    const uint2 x = __ldcg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    __stcg(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    __stcg(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                   *reinterpret_cast<const uint32_t*>(&b)));
  }
}

// --------------------------------------------------- float32 states
template <typename G, typename P>
__device__ void chunk32(const AdamwTensor& t, const Hyper& h, int64_t begin) {
  const G* g = static_cast<const G*>(t.grad);
  P* p = static_cast<P*>(t.param);
  float *m = static_cast<float*>(t.m), *v = static_cast<float*>(t.v);
  __nv_bfloat16* c = static_cast<__nv_bfloat16*>(t.copy);
  const int64_t end = min(begin + CHUNK, t.n);
  const int64_t wide = t.wide ? begin + (end - begin) / 4 * 4 : begin;
#pragma unroll 1
  for (int64_t i = begin + 4 * threadIdx.x; i < wide; i += 4 * THREADS) {
    float gg[4], pp[4], mm[4], vv[4];
    load4(g + i, gg);
    load4(p + i, pp);
    load4(m + i, mm);
    load4(v + i, vv);
#pragma unroll
    for (int k = 0; k < 4; ++k) update(h, gg[k], pp[k], mm[k], vv[k]);
    store4(p + i, pp);
    store4(m + i, mm);
    store4(v + i, vv);
    if (c) store4(c + i, pp);
  }
#pragma unroll 2
  for (int64_t i = wide + threadIdx.x; i < end; i += THREADS) {
    float pp = load1(p + i), mm = load1(m + i), vv = load1(v + i);
    update(h, load1(g + i), pp, mm, vv);
    store1(p + i, pp);
    store1(m + i, mm);
    store1(v + i, vv);
    if (c) store1(c + i, pp);
  }
}

// ----------------------------------------------------- 8-bit states
__device__ __forceinline__ float decode1(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}
__device__ __forceinline__ void decode4(uint32_t codes, float* v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2 x(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(codes >> (16 * k)), __NV_E4M3));
    const float2 f = __half22float2(x);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t encode4(const float* v) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The larger of a and |b|, NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}

// The largest of the warp's non-negative numbers, a NaN if there is one (its
// bits are larger than infinity's).
__device__ __forceinline__ float warp_largest(float most) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu));
}

// Codes of x / scale for the e4m3 numbers of a block.  They are wanted exactly:
// a code that fell on the other side of a rounding border would change the
// moment by a sixteenth, and what follows from it.  So x is multiplied with a
// number just above and one just below 1 / scale, and where the two products
// have the same code (all but one lane in some thousand) that is the quotient's.
struct Coder {
  float scale, up, down;
  __device__ __forceinline__ explicit Coder(float most) {
    scale = most / E4M3_MAX;
    if (scale < TINY) scale = 0.0f;
    const float inv = scale > 0.0f ? 1.0f / scale : 0.0f;
    up = inv * (1.0f + 0x1p-20f);
    down = inv * (1.0f - 0x1p-20f);
  }
  // x may be off by 2^-22 of itself; false where that could matter
  __device__ __forceinline__ bool codes(const float (&x)[8], uint2& out) const {
    float a[8], b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = x[k] * up;
      b[k] = x[k] * down;
    }
    out = make_uint2(encode4(a), encode4(a + 4));
    return out.x == encode4(b) && out.y == encode4(b + 4);
  }
  __device__ __forceinline__ void quotients(float (&x)[8]) const {
#pragma unroll 1
    for (int k = 0; k < 8; ++k) x[k] = scale > 0.0f ? x[k] / scale : 0.0f;
  }
};

// The root without its last half ulp (2^-23 of itself), and the reciprocal so:
// with correctly rounded ones the step took 99 instructions an element and was
// bound by them.
__device__ __forceinline__ float root_of(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float moved_fast(const Hyper& h, float p, float m, float root) {
  // the denominator is 0 or a normal number: a root of a float is, and eps is held to that
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(root, h.rbc2, h.eps)));
  return fmaf(p, h.decay, -h.step * (m * inv));
}

// Four elements as they come from memory.
template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 w;
  __device__ __forceinline__ void load(const float* p) { w = __ldcg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldcg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
};

// What a lane reads of a block: elements 4l .. 4l + 3 of each half, so that an
// access of the warp covers whole sectors.
template <typename G, typename P>
struct Block8 {
  Four<G> g[2];
  Four<P> p[2];
  uint32_t m[2], r[2];
  float ms, rs;
  __device__ __forceinline__ void load(const AdamwTensor& t, int64_t blk) {
    const int64_t at = blk * BLOCK8 + 4 * (threadIdx.x & 31);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[k] = __ldcg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + at + 128 * k));
      r[k] = __ldcg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + at + 128 * k));
      g[k].load(static_cast<const G*>(t.grad) + at + 128 * k);
      p[k].load(static_cast<const P*>(t.param) + at + 128 * k);
    }
    ms = __ldcg(t.m_scale + blk);
    rs = __ldcg(t.v_scale + blk);
  }
};

// One warp, one block of 256, held as above (WIDE) or element by element,
// l, l + 32, ... to a lane (the last block, and tensors that are not aligned
// for wide accesses).
template <typename G, typename P, bool WIDE>
__device__ __forceinline__ void block8(const AdamwTensor& t, const Hyper& h, int64_t blk,
                                       const Block8<G, P>* held = nullptr) {
  const int lane = threadIdx.x & 31;
  const int64_t first = blk * BLOCK8;
  const G* g = static_cast<const G*>(t.grad) + first;
  P* p = static_cast<P*>(t.param) + first;
  uint8_t *mc = static_cast<uint8_t*>(t.m) + first, *rc = static_cast<uint8_t*>(t.v) + first;
  __nv_bfloat16* c = t.copy ? static_cast<__nv_bfloat16*>(t.copy) + first : nullptr;
  const int left = static_cast<int>(min(t.n - first, static_cast<int64_t>(BLOCK8)));
  float gg[8], pp[8], mm[8], rr[8], vv[8];
  const int at = 4 * lane;
  float ms, rs;
  if constexpr (WIDE) {
    ms = held->ms;
    rs = held->rs;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      held->g[k].get(gg + 4 * k);
      held->p[k].get(pp + 4 * k);
      decode4(held->m[k], mm + 4 * k);
      decode4(held->r[k], rr + 4 * k);
    }
  } else {
    ms = __ldcg(t.m_scale + blk);
    rs = __ldcg(t.v_scale + blk);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = lane + 32 * k;
      const bool in = i < left;
      gg[k] = in ? load1(g + i) : 0.0f;
      pp[k] = in ? load1(p + i) : 0.0f;
      mm[k] = in ? decode1(__ldcg(mc + i)) : 0.0f;
      rr[k] = in ? decode1(__ldcg(rc + i)) : 0.0f;
    }
  }
  float mmost = 0.0f, vmost = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = gg[k] * h.coef, r = rr[k] * rs;
    float m = next_m(h, mm[k] * ms, x), v = next_v(h, r * r, x);
    // an element behind the end is 0 whatever the scales are
    if (!WIDE && lane + 32 * k >= left) m = v = 0.0f;
    mm[k] = m;
    vv[k] = v;
    rr[k] = root_of(v);
    pp[k] = moved_fast(h, pp[k], m, rr[k]);
    mmost = larger(mmost, m);
    vmost = larger(vmost, v);
  }
  if constexpr (WIDE) {
    store4(p + at, pp);
    store4(p + at + 128, pp + 4);
    if (c) {
      store4(c + at, pp);
      store4(c + at + 128, pp + 4);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (lane + 32 * k < left) {
        store1(p + lane + 32 * k, pp[k]);
        if (c) store1(c + lane + 32 * k, pp[k]);
      }
  }
  const Coder mcoder(warp_largest(mmost)), rcoder(sqrtf(warp_largest(vmost)));
  // no positive root becomes zero
  const float least = rcoder.scale * E4M3_MIN;
#pragma unroll
  for (int k = 0; k < 8; ++k) rr[k] = rr[k] > 0.0f ? fmaxf(rr[k], least) : rr[k];
  uint2 mq, rq;
  if (!mcoder.codes(mm, mq)) {
    mcoder.quotients(mm);
    mq = make_uint2(encode4(mm), encode4(mm + 4));
  }
  if (!rcoder.codes(rr, rq)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) rr[k] = sqrtf(vv[k]);
    rcoder.quotients(rr);
#pragma unroll
    for (int k = 0; k < 8; ++k) rr[k] = rr[k] > 0.0f ? fmaxf(rr[k], E4M3_MIN) : rr[k];
    rq = make_uint2(encode4(rr), encode4(rr + 4));
  }
  if constexpr (WIDE) {
    __stcg(reinterpret_cast<uint32_t*>(mc + at), mq.x);
    __stcg(reinterpret_cast<uint32_t*>(mc + at + 128), mq.y);
    __stcg(reinterpret_cast<uint32_t*>(rc + at), rq.x);
    __stcg(reinterpret_cast<uint32_t*>(rc + at + 128), rq.y);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = lane + 32 * k;
      if (i < left) {
        __stcg(mc + i, static_cast<uint8_t>((k < 4 ? mq.x : mq.y) >> (8 * (k & 3))));
        __stcg(rc + i, static_cast<uint8_t>((k < 4 ? rq.x : rq.y) >> (8 * (k & 3))));
      }
    }
  }
  if (lane == 0) {
    __stcg(t.m_scale + blk, mcoder.scale);
    __stcg(t.v_scale + blk, rcoder.scale);
  }
}

template <typename G, typename P, int PER_WARP>
__device__ void chunk8(const AdamwTensor& t, const Hyper& h, int64_t begin) {
  const int64_t last = (min(begin + PER_WARP * CHUNK, t.n) + BLOCK8 - 1) / BLOCK8;
  const int64_t b = begin / BLOCK8 + (threadIdx.x >> 5) * PER_WARP;
  if (t.wide && (b + PER_WARP) * BLOCK8 <= t.n) {
    Block8<G, P> held[PER_WARP];
#pragma unroll
    for (int k = 0; k < PER_WARP; ++k) held[k].load(t, b + k);
#pragma unroll
    for (int k = 0; k < PER_WARP; ++k) block8<G, P, true>(t, h, b + k, &held[k]);
    return;
  }
#pragma unroll 1
  for (int k = 0; k < PER_WARP && b + k < last; ++k) {
    if (t.wide && (b + k + 1) * BLOCK8 <= t.n) {
      Block8<G, P> held;
      held.load(t, b + k);
      block8<G, P, true>(t, h, b + k, &held);
    } else {
      block8<G, P, false>(t, h, b + k);
    }
  }
}

// The tensor of this CTA: the last whose first CTA is not behind it.
template <int CAP>
__device__ __forceinline__ int find(const int (&first)[CAP], int n, int block) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= block) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace

// BLOCKS: 8-bit blocks of one warp, 0 with float32 states
template <int CAP, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS == 2 ? 7 : 8) relkl_adamw_kernel(const __grid_constant__ AdamwParams<CAP> p) {
  const int k = find(p.first, p.n, blockIdx.x);
  const AdamwTensor& t = p.t[k];
  const Hyper h = hyper(p.plan, t);
  if (h.skip) return;
  const int64_t begin = static_cast<int64_t>(blockIdx.x - p.first[k]) * (BLOCKS == 2 ? 2 * CHUNK : CHUNK);
  using H = __nv_bfloat16;
#define RELKL_CHUNK(G, P)                \
  do {                                   \
    if constexpr (BLOCKS > 0)            \
      chunk8<G, P, BLOCKS>(t, h, begin); \
    else                                 \
      chunk32<G, P>(t, h, begin);        \
  } while (0)
  if (t.grad_bf16) {
    if (t.param_bf16) RELKL_CHUNK(H, H); else RELKL_CHUNK(H, float);
  } else {
    if (t.param_bf16) RELKL_CHUNK(float, H); else RELKL_CHUNK(float, float);
  }
#undef RELKL_CHUNK
}

// ------------------------------------------------------- gradient norm
// sqrt(sum of g^2) over all tensors.  The squares of 16 bytes are summed in
// float32, or where that leaves float32's range in double precision, as is the
// rest, in an order that depends on the sizes and the grid only, so the same gradients
// give the same bits.  An element from 2^64 on, whose square float32 does not
// hold, counts as infinite: such a step is left out by its clipping factor.
namespace {

constexpr int NORM_THREADS = 512, NORM_HOLD = 4;
constexpr int NORM_CHUNK = 16 * NORM_HOLD * NORM_THREADS;   // bytes
constexpr float NORM_MOST = 0x1p64f;

template <typename G>
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[16 / sizeof(G)]) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(G) == 4) {
      x[k] = __uint_as_float(a[k]);
    } else {
      x[2 * k] = __uint_as_float(a[k] << 16);
      x[2 * k + 1] = __uint_as_float(a[k] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ double square(float x) {
  return fabsf(x) < NORM_MOST ? static_cast<double>(x) * x : static_cast<double>(x * x);
}

// A chunk: consecutive elements of one tensor, of which a thread holds four
// accesses of 16 bytes (a warp's are next to one another).  201 M elements from
// HBM take 84 to 87 us in bf16 and 145 to 147 us in float32, 4.7 and 5.5 TB/s, of
// which some 7 us are a graph's start and the two launches (5.1 and 5.8 TB/s
// without them); where the end of the gradients is still in L2, 63 and 116 us.
// What holds bf16 at 1.3 times its bytes' time is not known.  A thread one of whose four
// accesses sums up to less than 1e-30, as zeros do, reads and sums them again: with
// every other row zero 105 and 160 us instead of 63 and 116.  With eight elements to a thread at a time, in accesses whose halves of sectors
// came twice, 129 and 190 us.  256 threads a CTA, two or eight accesses, or the
// next chunk's loads before this one's sums: 85 to 98 and 145 to 168 us.
struct Chunk {
  const char* at;
  int bytes, wide;      // `wide` of them come in such accesses
  bool bf16;
  uint4 w[NORM_HOLD];
};

template <int CAP>
__device__ __forceinline__ void load_chunk(const NormParams<CAP>& p, int chunk, Chunk& c) {
  const int k = find(p.first, p.n, chunk);
  const NormTensor& t = p.t[k];
  const int64_t begin = static_cast<int64_t>(chunk - p.first[k]) * NORM_CHUNK;
  c.at = static_cast<const char*>(t.grad) + begin;
  c.bf16 = t.bf16;
  c.bytes = static_cast<int>(min(t.n * (t.bf16 ? 2 : 4) - begin, static_cast<int64_t>(NORM_CHUNK)));
  c.wide = t.wide ? c.bytes / 16 * 16 : 0;
#pragma unroll
  for (int h = 0; h < NORM_HOLD; ++h) {
    const int i = 16 * (h * NORM_THREADS + threadIdx.x);
    c.w[h] = i < c.wide ? __ldcg(reinterpret_cast<const uint4*>(c.at + i)) : make_uint4(0, 0, 0, 0);
  }
}

template <typename G>
__device__ __forceinline__ double squares(const Chunk& c) {
  constexpr int PER = 16 / sizeof(G);
  float s[NORM_HOLD];
  double sum = 0.0;
  bool plain = true;
#pragma unroll
  for (int h = 0; h < NORM_HOLD; ++h) {
    float x[PER];
    unpack<G>(c.w[h], x);
    s[h] = 0.0f;
#pragma unroll
    for (int k = 0; k < PER; ++k) s[h] = fmaf(x[k], x[k], s[h]);
    plain = plain && s[h] >= 1e-30f && isfinite(s[h]);
  }
  if (plain) {
#pragma unroll
    for (int h = 0; h < NORM_HOLD; ++h) sum += s[h];
  } else {   // read again: few chunks need it, and registers are short
#pragma unroll 1
    for (int i = 16 * threadIdx.x; i < c.wide; i += 16 * NORM_THREADS) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(c.at + i));
      if ((v.x | v.y | v.z | v.w) == 0) continue;
      float x[PER];
      unpack<G>(v, x);
#pragma unroll
      for (int k = 0; k < PER; ++k) sum += square(x[k]);
    }
  }
  const G* g = reinterpret_cast<const G*>(c.at);
  for (int i = c.wide / static_cast<int>(sizeof(G)) + threadIdx.x; i < c.bytes / static_cast<int>(sizeof(G));
       i += NORM_THREADS)
    sum += square(load1(g + i));
  return sum;
}

__device__ double block_sum(double v) {
  __shared__ double part[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = threadIdx.x < blockDim.x / 32 ? part[threadIdx.x] : 0.0;
  if (threadIdx.x < 32)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  return v;   // thread 0's
}

// out[0]: the norm; out[1]: what gradients are multiplied by so that their norm
// is at most max_norm, NaN where the norm is no finite number.
__device__ void write_norm(float* out, double squares, float max_norm) {
  const float norm = static_cast<float>(sqrt(squares));
  out[0] = norm;
  const double coef = static_cast<double>(max_norm) / (static_cast<double>(norm) + 1e-6);
  out[1] = isfinite(norm) ? static_cast<float>(coef < 1.0 ? coef : 1.0) : __int_as_float(0x7fc00000);
}

}  // namespace

template <int CAP>
__global__ void __launch_bounds__(NORM_THREADS, 3) relkl_grad_norm_kernel(const __grid_constant__ NormParams<CAP> p) {
  double sum = 0.0;
  for (int chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
    Chunk c;
    load_chunk(p, chunk, c);
    sum += c.bf16 ? squares<__nv_bfloat16>(c) : squares<float>(c);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    if (p.out)
      write_norm(p.out, sum, p.max_norm);
    else
      p.partial[blockIdx.x] = sum;
  }
}

__global__ void __launch_bounds__(NORM_THREADS)
relkl_norm_finish_kernel(const double* partial, int n, float max_norm, float* out) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) sum += partial[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) write_norm(out, sum, max_norm);
}

// ------------------------------------------------------------- launches
int64_t norm_chunks(int64_t n, bool bf16) { return (n * (bf16 ? 2 : 4) + NORM_CHUNK - 1) / NORM_CHUNK; }

namespace {

template <int CAP, int BLOCKS>
cudaError_t adamw_group(const AdamwTensor* t, int n, const AdamwPlan& plan, cudaStream_t stream) {
  AdamwParams<CAP> p;
  p.plan = plan;
  p.n = n;
  int64_t blocks = 0;
  constexpr int chunk = BLOCKS == 2 ? 2 * CHUNK : CHUNK;
  for (int k = 0; k < n; ++k) {
    p.t[k] = t[k];
    p.first[k] = static_cast<int>(blocks);
    blocks += (t[k].n + chunk - 1) / chunk;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  }
  relkl_adamw_kernel<CAP, BLOCKS><<<static_cast<unsigned>(blocks), THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

// Elements from which a warp takes two 8-bit blocks.  It loads both before it
// works on the first, and looks up tensor and scalars once: 201 M elements take
// 500 us instead of 536 (float32 weights, bf16 gradients and copies), 406
// instead of 465 (all bf16), 485 instead of 521 (all float32).  Seven CTAs an SM
// leave 72 registers, and 30 words spill: 491, 404 and 474 us; with 8 CTAs 488,
// 397 and 502, with 6 516, 421 and 486, with 5, where nothing spills, 547, 480 and
// 528.  Fewer fill the
// SMs worse that way: 34 M 96, 74, 94 and 94, 82, 96 us, 12.6 M 47, 33, 47 and 41,
// 37, 45, 3.1 M 25, 14, 25 and 16, 14, 18.
constexpr int64_t kAdamwTwoBlocks = int64_t(1) << 25;

template <int BLOCKS>
cudaError_t adamw_blocks(const AdamwTensor* t, int n, const AdamwPlan& plan, cudaStream_t stream) {
  if (n <= kAdamwFew) return adamw_group<kAdamwFew, BLOCKS>(t, n, plan, stream);
  if (n <= kAdamwSome) return adamw_group<kAdamwSome, BLOCKS>(t, n, plan, stream);
  return adamw_group<kAdamwMost, BLOCKS>(t, n, plan, stream);
}

template <int CAP>
cudaError_t norm_group(const NormTensor* t, int n, int64_t chunks, int grid, double* partial,
                       float* out, float max_norm, cudaStream_t stream) {
  NormParams<CAP> p;
  p.n = n;
  p.chunks = static_cast<int>(chunks);
  p.partial = partial;
  p.out = out;
  p.max_norm = max_norm;
  int64_t at = 0;
  for (int k = 0; k < n; ++k) {
    p.t[k] = t[k];
    p.first[k] = static_cast<int>(at);
    at += norm_chunks(t[k].n, t[k].bf16);
  }
  relkl_grad_norm_kernel<CAP><<<grid, NORM_THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Tensors are those with elements, at most kAdamwMost of them.
cudaError_t launch_adamw(const AdamwTensor* t, int n, const AdamwPlan& plan, bool bits8,
                         cudaStream_t stream) {
  if (!bits8) return adamw_blocks<0>(t, n, plan, stream);
  int64_t all = 0;
  for (int k = 0; k < n; ++k) all += t[k].n;
  return all >= kAdamwTwoBlocks ? adamw_blocks<2>(t, n, plan, stream) : adamw_blocks<1>(t, n, plan, stream);
}

// One group's sum: into `out` as a norm where one CTA does all (grid 1), else
// `grid` partial sums.
cudaError_t launch_grad_norm(const NormTensor* t, int n, int64_t chunks, int grid, double* partial,
                             float* out, float max_norm, cudaStream_t stream) {
  if (n <= kAdamwFew) return norm_group<kAdamwFew>(t, n, chunks, grid, partial, out, max_norm, stream);
  if (n <= kAdamwSome) return norm_group<kAdamwSome>(t, n, chunks, grid, partial, out, max_norm, stream);
  return norm_group<kAdamwMost>(t, n, chunks, grid, partial, out, max_norm, stream);
}

cudaError_t launch_norm_finish(const double* partial, int n, float max_norm, float* out,
                               cudaStream_t stream) {
  relkl_norm_finish_kernel<<<1, NORM_THREADS, 0, stream>>>(partial, n, max_norm, out);
  return cudaGetLastError();
}

}  // namespace relkl
