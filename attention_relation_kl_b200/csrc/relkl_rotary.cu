// Rotary positions of the relation inputs, in either direction:
//
//   forward:   (a, b) -> m (a cos t - b sin t, b cos t + a sin t)
//   gradient:  (a, b) -> m (a cos t + b sin t, b cos t - a sin t)
//
// for the pairs of the first `rot` entries of every head, t = pos(b, n) f_i,
// with the pair frequencies f_i and the factor m given by the caller; the
// other entries of a head, and tensors that carry no rotation (V), are moved
// to the output's layout and type unchanged.
//
// What bounds it: every element is read once and written once, so HBM.  The
// angles are formed in double precision (positions reach 10^5 and more), which
// costs far more than the rotation, so one thread keeps the cosines and sines
// of its few pairs of one token in registers and runs over the heads of a
// group with them; no table is read or written.
//
// Measured (B200, copy bandwidth 6.56 TB/s; on the GPU, by a replayed graph):
// 32K tokens, Q, K and V of 32 heads of 128, bf16, tokens to heads: 269 us, 6.0
// TB/s; gradients of 2 x 16K tokens, 32 + 8 + 8 heads, fp32 heads to bf16
// tokens: 182 us, 6.7 TB/s.  What made the difference was how many rows are in
// flight, not how many bytes a thread has: one head at a time at 8 blocks an SM
// against four heads at 3 blocks: 285 and 321 us; loads past L1 against streaming
// ones: 273 and 279 us (182 and 193 us for the gradients).  8 blocks leave a
// thread 32 registers, in which half of the variants spill (bf16 in both, halves,
// 8 entries wide, which the 32K inputs take, 60 bytes stored and 72 loaded before
// the loop over heads); with 6, 5 and 4 blocks they took 280, 297 and 332 us, the
// gradients 202, 221 and 246.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "relkl_params.h"

namespace relkl {

namespace {

// m cos(pos f) and m sin(pos f).  The angle is reduced by whole turns in
// double precision, in units of pi; its float part goes through sincospif and
// the rest enters by the first-order term, so both are off by an ulp of 1 at
// most, and by what the angle itself is off: its position, two products and 1 /
// pi round, 4 * 2^-53 of the angle, which reaches that ulp at angles of 2^27
// (past a position of 10^8 for the fastest pair).
__device__ __forceinline__ void pair_angle(double pos, double f, float m, float& c, float& s) {
  const double u = pos * f * 0.31830988618379067154;   // half turns: angle / pi
  const double r = fma(-2.0, rint(0.5 * u), u);        // exact, in [-1, 1]
  const float hi = static_cast<float>(r);
  const float lo = static_cast<float>((r - static_cast<double>(hi)) * 3.14159265358979323846);
  float sh, ch;
  sincospif(hi, &sh, &ch);
  c = fmaf(-sh, lo, ch) * m;
  s = fmaf(ch, lo, sh) * m;
}

// V consecutive elements as floats, in accesses of at most 16 bytes: loads
// keep out of L1, where nothing is read twice, stores are the first to leave L2.
template <typename T, int V>
struct Vec {
  static constexpr int kBytes = V * static_cast<int>(sizeof(T));
  uint32_t w[(kBytes + 3) / 4];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x; w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      w[0] = __ldcg(reinterpret_cast<const unsigned int*>(p));
    } else {
      w[0] = __ldcg(reinterpret_cast<const unsigned short*>(p));
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        __stcs(reinterpret_cast<uint4*>(p) + i,
               make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
    } else if constexpr (kBytes == 8) {
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    } else if constexpr (kBytes == 4) {
      __stcs(reinterpret_cast<unsigned int*>(p), w[0]);
    } else {
      __stcs(reinterpret_cast<unsigned short*>(p), static_cast<unsigned short>(w[0]));
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
  }
  // rounded once, to nearest even
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (V == 1) {
      w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
  }
};

template <typename T, typename U, int V>
__device__ __forceinline__ void move_heads(const T* x, U* y, int64_t xh, int64_t yh, int heads) {
#pragma unroll 1
  for (int h = 0; h < heads; ++h) {
    Vec<T, V> a;
    a.load(x + h * xh);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = a.get(i);
    Vec<U, V> o;
    o.set(v);
    o.store(y + h * yh);
  }
}

// The entries that do not turn, or a tensor that does not: `width` of them to
// a thread, whatever the rotated part's width is.
template <typename T, typename U>
__device__ __forceinline__ void move_chunk(const T* x, U* y, int64_t xh, int64_t yh, int heads, int width) {
  switch (width) {
    case 8: move_heads<T, U, 8>(x, y, xh, yh, heads); break;
    case 4: move_heads<T, U, 4>(x, y, xh, yh, heads); break;
    case 2: move_heads<T, U, 2>(x, y, xh, yh, heads); break;
    default: move_heads<T, U, 1>(x, y, xh, yh, heads);
  }
}

}  // namespace

// Thread = (token, chunk): a chunk is V pairs of the `half` layout (V entries
// of each half), V / 2 pairs of the interleaved layout (V neighbouring
// entries; with V = 1 one pair, entry by entry), or some entries that do not
// turn.  blockIdx.y = head group of a tensor.
template <typename T, typename U, int V, bool HALVES>
__global__ void __launch_bounds__(256, 8) relkl_rotary_kernel(const __grid_constant__ RotaryParams p) {
  // the group's tensor and first head
  int g = blockIdx.y, r = 0;
  while (g >= p.t[r].groups) g -= p.t[r++].groups;
  const RotaryTensor& t = p.t[r];
  const int64_t item = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t tok = item / t.chunks;
  const int chunk = static_cast<int>(item - tok * t.chunks);
  if (tok >= p.tokens) return;
  const int64_t b = tok / p.N, n = tok - b * p.N;
  const int h0 = g * p.heads_per_group;
  const int heads = min(p.heads_per_group, t.H - h0);
  const T* x = static_cast<const T*>(t.x) + b * t.xs[0] + h0 * t.xs[1] + n * t.xs[2];
  U* y = static_cast<U*>(t.y) + b * t.ys[0] + h0 * t.ys[1] + n * t.ys[2];
  const int64_t xh = t.xs[1], yh = t.ys[1];

  if (chunk >= t.rot_chunks) {
    const int at = (t.apply ? p.rot : 0) + (chunk - t.rot_chunks) * t.width;
    move_chunk<T, U>(x + at, y + at, xh, yh, heads, t.width);
    return;
  }
  constexpr bool SPLIT = HALVES || V == 1;   // a pair's entries are loaded apart
  const int at = (!HALVES && V == 1) ? 2 * chunk : chunk * V;
  const int far = HALVES ? p.rot / 2 : 1;

  double pos;
  if (p.positions) {
    const int64_t i = b * p.pos_stride[0] + n * p.pos_stride[1];
    pos = p.pos_bytes == 8
              ? static_cast<double>(static_cast<const long long*>(p.positions)[i])
              : static_cast<double>(static_cast<const int*>(p.positions)[i]);
  } else {
    pos = static_cast<double>(n);
  }
  pos = fma(pos, p.pos_scale, p.pos_offset);
  constexpr int P = SPLIT ? V : V / 2;
  float c[P], s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    pair_angle(pos, p.inv_freq[chunk * P + i], p.mscale, c[i], s[i]);
    if (p.inverse) s[i] = -s[i];
  }

  x += at;
  y += at;
  if constexpr (SPLIT) {
#pragma unroll 1
    for (int h = 0; h < heads; ++h) {
      Vec<T, V> lo, hi;
      lo.load(x + h * xh);
      hi.load(x + h * xh + far);
      float ya[V], yb[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float a = lo.get(i), q = hi.get(i);
        ya[i] = fmaf(a, c[i], -q * s[i]);
        yb[i] = fmaf(q, c[i], a * s[i]);
      }
      Vec<U, V> o0, o1;
      o0.set(ya);
      o1.set(yb);
      o0.store(y + h * yh);
      o1.store(y + h * yh + far);
    }
  } else {
#pragma unroll 1
    for (int h = 0; h < heads; ++h) {
      Vec<T, V> in;
      in.load(x + h * xh);
      float v[V];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float a = in.get(2 * i), q = in.get(2 * i + 1);
        v[2 * i] = fmaf(a, c[i], -q * s[i]);
        v[2 * i + 1] = fmaf(q, c[i], a * s[i]);
      }
      Vec<U, V> o;
      o.set(v);
      o.store(y + h * yh);
    }
  }
}

namespace {

// Largest of 8, 4, 2, 1, at most `most`, that divides `entries` and whose
// accesses, of at most 16 bytes, are aligned at entry `at` of every head.  The
// rotated parts of a launch share one width, whatever does not turn has its
// own: 8192 tokens of 32 + 8 + 8 heads in bf16 took, with one width for all,
// 40.5 (40 of 80 entries turn), 55.1 (24 of 96) and 96.5 us (20 of 128), and
// take 29.9, 37.8 and 60.6; where all of a head turns, 41.6 and 39.7.
int vector_width(const RotaryTensor& t, int most, int at, int entries, int xsize, int ysize) {
  for (int v = most; v > 1; v /= 2) {
    const int64_t xa = v * xsize < 16 ? v * xsize : 16, ya = v * ysize < 16 ? v * ysize : 16;
    bool ok = entries % v == 0 && at * xsize % xa == 0 && at * ysize % ya == 0 &&
              reinterpret_cast<uintptr_t>(t.x) % xa == 0 && reinterpret_cast<uintptr_t>(t.y) % ya == 0;
    for (int i = 0; i < 3; ++i) ok = ok && t.xs[i] * xsize % xa == 0 && t.ys[i] * ysize % ya == 0;
    if (ok) return v;
  }
  return 1;
}

template <typename T, typename U, int V, bool HALVES>
cudaError_t launch(RotaryParams& p, int num_sms, cudaStream_t stream) {
  p.tokens = static_cast<int64_t>(p.B) * p.N;
  int64_t blocks = 0;
  int most = 1;
  int64_t work = 0;     // blocks with one head to a thread
  for (int r = 0; r < p.n; ++r) {
    RotaryTensor& t = p.t[r];
    const int turned = t.apply ? p.rot : 0;
    t.rot_chunks = (HALVES || V == 1) ? turned / 2 / V : turned / V;
    t.width = vector_width(t, (sizeof(T) == 2 && sizeof(U) == 2) ? 8 : 4, turned, p.d - turned, sizeof(T), sizeof(U));
    t.chunks = t.rot_chunks + (p.d - turned) / t.width;
    const int64_t own = (p.tokens * t.chunks + 255) / 256;
    blocks = own > blocks ? own : blocks;
    work += own * t.H;
    most = t.H > most ? t.H : most;
  }
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // As many heads for one thread as leave the SMs two waves of blocks, but at
  // most 4: with 1, 2, 4, 8, 16 heads the 32K inputs took 520, 326, 269, 272,
  // 271 us, the gradients 367, 219, 182, 181, 181 (angles weigh on the left; on
  // the right nothing is gained, and fewer blocks fill the last wave worse).
  int64_t hg = work / (static_cast<int64_t>(num_sms) * 16);
  hg = hg < 1 ? 1 : (hg > 4 ? 4 : hg);
  while ((most + hg - 1) / hg * p.n > 65535) hg *= 2;   // the grid's y extent
  p.heads_per_group = static_cast<int>(hg);
  int groups = 0;
  for (int r = 0; r < p.n; ++r) {
    p.t[r].groups = (p.t[r].H + p.heads_per_group - 1) / p.heads_per_group;
    groups += p.t[r].groups;
  }
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
  relkl_rotary_kernel<T, U, V, HALVES><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, typename U, bool HALVES>
cudaError_t pick(RotaryParams& p, int num_sms, cudaStream_t stream) {
  // 16 bytes of the wider type in one access
  constexpr int most = (sizeof(T) == 2 && sizeof(U) == 2) ? 8 : 4;
  int v = most;
  for (int r = 0; r < p.n; ++r)
    if (p.t[r].apply) v = vector_width(p.t[r], v, 0, HALVES ? p.rot / 2 : p.rot, sizeof(T), sizeof(U));
  if constexpr (most == 8)
    if (v == 8) return launch<T, U, 8, HALVES>(p, num_sms, stream);
  if (v == 4) return launch<T, U, 4, HALVES>(p, num_sms, stream);
  if (v == 2) return launch<T, U, 2, HALVES>(p, num_sms, stream);
  return launch<T, U, 1, HALVES>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rotary(RotaryParams& p, bool x_bf16, bool y_bf16, bool interleaved,
                          int num_sms, cudaStream_t stream) {
  using H = __nv_bfloat16;
#define RELKL_ROTARY(T, U) \
  return interleaved ? pick<T, U, false>(p, num_sms, stream) : pick<T, U, true>(p, num_sms, stream)
  if (x_bf16 && y_bf16) RELKL_ROTARY(H, H);
  if (x_bf16) RELKL_ROTARY(H, float);
  if (y_bf16) RELKL_ROTARY(float, H);
  RELKL_ROTARY(float, float);
#undef RELKL_ROTARY
}

}  // namespace relkl
