// The norm over many gradients and their scaling to a largest norm (gfx950,
// wave64):
//   norm = sqrt(sum over all tensors of g^2),  out = g min(1, max_norm / (norm + eps))
// Bound by HBM: one pass reads all gradients and leaves a sum a workgroup, the
// next one adds those in a fixed order (every workgroup for itself: a launch of
// its own between the two would cost more) and scales.  Sums are of 64 bits: a
// product and an addition of doubles for each element stay below the time of
// its bytes, and no size of a gradient overflows or vanishes in them.
//
// The tensors' addresses travel as arguments of the launch, so that a call needs
// no copy to the device and may be captured; they are cut into pieces of 32768
// elements that the workgroups take in turn.  The scaling pass goes backwards:
// what the first one read last is still in the last-level cache.
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int CT = 256;           // threads
constexpr int CU = 4;             // 16-byte loads of a thread in flight
constexpr int64_t PIECE = 32768;  // elements

// sum over the workgroup; all threads get it
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < CT / 64; ++w) v += lds[w];
  return v;
}

// The tensor that holds piece i.
__device__ __forceinline__ int find_tensor(const GradTable& t, int64_t i) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <class T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}
template <>
__device__ __forceinline__ float value(float v) {
  return v;
}

// squares of elements [a, b) of p, this thread's share
template <class T>
__device__ __forceinline__ double squares(const T* p, int64_t a, int64_t b) {
  constexpr int EC = 16 / sizeof(T);
  p += a;
  const int n = (int)(b - a);
  int head = (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T));
  head = head < n ? head : n;
  const int vecs = (n - head) / EC;
  double s = 0.0;
  if ((int)threadIdx.x < head) {
    const double f = value(p[threadIdx.x]);
    s = f * f;
  }
  const int rest = head + vecs * EC + (int)threadIdx.x;
  if (rest < n) {
    const double f = value(p[rest]);
    s = fma(f, f, s);
  }
  const u32x4_t* v = (const u32x4_t*)(p + head);
  for (int i = threadIdx.x; i < vecs; i += CT * CU) {
    u32x4_t q[CU];
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      q[u] = u32x4_t{0, 0, 0, 0};
      if (i + u * CT < vecs) q[u] = v[i + u * CT];
    }
#pragma unroll
    for (int u = 0; u < CU; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          const double f = __uint_as_float(q[u][j]);
          s = fma(f, f, s);
        } else {
          const double f = bf16_lo(q[u][j]), g = bf16_hi(q[u][j]);
          s = fma(f, f, s);
          s = fma(g, g, s);
        }
      }
  }
  return s;
}

__global__ __launch_bounds__(CT) void k_squares(GradTable t, double* part) {
  __shared__ double lds[CT / 64];
  double s = 0.0;
  for (int64_t i = blockIdx.x; i < t.pieces; i += gridDim.x) {
    const int j = find_tensor(t, i);
    const int64_t a = (i - t.first[j]) * PIECE, b = a + PIECE < t.n[j] ? a + PIECE : t.n[j];
    s += t.type(j, 0) ? squares((const float*)t.in[j], a, b) : squares((const uint16_t*)t.in[j], a, b);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double join(const double* part, int parts, double* lds) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += CT) s += part[i];
  return block_sum(s, lds);
}

__global__ __launch_bounds__(CT) void k_norm(const double* part, int parts, float* norm) {
  __shared__ double lds[CT / 64];
  const double s = join(part, parts, lds);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

// elements [a, b) of in times c; 16 bytes of in at a time where out then lies at a whole chunk too
template <class TI, class TO>
__device__ __forceinline__ void scale(const TI* in, TO* out, int64_t a, int64_t b, float c) {
  constexpr int EC = 16 / sizeof(TI);
  in += a;
  out += a;
  const int n = (int)(b - a);
  int head = (int)(((16 - ((uintptr_t)in & 15)) & 15) / sizeof(TI));
  head = head < n ? head : n;
  int vecs = (n - head) / EC;
  if (((uintptr_t)(out + head) & (EC * sizeof(TO) < 16 ? EC * sizeof(TO) - 1 : 15)) != 0) vecs = 0;
  auto put = [&](int i) {
    const float f = value(in[i]) * c;
    if constexpr (sizeof(TO) == 4)
      out[i] = f;
    else
      out[i] = (TO)f32_to_bf16(f);
  };
  if ((int)threadIdx.x < head) put(threadIdx.x);
  for (int i = head + vecs * EC + (int)threadIdx.x; i < n; i += CT) put(i);
  const u32x4_t* v = (const u32x4_t*)(in + head);
  for (int i = threadIdx.x; i < vecs; i += CT * CU) {
    u32x4_t q[CU];
#pragma unroll
    for (int u = 0; u < CU; ++u)
      if (i + u * CT < vecs) q[u] = v[i + u * CT];
#pragma unroll
    for (int u = 0; u < CU; ++u) {
      if (i + u * CT >= vecs) continue;
      float f[EC];
#pragma unroll
      for (int j = 0; j < EC; ++j)
        f[j] = c * (sizeof(TI) == 4 ? __uint_as_float(q[u][j]) : (j & 1) ? bf16_hi(q[u][j >> 1]) : bf16_lo(q[u][j >> 1]));
      TO* o = out + head + (int64_t)(i + u * CT) * EC;
      if constexpr (sizeof(TO) == 4) {
#pragma unroll
        for (int j = 0; j < EC; j += 4) *(f32x4_t*)(o + j) = f32x4_t{f[j], f[j + 1], f[j + 2], f[j + 3]};
      } else {
        uint32_t w[EC / 2];
#pragma unroll
        for (int j = 0; j < EC / 2; ++j) w[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
        if constexpr (EC == 8)
          *(u32x4_t*)o = u32x4_t{w[0], w[1], w[2], w[3]};
        else
          *(uint2*)o = uint2{w[0], w[1]};
      }
    }
  }
}

// part NULL: *norm is given; else the norm is the root of their sum, and stored by the first workgroup.
__global__ __launch_bounds__(CT) void k_clip(GradTable t, const double* part, int parts, float* norm, float max_norm,
                                             float eps, int store) {
  __shared__ double lds[CT / 64];
  float r;
  if (part) {
    r = (float)sqrt(join(part, parts, lds));
    if (store && blockIdx.x == 0 && threadIdx.x == 0) *norm = r;
  } else {
    r = *norm;
  }
  const double q = (double)max_norm / ((double)r + (double)eps);
  const float c = q >= 1.0 ? 1.0f : (float)q;  // a NaN stays one
  for (int64_t k = blockIdx.x; k < t.pieces; k += gridDim.x) {
    const int64_t i = t.pieces - 1 - k;
    const int j = find_tensor(t, i);
    if (c == 1.0f && t.in[j] == t.out[j]) continue;  // as it is
    const int64_t a = (i - t.first[j]) * PIECE, b = a + PIECE < t.n[j] ? a + PIECE : t.n[j];
    const bool fi = t.type(j, 0), fo = t.type(j, 1);
    if (fi && fo)
      scale((const float*)t.in[j], (float*)t.out[j], a, b, c);
    else if (fi)
      scale((const float*)t.in[j], (uint16_t*)t.out[j], a, b, c);
    else if (fo)
      scale((const uint16_t*)t.in[j], (float*)t.out[j], a, b, c);
    else
      scale((const uint16_t*)t.in[j], (uint16_t*)t.out[j], a, b, c);
  }
}

}  // namespace

int64_t clip_pieces(int64_t n) { return (n + PIECE - 1) / PIECE; }
int clip_groups(int64_t pieces) { return (int)(pieces < kClipGroups ? pieces : kClipGroups); }

hipError_t launch_squares(const GradTable& t, double* part, hipStream_t s) {
  return launch(Launch{s, nullptr, nullptr}, k_squares, dim3((unsigned)clip_groups(t.pieces)), dim3(CT), t, part);
}
hipError_t launch_norm(const double* part, int parts, float* norm, hipStream_t s) {
  return launch(Launch{s, nullptr, nullptr}, k_norm, dim3(1), dim3(CT), part, parts, norm);
}
hipError_t launch_clip(const GradTable& t, const double* part, int parts, float* norm, float max_norm, float eps,
                       bool store, hipStream_t s) {
  return launch(Launch{s, nullptr, nullptr}, k_clip, dim3((unsigned)clip_groups(t.pieces)), dim3(CT), t, part, parts, norm,
                max_norm, eps, (int)store);
}

}  // namespace moe
