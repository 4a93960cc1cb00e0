// The norm over many gradients and their scaling to a largest norm (gfx950,
// wave64):
//   norm = sqrt(sum over all tensors of g^2),  out = g min(1, max_norm / (norm + eps))
// Bound by HBM: one pass reads all gradients and leaves a sum a workgroup, the
// next one adds those in a fixed order (every workgroup for itself: a launch of
// its own between the two costs more while there are few, 1000 tensors of 65536
// elements 144 against 149 us; 4000 of them 662 against 543) and scales.  Sums are of 64 bits: a
// product and an addition of doubles for each element stay below the time of
// its bytes, and no size of a gradient overflows or vanishes in them.
//
// The tensors' addresses travel as arguments of the launch, so that a call needs
// no copy to the device and may be captured; they are cut into pieces of 2048 to
// at most 32768 elements that the workgroups take in turn.  The scaling pass goes backwards:
// what the first one read last is still in the last-level cache.  830 million bf16 elements: 313 and 621 us, 5.3
// TB/s both.
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int CT = 256;           // threads
constexpr int CU = 4;             // 16-byte loads of a thread in flight

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

// The table, the launch's first argument, two tensors a lane: one way to memory for all of it, where a
// search over the arguments takes one a step (61 tensors of 400 thousand elements in all: 6.5 and 7.7 us
// with it, 5.5 and 6.7 without).
struct Table {
  const char* in[2];
  char* out[2];
  int64_t n[2];
  int32_t first[2];
  uint32_t types[2];  // bit 0: in is fp32, bit 1: out
  int count;
};
__device__ __forceinline__ Table read_table(int count) {
  const GradTable* g = (const GradTable*)(const char*)__builtin_amdgcn_kernarg_segment_ptr();
  Table t;
  t.count = count;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = (int)(threadIdx.x & 63) + 64 * u, j = i < count ? i : 0;
    t.in[u] = (const char*)g->in[j];
    t.out[u] = (char*)g->out[j];
    t.n[u] = g->n[j];
    t.first[u] = i < count ? g->first[j] : 0x7FFFFFFF;
    t.types[u] = (g->types[0][j >> 5] >> (j & 31) & 1) | (g->types[1][j >> 5] >> (j & 31) & 1) << 1;
  }
  return t;
}
__device__ __forceinline__ int64_t pick(const int64_t (&v)[2], int j) {
  const int64_t x = j < 64 ? v[0] : v[1];
  return ((int64_t)__builtin_amdgcn_readlane((int)(x >> 32), j & 63) << 32) |
         (uint32_t)__builtin_amdgcn_readlane((int)x, j & 63);
}
// Elements [a, b) of the tensor that piece i is of.
struct Piece {
  const void* in;
  void* out;
  int64_t a, b;
  bool in32, out32;
};
__device__ __forceinline__ Piece find_piece(const Table& t, int i, int shift) {
  const int j = __builtin_popcountll(__ballot(t.first[0] <= i)) + __builtin_popcountll(__ballot(t.first[1] <= i)) - 1;
  const int64_t n = pick(t.n, j), in[2] = {(int64_t)t.in[0], (int64_t)t.in[1]},
                out[2] = {(int64_t)t.out[0], (int64_t)t.out[1]};
  const int first = __builtin_amdgcn_readlane(j < 64 ? t.first[0] : t.first[1], j & 63);
  const uint32_t types = (uint32_t)__builtin_amdgcn_readlane((int)(j < 64 ? t.types[0] : t.types[1]), j & 63);
  const int64_t a = (int64_t)(i - first) << shift, b = a + ((int64_t)1 << shift);
  return Piece{(const void*)pick(in, j), (void*)pick(out, j), a, b < n ? b : n, (types & 1) != 0, (types & 2) != 0};
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

__global__ __launch_bounds__(CT) void k_squares(GradTable g, double* part) {
  __shared__ double lds[CT / 64];
  double s = 0.0;
  const Table t = read_table(g.count);
  for (int i = blockIdx.x; i < g.pieces; i += gridDim.x) {
    const Piece p = find_piece(t, i, g.shift);
    s += p.in32 ? squares((const float*)p.in, p.a, p.b) : squares((const uint16_t*)p.in, p.a, p.b);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double join(const double* part, int parts, double* lds) {
  double s = 0.0;
#pragma unroll 8
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
__global__ __launch_bounds__(CT) void k_clip(GradTable g, const double* part, int parts, float* norm, float max_norm,
                                             float eps, int store) {
  __shared__ double lds[CT / 64];
  const Table t = read_table(g.count);
  float r;
  if (part) {
    r = (float)sqrt(join(part, parts, lds));
    if (store && blockIdx.x == 0 && threadIdx.x == 0) *norm = r;
  } else {
    r = *norm;
  }
  const double q = (double)max_norm / ((double)r + (double)eps);
  const float c = q >= 1.0 ? 1.0f : (float)q;  // a NaN stays one
  for (int k = blockIdx.x; k < g.pieces; k += gridDim.x) {
    const Piece p = find_piece(t, g.pieces - 1 - k, g.shift);
    if (c == 1.0f && p.in == p.out) continue;  // as it is
    if (p.in32 && p.out32)
      scale((const float*)p.in, (float*)p.out, p.a, p.b, c);
    else if (p.in32)
      scale((const float*)p.in, (uint16_t*)p.out, p.a, p.b, c);
    else if (p.out32)
      scale((const uint16_t*)p.in, (float*)p.out, p.a, p.b, c);
    else
      scale((const uint16_t*)p.in, (uint16_t*)p.out, p.a, p.b, c);
  }
}

}  // namespace

int64_t clip_pieces(int64_t n, int shift) { return (n + ((int64_t)1 << shift) - 1) >> shift; }
// As large as leaves every one of the kClipGroups workgroups a piece: a workgroup goes through one in
// steps that wait for each other (61 tensors of 400 thousand elements in all: pieces of 32768 5.5 and
// 6.7 us, of 2048 3.5 and 3.9).
int clip_shift(int64_t elements) {
  int shift = 11;
  while (shift < 15 && (elements >> shift) > kClipGroups) ++shift;
  return shift;
}
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
