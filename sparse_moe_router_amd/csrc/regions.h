// Which bytes a call's buffers take, and whether two buffers share any (host
// code without HIP).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

// Bytes of one buffer: n from the first to the last; with a pitch only `width`
// bytes of every `pitch` (the rows of a column slice).
struct Region {
  const void* p;
  size_t n;
  size_t pitch, width;  // pitch 0: all n bytes
};

inline Region bytes_at(const void* p, size_t n) { return Region{p, n, 0, n}; }

// A [rows][cols] matrix of es-byte elements whose rows are ld elements apart.
inline Region matrix_at(const void* p, int64_t rows, int64_t ld, int64_t cols, int es) {
  if (!p || rows <= 0) return Region{p, 0, 0, 0};
  const size_t width = (size_t)cols * es, pitch = (size_t)ld * es, n = (size_t)(rows - 1) * pitch + width;
  if (rows == 1 || pitch == width) return bytes_at(p, n);
  return Region{p, n, pitch, width};
}

// Column slices of one buffer lie side by side: rows of one pitch whose byte
// columns, counted from a's first, are [0, a.width) and [d, d + b.width) with
// nothing reaching into the next row.  Slices of different pitches count as
// overlapping wherever their extents do.
inline bool overlap(const Region& a, const Region& b) {
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  if (!a.n || !b.n || a0 >= b0 + b.n || b0 >= a0 + a.n) return false;
  const size_t pitch = a.pitch ? a.pitch : b.pitch;
  if (!pitch || (a.pitch && b.pitch && a.pitch != b.pitch)) return true;
  const size_t d = b0 >= a0 ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
  return d < a.width || d + b.width > pitch;
}

// The buffers of one call.  Every output must be disjoint from every input and
// from every other output.
struct Regions {
  Region in[8], out[12];
  int nin = 0, nout = 0;
  void input(const Region& r) {
    if (r.p && r.n) in[nin++] = r;
  }
  void output(const Region& r) {
    if (r.p && r.n) out[nout++] = r;
  }
  void input(const void* p, size_t n) { input(bytes_at(p, n)); }
  void output(const void* p, size_t n) { output(bytes_at(p, n)); }
  bool disjoint() const {
    for (int i = 0; i < nout; ++i) {
      for (int j = 0; j < nin; ++j)
        if (overlap(out[i], in[j])) return false;
      for (int j = i + 1; j < nout; ++j)
        if (overlap(out[i], out[j])) return false;
    }
    return true;
  }
};

}  // namespace moe
