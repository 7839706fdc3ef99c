// Argument checks and launch settings that the cache operators' entry points
// share (cache_ops.cu, page_ops.cu).  Host code.
#pragma once

#include <cuda_runtime.h>

#include <initializer_list>
#include <utility>

#include "../../include/psv.h"
#include "cache_kernels.h"

#define PSV_API extern "C" __attribute__((visibility("default")))

namespace psv {

inline int dtype_size(int dtype) {
  switch (dtype) {
    case PSV_DTYPE_F32: return 4;
    case PSV_DTYPE_BF16:
    case PSV_DTYPE_F16: return 2;
    default: return 0;
  }
}

inline int cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return PSV_OK;
  return cache_fail(PSV_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Device memory of the current device `dev` (managed memory counts).  A look at
// a pointer takes the host about 0.4 us, so that a call looks at its first
// input and its output: what is mixed up in practice is whole sets of tensors.
inline int check_device(int dev, const void* ptr, const char* name) {
  if (!ptr) return cache_fail(PSV_EINVAL, "%s is null", name);
  cudaPointerAttributes a;
  cudaError_t e = cudaPointerGetAttributes(&a, ptr);
  if (e != cudaSuccess) return cuda_status(e, name);
  if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
    return cache_fail(PSV_EINVAL, "%s is not device memory", name);
  if (a.type == cudaMemoryTypeDevice && a.device != dev)
    return cache_fail(PSV_EINVAL, "%s is on device %d, the current device is %d", name, a.device, dev);
  return PSV_OK;
}

// Whether every one of these pointers (null ones too) is on four bytes, as the
// kernels read and write ints and floats there one by one.
inline bool on4(std::initializer_list<const void*> ptrs) {
  uintptr_t at = 0;
  for (const void* p : ptrs) at |= reinterpret_cast<uintptr_t>(p);
  return (at & 3) == 0;
}

inline bool stride_ok(const int64_t* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] > (int64_t{1} << 40)) return false;
  return true;
}

// Whether the rows of an output [n0][n1][n2][width] are distinct: taken by
// growing stride, every index steps over all that lies inside it.
inline bool rows_distinct(const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int64_t width) {
  int64_t st[3] = {s[0], s[1], s[2]}, n[3] = {n0, n1, n2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        const int64_t a = st[i], c = n[i];
        st[i] = st[j], n[i] = n[j];
        st[j] = a, n[j] = c;
      }
  int64_t span = width;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < span) return false;
    span += st[i] * (n[i] - 1);
  }
  return true;
}

// Whether two tensors at one address have their rows in the same places (an index
// of extent one is never stepped).
inline bool same_rows(const int64_t* a, const int64_t* b, int64_t n0, int64_t n1, int64_t n2) {
  return (n0 == 1 || a[0] == b[0]) && (n1 == 1 || a[1] == b[1]) && (n2 == 1 || a[2] == b[2]);
}

// The bytes of a tensor: rows of `width` bytes, n[d] of them st[d] bytes apart
// along each of three indexes.
struct Area {
  const char* at;
  int64_t st[3], n[3], width;
  const char* name;
  const char* end;  // behind the last byte
};

inline Area tensor_area(const char* name, const void* at, const int64_t* s, int64_t n0, int64_t n1, int64_t n2,
                        int64_t width, int size) {
  const char* first = static_cast<const char*>(at);
  return Area{first, {s[0] * size, s[1] * size, s[2] * size}, {n0, n1, n2}, width * size, name,
              first + (s[0] * (n0 - 1) + s[1] * (n1 - 1) + s[2] * (n2 - 1) + width) * size};
}

// A contiguous one (null: none).
inline Area plain_area(const char* name, const void* at, int64_t bytes) {
  const char* first = static_cast<const char*>(at);
  return Area{first, {0, 0, 0}, {1, 1, 1}, at ? bytes : 0, name, first + (at ? bytes : 0)};
}

// Whether two areas, b `d` bytes behind a, may share a byte, from index `level`
// on.  Where their strides agree and hold what lies inside them, only copies next
// to each other can meet, so that tensors packed into one buffer are told apart;
// where they do not agree the whole stretches count.
inline bool areas_meet(const Area& a, const Area& b, int64_t d, int level) {
  int64_t ea = a.width, eb = b.width;
  for (int i = 2; i > level; --i) ea += a.st[i] * (a.n[i] - 1), eb += b.st[i] * (b.n[i] - 1);
  if (level == 3) return d < ea && d + eb > 0;
  const int64_t st = a.st[level], na = a.n[level], nb = b.n[level];
  if (d >= ea + a.st[level] * (na - 1) || d + eb + b.st[level] * (nb - 1) <= 0) return false;
  if (na == 1 && nb == 1) return areas_meet(a, b, d, level + 1);
  if (st != b.st[level] || ea > st || eb > st) return true;
  const int64_t k0 = d >= 0 ? d / st : -((-d + st - 1) / st);  // copy k of a starts at or before b's first
  for (int64_t k = k0; k <= k0 + 1; ++k)
    if (k > -nb && k < na && areas_meet(a, b, d - k * st, level + 1)) return true;
  return false;
}

inline bool areas_meet(Area a, Area b) {
  if (!a.width || !b.width) return false;
  for (int i = 0; i < 3; ++i) {
    if (a.st[i] == 0) a.n[i] = 1;  // (every copy the same)
    if (b.st[i] == 0) b.n[i] = 1;
    if (a.n[i] == 1) a.st[i] = b.n[i] == 1 ? 0 : b.st[i];  // an index of extent one is never stepped
    if (b.n[i] == 1) b.st[i] = a.st[i];
  }
  for (Area* x : {&a, &b})  // the largest stride first
    for (int i = 0; i < 3; ++i)
      for (int j = i + 1; j < 3; ++j)
        if (x->st[j] > x->st[i]) std::swap(x->st[i], x->st[j]), std::swap(x->n[i], x->n[j]);
  return areas_meet(a, b, b.at - a.at, 0);
}

// Refuses outputs that meet an input or one another.  (Almost always the whole
// stretches are apart, and a look at those first saves a call 0.2 to 0.5 us.)
inline int check_areas(std::initializer_list<Area> outs, std::initializer_list<Area> ins) {
  auto areas_meet = [](const Area& a, const Area& b) {
    return a.at < b.end && b.at < a.end && psv::areas_meet(a, b);
  };
  for (const Area* o = outs.begin(); o != outs.end(); ++o) {
    for (const Area& i : ins)
      if (areas_meet(*o, i)) return cache_fail(PSV_EINVAL, "%s overlaps %s", o->name, i.name);
    for (const Area* p = outs.begin(); p != o; ++p)
      if (areas_meet(*o, *p)) return cache_fail(PSV_EINVAL, "%s overlaps %s", o->name, p->name);
  }
  return PSV_OK;
}

inline bool overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + bbytes && y < x + abytes;
}

inline Strides3 strides3(const int64_t* s) { return Strides3{s[0], s[1], s[2]}; }

// Whether a tensor's base and the strides that are stepped are multiples of `bytes`
// (a power of two).
inline bool multiple_of(int bytes, const void* ptr, const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int size) {
  const int64_t n[3] = {n0, n1, n2};
  if (reinterpret_cast<uintptr_t>(ptr) & (bytes - 1)) return false;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] * size) % bytes != 0) return false;
  return true;
}

inline bool multiple16(const void* ptr, const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int size) {
  return multiple_of(16, ptr, s, n0, n1, n2, size);
}

// A launch that may begin while the kernel before it ends (it waits for that
// kernel's results itself).
inline cudaLaunchConfig_t pdl_config(dim3 grid, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace psv
