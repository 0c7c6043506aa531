// api_checks.h -- argument checks that the C entry points share.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "mssm.h"
#include "mssm_internal.h"

namespace mssm {
namespace api {

constexpr int64_t kMost = INT64_MAX / 16;  // elements of one array
constexpr int64_t kGrid = INT32_MAX;       // workgroups of one launch
constexpr int64_t kItems = UINT32_MAX;     // threads of one launch

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline int64_t blocks128(int64_t n) { return (n + 127) / 128; }
inline int64_t size_of(int32_t dtype) { return dtype == MSSM_BF16 ? 2 : 4; }
inline bool known(int32_t dtype) { return dtype == MSSM_F32 || dtype == MSSM_BF16; }

// a * b <= limit for positive a, b.
inline bool fits(int64_t a, int64_t b, int64_t limit = kMost) { return a > 0 && b > 0 && a <= limit / b; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range range(const void* p, int64_t bytes) {
  return p && bytes > 0 ? Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes} : Range{0, 0};
}
// Rows of `cols` elements, `stride` apart.
inline Range rows_range(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t size) {
  return range(p, ((rows - 1) * stride + cols) * size);
}
inline bool overlap(Range a, Range b) {
  return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi;
}
// Whether an output overlaps an input or another output.
inline bool aliased(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (overlap(*o, i)) return true;
    for (const Range* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
  }
  return false;
}
inline bool all_aligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (p && !aligned(p, a)) return false;
  return true;
}

inline int done(hipError_t e, const char* what) {
  if (e == hipSuccess) return MSSM_OK;
  mssm::set_hip_error(what, e);
  return MSSM_ERR_HIP;
}

}  // namespace api
}  // namespace mssm
