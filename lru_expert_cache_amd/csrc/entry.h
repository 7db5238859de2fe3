// What the C entry points of the operators share: argument checks, the device
// of the pointers and the stream, the layout of scratch memory.
#pragma once
#include <algorithm>
#include <initializer_list>

#include "common.h"

namespace ftmoe {

constexpr int32_t kMaxDim = (1 << 24) - 1;  // tokens and widths
constexpr int64_t kAlign = 256;             // parts of the scratch memory

template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {  // an error message that could not be stored
    return FT_E_HIP;
  }
}

inline int bad(const char* what) {
  set_error("%s", what);
  return FT_E_INVALID;
}

inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// scratch memory, handed out in order; the same code lays it out (base 0) and uses it
struct Carve {
  uint8_t* base;
  int64_t used = 0;
  uint8_t* take(int64_t bytes) {
    uint8_t* p = base + used;
    used += up(bytes, kAlign);
    return p;
  }
};

struct Arg {
  const void* p;
  int64_t align;  // of the element type
  const char* name;
};

// Every pointer is there, aligned for its elements and memory of one device,
// the stream's; that device is made current while the guard lives.
struct DeviceGuard {
  int back = -1;
  ~DeviceGuard() {
    if (back >= 0) (void)hipSetDevice(back);
  }
  int enter(hipStream_t s, std::initializer_list<Arg> args) {
    for (const Arg& a : args) {
      if (!a.p) {
        set_error("%s is NULL", a.name);
        return FT_E_INVALID;
      }
      if (reinterpret_cast<uintptr_t>(a.p) % uintptr_t(a.align)) {
        set_error("%s is not aligned to %lld bytes", a.name, (long long)a.align);
        return FT_E_INVALID;
      }
    }
    int cur = 0, dev = 0;
    FT_HIP_CHECK(hipGetDevice(&cur));
    dev = cur;
    if (s) FT_HIP_CHECK(hipStreamGetDevice(s, &dev));
    for (const Arg& a : args) {
      if (&a != args.begin() && a.p == args.begin()->p) continue;  // (arguments that are not there)
      hipPointerAttribute_t at;
      if (hipPointerGetAttributes(&at, a.p) != hipSuccess) {
        (void)hipGetLastError();
        at.type = hipMemoryTypeUnregistered;
      }
      if ((at.type != hipMemoryTypeDevice && at.type != hipMemoryTypeManaged) || at.device != dev) {
        set_error("%s is not memory of device %d, the stream's", a.name, dev);
        return FT_E_INVALID;
      }
    }
    if (dev != cur) {
      FT_HIP_CHECK(hipSetDevice(dev));
      back = cur;
    }
    return FT_OK;
  }
};

inline bool dim_ok(int64_t v, int64_t lo) { return v >= lo && v <= kMaxDim; }
// a row distance: 0 = the width; a limit keeps every byte offset within 64 bits
inline bool row_ok(int64_t& ld, int64_t width) {
  if (ld == 0) ld = width;
  return ld >= width && ld < (int64_t(1) << 32);
}

inline int64_t size_of(int dtype) { return dtype == FT_DT_F32 ? 4 : 2; }

inline bool same(const void* p, std::initializer_list<const void*> others) {
  for (const void* o : others)
    if (p && p == o) return true;
  return false;
}

// A matrix of a call, for the check of what lies where.
struct Rows {
  const void* p;
  int64_t rows, bytes, ld;  // bytes of a row, and from row to row
};
// the same rows
inline bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.bytes == b.bytes && a.ld == b.ld; }
// Whether two matrices share bytes.  Exact for rows at one distance (columns of
// one buffer); others count as overlapping where their spans do.
inline bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t la = uint64_t(a.rows - 1) * uint64_t(a.ld) + uint64_t(a.bytes);
  const uint64_t lb = uint64_t(b.rows - 1) * uint64_t(b.ld) + uint64_t(b.bytes);
  if (pa <= pb ? pb - pa >= la : pa - pb >= lb) return false;
  if (a.ld == b.ld && a.ld > 0) {
    const uint64_t ld = uint64_t(a.ld);
    const uint64_t off = pb >= pa ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;  // of b's rows within a's
    if (off >= uint64_t(a.bytes) && off + uint64_t(b.bytes) <= ld) return false;
  }
  return true;
}

inline int check_work(const void* work, int64_t have, int64_t need) {
  if (have < need || (need > 0 && !work)) {
    set_error("the call needs %lld bytes of scratch memory, %lld given", (long long)need,
              (long long)(work ? have : 0));
    return FT_E_INVALID;
  }
  return FT_OK;
}

}  // namespace ftmoe
