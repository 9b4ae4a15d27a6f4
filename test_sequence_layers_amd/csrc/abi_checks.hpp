// Argument checks that the C ABI layers of ttt_seq.h and ttt_lm.h share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ttt.h"
#include "internal.hpp"

namespace {

constexpr int kMaxB = 65535;

inline bool known(ttt_dtype dt) { return dt == TTT_F32 || dt == TTT_BF16; }
inline size_t elem_size(ttt_dtype dt) { return dt == TTT_BF16 ? 2 : 4; }
inline ttt_status from_hip(hipError_t e) { return e == hipSuccess ? TTT_OK : TTT_ERR_HIP; }

// The buffers of one call: alignment and presence are noted as they are added, overlaps (of any
// output with anything but itself) are looked for at the end.
class Buffers {
 public:
  void in(const void* p, size_t bytes, size_t align, bool needed = true) { add(p, bytes, align, needed, false); }
  void out(const void* p, size_t bytes, size_t align, bool needed = true) { add(p, bytes, align, needed, true); }
  // rows tokens of `width` elements, `stride` apart.
  void rows(const void* p, long long rows, long long stride, long long width, size_t e, bool needed = true) {
    if (p && (stride < width || (double)rows * (double)stride > (double)(1ll << 46))) bad_ = true;
    else in(p, ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * e, e, needed);
  }
  bool ok() const {
    if (bad_) return false;
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < i; ++j)
        if ((b_[i].out || b_[j].out) && b_[i].lo < b_[j].hi && b_[j].lo < b_[i].hi) return false;
    return true;
  }

 private:
  void add(const void* p, size_t bytes, size_t align, bool needed, bool out) {
    if (!p) {
      bad_ = bad_ || needed;
      return;
    }
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a & (align - 1)) bad_ = true;
    b_[n_++] = Buf{a, a + bytes, out};
  }
  struct Buf {
    uintptr_t lo, hi;
    bool out;
  };
  Buf b_[24];
  int n_ = 0;
  bool bad_ = false;
};

// Workspace: TTT_ERR_WORKSPACE when it is missing or small, otherwise added as an output (16-byte
// aligned) so that it overlaps nothing.
inline ttt_status add_workspace(Buffers& bufs, void* ws, size_t have, size_t need) {
  if (need == 0) return TTT_OK;
  if (!ws || have < need) return TTT_ERR_WORKSPACE;
  bufs.out(ws, need, 16);
  return TTT_OK;
}

}  // namespace
