// Argument checks that the C ABI's entry points share (host only, internal).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "gdn.h"

namespace gdn {
namespace check {

struct Tensor {
  const void* ptr;
  size_t bytes;
  size_t align;
  bool required;
};

inline bool overlap(const Tensor& a, const Tensor& b) {
  if (!a.ptr || !b.ptr || !a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.ptr), y = reinterpret_cast<uintptr_t>(b.ptr);
  return x < y ? y - x < a.bytes : x - y < b.bytes;
}

// NULL and alignment of every tensor, and no output may overlap another tensor.
inline gdn_status check_tensors(std::initializer_list<Tensor> ins, std::initializer_list<Tensor> outs) {
  for (const auto& set : {ins, outs})
    for (const Tensor& t : set) {
      if (!t.ptr) {
        if (t.required && t.bytes) return GDN_ERR_NULL;
        continue;
      }
      if (reinterpret_cast<uintptr_t>(t.ptr) % t.align) return GDN_ERR_ALIGN;
    }
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Tensor& t : ins)
      if (overlap(*o, t)) return GDN_ERR_ALIAS;
    for (auto q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return GDN_ERR_ALIAS;
  }
  return GDN_OK;
}

// Sequences of a dense (B rows of T tokens) or packed problem; *max_len is the
// longest one's length.
template <typename P>
gdn_status check_seqs(const P* p, int64_t* max_len) {
  if (p->cu_seqlens_host || p->cu_seqlens_dev) {
    if (!p->cu_seqlens_host || !p->cu_seqlens_dev) return GDN_ERR_NULL;
    if (p->B != 1) return GDN_ERR_SHAPE;
    const int32_t* cu = p->cu_seqlens_host;
    if (cu[0] != 0 || cu[p->num_seqs] != p->T) return GDN_ERR_SEQLENS;
    int64_t mx = 0;
    for (int32_t n = 0; n < p->num_seqs; ++n) {
      if (cu[n + 1] < cu[n]) return GDN_ERR_SEQLENS;
      mx = std::max<int64_t>(mx, cu[n + 1] - cu[n]);
    }
    *max_len = mx;
  } else {
    if (p->num_seqs != p->B) return GDN_ERR_SHAPE;
    *max_len = p->T;
  }
  return p->num_seqs > 65535 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

inline gdn_status hip_status(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

inline size_t up256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace check
}  // namespace gdn
