// Host-side argument checks shared by the entry points that stand beside the
// layer's own (embedding.cu, layer_norm.cu, cross_entropy.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "internal.h"

namespace moe {
namespace entry {

constexpr size_t kStatusBytes = 256;   // status region at the start of every workspace

inline size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// A required device pointer, and one that may be left out.
inline bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }
inline bool opt_ok(const void* p) { return aligned16(p); }

// Hidden sizes of these operators: rows of whole 16-byte words.
constexpr int kMaxH = 16384;
inline bool hidden_ok(int32_t H) { return H > 0 && H <= kMaxH && H % 8 == 0; }

inline moe_status status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace entry
}  // namespace moe
