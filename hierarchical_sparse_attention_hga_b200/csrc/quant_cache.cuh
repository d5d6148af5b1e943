// The 8-bit K/V cache: layout and helpers shared by its append, attention and
// eviction kernels.
//
// Keys and values are held per (sequence, KV head) as groups of 16 tokens, the
// unit the routing selects: 16 x D codes (e4m3 or int8) and one float32 scale
// per group and tensor.  Groups live in slots of one pool; table entry e of a
// (sequence, KV head) names the slot of its e-th live group, in position order.
// The rows of the group that is still open are kept, unrounded, in a tail.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace hga {

constexpr int kQuantGroup = 16;  // tokens per group (cfg group is 16)
constexpr int kQuantMaxGroups = 1 << 20;  // table entries per (sequence, KV head)
// Positions count evicted tokens too; the groups before them fit `evicted`, an int32.
constexpr int64_t kQuantMaxPos = (int64_t{1} << 35) - 2;
constexpr int64_t kQuantMaxSlots = (1 << 27) - 1;  // a slot's first row is an int32 coordinate

struct QuantCache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  void* k_tail;            // [B][Hkv][16][D] of the input type
  void* v_tail;
  const int32_t* table;    // [B][Hkv][max_groups]
  const int32_t* evicted;  // [B][Hkv] or null
  int64_t n_slots;
  int max_groups;
  int format;              // kQuantE4m3 or kQuantInt8
};

constexpr int kQuantE4m3 = 0, kQuantInt8 = 1;

// Groups and tail rows a (sequence, KV head) holds.
struct QuantItem {
  int closed;  // live groups in the pool
  int rest;    // rows of the open group (0..15)
  bool ok;     // false: the position or the count of evicted groups was bad
  __device__ __forceinline__ int units() const { return closed + (rest > 0); }
  __device__ __forceinline__ int tokens() const { return closed * kQuantGroup + rest; }
};

// The item's state at position pos (of its last token; -1: empty).  A position
// or eviction count that does not fit the table is flagged and reads as empty.
__device__ __forceinline__ QuantItem quant_item(const QuantCache& qc, int64_t pos, int64_t item,
                                                unsigned* err) {
  QuantItem it{0, 0, true};
  if (pos == -1) return it;
  if (pos < -1 || pos > kQuantMaxPos) {
    flag_error(err, kErrPos);
    it.ok = false;
    return it;
  }
  const int64_t gone = qc.evicted ? qc.evicted[item] : 0;
  const int64_t closed = ((pos + 1) >> 4) - gone;
  const int rest = static_cast<int>((pos + 1) & 15);
  if (gone < 0 || closed < 0 || closed + (rest > 0) > qc.max_groups) {
    flag_error(err, kErrPos);
    it.ok = false;
    return it;
  }
  it.closed = static_cast<int>(closed);
  it.rest = rest;
  return it;
}

// Two e4m3 codes (low byte first) as two halves: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

// Two floats in one register pair; each half of an operation is rounded as the
// scalar one, at half the instructions.
namespace f32x2 {
__device__ __forceinline__ uint64_t pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ uint64_t mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
}  // namespace f32x2

}  // namespace hga
