// Decode attention over the 8-bit K/V cache.
//
// One query token per sequence attends, exactly, every live group of its
// (sequence, KV head) and the open group's tail rows, or, given routed group
// ids, the sinks, the window and the routed groups (the sets of hga_attend):
//   s_t = (q . c_t) k_scale / sqrt(D),  p = softmax(s),  out = sum_t p_t v_scale c'_t
// with codes c, c'.  On request each group's weight, the sum of p over its
// tokens and the G query heads of the KV head, is added to an accumulator.
//
// Bound by HBM: 2 D bytes a token are read once, for 4 G D operations.  16 x 32K
// tokens of 8 KV heads, 4 query heads each: 178 us with the merge, 6.1 TB/s, 0.93 of
// a copy; 8 heads 180 us; 16 heads 235 us, there by the instructions; 8 x 128K int8
// 341 us, 380 under sustained load at the power limit.  Few or short items cost more than
// their bytes, by the partials and by what each item waits for: one 1K prompt 9 us, one of
// 32K 22 us (10.3 by its bytes), 128 short ones 28.5 us (11.8).  Each warp
// streams groups through a ring of its own in shared memory (one TMA box for a
// group's K, one for its V), reads the codes back in
// the very bytes that the matrix instruction's operand layout wants from each
// lane, widens them in registers to f16 (exact for both formats) and multiplies
// on mma.sync m16n8k16 with the TOKENS as the 16 rows and the query heads as the
// 8 columns: no wasted rows for few heads.  S^T = K Q^T lands with a lane holding
// two heads of two tokens; movmatrix turns it into the second product's operand
// (O^T += V^T P^T).  The order in which the D dimensions meet in a product is
// free as long as both operands agree, and so are the orders of a group's tokens
// and of O's rows; they are chosen so that a lane's bytes are consecutive ones of
// a row and no two lanes of a phase meet in a bank (see Tile).
//
// Precision.  f16 operands hold the codes exactly.  bf16 queries and tails are scaled by
// a power of two (a query's and a tail's own) and exact down to 2^-31 of their largest element;
// float32 ones are split into a high and a low half, 22 bits, without the product of the two
// low halves; either way no element is off by more than 2^-39 of the largest, where
// f16 ends.  The softmax weights, multiplied by v_scale, are split likewise: 22 bits of a
// weight down to 2^-14 of the largest p v_scale that the warp has met, below that an error of
// up to 2^-36 of that largest one (so a dimension that only such light groups feed has
// fewer bits than float32 would leave it; the row has not).  With at most four heads the
// low halves take the unused four columns, for free.  Exponentials are ex2.approx (2 ulp).
// References of the running softmax are integers, so every rescaling is exact, and v_scale
// enters as exponent and mantissa, so its size never costs bits.  A weight's reference
// (of p v_scale) is kept as its distance from the score's, and the exponents of
// weights are sums of distances: beyond 2^24 a score has no bits left to which an
// exponent could be added.  Each tile's product starts from zero and is added to the
// running sum in float32 (round to nearest): the matrix unit's own accumulation is
// never longer than a tile.
//
// Work.  A fixed grid; the units (groups, and one for a tail) of all items form
// one list, of which each warp takes an equal slice, whatever the sequences'
// lengths.  Every item stands there with kItemCost more units than it has, for
// what it costs beside its bytes (2, 4, 8: 128 short sequences 41, 37, 35 us, routed
// sets 29.5, 27.6, 26.5).  A warp leaves one partial (sum, references,
// denominator) per item it touches, at slot warp + item (distinct, since one of
// the two grows from each partial to the next); a second kernel merges them, in
// a fixed order.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "quant_cache.cuh"
#include "tmap.h"

namespace hga {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 2;             // units a warp works on at a time (1: 8 x 128K int8 384 us, 2: 340)
constexpr int kStages = 2;           // tiles in a warp's ring
static_assert(32 % kTile == 0, "a tile's slots come from one block of 32");
constexpr int kItemCost = 8;         // an item's fixed work, in units (see the slices)
constexpr int kMinSlice = 2;         // units a warp takes at least (a 1K prompt: 11.3 us, 4: 12.3, 8: 14.3)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kWaitLimit = 1u << 26;  // bounded mbarrier polls (and 50 ms)
constexpr float kNoRef = -3e38f;     // reference before the first score
constexpr float kHeadroom = 2.f;     // a raised reference exceeds the maximum by 2 to 3
constexpr float kWeightExp = 14.f;   // weights are below 2 * 2^14 in f16 (65504), one of them at least 2^11

// Resident CTAs per SM that the register use allows (shared memory may allow fewer:
// launch_attend).
__host__ __device__ constexpr int ctas_per_sm(int gm) { return gm == 16 ? 2 : 3; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t ex2_pair(uint64_t x) {
  const float2 v = f32x2::unpack(x);
  return f32x2::pack(ex2(v.x), ex2(v.y));
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero accumulators.
__device__ __forceinline__ void mma_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transposes an 8 x 8 matrix of halves held two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void load_shared(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t a, uint32_t (&r)[2]) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}

// One unit's codes in shared memory: K rows, then V rows, D bytes each, the
// 16-byte pieces of a row permuted as the copy's swizzle does it (128-byte rows:
// by the row's low three bits; 64-byte rows: by bits 1 and 2).  Row n of the
// matrix products is token token(n), so that
//  - K: the two rows that eight lanes read (n = 2m, 2m + 1; 64 bytes of each) lie
//    in different halves of the banks,
//  - V: the four rows (n = 2c, or 2c + 1) and the neighbouring pieces that a
//    phase's lanes read cover every bank once.
template <int D>
struct Tile {
  static constexpr int kUnitBytes = 2 * kQuantGroup * D;
  static __device__ __forceinline__ int token(int n) {
    const int c = (n & 7) >> 1;
    if (D == 128) return (n & 8) | ((n & 1) ? (2 * c) ^ 5 : 2 * c);
    const int even = (c & 1) | ((c & 2) << 1);
    return (n & 8) | ((n & 1) ? even ^ 3 : even);
  }
  static __device__ __forceinline__ int piece(int row, int i) {
    return row * D + ((i ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
  }
};

// Four codes as two pairs of halves: exact.  int8: 1024 + (code + 128) is a half
// whose low byte is code + 128; subtracting 1152 leaves the code.
template <int FORMAT>
__device__ __forceinline__ void widen4(uint32_t r, uint32_t& lo, uint32_t& hi) {
  if (FORMAT == kQuantE4m3) {
    lo = e4m3x2_to_half2(static_cast<uint16_t>(r));
    hi = e4m3x2_to_half2(static_cast<uint16_t>(r >> 16));
  } else {
    const uint32_t x = r ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
    const __half2 hb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&ha);
    hi = *reinterpret_cast<const uint32_t*>(&hb);
  }
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The remainder of (a, b) that pack_half2 left, as halves.
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_half2(a - f.x, b - f.y);
}

// 2^n for an integer n in [-126, 127].
__device__ __forceinline__ float exp2i(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }

// Exponent e (clamped to [-100, 127]) of the largest |value|'s bits, so that
// value * 2^(14 - e) is below 2^15; 0 for all-zero input.
__device__ __forceinline__ int scale_exponent(uint32_t top_bits) {
  return top_bits == 0 ? 0 : max(static_cast<int>(top_bits >> 23) - 127, -100);
}
constexpr uint32_t kInfBits = 0x7f800000u;

// The largest |element| of rows as bits (NaN above infinity above the finite ones),
// four at a time.
struct TopBf16 {
  uint32_t top = 0;
  __device__ __forceinline__ void add(const uint2& r) {
    asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(r.x & 0x7fff7fffu));
    asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(r.y & 0x7fff7fffu));
  }
  __device__ __forceinline__ uint32_t bits() const { return max(top << 16, top & 0xffff0000u); }
};
struct TopF32 {
  uint32_t top = 0;
  __device__ __forceinline__ void add(const float4& r) {
    top = max(max(top, __float_as_uint(r.x) & 0x7fffffffu), __float_as_uint(r.y) & 0x7fffffffu);
    top = max(max(top, __float_as_uint(r.z) & 0x7fffffffu), __float_as_uint(r.w) & 0x7fffffffu);
  }
  __device__ __forceinline__ uint32_t bits() const { return top; }
};

// v_scale as mant * 2^ex.
__device__ __forceinline__ void split_scale(float v, float& mant, float& ex) {
  const uint32_t u = __float_as_uint(v), e = (u >> 23) & 255;
  if (e == 0) {  // zero or subnormal
    mant = v * 0x1p126f;
    ex = -126.f;
  } else if (e == 255) {
    mant = v;
    ex = 0.f;
  } else {
    mant = __uint_as_float((u & 0x807fffffu) | 0x3f800000u);
    ex = static_cast<float>(static_cast<int>(e) - 127);
  }
}

// The units a query attends, as a virtual list: groups [0, a_end), groups
// [b_base, closed), the routed ids (entries that are not kept: -1), the tail.
struct Units {
  int a_end, b_base, fixed, groups, total;
  __device__ __forceinline__ int entry(int i, const int* routed) const {
    if (i < a_end) return i;
    if (i < fixed) return b_base + (i - a_end);
    return routed[i - fixed];
  }
};

// tokens: live ones of the item, those of the groups and of the tail
__device__ __forceinline__ Units units_of(const LayerParams& p, int tokens, bool routed) {
  const int closed = tokens / kQuantGroup, open = tokens % kQuantGroup > 0;
  Units u{0, 0, closed, closed, closed + open};
  if (routed && tokens) {  // nothing was evicted: the query is at position tokens - 1
    const int first = max(0, (tokens - 1) / p.C - p.local);
    u.a_end = min(p.sink, first) * p.Ng;
    u.b_base = first * p.Ng;
    u.fixed = u.a_end + closed - u.b_base;
    u.groups = u.fixed + p.kg;
    u.total = u.groups + open;
  }
  return u;
}

// Scratch of one call.
struct Workspace {
  int2* parts;     // [items]: first warp of the item, number of warps (0: no tokens)
  float* stat;     // [warps + items][16][4]: weight reference less the score's, score reference, denominator
  float* sum;      // [warps + items][G][D], dimensions in the kernel's order
  int warps;       // at most
  float2* group;   // [items][G][max_groups + kg]: each unit's sum (-1: a routed id that is not
                   // kept) and its reference, in the virtual list's order (weights only)
};

// The dimension at place i of a partial sum's row.
template <int D>
__device__ __forceinline__ int dim_of(int i) {
  return ((i >> 1) & 7) * (D / 8) + 2 * (i >> 4) + (i & 1);
}

// GM: query heads per KV head rounded up to 4, 8 or 16.
template <typename T, int D, int FORMAT, int GM>
struct Warp {
  static constexpr int NT = GM == 16 ? 2 : 1;          // 8-column tiles
  static constexpr int NK = D / 16;                    // k-steps, and 16-row tiles of O^T
  static constexpr bool kSplitQ = sizeof(T) == 4;      // a low half of the queries

  uint32_t qh[NT][NK][2], ql[kSplitQ ? NT : 1][kSplitQ ? NK : 1][2];
  float f[NT][2];                                      // score scale of this lane's columns (log2 units)
  uint64_t o[NK][NT][2];                               // pairs of columns: rows g, g + 8
  float ref_s[NT][2], lift[NT][2];                     // references: scores, and scores times v_scale less ref_s
  uint64_t l[NT];

  using Row = typename std::conditional<kSplitQ, float4, uint2>::type;  // four values
  using Top = typename std::conditional<kSplitQ, TopF32, TopBf16>::type;

  // Query heads of (b, h): column n of tile nt is head nt * 8 + n; with GM == 4
  // columns 4..7 repeat heads 0..3.
  __device__ __forceinline__ void fetch_q(const T* q, const LayerParams& p, int b, int h, Row (&raw)[NT][NK]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = GM == 4 ? g & 3 : nt * 8 + g;
      const T* row = q + (static_cast<int64_t>(b) * p.Hq + h * p.G + head) * D + c * 16;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks)
        raw[nt][ks] = head < p.G ? *reinterpret_cast<const Row*>(row + (ks >> 2) * 64 + (ks & 3) * 4) : Row{};
    }
  }
  __device__ __forceinline__ void load_q(const Row (&raw)[NT][NK]) {
    const int lane = threadIdx.x & 31, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Top most;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) most.add(raw[nt][ks]);
      uint32_t top = most.bits();
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = top < kInfBits ? scale_exponent(top) : 0;
      const float up = exp2i(14 - e);
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        float x[4];
        unpack(raw[nt][ks], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= up;
        qh[nt][ks][0] = pack_half2(x[0], x[1]);
        qh[nt][ks][1] = pack_half2(x[2], x[3]);
        if constexpr (kSplitQ) {
          ql[nt][ks][0] = pack_rest(x[0], x[1], qh[nt][ks][0]);
          ql[nt][ks][1] = pack_rest(x[2], x[3], qh[nt][ks][1]);
        }
      }
      // a query with an infinity or NaN makes its head NaN
      const float down = top < kInfBits ? exp2i(e - 14) * (kLog2e * rsqrtf(static_cast<float>(D))) : CUDART_NAN_F;
      f[nt][0] = __shfl_sync(0xffffffffu, down, 8 * c);       // column 2c is lane group g = 2c
      f[nt][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ref_s[nt][e] = kNoRef;
        lift[nt][e] = 0.f;
      }
      l[nt] = 0;  // a pair of zeros
#pragma unroll
      for (int mt = 0; mt < NK; ++mt) o[mt][nt][0] = o[mt][nt][1] = 0;
    }
  }

  // Softmax of U units' scores x (log2 units, -inf where there is no token):
  // raises the references if need be, adds to l, and leaves the weights times
  // v_scale (mant * 2^ex) as operands pb[u][nt][high, low][2].  group != null:
  // the sum of p per unit and head goes to group[head * stride + at[u]] (at >= 0).
  template <int U, bool WEIGHT>
  __device__ __forceinline__ void softmax(const float (&x)[U][NT][4], const float (&mant)[U],
                                          const float (&ex)[U], uint32_t (&pb)[U][NT][2][2],
                                          float2* group, int stride, const int (&at)[U],
                                          const bool (&kept)[U], int G) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a = -CUDART_INF_F, b = -CUDART_INF_F;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float y = fmaxf(x[u][nt][e], x[u][nt][e + 2]) - ref_s[nt][e];
          a = fmaxf(a, y);
          b = fmaxf(b, y + ex[u]);
        }
        raise |= a > 0.f || b > lift[nt][e];
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float corr[2], fall[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float a = -CUDART_INF_F, b = -CUDART_INF_F;
#pragma unroll
          for (int u = 0; u < U; ++u) a = fmaxf(a, fmaxf(x[u][nt][e], x[u][nt][e + 2]));
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
          const float na = a > ref_s[nt][e] ? ceilf(a) + kHeadroom : ref_s[nt][e];
#pragma unroll
          for (int u = 0; u < U; ++u) b = fmaxf(b, fmaxf(x[u][nt][e], x[u][nt][e + 2]) - na + ex[u]);
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, s));
          const float by = na - ref_s[nt][e];
          const float held = lift[nt][e] - by;  // the weight's reference where it was
          const float nb = b > held ? ceilf(b) + kHeadroom : held;
          fall[e] = ex2(-by);
          corr[e] = ex2(held - nb);  // integers: exact
          ref_s[nt][e] = na;
          lift[nt][e] = nb;
        }
        l[nt] = f32x2::mul(l[nt], f32x2::pack(fall[0], fall[1]));
#pragma unroll
        for (int mt = 0; mt < NK; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) o[mt][nt][i] = f32x2::mul(o[mt][nt][i], f32x2::pack(corr[0], corr[1]));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint64_t minus = f32x2::pack(-ref_s[nt][0], -ref_s[nt][1]);
        const uint64_t y0 = f32x2::add(f32x2::pack(x[u][nt][0], x[u][nt][1]), minus);
        const uint64_t y1 = f32x2::add(f32x2::pack(x[u][nt][2], x[u][nt][3]), minus);
        const float up = kWeightExp + ex[u];
        const uint64_t more = f32x2::pack(up - lift[nt][0], up - lift[nt][1]);
        const uint64_t m2 = f32x2::pack(mant[u], mant[u]);
        const uint64_t sum = f32x2::add(ex2_pair(y0), ex2_pair(y1));
        l[nt] = f32x2::add(l[nt], sum);
        const float2 w0 = f32x2::unpack(f32x2::mul(m2, ex2_pair(f32x2::add(y0, more))));
        const float2 w1 = f32x2::unpack(f32x2::mul(m2, ex2_pair(f32x2::add(y1, more))));
        const uint32_t h0 = pack_half2(w0.x, w0.y), h1 = pack_half2(w1.x, w1.y);
        const uint32_t r0 = pack_rest(w0.x, w0.y, h0), r1 = pack_rest(w1.x, w1.y, h1);
        if constexpr (GM == 4) {  // columns 0..3: high halves, 4..7: low halves
          pb[u][nt][0][0] = transpose8(c < 2 ? h0 : r0);
          pb[u][nt][0][1] = transpose8(c < 2 ? h1 : r1);
        } else {
          pb[u][nt][0][0] = transpose8(h0);
          pb[u][nt][0][1] = transpose8(h1);
          pb[u][nt][1][0] = transpose8(r0);
          pb[u][nt][1][1] = transpose8(r1);
        }
        if constexpr (WEIGHT) {
          const float2 both = f32x2::unpack(sum);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float s = e ? both.y : both.x;
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
            const int head = nt * 8 + 2 * c + e;
            if (g == 0 && head < G && at[u] >= 0 && (GM != 4 || c < 2))
              group[static_cast<int64_t>(head) * stride + at[u]] =
                  make_float2(kept[u] ? s : -1.f, ref_s[nt][e]);
          }
        }
      }
  }

  // Tail rows (rest of them valid) as one unit.  All loads come first.
  __device__ void tail(const T* kt, const T* vt, int rest, float2* group, int stride, int unit, int G) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    Row kr[2][NK], vr[4][D / 32];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        kr[r][ks] = Row{};
        if (g + 8 * r < rest)
          kr[r][ks] = *reinterpret_cast<const Row*>(kt + (g + 8 * r) * D + (ks >> 2) * 64 + c * 16 + (ks & 3) * 4);
      }
    // V: rows 2c, 2c + 1, 2c + 8, 2c + 9, this lane's D / 8 dimensions
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 2 * c + (r & 1) + 8 * (r >> 1);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        vr[r][j] = Row{};
        if (row < rest) vr[r][j] = *reinterpret_cast<const Row*>(vt + row * D + g * (D / 8) + 4 * j);
      }
    }
    Top most_k, most_v;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) most_k.add(kr[r][ks]);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) most_v.add(vr[r][j]);
    const uint32_t top_k = __reduce_max_sync(0xffffffffu, most_k.bits());
    const uint32_t top_v = __reduce_max_sync(0xffffffffu, most_v.bits());
    // as the group will once it is closed, a tail with an infinity or NaN makes NaN
    const bool finite = max(top_k, top_v) < kInfBits;
    const int e_k = finite ? scale_exponent(top_k) : 0, e_v = finite ? scale_exponent(top_v) : 0;
    float y[4];
    const float up_k = exp2i(14 - e_k), down_k = exp2i(e_k - 14), up_v = exp2i(14 - e_v);
    float x[1][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) x[0][nt][0] = x[0][nt][1] = x[0][nt][2] = x[0][nt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      uint32_t a[4], b[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        unpack(kr[r][ks], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= up_k;
        a[r] = pack_half2(y[0], y[1]);
        a[r + 2] = pack_half2(y[2], y[3]);
        if constexpr (kSplitQ) {
          b[r] = pack_rest(y[0], y[1], a[r]);
          b[r + 2] = pack_rest(y[2], y[3], a[r + 2]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma(x[0][nt], a[0], a[1], a[2], a[3], qh[nt][ks][0], qh[nt][ks][1]);
        if constexpr (kSplitQ) {
          mma(x[0][nt], a[0], a[1], a[2], a[3], ql[nt][ks][0], ql[nt][ks][1]);
          mma(x[0][nt], b[0], b[1], b[2], b[3], qh[nt][ks][0], qh[nt][ks][1]);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[0][nt][i] = !finite ? CUDART_NAN_F : g + 8 * (i >> 1) < rest ? x[0][nt][i] * (f[nt][i & 1] * down_k) : -CUDART_INF_F;
    const float mant[1] = {1.f}, ex[1] = {static_cast<float>(e_v - 14)};
    const int at[1] = {unit};
    const bool kept[1] = {true};
    uint32_t pb[1][NT][2][2];
    if (group) softmax<1, true>(x, mant, ex, pb, group, stride, at, kept, G);
    else softmax<1, false>(x, mant, ex, pb, group, stride, at, kept, G);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      float v[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        unpack(vr[r][j], v[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[r][i] *= up_v;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t a[4], b[4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const float y0 = v[2 * r][2 * half + d], y1 = v[2 * r + 1][2 * half + d];
            a[2 * r + d] = pack_half2(y0, y1);
            if constexpr (kSplitQ) b[2 * r + d] = pack_rest(y0, y1, a[2 * r + d]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s[4];
          mma_zero(s, a[0], a[1], a[2], a[3], pb[0][nt][0][0], pb[0][nt][0][1]);
          if constexpr (GM != 4) mma(s, a[0], a[1], a[2], a[3], pb[0][nt][1][0], pb[0][nt][1][1]);
          if constexpr (kSplitQ) mma(s, b[0], b[1], b[2], b[3], pb[0][nt][0][0], pb[0][nt][0][1]);
          add_to(2 * j + half, nt, s);
        }
      }
    }
  }

  __device__ __forceinline__ void add_to(int mt, int nt, const float (&s)[4]) {
    o[mt][nt][0] = f32x2::add(o[mt][nt][0], f32x2::pack(s[0], s[1]));
    o[mt][nt][1] = f32x2::add(o[mt][nt][1], f32x2::pack(s[2], s[3]));
  }

  static __device__ __forceinline__ void unpack(const float4& v, float (&y)[4]) {
    y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
  }
  static __device__ __forceinline__ void unpack(const uint2& v, float (&y)[4]) {
    y[0] = __uint_as_float(v.x << 16); y[1] = __uint_as_float(v.x & 0xffff0000u);
    y[2] = __uint_as_float(v.y << 16); y[3] = __uint_as_float(v.y & 0xffff0000u);
  }
};

template <typename T, int D, int FORMAT, int GM>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(GM))
quant_attend_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    LayerParams p, QuantCache qc, const T* q, const int64_t* pos,
                    const int32_t* group_idx, Workspace ws, unsigned* err) {
  using W = Warp<T, D, FORMAT, GM>;
  constexpr int NT = W::NT, NK = W::NK;
  constexpr int kUnitBytes = Tile<D>::kUnitBytes;
  constexpr int kRing = kStages * kTile * kUnitBytes;
  extern __shared__ uint8_t s_dyn[];                    // [kWarps][kRing], then [kWarps][kg] routed ids
  uint8_t* s_rings = s_dyn + (1024 - ptx::smem_u32(s_dyn) % 1024) % 1024;
  __shared__ uint64_t s_full[kWarps][kStages];
  // per unit, two blocks of 32: k_scale, v_scale as mantissa and exponent, state (1: in
  // the ring, 0: no tokens, -1: id not kept)
  __shared__ float4 s_units[kWarps][2][32];
  // list length before each thread's rows: used up before the first unit is staged
  static_assert(kThreads * sizeof(int64_t) <= sizeof(s_units), "where the units will stand");
  int64_t* s_before = reinterpret_cast<int64_t*>(s_units);
  __shared__ int64_t s_all;
  __shared__ int s_tokens[kThreads];                    // live tokens of each thread's row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = s_rings + warp * kRing;
  const uint32_t ring_at = ptx::smem_u32(ring);
  int* routed = reinterpret_cast<int*>(s_rings + kWarps * kRing) + warp * p.kg;
  const int items = p.B * p.Hkv;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < kStages; ++k) ptx::mbar_init(&s_full[warp][k], 1);
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&map_k);
    ptx::prefetch_tensormap(&map_v);
  }
  auto worker = [&]() { return static_cast<int64_t>(blockIdx.x) * kWarps + warp; };
  // The list's rows are the sequences, whose `same` KV heads have equal lengths, or,
  // where eviction may have made them differ, the items.
  const int same = qc.evicted ? 1 : p.Hkv, rows = qc.evicted ? items : p.B;
  auto tokens_of = [&](int row, unsigned* e) { return quant_item(qc, pos[qc.evicted ? row / p.Hkv : row], row, e).tokens(); };
  // A row's items' length in the list: their units, their fixed work in front.
  auto length_of = [&](int tokens) { return tokens ? units_of(p, tokens, group_idx != nullptr).total + kItemCost : 0; };
  const int per = (rows + kThreads - 1) / kThreads;  // rows a thread sums up
  // Every input may be what the kernel just before writes, positions and counts of
  // evicted groups too, and the scratch may still be read by an earlier call's merge: all
  // of it is used behind pdl_wait.  Where a thread has one row at most, the search for the
  // slice goes ahead of the wait by the positions that stand there then, and is done
  // again if behind it one has changed (calls back to back, 4 short float32 sequences: 11.8 us
  // with the search behind the wait, 10.2 so; a 1K prompt 10.0 and 9.0).
  bool waited = per > 1 || qc.evicted;
  if (waited) pdl_wait();
  // Where there are more rows, positions are read again below.  They do not change while a
  // call runs; if they do, its result is undefined, but every index stays in range and
  // the loops end: the two that look for items at the last one.
  int item;
  int skip;   // of the item's length, where the slice enters it
  int left;   // of the slice (at most the longest item's length, or a 1000th of the list)
  int slice;  // a whole one's length
  int b, h, tokens, u_lo, u_hi;  // of the item; the slice has its units [u_lo, u_hi)
  Units un;
  auto enter_item = [&]() {
    b = item / p.Hkv;
    h = item % p.Hkv;
    const int row = qc.evicted ? item : b;
    tokens = per == 1 ? s_tokens[row] : tokens_of(row, nullptr);
    un = units_of(p, tokens, group_idx != nullptr);
    u_lo = max(skip - kItemCost, 0);
    u_hi = min(skip + left - kItemCost, un.total);
  };
  for (;;) {
    int tokens = 0;
    int64_t mine = 0, seen = 0;
    if (!waited) {  // past L1, which must not keep what stands there now
      seen = tid < rows ? __ldcg(pos + tid) : -1;
      tokens = quant_item(qc, seen, tid, nullptr).tokens();
      mine = static_cast<int64_t>(length_of(tokens)) * same;
    }
    for (int i = min(rows, tid * per); waited && i < min(rows, (tid + 1) * per); ++i) {
      tokens = tokens_of(i, blockIdx.x == 0 ? err : nullptr);
      mine += static_cast<int64_t>(length_of(tokens)) * same;
    }
    s_before[tid] = mine;
    s_tokens[tid] = tokens;
    __syncthreads();
    if (warp == 0) {
      int64_t v[kWarps], sum = 0;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        v[j] = s_before[lane * kWarps + j];
        sum += v[j];
      }
      int64_t x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      int64_t run = x - sum;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        s_before[lane * kWarps + j] = run;
        run += v[j];
      }
      if (lane == 31) s_all = x;
    }
    __syncthreads();
    const int64_t all = s_all, slices = static_cast<int64_t>(gridDim.x) * kWarps;
    slice = max(kMinSlice, static_cast<int>((all + slices - 1) / slices));
    const int64_t lo = slice * worker();  // the slice is [lo, lo + left) of the list
    left = static_cast<int>(min(static_cast<int64_t>(slice), max(all - lo, static_cast<int64_t>(0))));
    item = 0;
    skip = 0;
    if (left > 0) {
      int owner = -1;  // the last thread whose rows begin at or before lo
#pragma unroll
      for (int j = 0; j < kWarps; ++j) owner += __popc(__ballot_sync(0xffffffffu, s_before[j * 32 + lane] <= lo));
      int64_t start = s_before[owner];  // where the row begins in the list
      auto enter = [&](int row, int length) {
        const int head = static_cast<int>(static_cast<uint64_t>(lo - start) / static_cast<uint32_t>(length));
        item = row * same + head;
        skip = static_cast<int>(lo - start - static_cast<int64_t>(head) * length);
      };
      if (per == 1) {  // its row is not empty: the next one would begin where it does
        enter(owner, length_of(s_tokens[owner]));
      } else {
        item = items;
        for (int row = owner * per; row < rows; row += 32) {
          const int n = row + lane < rows ? length_of(tokens_of(row + lane, nullptr)) : 0;
          int64_t x = static_cast<int64_t>(n) * same;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          const unsigned beyond = __ballot_sync(0xffffffffu, start + x > lo);
          if (beyond) {
            const int j = __ffs(beyond) - 1, length = __shfl_sync(0xffffffffu, n, j);
            start += __shfl_sync(0xffffffffu, x - static_cast<int64_t>(n) * same, j);
            enter(row + j, length);
            break;
          }
          start += __shfl_sync(0xffffffffu, x, 31);
        }
      }
      if (item < items) enter_item();
    }
    if (waited) {
      __syncthreads();  // every warp has searched
      break;
    }
    pdl_wait();
    waited = true;
    if (!__syncthreads_or(tid < rows && pos[tid] != seen)) {
      if (blockIdx.x == 0 && tid < rows) tokens_of(tid, err);  // flags what is wrong
      break;
    }
  }
  if (blockIdx.x == 0) {  // items without units have no partials
    for (int i = min(rows, tid * per); i < min(rows, (tid + 1) * per); ++i)
      if ((per == 1 ? s_tokens[i] : tokens_of(i, nullptr)) == 0)
        for (int k = 0; k < same; ++k) ws.parts[static_cast<int64_t>(i) * same + k] = make_int2(0, 0);
  }

  W w;
  int stage = 0;       // of the ring, and its phase
  uint32_t phase = 0;
  bool alive = true;   // no wait gave up
  const uint64_t limit_ns = p.debug & kDebugSkipQuantCopy ? 2000000ull : 50000000ull;
  for (bool entered = true; left > 0; ++item, entered = false) {
    if (item >= items) {
      flag_error(err, kErrPos);
      break;
    }
    if (!entered) enter_item();
    if (un.total == 0) continue;
    if (u_hi <= 0) break;  // only the item's fixed part
    left -= un.total + kItemCost - skip;
    skip = 0;
    typename W::Row q_raw[NT][NK];
    w.fetch_q(q, p, b, h, q_raw);  // on its way while the slots are
    pdl_trigger();  // once every CTA has come here or left, the merge may take the places that others leave
    if (lane == 0 && u_lo == 0) {  // this warp has the item's first unit; its last one is total - u_hi further on
      const int me = static_cast<int>(worker()), more = static_cast<int>((static_cast<unsigned>(max(0, -left)) + slice - 1) / slice);
      ws.parts[item] = make_int2(me, min(more, static_cast<int>(gridDim.x) * kWarps - 1 - me) + 1);
    }
    if (un.groups > un.fixed) {
      // kept: ids of candidate chunks, larger than all candidate ids before them
      const int32_t* ids = group_idx + static_cast<int64_t>(item) * p.kg;
      const int window = un.b_base / p.Ng;
      int before = -1;
      bool bad = false;
      for (int i0 = 0; i0 < p.kg; i0 += 32) {
        const int id = i0 + lane < p.kg ? ids[i0 + lane] : -1;
        const bool candidate = id >= 0 && id / p.Ng >= p.sink && id / p.Ng < window;
        int m = candidate ? id : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, m, o);
          if (lane >= o) m = max(m, y);
        }
        int prev = __shfl_up_sync(0xffffffffu, m, 1);
        prev = max(before, lane ? prev : -1);
        const bool keep = candidate && id > prev;
        bad |= id >= 0 && !keep;
        if (i0 + lane < p.kg) routed[i0 + lane] = keep ? id : -1;
        before = max(before, __shfl_sync(0xffffffffu, m, 31));
      }
      if (bad) flag_error(err, kErrGroupIdx);
      __syncwarp();
    }
    const int stride = qc.max_groups + p.kg;
    float2* group = ws.group ? ws.group + static_cast<int64_t>(item) * p.G * stride : nullptr;
    const int32_t* table = qc.table + static_cast<int64_t>(item) * qc.max_groups;
    const int g_hi = min(u_hi, un.groups);  // groups of the slice: [u_lo, g_hi)

    // The slots of the slice's units, 32 at a time: lane i has the one of unit
    // base + i, loaded (unchecked) a block ahead.  -1: no unit, or no slot, -2: id
    // not kept.
    auto load_slots = [&](int base) {
      const int e = base + lane < g_hi ? un.entry(base + lane, routed) : -1;
      return e >= 0 ? table[e] : -1;
    };
    auto checked = [&](int slot, int base) {
      if (base + lane >= g_hi) return -1;
      if (un.entry(base + lane, routed) < 0) return -2;
      if (slot >= 0 && slot < qc.n_slots) return slot;
      flag_error(err, kErrPage);
      return -1;
    };
    // The scales of a block's units, a lane each, are on their way from its first
    // copies to the tile behind them, and then in shared memory.
    int slots = 0, slots_next = load_slots(u_lo), issued = 0, staged = -1;
    float k_scale = 0.f, v_scale = 0.f;
    auto stage_scales = [&]() {
      if (staged >= 0) {
        float mant, ex;
        split_scale(v_scale, mant, ex);
        s_units[warp][(staged >> 5) & 1][lane] = make_float4(k_scale, mant, ex, slots >= 0 ? 1.f : static_cast<float>(slots + 1));
        staged = -1;
      }
    };
    // starts the copies of the slice's next tile, if there is one left
    auto issue = [&](int stage) {
      if (u_lo + issued < g_hi) {
        if ((issued & 31) == 0) {
          slots = checked(slots_next, u_lo + issued);
          slots_next = load_slots(u_lo + issued + 32);
          k_scale = slots >= 0 ? qc.k_scale[slots] : 0.f;
          v_scale = slots >= 0 ? qc.v_scale[slots] : 0.f;
          staged = issued;
        }
        uint8_t* dst = ring + stage * kTile * kUnitBytes;
        const bool copies = lane == 0 && !((p.debug & kDebugSkipQuantCopy) && item == 0 && u_lo == 0 && issued == 0);
        if (copies) ptx::mbar_expect_tx(&s_full[warp][stage], kTile * kUnitBytes);
#pragma unroll
        for (int j = 0; j < kTile; ++j) {
          const int slot = __shfl_sync(0xffffffffu, slots, (issued & 31) + j);
          if (copies) {  // a row before the first reads as zeros
            const int row = slot >= 0 ? slot * kQuantGroup : -kQuantGroup;
            ptx::tma_load_2d(dst + j * kUnitBytes, &map_k, &s_full[warp][stage], 0, row);
            ptx::tma_load_2d(dst + j * kUnitBytes + kUnitBytes / 2, &map_v, &s_full[warp][stage], 0, row);
          }
        }
        issued += kTile;
      }
    };

    if (alive) {
#pragma unroll
      for (int k = 0; k < kStages; ++k) issue((stage + k) % kStages);
    }
    w.load_q(q_raw);
    w.clear();
    if (u_hi > un.groups && alive) {
      const int64_t at = static_cast<int64_t>(item) * kQuantGroup * D;
      w.tail(static_cast<const T*>(qc.k_tail) + at, static_cast<const T*>(qc.v_tail) + at, tokens % kQuantGroup, group,
             stride, un.groups, p.G);
    }
    stage_scales();
    __syncwarp();
    for (int u = u_lo; u < g_hi && alive; u += kTile) {
      if (!__all_sync(0xffffffffu, ptx::mbar_wait_ns(&s_full[warp][stage], phase, kWaitLimit, limit_ns))) {
        // the warp starts no more copies; those under way, this stage's and the ones
        // behind it, get another millisecond each before it goes on
        alive = false;
        flag_error(err, kErrTimeout);
#pragma unroll 1
        for (int k = 0; k < kStages && u + k * kTile < u_lo + issued; ++k)
          ptx::mbar_wait_ns(&s_full[warp][(stage + k) % kStages], stage + k < kStages ? phase : phase ^ 1, kWaitLimit, 1000000ull);
        __syncwarp();
        break;
      }
      const uint32_t tile = ring_at + stage * kTile * kUnitBytes;
      float x[kTile][NT][4], mant[kTile], ex[kTile];
      int at[kTile];
      bool kept[kTile];
#pragma unroll
      for (int j = 0; j < kTile; ++j) {
        const uint32_t kt = tile + j * kUnitBytes;
        uint32_t k[2][D / 64][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < D / 64; ++i) load_shared(kt + Tile<D>::piece(Tile<D>::token(g + 8 * r), i * 4 + c), k[r][i]);
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
          uint32_t a0, a1, a2, a3;
          widen4<FORMAT>(k[0][ks >> 2][ks & 3], a0, a2);
          widen4<FORMAT>(k[1][ks >> 2][ks & 3], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (ks == 0) mma_zero(x[j][nt], a0, a1, a2, a3, w.qh[nt][ks][0], w.qh[nt][ks][1]);
            else mma(x[j][nt], a0, a1, a2, a3, w.qh[nt][ks][0], w.qh[nt][ks][1]);
            if constexpr (W::kSplitQ) mma(x[j][nt], a0, a1, a2, a3, w.ql[nt][ks][0], w.ql[nt][ks][1]);
          }
        }
        const int r = u - u_lo + j;
        const float4 unit = s_units[warp][(r >> 5) & 1][r & 31];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[j][nt][i] = unit.w > 0.f ? x[j][nt][i] * (w.f[nt][i & 1] * unit.x) : -CUDART_INF_F;
        mant[j] = unit.y;
        ex[j] = unit.z;
        at[j] = u + j < g_hi ? u + j : -1;
        kept[j] = unit.w >= 0.f;
      }
      uint32_t pb[kTile][NT][2][2];
      if (group) w.template softmax<kTile, true>(x, mant, ex, pb, group, stride, at, kept, p.G);
      else w.template softmax<kTile, false>(x, mant, ex, pb, group, stride, at, kept, p.G);
      uint32_t v[kTile][4][D / 32];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9; D / 8 bytes at g D / 8
#pragma unroll
      for (int j = 0; j < kTile; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = Tile<D>::token(2 * c + (r & 1) + 8 * (r >> 1));
          load_shared(tile + j * kUnitBytes + kQuantGroup * D + Tile<D>::piece(row, g * D / 128) + (D == 64 ? (g & 1) * 8 : 0), v[j][r]);
        }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t a[kTile][2][4];  // the two 16-row tiles of these four bytes
#pragma unroll
        for (int j = 0; j < kTile; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t lo16 = __byte_perm(v[j][2 * r][i], v[j][2 * r + 1][i], 0x5140);
            const uint32_t hi16 = __byte_perm(v[j][2 * r][i], v[j][2 * r + 1][i], 0x7362);
            widen4<FORMAT>(lo16, a[j][0][2 * r], a[j][0][2 * r + 1]);
            widen4<FORMAT>(hi16, a[j][1][2 * r], a[j][1][2 * r + 1]);
          }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float s[4];
#pragma unroll
            for (int j = 0; j < kTile; ++j) {
              const uint32_t(&y)[4] = a[j][half];
              if (j == 0) mma_zero(s, y[0], y[1], y[2], y[3], pb[j][nt][0][0], pb[j][nt][0][1]);
              else mma(s, y[0], y[1], y[2], y[3], pb[j][nt][0][0], pb[j][nt][0][1]);
              if constexpr (GM != 4) mma(s, y[0], y[1], y[2], y[3], pb[j][nt][1][0], pb[j][nt][1][1]);
            }
            w.add_to(2 * i + half, nt, s);
          }
      }
      stage_scales();
      __syncwarp();  // every lane has read the stage, and written its scales
      issue(stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }

    // this slice's partial of the item (empty, as are its units' weights, once a wait gave up)
    if (!alive) {
      w.clear();
      if (group)
        for (int i = u_lo + lane; i < u_hi; i += 32)
          for (int head = 0; head < p.G; ++head) group[static_cast<int64_t>(head) * stride + i] = make_float2(0.f, kNoRef);
    }
    const int64_t part = worker() + item;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = e ? f32x2::unpack(w.l[nt]).y : f32x2::unpack(w.l[nt]).x;
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
        const int head = nt * 8 + 2 * c + e;
        const bool mine = head < p.G && (GM != 4 || c < 2);
#pragma unroll
        for (int mt = 0; mt < NK; ++mt) {
          const float2 p0 = f32x2::unpack(w.o[mt][nt][0]), p1 = f32x2::unpack(w.o[mt][nt][1]);
          float y0 = e ? p0.y : p0.x, y1 = e ? p1.y : p1.x;
          if constexpr (GM == 4) {  // the low halves' columns
            y0 += __shfl_xor_sync(0xffffffffu, y0, 2);
            y1 += __shfl_xor_sync(0xffffffffu, y1, 2);
          }
          if (mine) *reinterpret_cast<float2*>(ws.sum + (part * p.G + head) * D + mt * 16 + g * 2) = make_float2(y0, y1);
        }
        if (mine && g == 0)
          *reinterpret_cast<float4*>(ws.stat + (part * 16 + head) * 4) =
              make_float4(w.lift[nt][e], w.ref_s[nt][e], l, 0.f);
      }
  }
}

// Merges an item's partials.  The first blocks along y: outputs and LSE of
// kMergeWarps / SPLIT query heads each, SPLIT warps sharing a head's partials;
// the blocks behind them: the weights of 1024 table entries each.
constexpr int kMergeEntries = 1024;
constexpr int merge_warps(int split) { return split > 1 ? split : 8; }
template <int D, typename TO, int SPLIT>
__global__ void __launch_bounds__(merge_warps(SPLIT) * 32)
quant_merge_kernel(LayerParams p, QuantCache qc, const int64_t* pos, Workspace ws,
                   const int32_t* group_idx, const float* weight_in,
                   float* weight_out, TO* __restrict__ out,
                   float* __restrict__ lse) {
  constexpr int kMergeWarps = merge_warps(SPLIT), kMergeThreads = kMergeWarps * 32;
  constexpr int kHeads = kMergeWarps / SPLIT;
  __shared__ float s_sum[SPLIT > 1 ? kMergeWarps : 1][D];
  __shared__ float4 s_warp[SPLIT > 1 ? kMergeWarps : 1];
  __shared__ float s_ref[16][2];
  __shared__ float s_add[kMergeEntries];
  const int64_t item = blockIdx.x;
  const int b = static_cast<int>(item / p.Hkv), h = static_cast<int>(item % p.Hkv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const int2 found = ws.parts[item];
  // only partials that exist, whatever the words hold
  const bool there = found.x >= 0 && found.y > 0 && found.y <= ws.warps - found.x;
  const int2 parts = there ? found : make_int2(0, 0);
  const int64_t first = parts.x + item;
  const float4* stat = reinterpret_cast<const float4*>(ws.stat) + first * 16;
  const int head_blocks = (p.G + kHeads - 1) / kHeads;
  if (static_cast<int>(blockIdx.y) < head_blocks) {
    const int head = blockIdx.y * kHeads + warp / SPLIT, share = warp % SPLIT;
    const bool on = head < p.G;
    float rw = 0.f, rs = kNoRef, acc[D / 32], l = 0.f;  // as in a partial: rw counts from rs
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] = 0.f;
    const float* rows = ws.sum + (first * p.G + head) * D + lane;
    const int count = on ? parts.y : 0;
    constexpr int kBatch = 4;  // partials on their way at a time
    for (int i0 = share; i0 < count; i0 += SPLIT * kBatch) {
      float4 s[kBatch];
      float x[kBatch][D / 32];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * SPLIT;
        s[k] = make_float4(0.f, kNoRef, 0.f, 0.f);
        if (i < count) s[k] = stat[i * 16 + head];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) x[k][j] = i < count ? rows[static_cast<int64_t>(i) * p.G * D + j * 32] : 0.f;
      }
      float ns = rs;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) ns = fmaxf(ns, s[k].y);
      const float held = rw + (rs - ns);
      float nw = held;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        s[k].x += s[k].y - ns;
        nw = fmaxf(nw, s[k].x);
      }
      const float fw = ex2(held - nw);
      l *= ex2(rs - ns);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) acc[j] *= fw;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float f = ex2(s[k].x - nw);
        l += s[k].z * ex2(s[k].y - ns);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) acc[j] += f * x[k][j];
      }
      rw = nw;
      rs = ns;
    }
    if constexpr (SPLIT > 1) {  // one head a block: its warps' sums
#pragma unroll
      for (int j = 0; j < D / 32; ++j) s_sum[warp][j * 32 + lane] = acc[j];
      if (lane == 0) s_warp[warp] = make_float4(rw, rs, l, 0.f);
      __syncthreads();
      if (share == 0) {
        static_assert(SPLIT <= 32, "a lane for every warp");
        const float4 s = lane < SPLIT ? s_warp[lane] : make_float4(0.f, kNoRef, 0.f, 0.f);
        rs = warp_max(s.y);
        const float above = s.x + (s.y - rs);
        rw = warp_max(above);
        l = warp_sum(s.z * ex2(s.y - rs));
        const float f = ex2(above - rw);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) acc[j] = 0.f;
#pragma unroll 8
        for (int k = 0; k < SPLIT; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
          for (int j = 0; j < D / 32; ++j) acc[j] += fk * s_sum[k][j * 32 + lane];
        }
      }
    }
    if (on && share == 0) {
      const int64_t row = static_cast<int64_t>(b) * p.Hq + h * p.G + head;
      // acc is in units of 2^(rs + rw - 14), l in units of 2^rs; two factors, since 2^rw
      // may be as small or large as the values
      const float inverse = l == 0.f ? 0.f : ex2(-kWeightExp) / l, scale = ex2(rw);
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
        store_out(out + row * D + dim_of<D>(j * 32 + lane), l == 0.f ? 0.f : acc[j] * inverse * scale);
      if (lse && lane == 0) lse[row] = l == 0.f ? -CUDART_INF_F : (rs + log2f(l)) * kLn2;
    }
  } else {
    const int e0 = (static_cast<int>(blockIdx.y) - head_blocks) * kMergeEntries;
    const QuantItem it = quant_item(qc, pos[b], item, nullptr);
    const int units = it.units();
    if (e0 < units) {
      for (int head = warp; head < p.G; head += kMergeWarps) {
        float rs = kNoRef, l = 0.f;
        for (int i = lane; i < parts.y; i += 32) rs = fmaxf(rs, stat[i * 16 + head].y);
        rs = warp_max(rs);
        for (int i = lane; i < parts.y; i += 32) {
          const float4 s = stat[i * 16 + head];
          l += s.z * ex2(s.y - rs);
        }
        l = warp_sum(l);
        if (lane == 0) {
          s_ref[head][0] = rs;
          s_ref[head][1] = l == 0.f ? 0.f : 1.f / l;
        }
      }
      __syncthreads();
      const Units un = units_of(p, it.tokens(), group_idx != nullptr);
      const int stride = qc.max_groups + p.kg;
      auto unit_weight = [&](int u) {
        float sum = 0.f;
        for (int head = 0; head < p.G; ++head) {
          const float2 s = ws.group[(item * p.G + head) * stride + u];
          sum += s.x * ex2(s.y - s_ref[head][0]) * s_ref[head][1];
        }
        return sum;
      };
      const int e1 = min(units, e0 + kMergeEntries);
      if (un.groups > un.fixed) {  // the routed ids of these entries
        for (int i = tid; i < kMergeEntries; i += kMergeThreads) s_add[i] = 0.f;
        __syncthreads();
        for (int i = tid; i < p.kg; i += kMergeThreads) {
          const int id = group_idx[item * p.kg + i];
          if (id >= e0 && id < e1 && ws.group[item * p.G * stride + un.fixed + i].x != -1.f)
            s_add[id - e0] = unit_weight(un.fixed + i);
        }
        __syncthreads();
      }
      for (int e = e0 + tid; e < e1; e += kMergeThreads) {
        float sum;
        if (e == it.closed) sum = unit_weight(un.groups);
        else if (e < un.a_end) sum = unit_weight(e);
        else if (e >= un.b_base) sum = unit_weight(un.a_end + e - un.b_base);
        else sum = s_add[e - e0];
        const int64_t at = item * qc.max_groups + e;
        weight_out[at] = weight_in[at] + sum;
      }
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int heads_rounded(const LayerParams& p) { return p.G <= 4 ? 4 : p.G <= 8 ? 8 : 16; }

// Scratch layout; base may be null (sizes only).
size_t layout(const LayerParams& p, int max_groups, bool weight, char* base, Workspace* ws) {
  const size_t items = static_cast<size_t>(p.B) * p.Hkv;
  ws->warps = device_sm_count() * ctas_per_sm(heads_rounded(p)) * kWarps;
  const size_t parts = items + ws->warps;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* x = base + at;
    at += align256(bytes);
    return x;
  };
  ws->stat = reinterpret_cast<float*>(take(parts * 16 * 4 * sizeof(float)));
  ws->sum = reinterpret_cast<float*>(take(parts * p.G * p.D * sizeof(float)));
  ws->parts = reinterpret_cast<int2*>(take(items * sizeof(int2)));
  ws->group = nullptr;
  if (weight)
    ws->group = reinterpret_cast<float2*>(take(items * p.G * (static_cast<size_t>(max_groups) + p.kg) * sizeof(float2)));
  return at;
}

template <typename T, int D, int FORMAT, int GM>
cudaError_t launch_attend(const LayerParams& p, const QuantCache& qc, const void* q, const int64_t* pos,
                          const int32_t* group_idx, const Workspace& ws, unsigned* err, cudaStream_t s) {
  // at most the resident CTAs, and no more than the largest possible list has slices
  const int64_t items = static_cast<int64_t>(p.B) * p.Hkv;
  int64_t most = qc.max_groups;
  if (group_idx) most = std::min(most, (static_cast<int64_t>(p.sink) + p.local + 1) * p.Ng) + p.kg + 1;
  const int64_t slices = (items * (most + kItemCost) + kMinSlice - 1) / kMinSlice;
  const size_t smem = 1024 + kWarps * (kStages * kTile * Tile<D>::kUnitBytes + (group_idx ? p.kg * sizeof(int) : 0));
  // An SM's 228 KB hold fewer CTAs where there are many routed ids (D = 128, from about
  // 350 on): slices for CTAs that only come in a second wave would be as long as the others.
  static const size_t fixed = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, quant_attend_kernel<T, D, FORMAT, GM>) == cudaSuccess ? a.sharedSizeBytes : 0;
  }();
  const int64_t fits = static_cast<int64_t>(228 * 1024 / (1024 + fixed + smem));
  const int64_t resident = device_sm_count() * std::min<int64_t>(fits, ctas_per_sm(GM));
  const unsigned grid = static_cast<unsigned>(std::min((slices + kWarps - 1) / kWarps, resident));
  CUtensorMap map_k, map_v;
  cudaError_t e = make_byte_map(&map_k, qc.k, qc.n_slots * kQuantGroup, D, kQuantGroup);
  if (e == cudaSuccess) e = make_byte_map(&map_v, qc.v, qc.n_slots * kQuantGroup, D, kQuantGroup);
  if (e != cudaSuccess) return e;
  e = ensure_smem<quant_attend_kernel<T, D, FORMAT, GM>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(quant_attend_kernel<T, D, FORMAT, GM>, dim3(grid), dim3(kThreads), smem, s, 1, map_k, map_v,
                    p, qc, static_cast<const T*>(q), pos,
                    group_idx, ws, err);
}

template <typename T, int D, int FORMAT>
cudaError_t launch_g(const LayerParams& p, const QuantCache& qc, const void* q, const int64_t* pos,
                     const int32_t* gi, const Workspace& ws, unsigned* err, cudaStream_t s) {
  switch (heads_rounded(p)) {
    case 4: return launch_attend<T, D, FORMAT, 4>(p, qc, q, pos, gi, ws, err, s);
    case 8: return launch_attend<T, D, FORMAT, 8>(p, qc, q, pos, gi, ws, err, s);
    default: return launch_attend<T, D, FORMAT, 16>(p, qc, q, pos, gi, ws, err, s);
  }
}

template <typename T>
cudaError_t launch_t(const LayerParams& p, const QuantCache& qc, const void* q, const int64_t* pos,
                     const int32_t* gi, const Workspace& ws, unsigned* err, cudaStream_t s) {
  if (qc.format == kQuantInt8)
    return p.D == 64 ? launch_g<T, 64, kQuantInt8>(p, qc, q, pos, gi, ws, err, s)
                     : launch_g<T, 128, kQuantInt8>(p, qc, q, pos, gi, ws, err, s);
  return p.D == 64 ? launch_g<T, 64, kQuantE4m3>(p, qc, q, pos, gi, ws, err, s)
                   : launch_g<T, 128, kQuantE4m3>(p, qc, q, pos, gi, ws, err, s);
}

template <int D, typename TO, int SPLIT>
cudaError_t launch_merge_split(const LayerParams& p, const QuantCache& qc, const int64_t* pos,
                               const Workspace& ws, const int32_t* group_idx, const float* weight_in,
                               float* weight_out, void* out, float* lse, cudaStream_t s) {
  constexpr int threads = merge_warps(SPLIT) * 32, heads = merge_warps(SPLIT) / SPLIT;
  const int blocks = (p.G + heads - 1) / heads + (weight_out ? (qc.max_groups + kMergeEntries - 1) / kMergeEntries : 0);
  return launch_pdl(quant_merge_kernel<D, TO, SPLIT>, dim3(static_cast<unsigned>(p.B * p.Hkv), blocks),
                    dim3(threads), 0, s, 1, p, qc, pos, ws, group_idx, weight_in, weight_out,
                    static_cast<TO*>(out), lse);
}

// Warps that share a head's partials, by how many partials an item has if all are
// alike: with 14 each (128 items, weights) 8 warps take 12 us and 32 warps, whose
// blocks need three waves, 19; with 7 each (256 items) one warp is 3 us faster than 8.
template <int D, typename TO>
cudaError_t launch_merge(const LayerParams& p, const QuantCache& qc, const int64_t* pos,
                         const Workspace& ws, const int32_t* gi, const float* wi, float* wo, void* out,
                         float* lse, cudaStream_t s) {
  const int64_t each = static_cast<int64_t>(device_sm_count()) * ctas_per_sm(heads_rounded(p)) * kWarps / (static_cast<int64_t>(p.B) * p.Hkv);
  auto* kernel = launch_merge_split<D, TO, 1>;
  if (each >= 8) kernel = launch_merge_split<D, TO, 8>;
  if (each >= 64) kernel = launch_merge_split<D, TO, 32>;
  return kernel(p, qc, pos, ws, gi, wi, wo, out, lse, s);
}

}  // namespace

size_t quant_attend_workspace_bytes(const LayerParams& p, int max_groups, bool weight) {
  Workspace ws;
  return layout(p, max_groups, weight, nullptr, &ws);
}

cudaError_t launch_quant_attend(const LayerParams& p, const QuantCache& qc, int dtype, int out_dtype,
                                const void* q, const int64_t* pos, const int32_t* group_idx,
                                const float* weight_in, float* weight_out, void* out, float* lse,
                                void* workspace, unsigned* err, cudaStream_t s) {
  using bf = __nv_bfloat16;
  Workspace ws;
  layout(p, qc.max_groups, weight_out != nullptr, static_cast<char*>(workspace), &ws);
  cudaError_t e = dtype == 0 ? launch_t<float>(p, qc, q, pos, group_idx, ws, err, s)
                             : launch_t<bf>(p, qc, q, pos, group_idx, ws, err, s);
  if (e != cudaSuccess) return e;
  if (p.D == 64)
    return out_dtype == 0 ? launch_merge<64, float>(p, qc, pos, ws, group_idx, weight_in, weight_out, out, lse, s)
                          : launch_merge<64, bf>(p, qc, pos, ws, group_idx, weight_in, weight_out, out, lse, s);
  return out_dtype == 0 ? launch_merge<128, float>(p, qc, pos, ws, group_idx, weight_in, weight_out, out, lse, s)
                        : launch_merge<128, bf>(p, qc, pos, ws, group_idx, weight_in, weight_out, out, lse, s);
}

}  // namespace hga
