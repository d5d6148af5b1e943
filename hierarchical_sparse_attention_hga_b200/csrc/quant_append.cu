// Append to the 8-bit K/V cache: new rows enter the tail, the groups they close
// are written in 8 bits, and (optionally) the RoPE-aware summary rows of those
// groups and of the chunks they close.
//
// A group x[16][D] is written once, when its last token arrives, from the
// unrounded rows (tail and new ones), so no code is ever rescaled:
//   amax = max |x|, inverse = peak / amax, scale = amax / peak (float32, rounded
//   to nearest), code = round-to-nearest-even(x * inverse), peak = 448 (e4m3) or
//   127 (int8).  amax < 2^-100 counts as zero (so neither quotient can overflow
//   or lose bits); a group that holds an infinity or NaN gets codes 0 and a NaN
//   scale, so that whatever attends it is NaN instead of silently finite.
//
// Summary rows use the batch builder's arithmetic (summary_math.cuh) on the
// unrounded rows.  A chunk row needs the raw sums of all its groups; those of
// groups closed by earlier calls are their stored rows times 16 (exact: a power
// of two), so token-by-token and batch appends give the batch builder's bits.
//
// One CTA per chunk (looping), one warp per group, which loads the group's K and V
// rows at once and holds them in registers: lane l has E = D / 32 consecutive
// dimensions of all 16 rows, so a row is one load and its codes one store of the
// warp.  The rotation of the summaries needs dimensions i and i + D/2 together;
// they are held by lanes l and l + 16, which trade half of their elements (one
// shuffle a row).
// Bound by HBM in a prompt (3 D bytes a token and tensor for bf16; 64K tokens of 8 KV
// heads: 61 us, as fast as a copy of the bytes, 70 with the summaries), by latency in a
// decode step (1.8 us for 128 heads).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "quant_cache.cuh"
#include "summary_math.cuh"

namespace hga {
namespace {

using summ::kGroup;

constexpr int kCtas4 = 4, kCtas8 = 2;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Sums of H rotated pairs over a group's rows, with the batch builder's roundings
// (summ::add_rotated): x += x c - y s, y += x s + y c.  High-frequency pairs have
// (c, s) = (1, 0), which leaves the bits of finite rows as a plain sum has them.
// table: per row and H pairs, cosines then sines.
template <int H> struct RotatedSum;
template <> struct RotatedSum<2> {
  uint64_t x = 0, y = 0;
  __device__ __forceinline__ void add(const float (&a)[2], const float (&b)[2], const float* table) {
    const float4 t = *reinterpret_cast<const float4*>(table);
    const uint64_t c = f32x2::pack(t.x, t.y), s = f32x2::pack(t.z, t.w), a2 = f32x2::pack(a[0], a[1]), b2 = f32x2::pack(b[0], b[1]);
    x = f32x2::add(x, f32x2::fma(a2, c, f32x2::mul(b2, s ^ 0x8000000080000000ull)));
    y = f32x2::add(y, f32x2::fma(a2, s, f32x2::mul(b2, c)));
  }
  __device__ __forceinline__ void get(float (&a)[2], float (&b)[2]) const {
    const float2 u = f32x2::unpack(x), v = f32x2::unpack(y);
    a[0] = u.x; a[1] = u.y; b[0] = v.x; b[1] = v.y;
  }
};
template <> struct RotatedSum<1> {
  float x = 0.f, y = 0.f;
  __device__ __forceinline__ void add(const float (&a)[1], const float (&b)[1], const float* table) {
    summ::add_rotated(x, y, a[0], b[0], *reinterpret_cast<const float2*>(table));
  }
  __device__ __forceinline__ void get(float (&a)[1], float (&b)[1]) const { a[0] = x; b[0] = y; }
};

// E consecutive elements of a row as they are stored.
template <typename T, int E> struct Piece;
template <> struct Piece<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  // the largest |x| so far, as bits: integer order, NaN above infinity
  static __device__ __forceinline__ void raise(uint32_t& top, const Piece& x) {
    top = max_u16x2(max_u16x2(top, x.v.x & 0x7fff7fffu), x.v.y & 0x7fff7fffu);
  }
  static __device__ __forceinline__ uint32_t float_bits(uint32_t top) { return max(top << 16, top & 0xffff0000u); }
  // the half of the elements that the partner lane needs, and back
  __device__ __forceinline__ void trade(bool upper, float (&x)[2], float (&y)[2]) const {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? v.x : v.y, 16), mine = upper ? v.y : v.x;
    const uint32_t wx = upper ? other : mine, wy = upper ? mine : other;
    x[0] = __uint_as_float(wx << 16); x[1] = __uint_as_float(wx & 0xffff0000u);
    y[0] = __uint_as_float(wy << 16); y[1] = __uint_as_float(wy & 0xffff0000u);
  }
};
template <> struct Piece<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
  static __device__ __forceinline__ void raise(uint32_t& top, const Piece& x) { top = max_u16x2(top, x.v & 0x7fff7fffu); }
  static __device__ __forceinline__ uint32_t float_bits(uint32_t top) { return max(top << 16, top & 0xffff0000u); }
  __device__ __forceinline__ void trade(bool upper, float (&x)[1], float (&y)[1]) const {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, v, 16);
    // lane l takes the pair of its first element, lane l + 16 that of its second
    x[0] = __uint_as_float(upper ? other & 0xffff0000u : v << 16);
    y[0] = __uint_as_float(upper ? v & 0xffff0000u : other << 16);
  }
};
template <> struct Piece<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ float at(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
  static __device__ __forceinline__ void raise(uint32_t& top, const Piece& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x.at(i)) & 0x7fffffffu);
  }
  static __device__ __forceinline__ uint32_t float_bits(uint32_t top) { return top; }
  __device__ __forceinline__ void trade(bool upper, float (&x)[2], float (&y)[2]) const {
    const float o0 = __shfl_xor_sync(0xffffffffu, upper ? v.x : v.z, 16);
    const float o1 = __shfl_xor_sync(0xffffffffu, upper ? v.y : v.w, 16);
    x[0] = upper ? o0 : v.x; x[1] = upper ? o1 : v.y;
    y[0] = upper ? v.z : o0; y[1] = upper ? v.w : o1;
  }
};
template <> struct Piece<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ float at(int i) const { return i ? v.y : v.x; }
  static __device__ __forceinline__ void raise(uint32_t& top, const Piece& x) {
    top = max(top, max(__float_as_uint(x.v.x) & 0x7fffffffu, __float_as_uint(x.v.y) & 0x7fffffffu));
  }
  static __device__ __forceinline__ uint32_t float_bits(uint32_t top) { return top; }
  __device__ __forceinline__ void trade(bool upper, float (&x)[1], float (&y)[1]) const {
    const float o = __shfl_xor_sync(0xffffffffu, upper ? v.x : v.y, 16);
    x[0] = upper ? o : v.x;
    y[0] = upper ? v.y : o;
  }
};

// E codes, the first in the lowest byte.
template <int FORMAT, int E>
__device__ __forceinline__ uint32_t quantise(const float (&y)[E]) {
  uint32_t r = 0;
  if (FORMAT == kQuantInt8) {
    // |y| <= 127 (1 + 2^-23): adding 1.5 * 2^23 rounds to the nearest even integer,
    // whose low byte is the code
    uint32_t w[E];
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = __float_as_uint(__fadd_rn(y[i], 12582912.f));
    r = __byte_perm(w[0], w[1], 0x0040);
    if (E == 4) r = __byte_perm(r, __byte_perm(w[E - 2], w[E - 1], 0x0040), 0x5410);
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      uint16_t h;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y[i + 1]), "f"(y[i]));
      r |= static_cast<uint32_t>(h) << (8 * i);
    }
  }
  return r;
}

__device__ __forceinline__ void store_codes(uint8_t* p, uint32_t r, std::integral_constant<int, 4>) {
  *reinterpret_cast<uint32_t*>(p) = r;
}
__device__ __forceinline__ void store_codes(uint8_t* p, uint32_t r, std::integral_constant<int, 2>) {
  *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(r);
}

// Resident CTAs per SM of 32 * NG threads that the launch bounds ask for.
constexpr int ctas_per_sm(int ng) { return ng == 4 ? kCtas4 : kCtas8; }

// Codes and scale of one group's rows (a lane's part), stored at the slot.
template <typename T, int D, int FORMAT>
__device__ __forceinline__ void write_group(const Piece<T, D / 32> (&x)[kGroup], uint8_t* codes,
                                            float* scales, int32_t slot) {
  constexpr int E = D / 32;
  constexpr float kPeak = FORMAT == kQuantInt8 ? 127.f : 448.f;
  const int lane = threadIdx.x & 31;
  uint32_t top = 0;
#pragma unroll
  for (int r = 0; r < kGroup; ++r) Piece<T, E>::raise(top, x[r]);
  top = __reduce_max_sync(0xffffffffu, Piece<T, E>::float_bits(top));
  const float amax = __uint_as_float(top);
  const bool finite = top < 0x7f800000u;
  const bool some = finite && amax >= 0x1p-100f;
  const float inverse = some ? __fdiv_rn(kPeak, amax) : 0.f;
  const float scale = some ? __fdiv_rn(amax, kPeak) : (finite ? 0.f : CUDART_NAN_F);
  const uint64_t inverse2 = f32x2::pack(inverse, inverse);
  uint8_t* dst = codes + static_cast<int64_t>(slot) * kGroup * D + lane * E;
#pragma unroll
  for (int r = 0; r < kGroup; ++r) {
    float y[E];
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 t = f32x2::unpack(f32x2::mul(f32x2::pack(x[r].at(i), x[r].at(i + 1)), inverse2));
      y[i] = t.x;
      y[i + 1] = t.y;
    }
    store_codes(dst + r * D, finite ? quantise<FORMAT, E>(y) : 0u, std::integral_constant<int, E>());
  }
  if (lane == 0) scales[slot] = scale;
}

template <typename T, int D, int FORMAT, int NG>
__global__ void __launch_bounds__(32 * NG, ctas_per_sm(NG))
quant_append_kernel(LayerParams p, QuantCache qc, const T* k_new, const T* v_new, int n_new,
                    const int32_t* counts, const int64_t* pos, float* chunk_sum, float* group_sum,
                    unsigned* err) {
  constexpr int P = D / 2, E = D / 32, H = E / 2;  // H: pairs of a lane
  __shared__ float s_gsum[2][NG][D];  // raw group sums of a chunk, by turns
  // rotations of a group's tokens (cosines, then sines, of H pairs at a time) and of a chunk's groups
  extern __shared__ __align__(16) float s_token[];            // [kGroup][D]
  float2* s_group = reinterpret_cast<float2*>(s_token + kGroup * D);  // [NG][n_lo]
  __shared__ double s_omega[P];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x;
  const int b = static_cast<int>(item / p.Hkv);
  // No input is const __restrict__: the kernel just before may still write it while this
  // one runs, so it may not be loaded as data that nobody writes.
  pdl_wait();
  pdl_trigger();  // dependents wait for the whole grid; they may be launched as its CTAs leave

  const int64_t pb = min(max(pos[b], int64_t{-2}), kQuantMaxPos + 1);  // out of range stays so
  const int64_t count = counts ? counts[b] : n_new;
  const int64_t p0 = pb - count + 1;  // position of the first new row
  const int64_t gone = qc.evicted ? qc.evicted[item] : 0;
  const int64_t u0 = p0 >> 4, u_end = (pb + 1) >> 4;  // groups [u0, u_end) close
  const int64_t open = (pb + 1) & 15 ? 1 : 0;
  if (count == 0) return;
  if (pb > kQuantMaxPos || count < 0 || count > n_new || p0 < 0 || gone < 0 || u0 < gone ||
      u_end + open - gone > qc.max_groups) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(err, kErrPos);
    return;
  }
  const bool sums = chunk_sum != nullptr;
  const int n_lo = P - p.n_high;
  const T* k_src = k_new + item * n_new * D + lane * E;
  const T* v_src = v_new + item * n_new * D + lane * E;
  T* k_tail = static_cast<T*>(qc.k_tail) + item * kGroup * D + lane * E;
  T* v_tail = static_cast<T*>(qc.v_tail) + item * kGroup * D + lane * E;

  if (u_end > u0) {
    const int64_t c_last = (u_end - 1) / NG;
    if (sums && u0 / NG + blockIdx.y <= c_last) {
      if (threadIdx.x < P)
        s_omega[threadIdx.x] = static_cast<int>(threadIdx.x) < p.n_high ? 0.0 : summ::pair_omega(p, D, threadIdx.x);
      __syncthreads();
      for (int i = threadIdx.x; i < kGroup * P; i += 32 * NG) {
        const int r = i / P, q = i % P;
        const float2 t = q < p.n_high ? make_float2(1.f, 0.f) : summ::rotation(summ::token_offset(r), s_omega[q]);
        float* to = s_token + r * D + q / H * (2 * H) + q % H;
        to[0] = t.x;
        to[H] = t.y;
      }
      for (int i = threadIdx.x; i < NG * n_lo; i += 32 * NG)
        s_group[i] = summ::rotation(summ::group_offset(p, i / n_lo), s_omega[p.n_high + i % n_lo]);
      __syncthreads();
    }
    // this lane's pairs: dims pair + j and pair + j + D/2
    const bool upper = lane >= 16;
    const int pair = (lane & 15) * E + (upper ? H : 0);
    int turn = 0;
    for (int64_t c = u0 / NG + blockIdx.y; c <= c_last; c += gridDim.y, turn ^= 1) {
      const int64_t u = c * NG + warp;
      const bool in_table = u < qc.max_groups;  // the summary tables' capacity
      if (u >= u0 && u < u_end) {
        const int32_t slot = qc.table[item * qc.max_groups + (u - gone)];
        Piece<T, E> k[kGroup], v[kGroup];
        const int64_t i0 = u * kGroup - p0;
        if (i0 >= 0) {
          const T *ks = k_src + i0 * D, *vs = v_src + i0 * D;
#pragma unroll
          for (int r = 0; r < kGroup; ++r) k[r].load(ks + r * D);
#pragma unroll
          for (int r = 0; r < kGroup; ++r) v[r].load(vs + r * D);
        } else {  // the rows before the first new one are in the tail
#pragma unroll
          for (int r = 0; r < kGroup; ++r) {
            k[r].load(i0 + r >= 0 ? k_src + (i0 + r) * D : k_tail + r * D);
            v[r].load(i0 + r >= 0 ? v_src + (i0 + r) * D : v_tail + r * D);
          }
        }
        const bool held = slot >= 0 && slot < qc.n_slots;
        if (!held && lane == 0) flag_error(err, kErrPage);
        if (held) write_group<T, D, FORMAT>(k, qc.k, qc.k_scale, slot);
        if (sums) {
          RotatedSum<H> sum;
#pragma unroll
          for (int r = 0; r < kGroup; ++r) {
            float px[H], py[H];
            k[r].trade(upper, px, py);
            sum.add(px, py, s_token + r * D + pair * 2);
          }
          float gx[H], gy[H];
          sum.get(gx, gy);
          if (in_table) {
            float* dst = group_sum + (item * qc.max_groups + u) * D;
#pragma unroll
            for (int j = 0; j < H; ++j) {
              dst[pair + j] = __fmul_rn(gx[j], 1.0f / kGroup);
              dst[P + pair + j] = __fmul_rn(gy[j], 1.0f / kGroup);
            }
          } else if (lane == 0) {
            flag_error(err, kErrPos);
          }
#pragma unroll
          for (int j = 0; j < H; ++j) {
            s_gsum[turn][warp][pair + j] = gx[j];
            s_gsum[turn][warp][P + pair + j] = gy[j];
          }
        }
        if (held) write_group<T, D, FORMAT>(v, qc.v, qc.v_scale, slot);
      } else if (sums && u < u0 && in_table) {  // a group an earlier call closed
        const float* row = group_sum + (item * qc.max_groups + u) * D;
        for (int i = lane; i < D; i += 32) s_gsum[turn][warp][i] = __fmul_rn(row[i], static_cast<float>(kGroup));
      }
      if (sums && (c + 1) * NG <= u_end) {  // the chunk closes: uniform over the CTA
        __syncthreads();  // the other turn's sums were last read before this
        if (c < p.n_chunks) {
          const float inv_c = 1.0f / p.C;
          float* dst = chunk_sum + (item * p.n_chunks + c) * D;
          for (int i = threadIdx.x; i < P; i += 32 * NG) {
            const float2 sc = summ::chunk_pair<D>(s_gsum[turn], s_group, NG, p.n_high, n_lo, i);
            dst[i] = __fmul_rn(sc.x, inv_c);
            dst[P + i] = __fmul_rn(sc.y, inv_c);
          }
        }
      }
    }
  }
  // The open group's new rows.  Only this CTA read the old tail (its first chunk
  // holds the first group), and it has finished.
  if (blockIdx.y == 0) {
    __syncthreads();
    const int64_t t0 = max(p0, u_end * kGroup);
    const int rows = static_cast<int>(pb + 1 - t0);
    for (int r = warp; r < rows; r += NG) {
      Piece<T, E> k, v;
      k.load(k_src + (t0 - p0 + r) * D);
      v.load(v_src + (t0 - p0 + r) * D);
      *reinterpret_cast<Piece<T, E>*>(k_tail + ((t0 & 15) + r) * D) = k;
      *reinterpret_cast<Piece<T, E>*>(v_tail + ((t0 & 15) + r) * D) = v;
    }
  }
}

template <typename T, int D, int FORMAT, int NG>
cudaError_t launch_t(const LayerParams& p, const QuantCache& qc, const void* k_new,
                     const void* v_new, int n_new, const int32_t* counts, const int64_t* pos,
                     float* chunk_sum, float* group_sum, unsigned* err, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(p.B) * p.Hkv;
  // A call's new rows touch at most this many chunks.  With summaries the CTAs that
  // fit at a time loop over them, so that each builds its rotations once; without, a
  // CTA takes one chunk, which evens out ragged batches (61 us for a 64K prompt,
  // four chunks a CTA 63 us).
  const int64_t chunks = (static_cast<int64_t>(n_new) + p.C - 2) / p.C + 1;
  int64_t gy = chunk_sum ? static_cast<int64_t>(device_sm_count()) * ctas_per_sm(NG) / items : std::min<int64_t>(chunks, 65535);
  gy = gy < 1 ? 1 : (gy > chunks ? chunks : gy);
  const size_t smem = chunk_sum ? kGroup * D * sizeof(float) + NG * (D / 2 - p.n_high) * sizeof(float2) : 0;
  return launch_pdl(quant_append_kernel<T, D, FORMAT, NG>, dim3(static_cast<unsigned>(items), static_cast<unsigned>(gy)),
                    dim3(32 * NG), smem, s, 1, p, qc, static_cast<const T*>(k_new),
                    static_cast<const T*>(v_new), n_new, counts, pos, chunk_sum, group_sum, err);
}

template <typename T, int D>
cudaError_t launch_f(const LayerParams& p, const QuantCache& qc, const void* k, const void* v, int n,
                     const int32_t* counts, const int64_t* pos, float* cs, float* gs, unsigned* err,
                     cudaStream_t s) {
  auto* kernel = qc.format == kQuantInt8 ? launch_t<T, D, kQuantInt8, 4> : launch_t<T, D, kQuantE4m3, 4>;
  if (p.Ng == 8) kernel = qc.format == kQuantInt8 ? launch_t<T, D, kQuantInt8, 8> : launch_t<T, D, kQuantE4m3, 8>;
  return kernel(p, qc, k, v, n, counts, pos, cs, gs, err, s);
}

}  // namespace

cudaError_t launch_quant_append(const LayerParams& p, const QuantCache& qc, int dtype,
                                const void* k_new, const void* v_new, int n_new,
                                const int32_t* counts, const int64_t* pos, float* chunk_sum,
                                float* group_sum, unsigned* err, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (dtype == 0)
    return p.D == 64 ? launch_f<float, 64>(p, qc, k_new, v_new, n_new, counts, pos, chunk_sum, group_sum, err, s)
                     : launch_f<float, 128>(p, qc, k_new, v_new, n_new, counts, pos, chunk_sum, group_sum, err, s);
  return p.D == 64 ? launch_f<bf, 64>(p, qc, k_new, v_new, n_new, counts, pos, chunk_sum, group_sum, err, s)
                   : launch_f<bf, 128>(p, qc, k_new, v_new, n_new, counts, pos, chunk_sum, group_sum, err, s);
}

}  // namespace hga
