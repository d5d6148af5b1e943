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
// One CTA per chunk (looping), one warp per (group, tensor), which reads each row
// once into registers: lane l holds E = D / 32 consecutive dimensions of all 16
// rows, so a row is one load and its codes one store of the warp.  The rotation
// of the summaries needs dimensions i and i + D/2 together; they are held by lanes
// l and l + 16, which trade half of their elements (one shuffle a row).
// Bound by HBM in a prompt (3 D bytes a token and tensor for bf16), by latency in
// a decode step.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "quant_cache.cuh"
#include "summary_math.cuh"

namespace hga {
namespace {

using summ::kGroup;

// E consecutive elements of a row as they are stored.
template <typename T, int E> struct Piece;
template <> struct Piece<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  // |x| of all elements as float bits: integer order, NaN above infinity
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t a = v.x & 0x7fff7fffu, b = v.y & 0x7fff7fffu;
    return max(max(a << 16, a & 0xffff0000u), max(b << 16, b & 0xffff0000u));
  }
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
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t a = v & 0x7fff7fffu;
    return max(a << 16, a & 0xffff0000u);
  }
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
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fffffffu;
    return max(max(__float_as_uint(v.x) & m, __float_as_uint(v.y) & m), max(__float_as_uint(v.z) & m, __float_as_uint(v.w) & m));
  }
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
  __device__ __forceinline__ uint32_t top() const {
    return max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu);
  }
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

// A barrier of the K warps alone.
__device__ __forceinline__ void k_barrier(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

template <typename T, int D, int FORMAT>
__global__ void __launch_bounds__(512)
quant_append_kernel(LayerParams p, QuantCache qc, const T* __restrict__ k_new,
                    const T* __restrict__ v_new, int n_new, const int32_t* __restrict__ counts,
                    const int64_t* __restrict__ pos, float* __restrict__ chunk_sum,
                    float* __restrict__ group_sum, unsigned* err) {
  constexpr int P = D / 2, E = D / 32, H = E / 2;  // H: pairs of a lane
  constexpr float kPeak = FORMAT == kQuantInt8 ? 127.f : 448.f;
  extern __shared__ float2 smem_tab[];
  __shared__ float s_gsum[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x;
  const int b = static_cast<int>(item / p.Hkv);
  pdl_wait();

  const int64_t pb = pos[b];
  const int64_t count = counts ? counts[b] : n_new;
  const int64_t p0 = pb - count + 1;  // position of the first new row
  const int64_t gone = qc.evicted ? qc.evicted[item] : 0;
  const int64_t u0 = p0 >> 4, u_end = (pb + 1) >> 4;  // groups [u0, u_end) close
  const int64_t open = (pb + 1) & 15 ? 1 : 0;
  if (count == 0) return;
  if (count < 0 || count > n_new || p0 < 0 || gone < 0 || u0 < gone ||
      u_end + open - gone > qc.max_groups) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(err, kErrPos);
    return;
  }
  const bool sums = chunk_sum != nullptr;
  const int n_lo = P - p.n_high;
  const bool is_v = warp >= p.Ng;
  const int w = is_v ? warp - p.Ng : warp;

  if (u_end > u0) {
    const int64_t c_last = (u_end - 1) / p.Ng;
    if (sums && u0 / p.Ng + blockIdx.y <= c_last) {
      for (int i = threadIdx.x; i < summ::table_entries(p, D); i += blockDim.x)
        smem_tab[i] = summ::table_entry(p, D, i);
      __syncthreads();
    }
    const T* src = (is_v ? v_new : k_new) + item * n_new * D + lane * E;
    const T* tail = static_cast<const T*>(is_v ? qc.v_tail : qc.k_tail) + item * kGroup * D + lane * E;
    uint8_t* codes = is_v ? qc.v : qc.k;
    float* scales = is_v ? qc.v_scale : qc.k_scale;
    // this lane's pairs: dims pair + j and pair + j + D/2
    const bool upper = lane >= 16;
    const int pair = (lane & 15) * E + (upper ? H : 0);
    for (int64_t c = u0 / p.Ng + blockIdx.y; c <= c_last; c += gridDim.y) {
      const int64_t u = c * p.Ng + w;
      const bool in_table = u < qc.max_groups;  // the summary tables' capacity
      if (u >= u0 && u < u_end) {
        const int32_t slot = qc.table[item * qc.max_groups + (u - gone)];
        Piece<T, E> x[kGroup];
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < kGroup; ++r) {
          const int64_t i = u * kGroup + r - p0;
          x[r].load(i >= 0 ? src + i * D : tail + r * D);
        }
#pragma unroll
        for (int r = 0; r < kGroup; ++r) top = max(top, x[r].top());
        top = __reduce_max_sync(0xffffffffu, top);
        const float amax = __uint_as_float(top);
        const bool finite = top < 0x7f800000u;
        const bool some = finite && amax >= 0x1p-100f;
        const float inverse = some ? __fdiv_rn(kPeak, amax) : 0.f;
        const float scale = some ? __fdiv_rn(amax, kPeak) : (finite ? 0.f : CUDART_NAN_F);
        if (slot >= 0 && slot < qc.n_slots) {
          uint8_t* dst = codes + static_cast<int64_t>(slot) * kGroup * D + lane * E;
#pragma unroll
          for (int r = 0; r < kGroup; ++r) {
            float y[E];
#pragma unroll
            for (int i = 0; i < E; ++i) y[i] = __fmul_rn(x[r].at(i), inverse);
            store_codes(dst + r * D, finite ? quantise<FORMAT, E>(y) : 0u, std::integral_constant<int, E>());
          }
          if (lane == 0) scales[slot] = scale;
        } else if (lane == 0) {
          flag_error(err, kErrPage);
        }
        if (sums && !is_v) {
          float gx[H], gy[H];
#pragma unroll
          for (int j = 0; j < H; ++j) gx[j] = gy[j] = 0.f;
#pragma unroll
          for (int r = 0; r < kGroup; ++r) {  // the batch builder's order and roundings
            float px[H], py[H];
            x[r].trade(upper, px, py);
#pragma unroll
            for (int j = 0; j < H; ++j) {
              const int i = pair + j;
              if (i < p.n_high) {
                gx[j] = __fadd_rn(gx[j], px[j]);
                gy[j] = __fadd_rn(gy[j], py[j]);
              } else {
                summ::add_rotated(gx[j], gy[j], px[j], py[j], smem_tab[r * n_lo + i - p.n_high]);
              }
            }
          }
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
            s_gsum[w][pair + j] = gx[j];
            s_gsum[w][P + pair + j] = gy[j];
          }
        }
      } else if (sums && !is_v && u < u0 && in_table) {  // a group an earlier call closed
        const float* row = group_sum + (item * qc.max_groups + u) * D;
        for (int i = lane; i < D; i += 32) s_gsum[w][i] = __fmul_rn(row[i], static_cast<float>(kGroup));
      }
      if (sums && !is_v && (c + 1) * p.Ng <= u_end) {  // the chunk closes: uniform over the K warps
        k_barrier(p.Ng * 32);
        if (c < p.n_chunks) {
          const float inv_c = 1.0f / p.C;
          float* dst = chunk_sum + (item * p.n_chunks + c) * D;
          for (int i = threadIdx.x; i < P; i += p.Ng * 32) {
            const float2 sc = summ::chunk_pair<D>(s_gsum, smem_tab + kGroup * n_lo, p.Ng, p.n_high, n_lo, i);
            dst[i] = __fmul_rn(sc.x, inv_c);
            dst[P + i] = __fmul_rn(sc.y, inv_c);
          }
        }
        k_barrier(p.Ng * 32);
      }
    }
  }
  // The open group's new rows.  Only this CTA read the old tail (its first chunk
  // holds the first group), and it has finished.
  if (blockIdx.y == 0) {
    __syncthreads();
    const int64_t t0 = max(p0, u_end * kGroup);
    const int rows = static_cast<int>(pb + 1 - t0);
    const T* from = (is_v ? v_new : k_new) + (item * n_new + (t0 - p0)) * D;
    T* to = static_cast<T*>(is_v ? qc.v_tail : qc.k_tail) + (item * kGroup + (t0 & 15)) * D;
    for (int r = w; r < rows; r += p.Ng) {
      Piece<T, E> x;
      x.load(from + r * D + lane * E);
      *reinterpret_cast<Piece<T, E>*>(to + r * D + lane * E) = x;
    }
  }
  pdl_trigger();
}

template <typename T, int D, int FORMAT>
cudaError_t launch_t(const LayerParams& p, const QuantCache& qc, const void* k_new,
                     const void* v_new, int n_new, const int32_t* counts, const int64_t* pos,
                     float* chunk_sum, float* group_sum, unsigned* err, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(p.B) * p.Hkv;
  // a call's new rows touch at most this many chunks; ~8 CTAs per SM, each looping
  const int64_t chunks = (n_new + p.C - 2) / p.C + 1;
  int64_t gy = (device_sm_count() * 8LL + items - 1) / items;
  gy = gy < 1 ? 1 : (gy > chunks ? chunks : gy);
  const size_t smem = chunk_sum ? summ::table_entries(p, D) * sizeof(float2) : 0;
  return launch_pdl(quant_append_kernel<T, D, FORMAT>, dim3(static_cast<unsigned>(items), static_cast<unsigned>(gy)),
                    dim3(64 * p.Ng), smem, s, 1, p, qc, static_cast<const T*>(k_new),
                    static_cast<const T*>(v_new), n_new, counts, pos, chunk_sum, group_sum, err);
}

template <typename T, int D>
cudaError_t launch_f(const LayerParams& p, const QuantCache& qc, const void* k_new,
                     const void* v_new, int n_new, const int32_t* counts, const int64_t* pos,
                     float* chunk_sum, float* group_sum, unsigned* err, cudaStream_t s) {
  return qc.format == kQuantInt8
             ? launch_t<T, D, kQuantInt8>(p, qc, k_new, v_new, n_new, counts, pos, chunk_sum, group_sum, err, s)
             : launch_t<T, D, kQuantE4m3>(p, qc, k_new, v_new, n_new, counts, pos, chunk_sum, group_sum, err, s);
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
