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
// One CTA per chunk (looping), one warp per (group, tensor): a lane owns the
// pairs (i, i + D/2) that the summary needs and holds the group's 16 rows of
// them in registers, so every row is read once.
#include "common.cuh"
#include "kernels.h"
#include "quant_cache.cuh"
#include "summary_math.cuh"

namespace hga {
namespace {

using summ::kGroup;

template <int FORMAT>
__device__ __forceinline__ uint32_t quantise2(float a, float b) {  // two codes, a in the low byte
  if (FORMAT == kQuantInt8) {
    // |a|, |b| <= 127 (1 + 2^-23): rounds to at most 127
    const int ia = __float2int_rn(a), ib = __float2int_rn(b);
    return (ia & 0xff) | ((ib & 0xff) << 8);
  }
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <typename T, int D, int FORMAT>
__global__ void __launch_bounds__(512)
quant_append_kernel(LayerParams p, QuantCache qc, const T* __restrict__ k_new,
                    const T* __restrict__ v_new, int n_new, const int32_t* __restrict__ counts,
                    const int64_t* __restrict__ pos, float* __restrict__ chunk_sum,
                    float* __restrict__ group_sum, unsigned* err) {
  constexpr int P = D / 2, PPL = P / 32;
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
  const T* src = (is_v ? v_new : k_new) + item * n_new * D;
  T* tail = static_cast<T*>(is_v ? qc.v_tail : qc.k_tail) + item * kGroup * D;
  uint8_t* codes = is_v ? qc.v : qc.k;
  float* scales = is_v ? qc.v_scale : qc.k_scale;

  if (u_end > u0) {
    if (sums) {
      for (int i = threadIdx.x; i < summ::table_entries(p, D); i += blockDim.x)
        smem_tab[i] = summ::table_entry(p, D, i);
      __syncthreads();
    }
    const int64_t c_last = (u_end - 1) / p.Ng;
    for (int64_t c = u0 / p.Ng + blockIdx.y; c <= c_last; c += gridDim.y) {
      const int64_t u = c * p.Ng + w;
      const bool in_table = u < qc.max_groups;  // the summary tables' capacity
      if (u >= u0 && u < u_end) {
        float x[kGroup][PPL], y[kGroup][PPL];
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < kGroup; ++r) {
          const int64_t i = u * kGroup + r - p0;
          const T* row = (i >= 0 ? src + i * D : tail + r * D) + lane * PPL;
#pragma unroll
          for (int e = 0; e < PPL; ++e) {
            x[r][e] = to_f32(row[e]);
            y[r][e] = to_f32(row[P + e]);
          }
        }
#pragma unroll
        for (int r = 0; r < kGroup; ++r)
#pragma unroll
          for (int e = 0; e < PPL; ++e)
            top = max(top, max(__float_as_uint(x[r][e]) & 0x7fffffffu,
                               __float_as_uint(y[r][e]) & 0x7fffffffu));
        top = __reduce_max_sync(0xffffffffu, top);  // as integers, NaN > inf > finite
        const float amax = __uint_as_float(top);
        const bool finite = top < 0x7f800000u;
        const bool some = finite && amax >= 0x1p-100f;
        const float inverse = some ? __fdiv_rn(kPeak, amax) : 0.f;
        const float scale = some ? __fdiv_rn(amax, kPeak) : (finite ? 0.f : CUDART_NAN_F);
        const int32_t slot = qc.table[item * qc.max_groups + (u - gone)];
        if (slot >= 0 && slot < qc.n_slots) {
          uint8_t* dst = codes + static_cast<int64_t>(slot) * kGroup * D + lane * PPL;
#pragma unroll
          for (int r = 0; r < kGroup; ++r) {
            if constexpr (PPL == 2) {
              const uint32_t cx = finite ? quantise2<FORMAT>(__fmul_rn(x[r][0], inverse), __fmul_rn(x[r][1], inverse)) : 0u;
              const uint32_t cy = finite ? quantise2<FORMAT>(__fmul_rn(y[r][0], inverse), __fmul_rn(y[r][1], inverse)) : 0u;
              *reinterpret_cast<uint16_t*>(dst + r * D) = static_cast<uint16_t>(cx);
              *reinterpret_cast<uint16_t*>(dst + r * D + P) = static_cast<uint16_t>(cy);
            } else {
              const uint32_t cxy = finite ? quantise2<FORMAT>(__fmul_rn(x[r][0], inverse), __fmul_rn(y[r][0], inverse)) : 0u;
              dst[r * D] = static_cast<uint8_t>(cxy);
              dst[r * D + P] = static_cast<uint8_t>(cxy >> 8);
            }
          }
          if (lane == 0) scales[slot] = scale;
        } else if (lane == 0) {
          flag_error(err, kErrPage);
        }
        if (sums && !is_v) {
          float gx[PPL], gy[PPL];
          summ::group_raw_sum<PPL>(x, y, smem_tab, p.n_high, n_lo, lane, gx, gy);
          if (in_table) {
            float* dst = group_sum + (item * qc.max_groups + u) * D;
#pragma unroll
            for (int e = 0; e < PPL; ++e) {
              dst[lane * PPL + e] = __fmul_rn(gx[e], 1.0f / kGroup);
              dst[P + lane * PPL + e] = __fmul_rn(gy[e], 1.0f / kGroup);
            }
          } else if (lane == 0) {
            flag_error(err, kErrPos);
          }
#pragma unroll
          for (int e = 0; e < PPL; ++e) {
            s_gsum[w][lane * PPL + e] = gx[e];
            s_gsum[w][P + lane * PPL + e] = gy[e];
          }
        }
      } else if (sums && !is_v && u < u0 && in_table) {  // a group an earlier call closed
        const float* row = group_sum + (item * qc.max_groups + u) * D;
        for (int i = lane; i < D; i += 32) s_gsum[w][i] = __fmul_rn(row[i], static_cast<float>(kGroup));
      }
      if (sums && (c + 1) * p.Ng <= u_end) {  // the chunk closes: uniform over the CTA
        __syncthreads();
        if (c < p.n_chunks) {
          const float inv_c = 1.0f / p.C;
          float* dst = chunk_sum + (item * p.n_chunks + c) * D;
          for (int i = threadIdx.x; i < P; i += blockDim.x) {
            const float2 sc = summ::chunk_pair<D>(s_gsum, smem_tab + kGroup * n_lo, p.Ng, p.n_high, n_lo, i);
            dst[i] = __fmul_rn(sc.x, inv_c);
            dst[P + i] = __fmul_rn(sc.y, inv_c);
          }
        }
        __syncthreads();
      }
    }
  }
  // The open group's new rows.  Only this CTA read the old tail (its first chunk
  // holds the first group), and it has finished.
  if (blockIdx.y == 0) {
    __syncthreads();
    const int64_t t0 = max(p0, u_end * kGroup);
    const int rows = static_cast<int>(pb + 1 - t0);
    for (int i = threadIdx.x; i < 2 * rows * D; i += blockDim.x) {
      const int which = i / (rows * D), j = i % (rows * D), r = j / D, d = j % D;
      const T* from = (which ? v_new : k_new) + (item * n_new + (t0 - p0) + r) * D + d;
      T* to = static_cast<T*>(which ? qc.v_tail : qc.k_tail) + (item * kGroup + ((t0 + r) & 15)) * D + d;
      *to = *from;
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
