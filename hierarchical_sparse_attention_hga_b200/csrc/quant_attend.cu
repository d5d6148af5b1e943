// Decode attention over the 8-bit K/V cache.
//
// One query token per sequence attends, exactly, every live group of its
// (sequence, KV head) and the open group's tail rows, or, given routed group
// ids, the sinks, the window and the routed groups (the sets of hga_attend):
//   s_t = (q . c_t) * k_scale / sqrt(D),  p = softmax(s),  out = sum_t p_t v_scale c'_t
// with codes c, c'.  On request each group's weight, the sum of p over its
// tokens and the G query heads of the KV head, is added to an accumulator.
#include "common.cuh"
#include "kernels.h"
#include "quant_cache.cuh"

namespace hga {
namespace {

constexpr int kThreads = 128;
constexpr int kGMax = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Table entries a query attends, as a virtual list: [0, a_end), then
// [b_base, closed), then the routed ids (kept ones; -1 where an entry is not).
struct Units {
  int a_end, b_base, fixed, total;
  __device__ __forceinline__ int entry(int i, const int* routed) const {
    if (i < a_end) return i;
    if (i < fixed) return b_base + (i - a_end);
    return routed[i - fixed];
  }
};

template <typename T, int D, int FORMAT, typename TO>
__global__ void __launch_bounds__(kThreads)
quant_attend_kernel(LayerParams p, QuantCache qc, const T* __restrict__ q,
                    const int64_t* __restrict__ pos, const int32_t* __restrict__ group_idx,
                    const float* weight_in, float* weight_out, TO* __restrict__ out,
                    float* __restrict__ lse, float* __restrict__ ws, unsigned* err) {
  __shared__ float s_k[kQuantGroup][D + 1], s_v[kQuantGroup][D + 1];
  __shared__ float s_q[kGMax][D + 1];
  __shared__ float s_p[kGMax][kQuantGroup], s_m[kGMax], s_l[kGMax], s_scale[kGMax];
  extern __shared__ int s_routed[];
  const int64_t item = blockIdx.x;
  const int b = static_cast<int>(item / p.Hkv), h = static_cast<int>(item % p.Hkv);
  const int tid = threadIdx.x;
  pdl_wait();
  const int64_t pb = pos[b];
  const QuantItem it = quant_item(qc, pb, item, tid == 0 ? err : nullptr);
  Units un{0, 0, it.closed, it.closed};
  if (group_idx && it.units()) {
    const int cur = static_cast<int>(pb / p.C);
    const int first = max(0, cur - p.local);
    un.a_end = min(p.sink, first) * p.Ng;
    un.b_base = first * p.Ng;
    un.fixed = un.a_end + it.closed - un.b_base;
    un.total = un.fixed + p.kg;
    for (int i = tid; i < p.kg; i += kThreads) s_routed[i] = group_idx[item * p.kg + i];
    __syncthreads();
    if (tid == 0) {
      int prev = -1;
      bool bad = false;
      for (int i = 0; i < p.kg; ++i) {
        const int id = s_routed[i];
        if (id < 0) { s_routed[i] = -1; continue; }
        const int c = id / p.Ng;
        if (c < p.sink || c >= first || id <= prev) { bad = true; s_routed[i] = -1; continue; }
        prev = id;
      }
      if (bad) flag_error(err, kErrGroupIdx);
    }
  }
  const float scale = kLog2e * rsqrtf(static_cast<float>(D));
  for (int i = tid; i < p.G * D; i += kThreads)
    s_q[i / D][i % D] = to_f32(q[(static_cast<int64_t>(b) * p.Hq + h * p.G) * D + i]) * scale;
  if (tid < kGMax) { s_m[tid] = -CUDART_INF_F; s_l[tid] = 0.f; }
  __syncthreads();
  float* lu = ws + item * p.G * qc.max_groups;  // log2 of each group's sum, per query head
  if (weight_out)
    for (int i = tid; i < p.G * qc.max_groups; i += kThreads) lu[i] = -CUDART_INF_F;
  float acc[kGMax];
#pragma unroll
  for (int j = 0; j < kGMax; ++j) acc[j] = 0.f;
  const int d = tid % D;
  constexpr int HS = kThreads / D;
  for (int u = 0; u < un.total + (it.rest > 0); ++u) {
    const bool tail = u == un.total;
    const int e = tail ? it.closed : un.entry(u, s_routed);
    __syncthreads();
    if (e < 0) continue;
    int rows = kQuantGroup;
    if (tail) {
      rows = it.rest;
      const T* kt = static_cast<const T*>(qc.k_tail) + item * kQuantGroup * D;
      const T* vt = static_cast<const T*>(qc.v_tail) + item * kQuantGroup * D;
      for (int i = tid; i < rows * D; i += kThreads) {
        s_k[i / D][i % D] = to_f32(kt[i]);
        s_v[i / D][i % D] = to_f32(vt[i]);
      }
    } else {
      const int32_t slot = qc.table[item * qc.max_groups + e];
      if (slot < 0 || slot >= qc.n_slots) {
        if (tid == 0) flag_error(err, kErrPage);
        continue;
      }
      const int64_t base = static_cast<int64_t>(slot) * kQuantGroup * D;
      const float ks = qc.k_scale[slot], vs = qc.v_scale[slot];
      for (int i = tid; i < kQuantGroup * D; i += kThreads) {
        s_k[i / D][i % D] = code_to_f32<FORMAT>(qc.k[base + i]) * ks;
        s_v[i / D][i % D] = code_to_f32<FORMAT>(qc.v[base + i]) * vs;
      }
    }
    __syncthreads();
    for (int i = tid; i < p.G * kQuantGroup; i += kThreads) {
      const int hh = i / kQuantGroup, t = i % kQuantGroup;
      float s = -CUDART_INF_F;
      if (t < rows) {
        s = 0.f;
        for (int x = 0; x < D; ++x) s += s_q[hh][x] * s_k[t][x];
      }
      s_p[hh][t] = s;
    }
    __syncthreads();
    if (tid < p.G) {
      float m = s_m[tid], mu = -CUDART_INF_F, sum = 0.f;
      for (int t = 0; t < rows; ++t) mu = fmaxf(mu, s_p[tid][t]);
      const float mn = fmaxf(m, mu), ref = mn == -CUDART_INF_F ? 0.f : mn;
      for (int t = 0; t < rows; ++t) {
        const float x = exp2f(s_p[tid][t] - ref);
        s_p[tid][t] = x;
        sum += x;
      }
      s_scale[tid] = m == -CUDART_INF_F ? 0.f : exp2f(m - ref);
      s_l[tid] = s_l[tid] * s_scale[tid] + sum;
      s_m[tid] = mn;
      if (weight_out) lu[tid * qc.max_groups + e] = log2f(sum) + ref;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kGMax; ++j) {
      const int hh = tid / D + j * HS;
      if (hh >= p.G) continue;
      acc[j] *= s_scale[hh];
      for (int t = 0; t < rows; ++t) acc[j] += s_p[hh][t] * s_v[t][d];
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kGMax; ++j) {
    const int hh = tid / D + j * HS;
    if (hh >= p.G) continue;
    const float m = s_m[hh], l = s_l[hh];
    const int64_t row = static_cast<int64_t>(b) * p.Hq + h * p.G + hh;
    store_out(out + row * D + d, l == 0.f ? 0.f : acc[j] / l);
    if (lse && d == 0) lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
  }
  if (weight_out) {
    for (int e = tid; e < it.units(); e += kThreads) {
      float sum = 0.f;
      for (int hh = 0; hh < p.G; ++hh)
        if (s_l[hh] != 0.f) sum += exp2f(lu[hh * qc.max_groups + e] - (s_m[hh] + log2f(s_l[hh])));
      const int64_t at = item * qc.max_groups + e;
      weight_out[at] = weight_in[at] + sum;
    }
  }
  pdl_trigger();
}

template <typename T, int D, int FORMAT, typename TO>
cudaError_t launch_t(const LayerParams& p, const QuantCache& qc, const void* q, const int64_t* pos,
                     const int32_t* group_idx, const float* weight_in, float* weight_out, void* out,
                     float* lse, void* ws, unsigned* err, cudaStream_t s) {
  return launch_pdl(quant_attend_kernel<T, D, FORMAT, TO>, dim3(static_cast<unsigned>(p.B * p.Hkv)),
                    dim3(kThreads), static_cast<size_t>(group_idx ? p.kg : 0) * sizeof(int), s, 1, p,
                    qc, static_cast<const T*>(q), pos, group_idx, weight_in, weight_out,
                    static_cast<TO*>(out), lse, static_cast<float*>(ws), err);
}

template <typename T, int D>
cudaError_t launch_f(const LayerParams& p, const QuantCache& qc, int out_dtype, const void* q,
                     const int64_t* pos, const int32_t* group_idx, const float* wi, float* wo,
                     void* out, float* lse, void* ws, unsigned* err, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (qc.format == kQuantInt8)
    return out_dtype == 0 ? launch_t<T, D, kQuantInt8, float>(p, qc, q, pos, group_idx, wi, wo, out, lse, ws, err, s)
                          : launch_t<T, D, kQuantInt8, bf>(p, qc, q, pos, group_idx, wi, wo, out, lse, ws, err, s);
  return out_dtype == 0 ? launch_t<T, D, kQuantE4m3, float>(p, qc, q, pos, group_idx, wi, wo, out, lse, ws, err, s)
                        : launch_t<T, D, kQuantE4m3, bf>(p, qc, q, pos, group_idx, wi, wo, out, lse, ws, err, s);
}

}  // namespace

size_t quant_attend_workspace_bytes(const LayerParams& p, int max_groups, bool weight) {
  return weight ? static_cast<size_t>(p.B) * p.Hq * max_groups * sizeof(float) : 0;
}

cudaError_t launch_quant_attend(const LayerParams& p, const QuantCache& qc, int dtype, int out_dtype,
                                const void* q, const int64_t* pos, const int32_t* group_idx,
                                const float* weight_in, float* weight_out, void* out, float* lse,
                                void* ws, unsigned* err, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (dtype == 0)
    return p.D == 64 ? launch_f<float, 64>(p, qc, out_dtype, q, pos, group_idx, weight_in, weight_out, out, lse, ws, err, s)
                     : launch_f<float, 128>(p, qc, out_dtype, q, pos, group_idx, weight_in, weight_out, out, lse, ws, err, s);
  return p.D == 64 ? launch_f<bf, 64>(p, qc, out_dtype, q, pos, group_idx, weight_in, weight_out, out, lse, ws, err, s)
                   : launch_f<bf, 128>(p, qc, out_dtype, q, pos, group_idx, weight_in, weight_out, out, lse, ws, err, s);
}

}  // namespace hga
