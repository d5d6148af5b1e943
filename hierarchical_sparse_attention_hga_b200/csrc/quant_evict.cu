// Eviction from the 8-bit K/V cache by accumulated attention weight.
//
// Per (sequence, KV head) with n live groups and a budget of `keep`: the first
// `sink` and the last `recent` groups stay, and of those between them the
// keep - sink - recent with the largest weights (equal weights: the earlier
// group).  No key or value moves: the table is a permutation of the item's
// slots, so a stable partition of it (kept entries, then the freed ones, then
// the ones that were free) evicts and hands the freed slots to later appends.
//
// One CTA per item, thread t owning a contiguous run of entries.  The weights
// are read once into shared memory and become order-preserving integers; the
// threshold (the smallest kept key) is found digit by digit with shared-memory
// histograms, and one block scan of (above, equal) counts gives every entry its
// place.  All reads of a row come before its first write, so the outputs may be
// the inputs.
#include "common.cuh"
#include "kernels.h"
#include "quant_cache.cuh"

namespace hga {
namespace {

constexpr int kThreads = 512;

// Larger key = kept first.  NaN counts as least; -0 and +0 are equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct ScanSmem {
  unsigned long long part[kThreads / 32];
};

// Exclusive block scan of a pair of counts packed in one 64-bit word.
__device__ __forceinline__ unsigned long long block_exclusive(unsigned long long v, ScanSmem& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm.part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = lane < kThreads / 32 ? sm.part[lane] : 0ull;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < kThreads / 32) sm.part[lane] = s;
  }
  __syncthreads();
  return x - v + (warp ? sm.part[warp - 1] : 0ull);
}

__global__ void __launch_bounds__(kThreads)
quant_evict_kernel(int Hkv, QuantCache qc, const int64_t* __restrict__ pos, int keep, int sink,
                   int recent, const float* weight_in, float* weight_out, int32_t* table_out,
                   int32_t* evicted_out, unsigned* err) {
  extern __shared__ uint32_t s_row[];  // [max_groups]: the weights, then the table
  __shared__ unsigned s_hist[256];
  __shared__ ScanSmem s_scan;
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int64_t item = blockIdx.x;
  const int tid = threadIdx.x;
  pdl_wait();

  const QuantItem it = quant_item(qc, pos[item / Hkv], item, tid == 0 ? err : nullptr);
  const int n = it.closed, max_groups = qc.max_groups;
  const float* w_in = weight_in + item * max_groups;
  float* w_out = weight_out + item * max_groups;
  const int32_t* t_in = qc.table + item * max_groups;
  int32_t* t_out = table_out + item * max_groups;
  const int gone = qc.evicted ? qc.evicted[item] : 0;
  if (!it.ok) {  // flagged: nothing is evicted
    for (int i = tid; i < max_groups; i += kThreads) {
      w_out[i] = w_in[i];
      t_out[i] = t_in[i];
    }
    if (tid == 0) evicted_out[item] = gone;
    return;
  }
  for (int i = tid; i < max_groups; i += kThreads) s_row[i] = __float_as_uint(w_in[i]);
  __syncthreads();

  const int lo = sink, hi = n - recent;   // candidates [lo, hi)
  const bool evicts = n > keep;           // then hi - lo > keep - sink - recent >= 0
  const int want = keep - sink - recent;  // candidates that stay
  uint32_t threshold = 0xffffffffu;       // no finite or infinite weight has this key
  int ties = 0;
  if (evicts && want > 0) {
    if (tid == 0) {
      s_prefix = 0;
      s_need = want;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      for (int i = lo + tid; i < hi; i += kThreads) {
        const uint32_t key = weight_key(__uint_as_float(s_row[i]));
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&s_hist[(key >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int need = s_need, d = 255;
        while (static_cast<int>(s_hist[d]) < need) need -= s_hist[d--];
        s_need = need;
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      }
      __syncthreads();
    }
    threshold = s_prefix;
    ties = s_need;  // entries equal to the threshold that stay, the earliest ones
  }

  // thread t owns entries [i0, i1); an odd run length spreads the banks
  const int run = ((max_groups + kThreads - 1) / kThreads) | 1;
  const int i0 = min(tid * run, max_groups), i1 = min(i0 + run, max_groups);
  unsigned long long mine = 0;  // low word: kept whatever the ties, high word: equal to the threshold
  for (int i = i0; i < min(i1, n); ++i) {
    if (!evicts || i < lo || i >= hi) {
      mine += 1;
    } else {
      const uint32_t key = weight_key(__uint_as_float(s_row[i]));
      if (key > threshold) mine += 1;
      else if (key == threshold) mine += 1ull << 32;
    }
  }
  const unsigned long long before = block_exclusive(mine, s_scan);
  const int kept_n = evicts ? keep : n;
  int kept = static_cast<int>(before & 0xffffffffu);
  int equal = static_cast<int>(before >> 32);
  int place = kept + min(equal, ties);  // kept entries before this thread's run
  unsigned long long mask[2] = {0, 0};  // which of the run's entries are kept (run <= 97)
  const int place0 = place;
  for (int i = i0; i < i1; ++i) {
    bool stay = i >= n;
    if (i < n) {
      if (!evicts || i < lo || i >= hi) {
        stay = true;
      } else {
        const uint32_t key = weight_key(__uint_as_float(s_row[i]));
        stay = key > threshold || (key == threshold && equal++ < ties);
      }
      if (stay) w_out[place++] = __uint_as_float(s_row[i]);
    }
    if (stay) mask[(i - i0) >> 6] |= 1ull << ((i - i0) & 63);
  }
  // the open group's weight follows the last kept one; entries behind it start at 0
  for (int i = kept_n + tid; i < max_groups; i += kThreads)
    w_out[i] = i == kept_n && n < max_groups ? __uint_as_float(s_row[n]) : 0.f;
  __syncthreads();

  for (int i = tid; i < max_groups; i += kThreads) s_row[i] = static_cast<uint32_t>(t_in[i]);
  __syncthreads();
  place = place0;
  for (int i = i0; i < i1; ++i) {
    const bool stay = mask[(i - i0) >> 6] >> ((i - i0) & 63) & 1;
    int to = i;
    if (i < n) to = stay ? place++ : kept_n + (i - place);
    t_out[to] = static_cast<int32_t>(s_row[i]);
  }
  if (tid == 0) evicted_out[item] = gone + (n - kept_n);
  pdl_trigger();
}

}  // namespace

cudaError_t launch_quant_evict(const LayerParams& p, const QuantCache& qc, const int64_t* pos,
                               int keep, int sink, int recent, const float* weight_in,
                               float* weight_out, int32_t* table_out, int32_t* evicted_out,
                               unsigned* err, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(qc.max_groups) * sizeof(uint32_t);
  cudaError_t e = ensure_smem<quant_evict_kernel>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(quant_evict_kernel, dim3(static_cast<unsigned>(p.B * p.Hkv)), dim3(kThreads),
                    smem, s, 1, p.Hkv, qc, pos, keep, sink, recent, weight_in, weight_out,
                    table_out, evicted_out, err);
}

}  // namespace hga
