// Eviction from the 8-bit K/V cache by accumulated attention weight.
//
// Per (sequence, KV head) with n live groups and a budget of `keep`: the first
// `sink` and the last `recent` groups stay, and of those between them the
// keep - sink - recent with the largest weights (equal weights: the earlier
// group).  No key or value moves: the table is a permutation of the item's
// slots, so a stable partition of it (kept entries, then the freed ones, then
// the ones that were free) evicts and hands the freed slots to later appends.
//
// One CTA per item; 16 bytes an entry, so a call is a chain of latencies (6.2 us
// for 128 rows of 513 groups, 12.8 us for 64 rows of 8192, where it is the CTA's own
// instructions: 0.6 of its issue slots).  The
// weights become order-preserving integers; the threshold (the smallest kept
// key) is found in three digits of 11, 11 and 10 bits with shared-memory
// histograms (the first digit holds sign, exponent and two more bits, so that
// weights of one size do not all meet in one counter).  Then 32 entries at a
// time become two masks (above, equal), one block scan over the masks' counts
// gives each its place, and kept and freed entries are written in order.  All
// reads of a row come before its first write, so the outputs may be the inputs.
#include "common.cuh"
#include "kernels.h"
#include "quant_cache.cuh"

namespace hga {
namespace {

constexpr int kBins = 2048;

// Larger key = kept first.  NaN counts as least; -0 and +0 are equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive block scan; `total` gets the sum.
template <int NT>
__device__ __forceinline__ unsigned block_exclusive(unsigned v, unsigned* part, unsigned& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // part may still be read from the last scan
  if (lane == 31) part[warp] = x;
  __syncthreads();
  unsigned s = lane < NT / 32 ? part[lane] : 0u;  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const unsigned before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return x - v + (warp ? before : 0u);
}

// Bytes of shared memory: one or both rows, then masks and places (or the histogram).
__host__ __device__ inline int mask_words(int max_groups) { return (max_groups + 31) / 32; }
__host__ __device__ inline size_t scratch_bytes(int max_groups) {
  const size_t places = static_cast<size_t>(mask_words(max_groups)) * 4;
  return mask_words(max_groups) * 8ull + (places > kBins * 4 ? places : kBins * 4);
}
size_t smem_bytes(int max_groups, int rows) {
  return (static_cast<size_t>(max_groups) * rows * 4 + 15) / 16 * 16 + scratch_bytes(max_groups);
}

// ROWS: rows in shared memory at a time (the weights, or the weights and the table).
template <int NT, int ROWS>
__global__ void __launch_bounds__(NT)
quant_evict_kernel(int Hkv, QuantCache qc, const int64_t* pos, int keep, int sink,
                   int recent, const float* weight_in, float* weight_out, int32_t* table_out,
                   int32_t* evicted_out, unsigned* err) {
  extern __shared__ __align__(16) uint32_t s_mem[];
  __shared__ unsigned s_part[NT / 32];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  const int max_groups = qc.max_groups, words = mask_words(max_groups);
  uint32_t* s_weight = s_mem;
  uint32_t* s_table = ROWS == 2 ? s_mem + max_groups : s_mem;
  uint32_t* s_above = s_mem + (max_groups * ROWS + 3) / 4 * 4;
  uint32_t* s_equal = s_above + words;
  unsigned* s_place = s_equal + words;
  unsigned* s_hist = s_place;  // before there are places
  const int64_t item = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* w_in = weight_in + item * max_groups;
  float* w_out = weight_out + item * max_groups;
  const int32_t* t_in = qc.table + item * max_groups;
  int32_t* t_out = table_out + item * max_groups;
  pdl_wait();  // the position too may be what the kernel just before writes
  pdl_trigger();  // dependents wait for the whole grid; they may be launched as its CTAs leave

  const int64_t pb = pos[item / Hkv];
  const int gone = qc.evicted ? qc.evicted[item] : 0;  // on its way with the rows
#pragma unroll 4
  for (int i = tid; i < max_groups; i += NT) {
    s_weight[i] = __float_as_uint(w_in[i]);
    if (ROWS == 2) s_table[i] = static_cast<uint32_t>(t_in[i]);
  }
  const QuantItem it = quant_item(qc, pb, item, tid == 0 ? err : nullptr);
  const int n = it.closed;
  const int lo = sink, hi = n - recent;      // candidates [lo, hi)
  const bool evicts = n > keep;              // then hi - lo > keep - sink - recent >= 0
  const int want = keep - sink - recent;     // candidates that stay
  uint32_t threshold = 0xffffffffu;          // no weight has this key
  int ties = 0;
  __syncthreads();
  if (evicts && want > 0) {
    uint32_t prefix = 0;
    int need = want;
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
      const int bits = shift == 0 ? 10 : 11;
      for (int i = tid; i < kBins; i += NT) s_hist[i] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += NT) {
        const uint32_t key = weight_key(__uint_as_float(s_weight[i]));
        if (shift == 21 || (key >> (shift + bits)) == (prefix >> (shift + bits)))
          atomicAdd(&s_hist[(key >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // thread t holds the bins from the top: kBins - 1 - t * each and below
      constexpr int kEach = kBins / NT;
      unsigned mine = 0, total;
#pragma unroll
      for (int j = 0; j < kEach; ++j) mine += s_hist[kBins - 1 - tid * kEach - j];
      unsigned before = block_exclusive<NT>(mine, s_part, total);
      if (before < static_cast<unsigned>(need) && before + mine >= static_cast<unsigned>(need)) {
        int j = 0;
        unsigned c;
        while (before + (c = s_hist[kBins - 1 - tid * kEach - j]) < static_cast<unsigned>(need)) {
          before += c;
          ++j;
        }
        s_digit = kBins - 1 - tid * kEach - j;
        s_need = need - static_cast<int>(before);
      }
      __syncthreads();
      prefix |= s_digit << shift;
      need = s_need;
    }
    threshold = prefix;
    ties = need;  // entries equal to the threshold that stay, the earliest ones
    __syncthreads();
  }

  for (int w = warp; w < words; w += NT / 32) {
    const int i = w * 32 + lane;
    bool above = false, equal = false;
    if (i < n) {
      above = !evicts || i < lo || i >= hi;
      if (!above) {
        const uint32_t key = weight_key(__uint_as_float(s_weight[i]));
        above = key > threshold;
        equal = key == threshold;
      }
    }
    const unsigned a = __ballot_sync(0xffffffffu, above), e = __ballot_sync(0xffffffffu, equal);
    if (lane == 0) {
      s_above[w] = a;
      s_equal[w] = e;
    }
  }
  __syncthreads();
  // counts (above in the low half, equal in the high one: at most 49152 each) before
  // each mask
  static_assert(kQuantEvictMax < 1 << 16, "two counts in a word");
  unsigned carry = 0;
  for (int w0 = 0; w0 < words; w0 += NT) {
    const int w = w0 + tid;
    const unsigned c = w < words ? __popc(s_above[w]) | __popc(s_equal[w]) << 16 : 0u;
    unsigned total;
    const unsigned x = block_exclusive<NT>(c, s_part, total);
    if (w < words) s_place[w] = carry + x;
    carry += total;
  }
  __syncthreads();

  const int kept_n = evicts ? keep : n;
  // Writes every entry to its place: the weights, the table, or both.
  auto write = [&](bool weights, bool table) {
    const unsigned below = (1u << lane) - 1;
    for (int w = warp; w < words; w += NT / 32) {
      const int i = w * 32 + lane;
      const unsigned a = s_above[w], e = s_equal[w], at = s_place[w];
      const int equal = static_cast<int>(at >> 16) + __popc(e & below);
      const int kept = static_cast<int>(at & 0xffffu) + __popc(a & below) + min(equal, ties);
      const bool stay = (a >> lane & 1) || ((e >> lane & 1) && equal < ties);
      if (weights && stay) w_out[kept] = __uint_as_float(s_weight[i]);  // only live entries stay
      if (table && i < max_groups) t_out[i >= n ? i : stay ? kept : kept_n + (i - kept)] = static_cast<int32_t>(s_table[i]);
    }
  };
  write(true, ROWS == 2);
  // the open group's weight follows the last kept one; entries behind it start at 0;
  // a flagged item is passed through
  for (int i = kept_n + tid; i < max_groups; i += NT)
    w_out[i] = !it.ok ? __uint_as_float(s_weight[i]) : i == kept_n && n < max_groups ? __uint_as_float(s_weight[n]) : 0.f;
  if (ROWS == 1) {
    __syncthreads();
    for (int i = tid; i < max_groups; i += NT) s_table[i] = static_cast<uint32_t>(t_in[i]);
    __syncthreads();
    write(false, true);
  }
  if (tid == 0) evicted_out[item] = gone + (n - kept_n);
}

template <int NT, int ROWS>
cudaError_t launch(const LayerParams& p, const QuantCache& qc, const int64_t* pos, int keep, int sink,
                   int recent, const float* weight_in, float* weight_out, int32_t* table_out,
                   int32_t* evicted_out, unsigned* err, cudaStream_t s) {
  const size_t smem = smem_bytes(qc.max_groups, ROWS);
  cudaError_t e = ensure_smem<quant_evict_kernel<NT, ROWS>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(quant_evict_kernel<NT, ROWS>, dim3(static_cast<unsigned>(p.B * p.Hkv)), dim3(NT),
                    smem, s, 1, p.Hkv, qc, pos, keep, sink, recent, weight_in, weight_out, table_out,
                    evicted_out, err);
}

}  // namespace

cudaError_t launch_quant_evict(const LayerParams& p, const QuantCache& qc, const int64_t* pos,
                               int keep, int sink, int recent, const float* weight_in,
                               float* weight_out, int32_t* table_out, int32_t* evicted_out,
                               unsigned* err, cudaStream_t s) {
  // Rows of 520 entries: 512 threads 6.2 us, 256 take 7.3, 1024 6.3.  Both rows in
  // shared memory while they fit (about 27,000 entries), else one after the other.
  auto* kernel = launch<512, 2>;
  if (qc.max_groups > 1024) kernel = launch<1024, 2>;
  if (smem_bytes(qc.max_groups, 2) > 220 * 1024) kernel = launch<1024, 1>;
  return kernel(p, qc, pos, keep, sink, recent, weight_in, weight_out, table_out, evicted_out, err, s);
}

}  // namespace hga
