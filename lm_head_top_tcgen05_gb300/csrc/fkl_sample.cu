// The sampler of a generation step (fkl_sample): temperature, top-k, top-p, min-p and the
// draw, from given random numbers.
//
// Every sum is one of whole numbers, w_v = floor(2^40 exp(z_v)), so it is exact and does not
// depend on how the row is split.  The logits that a filter keeps are the ones before a
// boundary in the order (logit descending, id ascending), so a row is never sorted: a boundary
// is searched for, and the draw then walks the ids in their own order.
//
// One cluster of 1 to 8 CTAs per row.  Each CTA reads its slice of the row once into shared
// memory, where all further passes run; the CTAs exchange a few sums through distributed
// shared memory.  After the load every CTA knows the row's largest logit m.  Then
//
//   no top-k, no top-p   one pass sums the weights (of what min-p keeps) per warp, and the draw
//                        looks up the id in the one warp's stretch that holds it;
//   top-k up to 512      a list: tau is a lower bound of the k-th largest logit (the least, over the
//                        CTAs, of the k / C-th largest of their threads' maxima), the logits
//                        >= tau, not many more than k, are gathered and the first CTA finishes;
//   otherwise            a histogram over bins of equal width in z (of counts for top-k, of weights
//                        in 17 bits for top-p, beside their exact sum) gives the bin of the
//                        boundary; a second pass sums the exact weights above that bin per
//                        warp and lists the bin's logits, from which the first CTA takes the
//                        boundary.  The rounded histogram only proposes the bin: the exact sums
//                        confirm it.
//
// When the list or the bin holds too many logits (many ties, a temperature so high that a bin is
// most of the row), or the bin is not confirmed, the boundary is found from exact histograms,
// first in z and then of the logits' bits, until what is left fits a list or is all equal.
//
// What bounds it (GB300): a row is 11 to 26 us from its load to its token, in which it is read
// once (2 to 5 us) and passed over once or twice in shared memory (a draw without filters
// executes 36 instructions a logit in all, top-p 0.9 of flat rows 101), with cluster barriers of about
// 1 us between: 3 with a list, 4 without filters, 10 with top-p, up to 18 with a top-k too large for
// a list before it; 36 rows of 201088 fp32 fit the device's shared memory at once.  On the
// device 64 such rows take 29 us without filters, 28 us with top-k 50, 68 us with top-p 0.9; one row
// 11, 12 and 26 us.
#include <atomic>
#include <climits>
#include <cmath>

#include "fkl_generate.cuh"
#include "fkl_types.cuh"

namespace fkl {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxSampleV = int64_t{1} << 22;  // 2^22 weights of 2^40 stay below 2^63
constexpr int kBins = 1024;
constexpr int kListCap = 1024;
// The first histogram, over z: 64 bins to each halving of the weight, 36 halvings.  Smaller weights
// belong to the last bin, which is not kept: a sharp row's logits are mostly there, and adding
// them to one address is slow (512 sharp rows of 32000, top-p 0.9: 69 us with, 62 us without).  A
// boundary in it is left to the exact histograms.
constexpr int kOctaveBits = 6, kOctaves = 36;
constexpr int kZBins = kOctaves << kOctaveBits;
constexpr float kZBinWidth = 0.6931471806f / 64.f;
constexpr int kFineBins = 2048;        // of the second histogram, over one bin of the first
constexpr int kGroups = 32;            // groups of bins that are added up before they are exchanged
constexpr int kFew = 32;
constexpr int kCountingMax = 160;      // longest list that is ranked by counting, not sorted (see kTwoSlice)

using u64 = unsigned long long;

// Order-preserving bits of a logit (-0 and +0 are the same logit) and back.
__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// floor(2^40 e) for 0 <= e <= 1 in two words: hi = floor(2^17 e) and the rest's lo = floor(2^40 rest)
// < 2^23.  Adding 64, whose last place is 2^-17, with rounding down leaves hi in the low bits of
// the sum; the rest e - hi 2^-17 is exact, and adding 2^-17, whose last place is 2^-40, to it
// leaves lo in the same way.
constexpr uint32_t kHiBias = 0x42800000u, kLoBias = 0x37000000u;  // bits of 64 and of 2^-17
__device__ __forceinline__ void split_weight(float e, uint32_t& hi, uint32_t& lo) {  // biased
  const float t = __fadd_rd(e, 64.f);
  const float rest = __fsub_rn(e, __fsub_rn(t, 64.f));
  hi = __float_as_uint(t);
  lo = __float_as_uint(__fadd_rd(rest, 7.62939453125e-6f));
}
__device__ __forceinline__ u64 fixed_point(float e) {
  uint32_t hi, lo;
  split_weight(e, hi, lo);
  return (static_cast<u64>(hi - kHiBias) << 23) + (lo - kLoBias);
}

// Exact sum of up to kMaxAdds weights in two words (the biases are taken off at the end).
struct WeightSum {
  static constexpr int kMaxAdds = 512;
  uint32_t hi = 0, lo = 0, n = 0;
  __device__ __forceinline__ void add(float e) {
    uint32_t h, l;
    split_weight(e, h, l);
    hi += h;
    lo += l;
    ++n;
  }
  __device__ __forceinline__ u64 total() const {
    return (static_cast<u64>(hi - n * kHiBias) << 23) + (lo - n * kLoBias);
  }
};

// The row's largest logit and its scale.  kPlain: m and 1/T are ordinary numbers, so (x - m) / T
// needs no special cases.
template <bool kPlain>
struct RowScale {
  float m, inv_t;
  __device__ __forceinline__ float z(float x) const {  // the product is rounded by itself
    if (kPlain) return __fmul_rn(x - m, inv_t);
    return x == m ? 0.f : __fmul_rn(x - m, inv_t);
  }
  // exp(z); 0 for -inf (and where infinities leave no number)
  __device__ __forceinline__ float e(float x) const {
    const float v = expf(z(x));
    if (kPlain) return v;
    return x > -INFINITY && v > 0.f ? v : 0.f;
  }
  __device__ __forceinline__ u64 weight(float x) const { return fixed_point(e(x)); }
  // Bin of the first histogram as a float 2^23 + bin; falls as x rises.
  __device__ __forceinline__ float z_bin_of(float z) const {
    const float u = __fmaf_rd(z, -1.f / kZBinWidth, 8388608.f);  // rounded down to a whole number
    return fminf(u, 8388608.f + static_cast<float>(kZBins - 1));
  }
  __device__ __forceinline__ float z_bin(float x) const { return z_bin_of(z(x)); }
  // Bin of the second histogram, within `bin` of the first; depends on z alone too.  Its loops must all
  // get the same bin, as one counts the entries that another writes, so each rounding is spelled
  // out: contracted or not, the plain expression gives other bins for one logit in some hundreds.
  __device__ __forceinline__ int fine_bin(float x, int bin) const {
    const float u = __fmul_rn(__fmaf_rn(static_cast<float>(bin), kZBinWidth, z(x)), -static_cast<float>(kFineBins) / kZBinWidth);
    return static_cast<int>(fminf(fmaxf(u, 0.f), static_cast<float>(kFineBins - 1)));
  }
};
__device__ __forceinline__ int bin_number(float z_bin) { return static_cast<int>(__float_as_uint(z_bin) - 0x4b000000u); }

// A boundary in the order (logit descending, id ascending): the last logit that is kept, with its
// id.  -0 and +0 compare equal, as in the order.
struct Boundary {
  float x;
  int id;
  __device__ __forceinline__ bool keeps(float v, int i) const { return v > x || (v == x && i <= id); }
};
__device__ __forceinline__ Boundary no_boundary() { return Boundary{-INFINITY, INT_MAX}; }

// Weights (41 bits) are added to the exact histograms in pieces, each into 32 bits: 3 of 14 bits
// for a slice in shared memory (at most 2^17 logits), 4 of 12 bits for longer ones (at most 2^19).
template <bool kResident>
struct Pieces {
  static constexpr int kCount = kResident ? 3 : 4, kBits = kResident ? 14 : 12;
  static constexpr int kMaxSlice = 1 << (32 - 1 - kBits);
};
static_assert(Pieces<false>::kMaxSlice * kMaxCluster >= kMaxSampleV, "a piece sum stays below 2^31");

template <bool kResident>
struct SampleShared {
  union {
    struct {
      union {
        uint32_t fine[kFineBins];
        u64 list[kListCap];  // the first CTA's list of the whole row: (key, ~id)
      };
      uint32_t near_ids[kListCap];  // this CTA's gathered ids
    };
    uint32_t zhist[kZBins];
    uint32_t hist[Pieces<kResident>::kCount][kBins];  // exact histograms
  } work;
  u64 warp_sum[kSampleWarps];
  u64 groups[kGroups];  // exchanged: this CTA's sums of each group of bins
  u64 kept_sum[kSampleWarps];  // weight that the draw can reach, per warp's stretch of the row
  // exchanged between the CTAs of the cluster (written before a cluster barrier, read after)
  u64 part[4];
  uint32_t count, key_lo, key_hi;
  float cta_max, tau;
  Boundary bound;
  int found;
  // this CTA only
  float warp_max[kSampleWarps];
  uint32_t warp_lo[kSampleWarps], warp_hi[kSampleWarps];
  uint32_t list_count, lo, hi;
  int bin;
  u64 before, want, draw;
  u64 group_sum[kGroups];
  u64 few[kFew], few_weights[kFew];
};

// Barrier of the cluster's threads: shared memory written before it is seen by every CTA after.
__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  cluster_sync();
}

// The barrier's two halves.
__device__ __forceinline__ void arrive_cluster() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_cluster() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same shared-memory object in CTA `rank` of the cluster.
template <class P>
__device__ __forceinline__ P* peer(P* p, int rank) {
  u64 a;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<u64>(p)), "r"(rank));
  return reinterpret_cast<P*>(a);
}
__device__ __forceinline__ int cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return static_cast<int>(n);
}

__device__ __forceinline__ u64 warp_add(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_prefix(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Inclusive prefix sum over the block's threads, and the total.
__device__ u64 block_prefix(u64 v, u64* warp_sum, u64& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_prefix(v, lane);
  __syncthreads();
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  const u64 sums = warp_prefix(lane < kSampleWarps ? warp_sum[lane] : 0ull, lane);
  total = __shfl_sync(0xffffffffu, sums, 31);
  const u64 before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0ull) + v;
}

// Sorts the first n (a power of two, at most 2 * kSampleThreads) keys in descending order with
// a bitonic network.  Steps of distance up to 32 stay within a warp's 64 keys.
__device__ void sort_descending(u64* keys, int n) {
  int last = 64;
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (j >= 64 || last >= 64)
        __syncthreads();
      else
        __syncwarp();
      last = j;
      const int q = threadIdx.x;
      if (q < n / 2) {
        const int i = 2 * q - (q & (j - 1));
        const u64 a = keys[i], b = keys[i + j];
        if ((a < b) == ((i & k) == 0)) {
          keys[i] = b;
          keys[i + j] = a;
        }
      }
    }
  }
  __syncthreads();
}

// The largest of a vector's logits, or NaN if one is NaN.
template <class T>
__device__ __forceinline__ float vector_max(const uint4& raw);
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <>
__device__ __forceinline__ float vector_max<float>(const uint4& raw) {
  const float w = __uint_as_float(raw.w);
  return max3_nan(max3_nan(__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z)), w, w);
}
template <>
__device__ __forceinline__ float vector_max<__nv_bfloat16>(const uint4& raw) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return __bfloat162float(__hmax_nan(m.x, m.y));
}
template <>
__device__ __forceinline__ float vector_max<__half>(const uint4& raw) {
  const __half2* h = reinterpret_cast<const __half2*>(&raw);
  const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}

// One CTA's slice of a row: ids [first, first + n), as 16-byte vectors of E logits.  Vectors are
// aligned in global memory, so the first and the last may be partial; the rest of them reads
// -inf, and so does NaN.  kResident: the vectors are held in shared memory.
template <class T, bool kResident>
struct Slice {
  static constexpr int E = 16 / sizeof(T);
  const T* g;
  uint4* s;
  int first, n, shift, nvec;
  int v0, v1;  // this warp's vectors (contiguous, so that warps are in the order of ids)

  __device__ __forceinline__ int id(int i, int j) const { return first + i * E + j - shift; }

  __device__ __forceinline__ bool inside(int i) const { return i * E >= shift && i * E - shift + E <= n; }
  // A vector at the slice's end, with -inf outside.
  __device__ __forceinline__ uint4 edge(int i) const {
    uint4 raw;
    T* e = reinterpret_cast<T*>(&raw);
    const int at = i * E - shift;
#pragma unroll
    for (int j = 0; j < E; ++j) e[j] = at + j >= 0 && at + j < n ? g[at + j] : from_float<T>(-INFINITY);
    return raw;
  }
  // The largest logit of a vector, in which NaN becomes -inf.  NaN is rare, so it is looked for in
  // the maximum, which it passes through.
  static __device__ __forceinline__ float settle(uint4& raw, bool& changed) {
    float most = vector_max<T>(raw);
    changed = most != most;
    if (changed) {
      float v[E];
      unpack16<T>(raw, v);
      T* e = reinterpret_cast<T*>(&raw);
      most = -INFINITY;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        v[j] = v[j] == v[j] ? v[j] : -INFINITY;
        most = fmaxf(most, v[j]);
        e[j] = from_float<T>(v[j]);
      }
    }
    return most;
  }
  // This thread's vectors (v0 + lane, every 32nd) into shared memory, and their largest logit.  All
  // of the copies are in flight at once: an SM then has 200 KB under way, which HBM's latency needs.
  __device__ __forceinline__ float load(int lane) const {
    float most = -INFINITY;
    bool changed;
    if constexpr (kResident) {
      for (int i = v0 + lane; i < v1; i += 32) {
        if (inside(i))
          copy16_async(s + i, g + (i * E - shift));
        else
          s[i] = edge(i);
      }
      copy_async_wait();
      for (int i = v0 + lane; i < v1; i += 32) {
        uint4 raw = s[i];
        most = fmaxf(most, settle(raw, changed));
        if (changed) s[i] = raw;
      }
    } else {
      for (int i = v0 + lane; i < v1; i += 32) {
        uint4 raw = inside(i) ? __ldg(reinterpret_cast<const uint4*>(g + (i * E - shift))) : edge(i);
        most = fmaxf(most, settle(raw, changed));
      }
    }
    return most;
  }
  __device__ __forceinline__ void get(int i, float (&v)[E]) const {
    unpack16<T>(raw(i), v);
  }
  __device__ __forceinline__ uint4 raw(int i) const {
    if (kResident) return s[i];
    uint4 v = inside(i) ? __ldg(reinterpret_cast<const uint4*>(g + (i * E - shift))) : edge(i);
    bool changed;
    settle(v, changed);
    return v;
  }
  // f(logit, id) for every element of this warp's vectors.
  template <class F>
  __device__ __forceinline__ void each(int lane, F f) const {
    for (int i = v0 + lane; i < v1; i += 32) {
      float v[E];
      get(i, v);
#pragma unroll
      for (int j = 0; j < E; ++j) f(v[j], id(i, j));
    }
  }
};

// u * W rounded down, within [0, W - 1]; NaN and negative numbers give 0.
__device__ __forceinline__ u64 draw_at(float u, u64 total) {
  const double rd = static_cast<double>(u) * static_cast<double>(total);
  if (!(rd >= 1.0)) return 0;
  return rd < static_cast<double>(total) ? min(static_cast<u64>(rd), total - 1) : total - 1;
}
// Weight that top-p keeps at least (at least the largest logit's); NaN and p <= 0 give 1.
__device__ __forceinline__ u64 top_p_weight(float p, u64 total) {
  const double lim = ceil(static_cast<double>(p) * static_cast<double>(total));
  return lim >= 1.0 ? static_cast<u64>(lim) : 1ull;
}
__device__ __forceinline__ float log_probability(float z, u64 total) {
  return z - logf(static_cast<float>(total) * 9.094947017729282e-13f);  // 2^-40
}

// State of one row, shared by the steps.
template <class T, bool kResident, bool kPlain>
struct RowCtx {
  static constexpr int E = Slice<T, kResident>::E;
  const Slice<T, kResident>& slice;
  SampleShared<kResident>& s;
  u64* counting;  // room for kCountingMax weights
  RowScale<kPlain> rs;
  int rank, ranks, warp, lane;

  // Sum of v over the block's threads, into s.part[slot] (visible to the cluster after its
  // next barrier); the warps' sums stay in `warps`.
  __device__ __forceinline__ void sum_to_part(u64 v, int slot, u64* warps) {
    v = warp_add(v);
    __syncthreads();
    if (lane == 0) warps[warp] = v;
    __syncthreads();
    if (warp == 0) add_warps(warps, slot);
  }
  // One warp: the sum of the warps' sums into s.part[slot].
  __device__ __forceinline__ void add_warps(const u64* warps, int slot) {
    const u64 t = warp_add(lane < kSampleWarps ? warps[lane] : 0ull);
    if (lane == 0) s.part[slot] = t;
  }
  // Sum of part[slot] over the cluster, and over the CTAs before this one.  Lane r of each warp
  // reads CTA r's, so that it takes one trip to their shared memory.
  __device__ __forceinline__ u64 total_of(int slot, u64* before = nullptr) {
    const u64 v = lane < ranks ? peer(&s, lane)->part[slot] : 0ull;
    const u64 run = warp_prefix(v, lane);
    if (before != nullptr) *before = __shfl_sync(0xffffffffu, run - v, rank);
    return __shfl_sync(0xffffffffu, run, 31);
  }
  __device__ __forceinline__ uint32_t total_count(uint32_t* before = nullptr) {
    const uint32_t v = lane < ranks ? peer(&s, lane)->count : 0u;
    if (before != nullptr) *before = __reduce_add_sync(0xffffffffu, lane < rank ? v : 0u);
    return __reduce_add_sync(0xffffffffu, v);
  }
  // A value that one thread computes in double (those units are few), for the block.
  template <class F>
  __device__ __forceinline__ u64 by_one_thread(u64& slot, F f) {
    if (threadIdx.x == 0) slot = f();
    __syncthreads();
    return slot;
  }

  // Exact sum of the weights f adds (f(x, id, sum)) over this thread's logits.
  template <class F>
  __device__ __forceinline__ u64 sum_weights(F f) {
    WeightSum sum;
    u64 total = 0;
    for (int i = slice.v0 + lane; i < slice.v1; i += 32) {
      float v[E];
      slice.get(i, v);
#pragma unroll
      for (int j = 0; j < E; ++j) f(v[j], slice.id(i, j), sum);
      if (!kResident && sum.n > WeightSum::kMaxAdds - E) {  // a resident slice has at most 256 a thread
        total += sum.total();
        sum = WeightSum();
      }
    }
    return total + sum.total();
  }

  // The same of every weight, two logits at a time where that is one instruction.
  __device__ __forceinline__ u64 sum_all() {
    if constexpr (!kPlain || !kResident) {
      return sum_weights([&](float x, int, WeightSum& w) { w.add(rs.e(x)); });
    } else {
      WeightSum sum;
      const float2 om = make_float2(-rs.m, -rs.m), it = make_float2(rs.inv_t, rs.inv_t);
      for (int i = slice.v0 + lane; i < slice.v1; i += 32) {
        float v[E];
        slice.get(i, v);
#pragma unroll
        for (int j = 0; j < E; j += 2) {
          const float2 z = fmul2(fadd2(make_float2(v[j], v[j + 1]), om), it);
          sum.add(expf(z.x));
          sum.add(expf(z.y));
        }
      }
      return sum.total();
    }
  }

  // Resets this CTA's list.
  __device__ __forceinline__ void clear_list() {
    __syncthreads();
    if (threadIdx.x == 0) s.list_count = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void append(int id) {
    const uint32_t at = atomicAdd(&s.list_count, 1u);
    if (at < kListCap) s.work.near_ids[at] = static_cast<uint32_t>(id);
  }
  __device__ __forceinline__ float logit(int id) const {
    if (kResident) {
      const int at = id - slice.first + slice.shift;
      return to_float(reinterpret_cast<const T*>(slice.s)[at]);
    }
    const float x = to_float(slice.g[id - slice.first]);
    return x == x ? x : -INFINITY;
  }
  __device__ __forceinline__ u64 entry(int id, float x) const {
    return (static_cast<u64>(logit_key(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
  }
  static __device__ __forceinline__ float entry_logit(u64 e) { return key_logit(static_cast<uint32_t>(e >> 32)); }
  static __device__ __forceinline__ int entry_id(u64 e) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)); }
  // Brings the CTAs' lists together in the first CTA, in the order of the CTAs.  Between two
  // cluster barriers; s.count is this CTA's number.
  __device__ __forceinline__ void push_list() {
    uint32_t at;
    total_count(&at);
    u64* to = rank == 0 ? &s.work.list[0] : peer(&s.work.list[0], 0);
    for (uint32_t i = threadIdx.x; i < s.count; i += kSampleThreads) {
      const int id = static_cast<int>(s.work.near_ids[i]);
      to[at + i] = entry(id, logit(id));
    }
  }
  // First CTA: pads the list's n entries to a power of two and sorts them.
  __device__ __forceinline__ void sort_list(u64* keys, int n) {
    int n2 = 1;
    while (n2 < n) n2 <<= 1;
    for (int i = n + threadIdx.x; i < n2; i += kSampleThreads) keys[i] = 0;
    sort_descending(keys, n2);
  }
  // First CTA: in the list of n entries, the one at which the running sum of amounts (1, or the
  // weights), in their order, reaches want, into s.bound; s.found tells whether there is one.
  __device__ __forceinline__ void bound_in_list(int n, bool by_mass, u64 want, u64* weights) {
    if (threadIdx.x == 0) s.found = 0;
    u64* list = s.work.list;
    auto found = [&](u64 c) {
      s.bound = Boundary{entry_logit(c), entry_id(c)};
      s.found = 1;
    };
    if (n <= kCountingMax) {
      for (int i = threadIdx.x; i < n; i += kSampleThreads) weights[i] = by_mass ? rs.weight(entry_logit(list[i])) : 1ull;
      __syncthreads();
      const int part = threadIdx.x % kShare;
      for (int i0 = 0; i0 < n; i0 += kSampleThreads / kShare) {
        const int i = i0 + static_cast<int>(threadIdx.x) / kShare;
        const u64 e = i < n ? list[i] : ~0ull;
        int rank_of;
        const u64 start = ahead_of(e, n, part, weights, rank_of);
        if (part == 0 && i < n && start < want && want <= start + weights[i]) found(e);
      }
      return;
    }
    // Longer: exact sums of 128 bins of the keys' range, then the bin's few entries by counting.
    constexpr int kKeyBins = 128;
    static_assert(kKeyBins <= kCountingMax && kListCap <= 2 * kSampleThreads, "the bins fit, two entries a thread");
    u64 mine[2] = {0, 0}, amount[2] = {0, 0};
    uint32_t klo = 0xffffffffu, khi = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = static_cast<int>(threadIdx.x) + j * kSampleThreads;
      if (i >= n) break;
      mine[j] = list[i];
      amount[j] = by_mass ? rs.weight(entry_logit(mine[j])) : 1ull;
      klo = min(klo, static_cast<uint32_t>(mine[j] >> 32));
      khi = max(khi, static_cast<uint32_t>(mine[j] >> 32));
    }
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    if (lane == 0) {
      s.warp_lo[warp] = klo;
      s.warp_hi[warp] = khi;
    }
    if (threadIdx.x < kKeyBins) weights[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
      s.bin = -1;
      s.list_count = 0;
    }
    __syncthreads();
    klo = __reduce_min_sync(0xffffffffu, s.warp_lo[lane % kSampleWarps]);
    khi = __reduce_max_sync(0xffffffffu, s.warp_hi[lane % kSampleWarps]);
    const int bits = 32 - __clz(khi - klo), shift = bits > 7 ? bits - 7 : 0;
    auto key_bin = [&](u64 e) { return static_cast<int>((khi - static_cast<uint32_t>(e >> 32)) >> shift); };
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (amount[j] != 0) atomicAdd(&weights[key_bin(mine[j])], amount[j]);
    __syncthreads();
    if (warp == 0) {
      u64 a[kKeyBins / 32], sum = 0;
#pragma unroll
      for (int j = 0; j < kKeyBins / 32; ++j) sum += a[j] = weights[kKeyBins / 32 * lane + j];
      u64 c = warp_prefix(sum, lane) - sum;
#pragma unroll
      for (int j = 0; j < kKeyBins / 32; ++j) {
        if (c < want && want <= c + a[j]) {
          s.bin = kKeyBins / 32 * lane + j;
          s.before = c;
        }
        c += a[j];
      }
    }
    __syncthreads();
    if (s.bin < 0) return;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (amount[j] != 0 && key_bin(mine[j]) == s.bin) {
        const uint32_t at = atomicAdd(&s.list_count, 1u);
        if (at < kFew) {
          s.few[at] = mine[j];
          s.few_weights[at] = amount[j];
        }
      }
    __syncthreads();
    const int m = static_cast<int>(s.list_count);
    if (m <= kFew) {
      if (static_cast<int>(threadIdx.x) < m) {
        const u64 e = s.few[threadIdx.x];
        u64 start = s.before;
        for (int j = 0; j < m; ++j)
          if (s.few[j] > e) start += s.few_weights[j];
        if (start < want && want <= start + s.few_weights[threadIdx.x]) found(e);
      }
      return;
    }
    sort_list(list, n);
    const int i0 = 2 * static_cast<int>(threadIdx.x);
    u64 w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) w[j] = i0 + j < n ? (by_mass ? rs.weight(entry_logit(list[i0 + j])) : 1ull) : 0ull;
    u64 total;
    const u64 upto = block_prefix(w[0] + w[1], s.warp_sum, total);
    const u64 start = upto - w[0] - w[1];
    if (start < want && want <= upto) found(list[i0 + (start + w[0] < want ? 1 : 0)]);
  }
  // Entries of the list (of n) ranked before e: their number and their weights' sum, counted by a
  // team of kShare lanes, each its share.
  static constexpr int kShare = 4;
  __device__ __forceinline__ u64 ahead_of(u64 e, int n, int part, const u64* weights, int& rank_of) {
    u64 mass = 0;
    rank_of = 0;
#pragma unroll 4
    for (int j = part; j < n; j += kShare) {
      const u64 c = s.work.list[j], w = weights[j];
      if (c > e) {
        ++rank_of;
        mass += w;
      }
    }
#pragma unroll
    for (int o = 1; o < kShare; o <<= 1) {
      rank_of += __shfl_xor_sync(0xffffffffu, rank_of, o);
      mass += __shfl_xor_sync(0xffffffffu, mass, o);
    }
    return mass;
  }

  // The bin of the CTAs' histograms together (read(other, bin) gives a bin's amount in one) at which
  // the running sum reaches `want`, and the sum before it; -1 if the sum stays below want.  want_of
  // gives want; one warp calls it, after the cluster barrier in here.  Called
  // when the block's histogram is complete; the histograms may be overwritten after the next
  // cluster barrier.  Each CTA adds its bins up in 32 groups; the group is found from
  // everyone's sums, and only its bins are read from the other CTAs.
  template <class W, class F>
  __device__ int find_in_bins(int bins, W want_of, u64& want, u64& before, F read) {
    const int per = bins / kGroups;
    __syncthreads();
    {
      constexpr int kTeam = kSampleThreads / kGroups;  // 16 threads per group
      const int g = static_cast<int>(threadIdx.x) / kTeam, at = static_cast<int>(threadIdx.x) % kTeam;
      u64 t = 0;
      for (int i = at; i < per; i += kTeam) t += read(&s, g * per + i);
#pragma unroll
      for (int o = kTeam / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (at == 0) s.groups[g] = t;
    }
    sync_cluster();
    if (threadIdx.x < kGroups * kMaxCluster) {
      const int g = static_cast<int>(threadIdx.x) / kMaxCluster, r = static_cast<int>(threadIdx.x) % kMaxCluster;
      u64 t = r < ranks ? peer(&s, r)->groups[g] : 0ull;
#pragma unroll
      for (int o = kMaxCluster / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (r == 0) s.group_sum[g] = t;
    }
    if (warp == kSampleWarps - 1) {
      const u64 w = want_of();
      if (lane == 0) s.want = w;
    }
    __syncthreads();
    want = s.want;
    const u64 mine = s.group_sum[lane];
    const u64 upto = warp_prefix(mine, lane);
    const int group = __ffs(__ballot_sync(0xffffffffu, upto >= want)) - 1;
    if (group < 0) return -1;
    const u64 run = __shfl_sync(0xffffffffu, upto - mine, group);
    static_assert(kZBins / kGroups <= kSampleThreads && kFineBins <= kZBins && kBins <= kZBins, "a thread per bin of a group");
    u64 v = 0;
    if (static_cast<int>(threadIdx.x) < per) {
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < ranks) v += read(peer(&s, r), group * per + static_cast<int>(threadIdx.x));
    }
    u64 total;
    const u64 c = run + block_prefix(v, s.warp_sum, total);
    if (c - v < want && want <= c) {
      s.bin = group * per + static_cast<int>(threadIdx.x);
      s.before = c - v;
    }
    __syncthreads();
    before = s.before;
    return s.bin;
  }

  // Exact histogram over the cluster of f's amounts (f(x, v, bin, amount) gives whether the logit
  // counts, its bin and its amount).
  template <class F>
  __device__ int find_bin(u64 want, u64& before, F f) {
    using P = Pieces<kResident>;
    __syncthreads();
    for (int i = threadIdx.x; i < P::kCount * kBins; i += kSampleThreads) s.work.hist[0][i] = 0;
    __syncthreads();
    slice.each(lane, [&](float x, int v) {
      uint32_t bin;
      u64 amount;
      if (f(x, v, bin, amount)) {
#pragma unroll
        for (int q = 0; q < P::kCount; ++q) {
          const uint32_t part = static_cast<uint32_t>(amount >> (q * P::kBits)) & ((1u << P::kBits) - 1);
          if (part) atomicAdd(&s.work.hist[q][bin], part);
        }
      }
    });
    const int bin = find_in_bins(kBins, [want] { return want; }, want, before, [](const SampleShared<kResident>* o, int i) {
      u64 t = 0;
#pragma unroll
      for (int q = 0; q < P::kCount; ++q) t += static_cast<u64>(o->work.hist[q][i]) << (q * P::kBits);
      return t;
    });
    sync_cluster();
    return bin;
  }

  // The id at which the running sum of f (over the ids, after `before` in the CTAs before) exceeds r,
  // when it lies in this CTA, in every lane of one warp; -1 elsewhere.  kept_sum holds f's sums per
  // warp's stretch.  The block's warps share the stretch that holds the id.
  template <class F>
  __device__ int locate(u64 before, u64 r, F f) {
    const u64 stretch = lane < kSampleWarps ? s.kept_sum[lane] : 0ull;
    const u64 upto = before + warp_prefix(stretch, lane);
    const int owner = before <= r ? __ffs(__ballot_sync(0xffffffffu, upto > r)) - 1 : -1;
    if (owner < 0) return -1;  // the same in the whole block
    before = __shfl_sync(0xffffffffu, upto - stretch, owner);
    const int per = (slice.nvec + kSampleWarps - 1) / kSampleWarps;
    const int w0 = min(slice.nvec, owner * per), w1 = min(slice.nvec, w0 + per);
    const int sub = (w1 - w0 + kSampleWarps - 1) / kSampleWarps;
    const int b = min(w1, w0 + warp * sub), e = min(w1, b + sub);
    u64 sum = 0;
    for (int i = b + lane; i < e; i += 32) {
      float v[E];
      slice.get(i, v);
#pragma unroll
      for (int j = 0; j < E; ++j) sum += f(v[j], slice.id(i, j));
    }
    sum = warp_add(sum);
    if (lane == 0) s.warp_sum[warp] = sum;
    __syncthreads();
    before += warp_add(lane < warp ? s.warp_sum[lane] : 0ull);
    if (!(before <= r && r < before + sum)) return -1;
    for (int i0 = b; i0 < e; i0 += 32) {
      const int i = i0 + lane;
      u64 a[E], mine = 0;
#pragma unroll
      for (int j = 0; j < E; ++j) a[j] = 0;
      if (i < e) {
        float v[E];
        slice.get(i, v);
#pragma unroll
        for (int j = 0; j < E; ++j) mine += a[j] = f(v[j], slice.id(i, j));
      }
      const u64 run = before + warp_prefix(mine, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, run > r);
      if (hit) {
        const int src = __ffs(hit) - 1;
        u64 c = run - mine;
        int id = -1;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          c += a[j];
          if (id < 0 && c > r) id = slice.id(i, j);
        }
        return __shfl_sync(0xffffffffu, id, src);
      }
      before = __shfl_sync(0xffffffffu, run, 31);
    }
    return -1;
  }

  // What min-p keeps of a logit above the boundaries.
  __device__ __forceinline__ bool min_p_keeps(float x, float e, float min_p) const { return x == rs.m || e >= min_p; }

  // The boundary of top-k (want logits) or top-p (a weight of want(total), by_mass), from the
  // histogram in z and the exact sums above its bin.  Leaves the weights that the draw can reach in
  // kept_sum, and their total without min-p in `kept`.  False, for the whole cluster: the bin
  // holds too many logits or is not the right one.
  __device__ bool z_boundary(const Boundary& keeps, bool by_mass, u64 count, float top_p, float min_p, Boundary& bound,
                             u64& kept) {
    const bool cut = keeps.x > -INFINITY;
    for (int i = threadIdx.x; i < kZBins; i += kSampleThreads) s.work.zhist[i] = 0;
    __syncthreads();
    if (by_mass) {
      auto count_in = [&](float z, float e, WeightSum& w) {
        w.add(e);
        // The weight relative to its octave, in 17 bits (its mantissa's; 1 counts as the number below
        // it, which has the octave's exponent), so that 2^15 add up in 32 bits; a longer slice's
        // bins wrap at worst, and the exact sums then refuse the bin.
        const uint32_t amount = ((((__float_as_uint(e) - 1u) & 0x7fffffu) | 0x800000u) + 64u) >> 7;
        const int b = bin_number(rs.z_bin_of(z));
        if (b < kZBins - 1) atomicAdd(&s.work.zhist[b], amount);
      };
      u64 sum;
      if (kPlain && kResident && !cut) {  // two logits at a time where that is one instruction
        WeightSum w;
        const float2 om = make_float2(-rs.m, -rs.m), it = make_float2(rs.inv_t, rs.inv_t);
        for (int i = slice.v0 + lane; i < slice.v1; i += 32) {
          float v[E];
          slice.get(i, v);
#pragma unroll
          for (int j = 0; j < E; j += 2) {
            const float2 z = fmul2(fadd2(make_float2(v[j], v[j + 1]), om), it);
            count_in(z.x, expf(z.x), w);
            count_in(z.y, expf(z.y), w);
          }
        }
        sum = w.total();
      } else {
        sum = sum_weights([&](float x, int v, WeightSum& w) {
          if (cut && !keeps.keeps(x, v)) return;
          count_in(rs.z(x), rs.e(x), w);
        });
      }
      sum_to_part(sum, 1, s.warp_sum);
    } else {
      slice.each(lane, [&](float x, int) {
        const int b = bin_number(rs.z_bin(x));
        if (b < kZBins - 1) atomicAdd(&s.work.zhist[b], 1u);
      });
    }
    u64 want, before = 0;
    auto want_of = [&] { return by_mass ? top_p_weight(top_p, total_of(1)) : count; };
    const int bin = find_in_bins(kZBins, want_of, want, before, [by_mass](const SampleShared<kResident>* o, int i) -> u64 {
      const u64 v = o->work.zhist[i];
      const int shift = 23 - (i >> kOctaveBits);  // to units of 2^-40
      return !by_mass ? v : shift >= 0 ? v << shift : v >> -shift;
    });
    sync_cluster();  // the lists overwrite the histograms
    if (bin < 0) return false;
    // the weights above the bin, and the bin's logits
    clear_list();
    const float edge = 8388608.f + static_cast<float>(bin);
    const bool filter = !(min_p <= 0.f);
    WeightSum open;
    u64 all = 0;
    u64 reach;
    if (kPlain && kResident && !cut && !filter) {  // two logits at a time where that is one instruction
      WeightSum w;
      const float2 om = make_float2(-rs.m, -rs.m), it = make_float2(rs.inv_t, rs.inv_t);
      // A logit below `low` is in a later bin (one bin to spare for the roundings), and a vector of
      // them is passed over.  Top-p 0.9 of 512 rows of 201088 bf16, without and with: sharp rows 272,
      // 225 us, flat rows, which keep most of theirs, 523, 526 us; one flat row of fp32 29, 31 us.
      // Top-k comes here for so many logits that most warps have some: looking first cost 3 % there.
      const float low = __fsub_rd(rs.m, static_cast<float>(bin + 2) * kZBinWidth / rs.inv_t);
      for (int i = slice.v0 + lane; i < slice.v1; i += 32) {
        if (by_mass && !(vector_max<T>(slice.raw(i)) >= low)) continue;
        float v[E];
        slice.get(i, v);
#pragma unroll
        for (int j = 0; j < E; j += 2) {
          const float2 z = fmul2(fadd2(make_float2(v[j], v[j + 1]), om), it);
          const float u0 = rs.z_bin_of(z.x), u1 = rs.z_bin_of(z.y);
          if (u0 < edge) w.add(expf(z.x));
          if (u1 < edge) w.add(expf(z.y));
          if (u0 == edge && v[j] > -INFINITY) append(slice.id(i, j));
          if (u1 == edge && v[j + 1] > -INFINITY) append(slice.id(i, j + 1));
        }
      }
      reach = w.total();
    } else {
      reach = sum_weights([&](float x, int v, WeightSum& w) {
        const float u = rs.z_bin(x);
        if (!(u <= edge)) return;
        if (cut && !keeps.keeps(x, v)) return;
        if (u == edge) {
          if (x > -INFINITY) append(v);
          return;
        }
        const float e = rs.e(x);
        if (filter) {
          open.add(e);
          if (!kResident && open.n >= WeightSum::kMaxAdds) {
            all += open.total();
            open = WeightSum();
          }
          if (!min_p_keeps(x, e, min_p)) return;
        }
        w.add(e);
      });
    }
    all = filter ? all + open.total() : reach;
    sum_to_part(reach, 3, s.kept_sum);
    sum_to_part(all, 2, s.warp_sum);
    if (threadIdx.x == 0) s.count = s.list_count;
    sync_cluster();
    const uint32_t n = total_count();
    const u64 above = total_of(2);
    const bool overfull = __ballot_sync(0xffffffffu, lane < ranks && peer(&s, lane)->count > kListCap) != 0;
    if (overfull || (by_mass && above >= want)) return false;
    u64 rest = want - (by_mass ? above : before);  // what is wanted of the bin
    int fine = -1;                                 // the second histogram's bin, if one was needed
    if (n > kListCap) {
      // too many for the first CTA's list: a second histogram of them alone
      // weights lose the bits that bring the bin's largest below 2^19: 2^13 of them add up in 32 bits
      const int shift = max(0, 41 - (bin >> kOctaveBits) - 19);
      for (int i = threadIdx.x; i < kFineBins; i += kSampleThreads) s.work.fine[i] = 0;
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < s.count; i += kSampleThreads) {
        const float x = logit(static_cast<int>(s.work.near_ids[i]));
        const uint32_t amount = by_mass ? static_cast<uint32_t>(rs.weight(x) >> shift) : 1u;
        atomicAdd(&s.work.fine[rs.fine_bin(x, bin)], amount);
      }
      u64 part_want = 0, ahead = 0;
      fine = find_in_bins(kFineBins, [&] { return by_mass ? max(rest >> shift, 1ull) : rest; }, part_want, ahead,
                          [](const SampleShared<kResident>* o, int i) { return static_cast<u64>(o->work.fine[i]); });
      if (fine < 0) {
        sync_cluster();
        return false;
      }
      u64 sum = 0, number = 0;
      for (uint32_t i = threadIdx.x; i < s.count; i += kSampleThreads) {
        const float x = logit(static_cast<int>(s.work.near_ids[i]));
        const int f = rs.fine_bin(x, bin);
        if (f < fine) sum += by_mass ? rs.weight(x) : 1ull;
        number += f == fine;
      }
      sum_to_part(sum, 2, s.warp_sum);
      sum_to_part(number, 3, s.warp_sum);
      sync_cluster();
      const u64 in_front = total_of(2);
      if (total_of(3) > kListCap || in_front >= rest) return false;
      rest -= in_front;
      u64 at = 0;
      total_of(3, &at);
      clear_list();
      u64* to = rank == 0 ? &s.work.list[0] : peer(&s.work.list[0], 0);
      for (uint32_t i = threadIdx.x; i < s.count; i += kSampleThreads) {
        const int id = static_cast<int>(s.work.near_ids[i]);
        const float x = logit(id);
        if (rs.fine_bin(x, bin) == fine) to[at + atomicAdd(&s.list_count, 1u)] = entry(id, x);
      }
    } else {
      push_list();
    }
    const int listed = fine < 0 ? static_cast<int>(n) : static_cast<int>(total_of(3));
    sync_cluster();
    if (rank == 0) bound_in_list(listed, by_mass, rest, counting);
    sync_cluster();
    if (!peer(&s, 0)->found) return false;
    bound = peer(&s, 0)->bound;
    // the bin's logits that stay join the sums of their stretches
    const int per = (slice.nvec + kSampleWarps - 1) / kSampleWarps;
    u64 more = 0;
    for (uint32_t i = threadIdx.x; i < s.count; i += kSampleThreads) {
      const int id = static_cast<int>(s.work.near_ids[i]);
      const float x = logit(id);
      if (!bound.keeps(x, id)) continue;
      const float e = rs.e(x);
      const u64 w = fixed_point(e);
      more += w;
      if (!filter || min_p_keeps(x, e, min_p))
        atomicAdd(&s.kept_sum[((id - slice.first + slice.shift) / E) / per], w);
    }
    if (!by_mass) {  // the weight that top-p takes its share of
      sum_to_part(more, 1, s.warp_sum);
      sync_cluster();
      kept = above + total_of(1);
    }
    return true;
  }

  // The boundary at which `want` logits (by_mass false) or a weight of `want` (by_mass true)
  // have been kept, among those that `keeps`, from exact histograms; want is at least 1 and at
  // most what there is.  The whole cluster.
  __device__ Boundary find_boundary(const Boundary& keeps, bool by_mass, u64 want) {
    auto amount_of = [&](float x) -> u64 { return by_mass ? rs.weight(x) : 1ull; };
    auto coarse = [&](float x) -> int { return bin_number(rs.z_bin(x)) * kBins / kZBins; };
    u64 before = 0;
    int bin = find_bin(want, before, [&](float x, int v, uint32_t& b, u64& amount) -> bool {
      if (!(x > -INFINITY) || !keeps.keeps(x, v)) return false;
      b = static_cast<uint32_t>(coarse(x));
      amount = amount_of(x);
      return true;
    });
    want -= before;
    gather_exact([&](float x, int v) { return x > -INFINITY && coarse(x) == bin && keeps.keeps(x, v); });
    for (;;) {
      sync_cluster();
      const uint32_t n = total_count();
      const uint32_t lo = __reduce_min_sync(0xffffffffu, lane < ranks ? peer(&s, lane)->key_lo : 0xffffffffu);
      const uint32_t hi = __reduce_max_sync(0xffffffffu, lane < ranks ? peer(&s, lane)->key_hi : 0u);
      if (n <= kListCap) {
        push_list();
        sync_cluster();
        if (rank == 0) bound_in_list(static_cast<int>(n), by_mass, want, counting);
        break;
      }
      if (lo == hi) {  // more equal logits than the list holds: the ids decide
        const float x0 = key_logit(lo);
        const u64 each = by_mass ? rs.weight(x0) : 1ull;
        const u64 skip = (want - 1) / each;  // equal logits kept before the last one
        auto tie = [&](float x, int v) -> u64 { return x == x0 && keeps.keeps(x, v) ? 1ull : 0ull; };
        u64 sum = 0, ahead = 0;
        slice.each(lane, [&](float x, int v) { sum += tie(x, v); });
        sum_to_part(sum, 0, s.kept_sum);
        sync_cluster();
        total_of(0, &ahead);
        const int id = locate(ahead, skip, tie);
        if (id >= 0 && lane == 0) peer(&s, 0)->bound = Boundary{x0, id};
        break;
      }
      const int bits = 32 - __clz(hi - lo);
      const int shift = bits > 10 ? bits - 10 : 0;
      static_assert(kBins == 1 << 10, "bins of the logits' bits");
      bin = find_bin(want, before, [&](float x, int v, uint32_t& b, u64& amount) -> bool {
        const uint32_t k = logit_key(x);
        if (k < lo || k > hi || !keeps.keeps(x, v)) return false;
        b = (hi - k) >> shift;
        amount = amount_of(x);
        return true;
      });
      want -= before;
      gather_exact([&](float x, int v) {
        const uint32_t k = logit_key(x);
        return k >= lo && k <= hi && static_cast<int>((hi - k) >> shift) == bin && keeps.keeps(x, v);
      });
    }
    sync_cluster();
    return peer(&s, 0)->bound;
  }

  // Lists the logits for which f holds; their number and the range of their keys go to s.count,
  // s.key_lo and s.key_hi.
  template <class F>
  __device__ void gather_exact(F f) {
    clear_list();
    if (threadIdx.x == 0) {
      s.lo = 0xffffffffu;
      s.hi = 0u;
    }
    __syncthreads();
    uint32_t lo = 0xffffffffu, hi = 0u;
    slice.each(lane, [&](float x, int v) {
      if (f(x, v)) {
        const uint32_t k = logit_key(x);
        lo = min(lo, k);
        hi = max(hi, k);
        append(v);
      }
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0 && lo <= hi) {
      atomicMin(&s.lo, lo);
      atomicMax(&s.hi, hi);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      s.count = s.list_count;
      s.key_lo = s.lo;
      s.key_hi = s.hi;
    }
  }

  // The first CTA's finish when the list holds everything that can be drawn: the top k, then
  // top-p and min-p among them, then the draw.  weights and by_id: room for kListCap each.
  __device__ void finish_list(int n, int k, bool need_p, float top_p, float min_p, float u, u64* weights, u64* by_id,
                              int32_t* token, float* logprob) {
    u64* list = s.work.list;
    if (n <= kCountingMax) {
      // Short: a thread per pair of an entry and a share of the list counts the entries ranked
      // before it and adds up their weights, then, of those kept, the weights of lower ids.
      for (int i = threadIdx.x; i < n; i += kSampleThreads) weights[i] = rs.weight(entry_logit(list[i]));
      __syncthreads();
      constexpr int kRound = kSampleThreads / kShare;  // entries per round
      static_assert(kCountingMax <= 2 * kRound, "two rounds of entries");
      const int part = threadIdx.x % kShare;
      u64 kept_w[2] = {0, 0}, ahead[2] = {0, 0}, top = 0;
      bool in_top[2] = {false, false};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q * kRound >= n) break;
        const int i = q * kRound + static_cast<int>(threadIdx.x) / kShare;
        int rank_of;
        ahead[q] = ahead_of(i < n ? list[i] : ~0ull, n, part, weights, rank_of);
        in_top[q] = i < n && rank_of < k;
        kept_w[q] = in_top[q] ? weights[i] : 0;
        if (part == 0) top += kept_w[q];
      }
      u64 total;
      block_prefix(top, s.warp_sum, total);
      const u64 want = need_p ? by_one_thread(s.want, [&] { return top_p_weight(top_p, total); }) : 0ull;
      u64 left = 0;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = q * kRound + static_cast<int>(threadIdx.x) / kShare;
        bool keep = in_top[q] && (!need_p || ahead[q] < want);
        if (keep) {
          const float x = entry_logit(list[i]);
          keep = min_p_keeps(x, rs.e(x), min_p);
        }
        if (!keep) kept_w[q] = 0;
        if (i < n && part == 0) by_id[i] = kept_w[q];
        if (part == 0) left += kept_w[q];
      }
      block_prefix(left, s.warp_sum, total);  // by_id is complete after its barriers
      const u64 r = by_one_thread(s.draw, [&] { return draw_at(u, total); });
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q * kRound >= n) break;
        const int i = q * kRound + static_cast<int>(threadIdx.x) / kShare;
        const int id = i < n ? entry_id(list[i]) : 0;
        u64 mass = 0;
#pragma unroll 4
        for (int j = part; j < n; j += kShare) {
          const u64 w = by_id[j];
          if (entry_id(list[j]) < id) mass += w;
        }
#pragma unroll
        for (int o = 1; o < kShare; o <<= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
        if (part == 0 && mass <= r && r < mass + kept_w[q]) {
          *token = id;
          if (logprob != nullptr) *logprob = log_probability(rs.z(entry_logit(list[i])), total);
        }
      }
      return;
    }
    sort_list(list, n);
    const int kk = min(k, n);
    const int i0 = 2 * static_cast<int>(threadIdx.x);
    u64 w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) w[j] = i0 + j < kk ? rs.weight(entry_logit(list[i0 + j])) : 0;
    u64 total;
    u64 upto = block_prefix(w[0] + w[1], s.warp_sum, total);
    if (threadIdx.x == 0) s.bin = kk;
    __syncthreads();
    if (need_p) {
      const u64 want = by_one_thread(s.want, [&] { return top_p_weight(top_p, total); });
      const u64 start = upto - w[0] - w[1];
      if (start < want && want <= upto) s.bin = i0 + (start + w[0] < want ? 2 : 1);
      __syncthreads();
    }
    const int keep = s.bin;
    u64 left = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = i0 + j;
      if (i < keep) {
        const float x = entry_logit(list[i]);
        if (!min_p_keeps(x, rs.e(x), min_p)) w[j] = 0;
        weights[i] = w[j];
        left += w[j];
        by_id[i] = ~((static_cast<u64>(entry_id(list[i])) << 32) | static_cast<uint32_t>(i));
      }
    }
    block_prefix(left, s.warp_sum, total);
    sort_list(by_id, keep);  // complements in descending order: ids in ascending order
    const u64 r = by_one_thread(s.draw, [&] { return draw_at(u, total); });
    u64 y[2] = {0, 0}, all;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (i0 + j < keep) y[j] = weights[static_cast<uint32_t>(~by_id[i0 + j])];
    upto = block_prefix(y[0] + y[1], s.warp_sum, all);
    const u64 start = upto - y[0] - y[1];
    if (start <= r && r < upto) {
      const u64 e = ~by_id[i0 + (start + y[0] <= r ? 1 : 0)];
      *token = static_cast<int32_t>(e >> 32);
      if (logprob != nullptr) *logprob = log_probability(rs.z(entry_logit(list[static_cast<uint32_t>(e)])), total);
    }
  }

  // Everything after the load.
  __device__ void run(int V, int k, bool list_first, float tau, float top_p, float min_p, float u, u64* scratch,
                      int32_t* token, float* logprob) {
    const bool need_k = k < V, need_p = !(top_p >= 1.f);
    if (list_first) {
      clear_list();
      for (int i = slice.v0 + lane; i < slice.v1; i += 32) {
        float v[E];
        slice.get(i, v);
        float most = v[0];
#pragma unroll
        for (int j = 1; j < E; ++j) most = fmaxf(most, v[j]);
        if (most >= tau) {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (v[j] >= tau && v[j] > -INFINITY) append(slice.id(i, j));
        }
      }
      __syncthreads();
      if (threadIdx.x == 0) s.count = s.list_count;
      sync_cluster();
      const uint32_t n = total_count();
      if (n <= kListCap) {
        push_list();
        sync_cluster();
        if (rank == 0)  // the slice is no longer needed
          finish_list(static_cast<int>(n), k, need_p, top_p, min_p, u, scratch, scratch + kListCap, token, logprob);
        return;
      }
    }
    Boundary bound = no_boundary();
    u64 kept = 0;
    bool sums = false, have_kept = false;  // kept_sum is up to date; kept is top-p's total
    if (need_k) {
      u64 valid = 0;
      slice.each(lane, [&](float x, int) { valid += x > -INFINITY; });
      sum_to_part(valid, 1, s.warp_sum);
      sync_cluster();
      const u64 n = total_of(1);
      if (static_cast<u64>(k) < n) {
        sync_cluster();
        sums = have_kept = z_boundary(bound, false, static_cast<u64>(k), top_p, min_p, bound, kept);
        if (!sums) {
          sync_cluster();
          bound = find_boundary(no_boundary(), false, static_cast<u64>(k));
        }
      }
    }
    if (need_p) {
      sync_cluster();
      sums = z_boundary(bound, true, 0, top_p, min_p, bound, kept);
      if (!sums) {
        sync_cluster();
        if (!have_kept) {
          const u64 sum = sum_weights([&](float x, int v, WeightSum& w) {
            if (bound.keeps(x, v)) w.add(rs.e(x));
          });
          sum_to_part(sum, 1, s.warp_sum);
          sync_cluster();
          kept = total_of(1);
        }
        bound = find_boundary(bound, true, by_one_thread(s.want, [&] { return top_p_weight(top_p, kept); }));
      }
    }
    // ---- draw
    const bool cut = bound.x > -INFINITY, filter = !(min_p <= 0.f);
    if (!sums) {
      sync_cluster();
      u64 sum;
      if (!cut && !filter)
        sum = sum_all();
      else
        sum = sum_weights([&](float x, int v, WeightSum& w) {
          if (cut && !bound.keeps(x, v)) return;
          const float e = rs.e(x);
          if (!filter || min_p_keeps(x, e, min_p)) w.add(e);
        });
      sum_to_part(sum, 1, s.kept_sum);
    } else {
      sync_cluster();
      if (warp == 0) add_warps(s.kept_sum, 1);
    }
    sync_cluster();
    u64 before = 0;
    const u64 total = total_of(1, &before);
    arrive_cluster();  // nothing of another CTA is read from here on
    const u64 r = by_one_thread(s.draw, [&] { return draw_at(u, total); });
    const int id = locate(before, r, [&](float x, int v) -> u64 {
      if (cut && !bound.keeps(x, v)) return 0;
      const float e = rs.e(x);
      return !filter || min_p_keeps(x, e, min_p) ? fixed_point(e) : 0;
    });
    if (id >= 0 && lane == 0) {
      *token = id;
      if (logprob != nullptr) *logprob = log_probability(rs.z(logit(id)), total);
    }
    wait_cluster();  // no CTA leaves while another reads its shared memory
  }
};

// A lower bound of the want-th largest of the block's thread maxima (-inf if fewer have a logit).
// 256 bins of equal width between the least and the largest; then the least maximum of the bins
// that hold the first `want`.
template <bool kResident>
__device__ float block_tau(float tmax, int want, SampleShared<kResident>& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool valid = tmax > -INFINITY;
  const uint32_t key = logit_key(tmax);
  const uint32_t whi = __reduce_max_sync(0xffffffffu, valid ? key : 0u);
  const uint32_t wlo = __reduce_min_sync(0xffffffffu, valid ? key : 0xffffffffu);
  if (lane == 0) {
    s.warp_hi[warp] = whi;
    s.warp_lo[warp] = wlo;
  }
  if (threadIdx.x < 256) s.work.zhist[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    s.bin = -1;
    s.lo = 0xffffffffu;
  }
  __syncthreads();
  const uint32_t hi = __reduce_max_sync(0xffffffffu, s.warp_hi[lane % kSampleWarps]);
  const uint32_t lo = __reduce_min_sync(0xffffffffu, s.warp_lo[lane % kSampleWarps]);
  const float x_hi = key_logit(hi), width = x_hi - key_logit(lo);
  const bool spread = lo < hi && width > 0.f && width < INFINITY;  // the same for the block
  const int bin = !valid || !spread ? 0 : static_cast<int>(fminf((x_hi - tmax) * (256.f / width), 255.f));
  if (valid) atomicAdd(&s.work.zhist[bin], 1u);
  __syncthreads();
  if (warp == 0) {
    u64 mine = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mine += s.work.zhist[8 * lane + j];
    u64 c = warp_prefix(mine, lane) - mine;
    if (c < static_cast<u64>(want) && static_cast<u64>(want) <= c + mine) {
      for (int j = 0; j < 8; ++j) {
        c += s.work.zhist[8 * lane + j];
        if (c >= static_cast<u64>(want)) {
          s.bin = 8 * lane + j;
          break;
        }
      }
    }
  }
  __syncthreads();
  const int last = s.bin;
  const uint32_t least = __reduce_min_sync(0xffffffffu, valid && bin <= last ? key : 0xffffffffu);
  if (lane == 0) atomicMin(&s.lo, least);
  __syncthreads();
  return last < 0 ? -INFINITY : key_logit(s.lo);
}

template <class T, bool kResident>
__global__ void __launch_bounds__(kSampleThreads, 2)
    sample_kernel(const T* __restrict__ logits, int V, int64_t ld, int per, const float* __restrict__ u,
                  const fkl_sample_params p, int32_t* __restrict__ token, float* __restrict__ logprob) {
  constexpr int E = Slice<T, kResident>::E;
  extern __shared__ uint4 dyn[];
  __shared__ SampleShared<kResident> s;
  const int ranks = cluster_size(), rank = static_cast<int>(cluster_ctarank());
  const int64_t b = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  u64* const counting = reinterpret_cast<u64*>(dyn);
  Slice<T, kResident> sl;
  sl.first = min(V, rank * per);
  sl.n = min(V, sl.first + per) - sl.first;
  sl.g = logits + b * ld + sl.first;
  sl.s = dyn + kCountingMax * sizeof(u64) / sizeof(uint4);
  sl.shift = static_cast<int>((reinterpret_cast<uintptr_t>(sl.g) % 16) / sizeof(T));
  sl.nvec = sl.n > 0 ? (sl.n + sl.shift + E - 1) / E : 0;
  const int per_warp = (sl.nvec + kSampleWarps - 1) / kSampleWarps;
  sl.v0 = min(sl.nvec, warp * per_warp);
  sl.v1 = min(sl.nvec, sl.v0 + per_warp);

  int k = p.top_k_rows != nullptr ? p.top_k_rows[b] : p.top_k;
  const float t = p.temperature_rows != nullptr ? p.temperature_rows[b] : p.temperature;
  const float top_p = p.top_p_rows != nullptr ? p.top_p_rows[b] : p.top_p;
  const float min_p = p.min_p_rows != nullptr ? p.min_p_rows[b] : p.min_p;
  const bool greedy = !(t > 0.f);
  if (greedy) k = 1;
  if (k <= 0 || k > V) k = V;

  // ---- load
  const float tmax = sl.load(lane);
  {
    float m = tmax;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s.warp_max[warp] = m;
  }
  // With w of n threads wanted the list holds about n log(n / (n - w)) logits.
  const bool list_first = k > 1 && k < V && k <= min(kListCap / 2, kSampleThreads * 3 / 4 * ranks);
  const float own_tau = list_first ? block_tau(tmax, (k + ranks - 1) / ranks, s) : -INFINITY;
  __syncthreads();
  if (warp == 0) {
    float m = lane < kSampleWarps ? s.warp_max[lane] : -INFINITY;
#pragma unroll
    for (int o = kSampleWarps / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) {
      s.cta_max = m;
      s.tau = own_tau;
    }
  }
  sync_cluster();
  float m = lane < ranks ? peer(&s, lane)->cta_max : -INFINITY;
  float tau = lane < ranks ? peer(&s, lane)->tau : INFINITY;
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    tau = fminf(tau, __shfl_xor_sync(0xffffffffu, tau, o));
  }
  m = __shfl_sync(0xffffffffu, m, 0);
  tau = __shfl_sync(0xffffffffu, tau, 0);
  float* const lp = logprob != nullptr ? logprob + b : nullptr;
  if (!(m > -INFINITY)) {  // nothing to draw
    if (rank == 0 && threadIdx.x == 0) {
      token[b] = -1;
      if (lp != nullptr) *lp = NAN;
    }
    sync_cluster();
    return;
  }
  if (k == 1) {  // the largest logit's first id
    int first = INT_MAX;
    if (s.cta_max == m)
      sl.each(lane, [&](float x, int v) {
        if (x == m) first = min(first, v);
      });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) s.warp_hi[warp] = static_cast<uint32_t>(first);
    __syncthreads();
    const uint32_t own = __reduce_min_sync(0xffffffffu, s.warp_hi[lane % kSampleWarps]);
    if (threadIdx.x == 0) s.count = own;
    sync_cluster();
    if (rank == 0 && warp == 0) {
      const uint32_t f = __reduce_min_sync(0xffffffffu, lane < ranks ? peer(&s, lane)->count : 0xffffffffu);
      if (lane == 0) {
        token[b] = static_cast<int32_t>(f);
        if (lp != nullptr) *lp = 0.f;
      }
    }
    sync_cluster();
    return;
  }
  const float inv_t = 1.f / t;
  u64* const scratch = reinterpret_cast<u64*>(dyn);
  if (m < INFINITY && inv_t > 0.f && inv_t < INFINITY) {
    RowCtx<T, kResident, true> c{sl, s, counting, RowScale<true>{m, inv_t}, rank, ranks, warp, lane};
    c.run(V, k, list_first, tau, top_p, min_p, u[b], scratch, token + b, lp);
  } else {
    RowCtx<T, kResident, false> c{sl, s, counting, RowScale<false>{m, inv_t}, rank, ranks, warp, lane};
    c.run(V, k, list_first, tau, top_p, min_p, u[b], scratch, token + b, lp);
  }
}

// ---------------------------------------------------------------- launch
// CTAs per row: the fewest whose slices fit two to an SM, or one to an SM, in shared memory;
// more (up to 8) as long as all rows still run at once.  Rows beyond what 8 CTAs hold are read
// again by each pass instead.
struct SamplePlan {
  int ranks, per;
  bool resident;
  size_t smem;
};

// Dynamic shared memory of each of n CTAs on an SM (227 KB to one, 228 KB less 1 KB a CTA to
// several), beside the static part.
template <bool kResident>
constexpr size_t max_dynamic(int n) {
  return ((n == 1 ? 227 * 1024 : 228 * 1024 / n - 1024) - sizeof(SampleShared<kResident>)) / 16 * 16;
}

// The longest slice, in bytes, of which an SM holds two beside the counted entries' weights and a
// vector that it may start inside: 8 of them are a row of 201088 fp32 logits.  Longer rows have one
// CTA to an SM, half as many rows at once.  On the device, 64 rows of 201088 and of 201089 fp32: 29
// and 44 us without filters, 28 and 44 with top-k 50, 74 and 128 with flat rows' top-p 0.9; 16 rows: 14
// and 19, 15 and 19, 36 and 52.  A larger SampleShared or kCountingMax moves that step to shorter rows.
constexpr size_t kTwoSlice = 100544;
static_assert(max_dynamic<true>(2) >= kCountingMax * sizeof(u64) + kTwoSlice + sizeof(uint4), "two such slices to an SM");

// Fewest logits that a CTA gets a slice of.
constexpr int64_t kMinSlice = 4096;

// Clusters of `ranks` CTAs (1, 2, 4 or 8) of one kernel that run at once, two CTAs to an SM, on the
// current device; asked of the driver once.
template <class Kern>
static int clusters_at_once(Kern kern, int ranks, int sms) {
  static std::atomic<int> known[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 2 * sms / ranks;
  std::atomic<int>& slot = known[dev][ranks == 1 ? 0 : ranks == 2 ? 1 : ranks == 4 ? 2 : 3];
  int n = slot.load();
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ranks));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = 64 * 1024;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ranks);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 2 * sms / ranks;
  }
  slot.store(n);
  return n;
}

template <class T>
static SamplePlan plan_sample(int64_t B, int64_t V, int sms) {
  constexpr size_t kScratch = 2 * kListCap * sizeof(u64);  // the list's weights and ids
  constexpr size_t kOne = max_dynamic<true>(1), kTwo = max_dynamic<true>(2);
  constexpr int64_t vec = 16 / sizeof(T);
  SamplePlan p{};
  for (p.ranks = 1;; p.ranks *= 2) {
    const int64_t per = ((V + p.ranks - 1) / p.ranks + vec - 1) / vec * vec;
    p.per = static_cast<int>(per);
    // the counted entries' weights and the slice, which may start inside a vector
    const size_t need = kCountingMax * sizeof(u64) + static_cast<size_t>(per) * sizeof(T) + 16;
    p.resident = need <= kOne && per <= Pieces<true>::kMaxSlice;
    p.smem = p.resident && need > kScratch ? need : kScratch;
    const bool wide = need <= kTwo && per <= Pieces<true>::kMaxSlice;
    if (p.ranks == kMaxCluster) return p;
    if (wide && (V < 2 * kMinSlice * p.ranks || B > clusters_at_once(sample_kernel<T, true>, 2 * p.ranks, sms))) return p;
  }
}

// Raises the kernels' shared-memory limits, once per device.
template <class T>
static cudaError_t raise_limits() {
  static std::atomic<uint64_t> raised[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (raised[(dev >> 6) & 1].load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(sample_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(max_dynamic<true>(1)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(sample_kernel<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(max_dynamic<false>(1)));
  if (e == cudaSuccess) raised[(dev >> 6) & 1].fetch_or(bit);
  return e;
}

template <class T, bool kResident>
static cudaError_t launch_sample(const void* logits, int64_t B, int64_t V, int64_t ld, const float* u,
                                 const fkl_sample_params& params, int32_t* token, float* logprob, const SamplePlan& pl,
                                 cudaStream_t st) {
  auto kern = sample_kernel<T, kResident>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * pl.ranks));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(pl.ranks);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(logits), static_cast<int>(V), ld, pl.per, u, params,
                            token, logprob);
}

static fkl_status sample_fail(fkl_status s, const char* msg) {
  set_last_error_message(msg);
  return s;
}

}  // namespace fkl

using namespace fkl;

extern "C" fkl_status fkl_sample(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld, const float* u,
                                 const fkl_sample_params* params, int32_t* token, float* logprob, void* stream) {
  set_last_error_message("");
  if (!type_ok(type)) return sample_fail(FKL_ERR_INVALID_ARG, "type must be one of FKL_TYPE_*");
  if (B < 0 || B > INT32_MAX || V < 1 || V > kMaxSampleV || ld < V)
    return sample_fail(FKL_ERR_INVALID_ARG, "need 0 <= B < 2^31, 1 <= V <= 2^22 and ld >= V");
  if (params == nullptr || (B > 0 && (logits == nullptr || u == nullptr || token == nullptr)))
    return sample_fail(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  const uintptr_t four = reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(token) |
                         reinterpret_cast<uintptr_t>(logprob) | reinterpret_cast<uintptr_t>(params->temperature_rows) |
                         reinterpret_cast<uintptr_t>(params->top_k_rows) |
                         reinterpret_cast<uintptr_t>(params->top_p_rows) |
                         reinterpret_cast<uintptr_t>(params->min_p_rows);
  if (reinterpret_cast<uintptr_t>(logits) % type_bytes(type) != 0 || four % 4 != 0)
    return sample_fail(FKL_ERR_ALIGNMENT, "logits must be aligned to their type, everything else to 4 bytes");
  int sms = 0;
  if (const int s = require_device(&sms); s != FKL_OK) return static_cast<fkl_status>(s);
  if (B == 0) return FKL_OK;
  const NamedPtr ptrs[] = {{logits, "logits"}, {u, "u"}, {token, "token"}, {logprob, "logprob"},
                           {params->temperature_rows, "temperature_rows"}, {params->top_k_rows, "top_k_rows"},
                           {params->top_p_rows, "top_p_rows"}, {params->min_p_rows, "min_p_rows"}};
  if (const int s = check_device_memory(ptrs); s != FKL_OK) return static_cast<fkl_status>(s);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = with_type(type, [&](auto t) {
    using T = decltype(t);
    if (const cudaError_t e = raise_limits<T>(); e != cudaSuccess) return e;
    const SamplePlan pl = plan_sample<T>(B, V, sms);
    return pl.resident ? launch_sample<T, true>(logits, B, V, ld, u, *params, token, logprob, pl, st)
                       : launch_sample<T, false>(logits, B, V, ld, u, *params, token, logprob, pl, st);
  });
  if (e != cudaSuccess) {
    cudaGetLastError();
    return sample_fail(FKL_ERR_CUDA, cudaGetErrorString(e));
  }
  return FKL_OK;
}
