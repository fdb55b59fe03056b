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
// shared memory.  The steps:
//
//   1. load      the slice, each thread's largest logit, the row's largest m, and tau, a lower
//                bound of the target-th largest logit: the least, over the CTAs, of the
//                ceil(target / C)-th largest of their threads' maxima;
//   2. gather    the logits >= tau into a list (and, for top-p alone, the total weight).  The
//                list holds the top k by construction, or is checked to hold the top-p weight;
//   3. finish    the first CTA sorts the list (some hundreds of entries), cuts it, sorts what
//                stays by id and draws.
//
// When the list cannot hold the answer (a flat row whose top-p set has thousands of ids, a
// large k, many ties) the boundary is found from histograms instead: 1024 bins of equal width
// in z, then of the logits' bits within the bin that holds the boundary, until its logits fit
// the list or are all equal; then the draw makes two more passes over the slices.  Without
// top-k and top-p only the draw remains.
#include <atomic>
#include <climits>
#include <cmath>

#include "fkl_ptx.cuh"
#include "fkl_types.cuh"

namespace fkl {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxSampleV = int64_t{1} << 22;  // 2^22 weights of 2^40 stay below 2^63
constexpr int kBins = 1024;
constexpr int kListCap = 1024;
constexpr int kTopPTarget = 192;  // list entries aimed at for top-p alone

using u64 = unsigned long long;

// Order-preserving bits of a logit (-0 and +0 are the same logit) and back.
__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// floor(2^40 e) for 0 <= e <= 1, from e's bits.
__device__ __forceinline__ u64 fixed_point(float e) {
  const uint32_t b = __float_as_uint(e);
  const int s = static_cast<int>(b >> 23) - 110;  // 2^40 e = mantissa * 2^s
  const uint32_t mant = (b & 0x7fffffu) | 0x800000u;
  return static_cast<u64>(mant >> min(max(-s, 0), 31)) * (1u << max(s, 0));
}

// The row's largest logit and its scale.
struct RowScale {
  float m, inv_t;
  bool plain;  // m and 1/T are ordinary numbers: (x - m) / T needs no special cases
  __device__ __forceinline__ float z(float x) const {
    if (plain) return (x - m) * inv_t;
    return x == m ? 0.f : (x - m) * inv_t;
  }
  // exp(z); 0 for -inf (and where infinities leave no number)
  __device__ __forceinline__ float e(float x) const {
    const float v = expf(z(x));
    if (plain) return v;
    return x > -INFINITY && v > 0.f ? v : 0.f;
  }
  __device__ __forceinline__ u64 weight(float x) const { return fixed_point(e(x)); }
};

// A boundary in the order (logit descending, id ascending).
struct Boundary {
  uint32_t key;
  int id;
  __device__ __forceinline__ bool keeps(uint32_t k, int v) const { return k > key || (k == key && v <= id); }
};

// Weights (41 bits) are added to the histograms in pieces, each into 32 bits: 3 of 14 bits for
// a slice in shared memory (at most 2^17 logits), 4 of 12 bits for longer ones (at most 2^19).
template <bool kResident>
struct Pieces {
  static constexpr int kCount = kResident ? 3 : 4, kBits = kResident ? 14 : 12;
  static constexpr int kMaxSlice = 1 << (32 - 1 - kBits);
};
static_assert(Pieces<false>::kMaxSlice * kMaxCluster >= kMaxSampleV, "a piece sum stays below 2^31");

template <bool kResident>
struct SampleShared {
  // a histogram, then the list of gathered logits, in the same place
  union {
    uint32_t hist[Pieces<kResident>::kCount][kBins];
    u64 list[kListCap];
  } work;
  u64 warp_sum[kSampleWarps];
  // exchanged between the CTAs of the cluster (written before a cluster barrier, read after)
  u64 part[2];
  uint32_t count, key_lo, key_hi;
  float cta_max, tau;
  Boundary bound;
  // this CTA only
  float warp_max[kSampleWarps];
  uint32_t list_count, lo, hi;
  int bin;
  u64 before;
};

// Barrier of the cluster's threads: shared memory written before it is seen by every CTA after.
__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  cluster_sync();
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
  u64 before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSampleWarps; ++w) {
    if (w == warp) before = total;
    total += warp_sum[w];
  }
  return before + v;
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

  __device__ __forceinline__ void read_global(int i, float (&v)[E]) const {
    const int at = i * E - shift;
    if (at >= 0 && at + E <= n) {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(g + at));
      unpack16<T>(raw, v);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = at + j >= 0 && at + j < n ? to_float(g[at + j]) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = v[j] == v[j] ? v[j] : -INFINITY;
  }
  __device__ __forceinline__ void put(int i, const float (&v)[E]) const {
    uint4 raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int j = 0; j < E; ++j) e[j] = from_float<T>(v[j]);  // exact: the values came from T
    s[i] = raw;
  }
  __device__ __forceinline__ void get(int i, float (&v)[E]) const {
    if (kResident)
      unpack16<T>(s[i], v);
    else
      read_global(i, v);
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

// State of one row, shared by the steps.
template <class T, bool kResident>
struct RowCtx {
  Slice<T, kResident> slice;
  SampleShared<kResident>& s;
  u64* merged;  // this CTA's share of the merged histogram: kBins / ranks sums
  RowScale rs;
  int rank, ranks, warp, lane;

  // Sum of v over the block's threads, into s.part[slot] (visible to the cluster after its
  // next barrier).
  __device__ __forceinline__ void sum_to_part(u64 v, int slot) {
    v = warp_add(v);
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 t = 0;
      for (int w = 0; w < kSampleWarps; ++w) t += s.warp_sum[w];
      s.part[slot] = t;
    }
  }
  // Sum of part[slot] over the cluster, and over the CTAs before this one.
  __device__ __forceinline__ u64 total_of(int slot, u64* before = nullptr) {
    u64 t = 0;
    for (int r = 0; r < ranks; ++r) {
      if (r == rank && before != nullptr) *before = t;
      t += peer(&s, r)->part[slot];
    }
    return t;
  }
  __device__ __forceinline__ uint32_t total_count() {
    uint32_t t = 0;
    for (int r = 0; r < ranks; ++r) t += peer(&s, r)->count;
    return t;
  }

  // Appends the logits for which f holds to this CTA's list; their number (which may exceed
  // the list) and the range of their keys go to s.count, s.key_lo and s.key_hi.
  template <class F>
  __device__ void gather(F f) {
    __syncthreads();
    if (threadIdx.x == 0) {
      s.list_count = 0;
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
        const uint32_t at = atomicAdd(&s.list_count, 1u);
        if (at < kListCap) s.work.list[at] = (static_cast<u64>(k) << 32) | (0xffffffffu - static_cast<uint32_t>(v));
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
  // Moves this CTA's list behind those of the CTAs before it, in the first CTA.  Between two
  // cluster barriers.
  __device__ __forceinline__ void push_list() {
    if (rank == 0) return;
    uint32_t at = 0;
    for (int r = 0; r < rank; ++r) at += peer(&s, r)->count;
    u64* to = peer(&s.work.list[0], 0);
    for (uint32_t i = threadIdx.x; i < s.count; i += kSampleThreads) to[at + i] = s.work.list[i];
  }
  // First CTA: pads the list's n entries to a power of two and sorts them.
  __device__ __forceinline__ void sort_list(u64* keys, int n) {
    int n2 = 1;
    while (n2 < n) n2 <<= 1;
    for (int i = n + threadIdx.x; i < n2; i += kSampleThreads) keys[i] = 0;
    sort_descending(keys, n2);
  }

  // Histogram over the cluster of f's amounts (f(x, v, bin, amount) gives whether the logit
  // counts, its bin and its amount): the bin at which the running sum reaches `want`, and the
  // sum before it.
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
    sync_cluster();
    // this CTA merges its share of the bins
    const int per = kBins / ranks;
    u64 sum = 0;
    for (int i = threadIdx.x; i < per; i += kSampleThreads) {
      u64 t = 0;
      for (int r = 0; r < ranks; ++r) {
        const SampleShared<kResident>* o = peer(&s, r);
#pragma unroll
        for (int q = 0; q < P::kCount; ++q) t += static_cast<u64>(o->work.hist[q][rank * per + i]) << (q * P::kBits);
      }
      merged[i] = t;
      sum += t;
    }
    sum_to_part(sum, 0);
    sync_cluster();
    // the share that holds the boundary, then the bin within it
    u64 run = 0;
    int owner = ranks - 1;
    for (int r = 0; r < ranks; ++r) {
      const u64 t = peer(&s, r)->part[0];
      if (run + t >= want) {
        owner = r;
        break;
      }
      if (r + 1 < ranks) run += t;
    }
    const u64* m = peer(merged, owner);
    const int i0 = 2 * static_cast<int>(threadIdx.x);
    const u64 a = i0 < per ? m[i0] : 0, b = i0 + 1 < per ? m[i0 + 1] : 0;
    u64 total;
    const u64 upto = run + block_prefix(a + b, s.warp_sum, total);
    if (threadIdx.x == 0) s.bin = -1;
    __syncthreads();
    const u64 start = upto - a - b;
    if (start < want && want <= upto) {
      const bool second = start + a < want;
      s.bin = owner * per + i0 + (second ? 1 : 0);
      s.before = start + (second ? a : 0);
    }
    __syncthreads();
    before = s.before;
    return s.bin;
  }

  // Sum of f over the ids before, and the id at which the running sum exceeds r, when it lies in
  // this CTA: each warp's sum must be in s.warp_sum and `before` be the sum of the CTAs before.
  // Returns the id in every lane of the warp that holds it, -1 elsewhere.
  template <class F>
  __device__ __forceinline__ int locate(u64 before, u64 r, F f) {
    constexpr int E = Slice<T, kResident>::E;
    for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
    if (!(before <= r && r < before + s.warp_sum[warp])) return -1;
    for (int i0 = slice.v0; i0 < slice.v1; i0 += 32) {
      const int i = i0 + lane;
      u64 a[E], sum = 0;
#pragma unroll
      for (int j = 0; j < E; ++j) a[j] = 0;
      if (i < slice.v1) {
        float v[E];
        slice.get(i, v);
#pragma unroll
        for (int j = 0; j < E; ++j) sum += a[j] = f(v[j], slice.id(i, j));
      }
      const u64 run = before + warp_prefix(sum, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, run > r);
      if (hit) {
        const int src = __ffs(hit) - 1;
        u64 c = run - sum;
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

  // The boundary at which `want` logits (by_mass false) or a weight of `want` (by_mass true)
  // have been kept, among those that `keeps`; want is at least 1 and at most what there is.
  // The whole cluster.
  __device__ Boundary find_boundary(const Boundary& keeps, bool by_mass, u64 want) {
    // z of weight 1 (2^-40) is -27.7; logits further down share the last bin
    const float scale = static_cast<float>(kBins) / 27.8f;
    auto z_bin = [&](float x) -> uint32_t {  // falls as x rises; rounds to the nearest bin
      const float t = fminf(rs.z(x) * -scale, static_cast<float>(kBins - 1));
      return __float_as_uint(t + 8388608.f) & (kBins - 1);
    };
    auto amount_of = [&](float x) -> u64 { return by_mass ? rs.weight(x) : 1ull; };
    u64 before = 0;
    int bin = find_bin(want, before, [&](float x, int v, uint32_t& b, u64& amount) -> bool {
      if (!(x > -INFINITY) || !keeps.keeps(logit_key(x), v)) return false;
      b = z_bin(x);
      amount = amount_of(x);
      return true;
    });
    want -= before;
    gather([&](float x, int v) {
      return x > -INFINITY && static_cast<int>(z_bin(x)) == bin && keeps.keeps(logit_key(x), v);
    });
    for (;;) {
      sync_cluster();
      const uint32_t n = total_count();
      uint32_t lo = 0xffffffffu, hi = 0u;
      for (int r = 0; r < ranks; ++r) {
        lo = min(lo, peer(&s, r)->key_lo);
        hi = max(hi, peer(&s, r)->key_hi);
      }
      if (n <= kListCap) {
        push_list();
        sync_cluster();
        if (rank == 0) {
          sort_list(s.work.list, static_cast<int>(n));
          const int i0 = 2 * static_cast<int>(threadIdx.x);
          u64 w[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[j] = i0 + j < static_cast<int>(n) ? amount_of(key_logit(static_cast<uint32_t>(s.work.list[i0 + j] >> 32))) : 0;
          u64 total;
          const u64 upto = block_prefix(w[0] + w[1], s.warp_sum, total);
          const u64 start = upto - w[0] - w[1];
          if (start < want && want <= upto) {
            const u64 c = s.work.list[i0 + (start + w[0] < want ? 1 : 0)];
            s.bound = Boundary{static_cast<uint32_t>(c >> 32), static_cast<int>(0xffffffffu - static_cast<uint32_t>(c))};
          }
        }
        break;
      }
      if (lo == hi) {  // more equal logits than the list holds: the ids decide
        const u64 each = by_mass ? rs.weight(key_logit(lo)) : 1ull;
        const u64 skip = (want - 1) / each;  // equal logits kept before the last one
        auto tie = [&](float x, int v) -> u64 { return logit_key(x) == lo && keeps.keeps(lo, v) ? 1ull : 0ull; };
        u64 sum = 0, ahead = 0;
        slice.each(lane, [&](float x, int v) { sum += tie(x, v); });
        sum_to_part(sum, 0);
        sync_cluster();
        total_of(0, &ahead);
        const int id = locate(ahead, skip, tie);
        if (id >= 0 && lane == 0) peer(&s, 0)->bound = Boundary{lo, id};
        break;
      }
      const int bits = 32 - __clz(hi - lo);
      const int shift = bits > 10 ? bits - 10 : 0;
      static_assert(kBins == 1 << 10, "bins of the logits' bits");
      bin = find_bin(want, before, [&](float x, int v, uint32_t& b, u64& amount) -> bool {
        const uint32_t k = logit_key(x);
        if (k < lo || k > hi || !keeps.keeps(k, v)) return false;
        b = (hi - k) >> shift;
        amount = amount_of(x);
        return true;
      });
      want -= before;
      gather([&](float x, int v) {
        const uint32_t k = logit_key(x);
        return k >= lo && k <= hi && static_cast<int>((hi - k) >> shift) == bin && keeps.keeps(k, v);
      });
    }
    sync_cluster();
    return peer(&s, 0)->bound;
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

  u64* const merged = reinterpret_cast<u64*>(dyn);
  Slice<T, kResident> sl;
  sl.first = min(V, rank * per);
  sl.n = min(V, sl.first + per) - sl.first;
  sl.g = logits + b * ld + sl.first;
  sl.s = dyn + kBins / ranks * sizeof(u64) / sizeof(uint4);
  sl.shift = static_cast<int>((reinterpret_cast<uintptr_t>(sl.g) % 16) / sizeof(T));
  sl.nvec = sl.n > 0 ? (sl.n + sl.shift + E - 1) / E : 0;
  const int per_warp = (sl.nvec + kSampleWarps - 1) / kSampleWarps;
  sl.v0 = min(sl.nvec, warp * per_warp);
  sl.v1 = min(sl.nvec, sl.v0 + per_warp);

  int k = p.top_k_rows != nullptr ? p.top_k_rows[b] : p.top_k;
  const float t = p.temperature_rows != nullptr ? p.temperature_rows[b] : p.temperature;
  const float top_p = p.top_p_rows != nullptr ? p.top_p_rows[b] : p.top_p;
  const float min_p = p.min_p_rows != nullptr ? p.min_p_rows[b] : p.min_p;
  const float draw = u[b];
  const bool greedy = !(t > 0.f);
  if (greedy) k = 1;
  if (k <= 0 || k > V) k = V;
  const bool need_k = k < V, need_p = !(top_p >= 1.f);

  // ---- 1. load
  float tmax = -INFINITY;
  constexpr int U = 4;  // vectors in flight per thread
  for (int i0 = sl.v0; i0 < sl.v1; i0 += 32 * U) {
    float v[U][E];
#pragma unroll
    for (int q = 0; q < U; ++q)
      if (i0 + 32 * q + lane < sl.v1) sl.read_global(i0 + 32 * q + lane, v[q]);
#pragma unroll
    for (int q = 0; q < U; ++q)
      if (i0 + 32 * q + lane < sl.v1) {
#pragma unroll
        for (int j = 0; j < E; ++j) tmax = fmaxf(tmax, v[q][j]);
        if (kResident) sl.put(i0 + 32 * q + lane, v[q]);
      }
  }
  {
    float m = tmax;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s.warp_max[warp] = m;
  }
  // With w of n threads wanted the list holds about n log(n / (n - w)) logits.
  const bool list_first = k > 1 && (need_k ? k <= min(kListCap / 2, kSampleThreads * 3 / 4 * ranks) : need_p);
  float tau = -INFINITY;
  if (list_first) {
    // the upper 16 bits of the want-th largest thread maximum, bit by bit
    const int want = ((need_k ? k : kTopPTarget) + ranks - 1) / ranks;
    const uint32_t key = logit_key(tmax);
    uint32_t th = 0;
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t c = th | (1u << bit);
      if (__syncthreads_count(key >= c) >= want) th = c;
    }
    // below -inf's key when fewer threads than wanted have a logit: every logit is gathered
    tau = th > logit_key(-INFINITY) ? key_logit(th) : -INFINITY;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float m = s.warp_max[0];
    for (int w = 1; w < kSampleWarps; ++w) m = fmaxf(m, s.warp_max[w]);
    s.cta_max = m;
    s.tau = tau;
  }
  sync_cluster();
  float m = -INFINITY;
  for (int r = 0; r < ranks; ++r) {
    m = fmaxf(m, peer(&s, r)->cta_max);
    tau = fminf(tau, peer(&s, r)->tau);
  }
  if (!(m > -INFINITY)) {  // nothing to draw
    if (rank == 0 && threadIdx.x == 0) {
      token[b] = -1;
      if (logprob != nullptr) logprob[b] = NAN;
    }
    sync_cluster();
    return;
  }
  const float inv_t = greedy ? 1.f : 1.f / t;
  const RowScale rs{m, inv_t, m < INFINITY && inv_t > 0.f && inv_t < INFINITY};
  RowCtx<T, kResident> c{sl, s, merged, rs, rank, ranks, warp, lane};

  if (k == 1) {  // the largest logit's first id
    int first = INT_MAX;
    sl.each(lane, [&](float x, int v) {
      if (x == m) first = min(first, v);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) s.warp_sum[warp] = static_cast<u64>(first);
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 f = s.warp_sum[0];
      for (int w = 1; w < kSampleWarps; ++w) f = min(f, s.warp_sum[w]);
      s.part[0] = f;
    }
    sync_cluster();
    if (rank == 0 && threadIdx.x == 0) {
      u64 f = s.part[0];
      for (int r = 1; r < ranks; ++r) f = min(f, peer(&s, r)->part[0]);
      token[b] = static_cast<int32_t>(f);
      if (logprob != nullptr) logprob[b] = 0.f;
    }
    sync_cluster();
    return;
  }

  // ---- 2. gather
  u64 total = 0;      // weight that top-p takes its share of
  bool have_total = false;
  if (list_first) {
    u64 all = 0, listed = 0;
    const bool sum_all = !need_k;
    c.gather([&](float x, int) {
      const bool in = x >= tau && x > -INFINITY;
      if (sum_all) {
        const u64 w = rs.weight(x);
        all += w;
        if (in) listed += w;
      }
      return in;
    });
    if (sum_all) {
      c.sum_to_part(all, 0);
      c.sum_to_part(listed, 1);
    }
    sync_cluster();
    const uint32_t n = c.total_count();
    bool finish = n <= kListCap;
    if (sum_all) {
      total = c.total_of(0);
      have_total = true;
      finish = finish && c.total_of(1) >= top_p_weight(top_p, total);
    }
    if (finish) {
      // ---- 3. the first CTA finishes
      c.push_list();
      sync_cluster();
      if (rank != 0) return;
      u64* list = s.work.list;
      c.sort_list(list, static_cast<int>(n));
      u64* weights = reinterpret_cast<u64*>(dyn);  // the row's slice is no longer needed
      u64* by_id = weights + kListCap;
      const int kk = need_k ? min(k, static_cast<int>(n)) : static_cast<int>(n);
      const int i0 = 2 * static_cast<int>(threadIdx.x);
      u64 w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) w[j] = i0 + j < kk ? rs.weight(key_logit(static_cast<uint32_t>(list[i0 + j] >> 32))) : 0;
      u64 sum;
      u64 upto = block_prefix(w[0] + w[1], s.warp_sum, sum);
      if (need_k) total = sum;
      if (threadIdx.x == 0) s.bin = kk;
      __syncthreads();
      if (need_p) {
        const u64 want = top_p_weight(top_p, total);
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
          const uint32_t key = static_cast<uint32_t>(list[i] >> 32);
          const uint32_t id = 0xffffffffu - static_cast<uint32_t>(list[i]);
          const float x = key_logit(key);
          if (!(x == m) && !(rs.e(x) >= min_p)) w[j] = 0;
          weights[i] = w[j];
          left += w[j];
          by_id[i] = ~((static_cast<u64>(id) << 32) | static_cast<uint32_t>(i));
        }
      }
      block_prefix(left, s.warp_sum, sum);
      c.sort_list(by_id, keep);  // complements in descending order: ids in ascending order
      const u64 r = draw_at(draw, sum);
      u64 x2[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (i0 + j < keep) x2[j] = weights[static_cast<uint32_t>(~by_id[i0 + j])];
      u64 all2;
      upto = block_prefix(x2[0] + x2[1], s.warp_sum, all2);
      const u64 start = upto - x2[0] - x2[1];
      if (start <= r && r < upto) {
        const u64 e = ~by_id[i0 + (start + x2[0] <= r ? 1 : 0)];
        token[b] = static_cast<int32_t>(e >> 32);
        if (logprob != nullptr)
          logprob[b] = log_probability(rs.z(key_logit(static_cast<uint32_t>(list[static_cast<uint32_t>(e)] >> 32))), sum);
      }
      return;
    }
  }

  // ---- boundaries from histograms
  Boundary bound{0u, INT_MAX};
  if (need_k) {
    u64 valid = 0;
    sl.each(lane, [&](float x, int) { valid += x > -INFINITY; });
    c.sum_to_part(valid, 0);
    sync_cluster();
    const u64 n = c.total_of(0);
    if (static_cast<u64>(k) < n) bound = c.find_boundary(bound, false, static_cast<u64>(k));
  }
  if (need_p) {
    if (!have_total) {
      u64 sum = 0;
      sl.each(lane, [&](float x, int v) {
        if (bound.keeps(logit_key(x), v)) sum += rs.weight(x);
      });
      c.sum_to_part(sum, 1);  // part[0] may still be read
      sync_cluster();
      total = c.total_of(1);
    }
    bound = c.find_boundary(bound, true, top_p_weight(top_p, total));
  }

  // ---- draw
  const bool cut = need_k || need_p, filter = min_p > 0.f;
  auto kept = [&](float x, int v) -> u64 {
    if (cut && !bound.keeps(logit_key(x), v)) return 0;
    const float e = rs.e(x);
    if (filter && !(x == m) && !(e >= min_p)) return 0;
    return fixed_point(e);
  };
  u64 sum = 0, before = 0;
  sl.each(lane, [&](float x, int v) { sum += kept(x, v); });
  c.sum_to_part(sum, 1);
  sync_cluster();
  total = c.total_of(1, &before);
  const int id = c.locate(before, draw_at(draw, total), kept);
  if (id >= 0 && lane == 0) {
    const float x = to_float(logits[b * ld + id]);
    token[b] = id;
    if (logprob != nullptr) logprob[b] = log_probability(rs.z(x), total);
  }
  sync_cluster();  // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- launch
// CTAs per row: the fewest whose slices fit two to an SM, or one to an SM, in shared memory;
// more (up to 8) while the rows do not fill the device.  Rows beyond what 8 CTAs hold are read
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
  return (n == 1 ? 227 * 1024 : 228 * 1024 / n - 1024) / 128 * 128 - (sizeof(SampleShared<kResident>) + 255) / 128 * 128;
}

// Fewest logits that a CTA gets a slice of.
constexpr int64_t kMinSlice = 4096;

static SamplePlan plan_sample(int64_t B, int64_t V, size_t elem, int sms) {
  constexpr size_t kScratch = 2 * kListCap * sizeof(u64);  // the list's weights and ids
  constexpr size_t kOne = max_dynamic<true>(1), kTwo = max_dynamic<true>(2);
  const int64_t vec = static_cast<int64_t>(16 / elem);
  SamplePlan p{};
  for (p.ranks = 1;; p.ranks *= 2) {
    const int64_t per = ((V + p.ranks - 1) / p.ranks + vec - 1) / vec * vec;
    p.per = static_cast<int>(per);
    // the merged histogram and the slice, which may start inside a vector
    const size_t need = kBins / p.ranks * sizeof(u64) + static_cast<size_t>(per) * elem + 16;
    p.resident = need <= kOne && per <= Pieces<true>::kMaxSlice;
    p.smem = p.resident && need > kScratch ? need : kScratch;
    const bool wide = need <= kTwo && per <= Pieces<true>::kMaxSlice;
    if (p.ranks == kMaxCluster || (wide && (B * p.ranks > sms || V < 2 * kMinSlice * p.ranks))) return p;
  }
}

template <class T, bool kResident>
static cudaError_t launch_sample(const void* logits, int64_t B, int64_t V, int64_t ld, const float* u,
                                 const fkl_sample_params& params, int32_t* token, float* logprob, const SamplePlan& pl,
                                 cudaStream_t st) {
  auto kern = sample_kernel<T, kResident>;
  static std::atomic<uint64_t> raised[2];  // devices whose shared-memory limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (!(raised[(dev >> 6) & 1].load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(max_dynamic<kResident>(1)));
    if (e != cudaSuccess) return e;
    raised[(dev >> 6) & 1].fetch_or(bit);
  }
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
    const SamplePlan pl = plan_sample(B, V, sizeof(T), sms);
    return pl.resident ? launch_sample<T, true>(logits, B, V, ld, u, *params, token, logprob, pl, st)
                       : launch_sample<T, false>(logits, B, V, ld, u, *params, token, logprob, pl, st);
  });
  if (e != cudaSuccess) {
    cudaGetLastError();
    return sample_fail(FKL_ERR_CUDA, cudaGetErrorString(e));
  }
  return FKL_OK;
}
