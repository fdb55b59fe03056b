// Scores given tokens under rows of logits (fkl_token_logprobs) and the gradient in the logits.
//
// Forward.  One pass over a row keeps, per thread, a reference m, l = sum of e_v and u = sum of e_v a_v
// with a_v = (x_v - m) log2(e) / T and e_v = 2^a_v.  Then with M the row's largest logit and L, U the sums
// brought to it, log sum exp((x - M) / T) = log L and entropy = log L - ln 2 U / L, two terms of one sign, which
// do not cancel however sharp the row is.  A thread's reference follows its largest logit lazily (it moves
// when a logit exceeds it by 2^8 in weight), so the rescaling stays off the common path.
//
// Alternatives.  A thread also keeps its largest logit.  The top_n-th largest of these, rounded down to
// 16 bits, is a bound below the CTA's top_n-th largest logit, and only threads whose largest reaches it hold
// logits that do: not many more than top_n.  Only their shares are read again, all at once, and what reaches
// the bound is ranked by counting.  Where that is more than the list holds (many ties), the boundary is
// found by a radix selection over (logit, id) instead.
//
// A row is split over a cluster of CTAs where there are few rows; the others store their sums and lists
// into the first CTA's shared memory, which joins them.
//
// Backward.  dx_v = ( q_v (c0 + c1 log2 q_v) + a 1[v = v*] ) / T with c0 = -(a + b entropy), c1 = -b ln 2,
// q_v = 2^((x_v - M) log2(e) / T - log2 L), one pass that reads the logits and writes their gradient.
//
// What bounds it (GB300, on the device, logits in HBM).  Many rows: HBM for fp32 (512 x 201088: 61 us, 6.8 TB/s), for
// 16 bits the 9 instructions of a logit beside it (2048 x 128256 bf16: 87 us, 6.0 TB/s; 512 x 151936: 31 us, 5.0 TB/s,
// as all rows run at once and end together).  Few rows: latency (1 x 201088 fp32 5.5 us, with 20 alternatives 8.9; from
// L2 4.4 and 7.8).  The gradient runs at the rate of a copy (2048 x 128256 bf16: 150 us, 7.0 TB/s), if its rows lie in
// 16-byte vectors as the logits' do.  Where they do not (rows V + 1 apart in 16 bits) every element goes by itself: 804
// us.  Rows that the mask leaves out are read and written too, on a path without loads in flight (half of those rows: 187 us).
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/fkl_score.h"
#include "fkl_generate.cuh"
#include "fkl_score.cuh"
#include "fkl_types.cuh"

namespace fkl {
namespace {

using u64 = unsigned long long;

constexpr int kMostThreads = 512;
constexpr int kMaxRanks = 8;      // CTAs of a row
constexpr int kMaxTop = 128;
constexpr int kListCap = 1024;    // logits that reach the bound; where there are more, they are selected exactly
constexpr int kInFlight = 4;      // vectors that a thread loads before it uses the first
constexpr float kFloor = -200.f;  // exponents below it are 0: 2^-200 is below fp32, and 0 * -200 is 0 (0 * -inf is not)
constexpr int64_t kMaxV = int64_t{1} << 22;
static_assert(kListCap >= kMaxRanks * kMaxTop, "the lists of every CTA");

struct ScoreArgs {
  const void* logits;
  int64_t ld;
  int V, slice;  // slice: vectors of a row that one CTA reads
  TokenIds tokens;
  const uint8_t* mask;
  float temperature;
  const float* temperature_rows;
  int top_n;
  float *logprob, *entropy, *stats;
  int32_t* top_ids;
  float* top_logprobs;
};

// Order-preserving bits of a logit (-0 and +0 are the same logit) and back.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// Rank of a logit: descending keys are logits descending, then ids ascending.
__device__ __forceinline__ u64 rank_key(float x, int id) {
  return (static_cast<u64>(order_bits(x)) << 32) | static_cast<uint32_t>(~id);
}
__device__ __forceinline__ float key_logit(u64 k) { return order_value(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_id(u64 k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// A row as 16-byte vectors.  The row may start inside a vector (`skip` elements from its start) and end inside
// one: those two are read element by element, the others lie in [first, last).
template <class T>
struct RowView {
  static constexpr int kN = 16 / static_cast<int>(sizeof(T));
  const T* x;
  int V, skip, first, last, count;
  __device__ __forceinline__ RowView(const T* row, int v) : x(row), V(v) {
    skip = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    count = (skip + V + kN - 1) / kN;
    first = skip > 0 ? 1 : 0;
    last = (skip + V) / kN;
  }
  __device__ __forceinline__ int id(int vec) const { return vec * kN - skip; }
  __device__ __forceinline__ uint4 raw(int vec) const { return __ldcs(reinterpret_cast<const uint4*>(x + id(vec))); }
  __device__ __forceinline__ void load(int vec, float (&f)[kN]) const {
    const int at = id(vec);
    if (at >= 0 && at + kN <= V) {
      unpack16<T>(*reinterpret_cast<const uint4*>(x + at), f);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) f[j] = at + j >= 0 && at + j < V ? to_float(x[at + j]) : -INFINITY;
    }
  }
};

// A vector of -inf.
template <class T>
__device__ __forceinline__ uint4 none_vec() {
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

// Running sums of one thread (see the head of this file).
struct RowSum {
  float m = -FLT_MAX, largest = -INFINITY;
  float2 l = make_float2(0.f, 0.f), u = make_float2(0.f, 0.f);

  __device__ __forceinline__ void move_to(float to, float sc) {
    const float r = fmaxf((m - to) * sc, -1000.f), f = ex2_approx(r);
    u = fmul2(ffma2(make_float2(r, r), l, u), make_float2(f, f));
    l = fmul2(l, make_float2(f, f));
    m = to;
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float sc, float lead) {
    float c = fmax3(x[0], x[1], x[2]);
#pragma unroll
    for (int j = 3; j + 1 < N; j += 2) c = fmax3(c, x[j], x[j + 1]);
    if (N % 2 == 0) c = fmaxf(c, x[N - 1]);
    largest = fmaxf(largest, c);
    if (c > m + lead) move_to(c, sc);
    const float2 nm = make_float2(-m, -m), s2 = make_float2(sc, sc);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      float2 a = fmul2(fadd2(make_float2(x[j], x[j + 1]), nm), s2);
      a = make_float2(fmaxf(a.x, kFloor), fmaxf(a.y, kFloor));  // -inf, NaN and what underflows: weight 0
      const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
      l = fadd2(l, e);
      u = ffma2(e, a, u);
    }
  }
};

// What a CTA tells the first one of its cluster: its largest logit, its sums at it, its +inf logits and how many
// alternatives it lists.
struct Part {
  float largest, l, u;
  int infinite, listed;
};

template <bool kTop>
struct ScoreShared {
  Part part[kMaxRanks];  // in the first CTA: of every CTA
  float warp_max[kMostThreads / 32], warp_l[kMostThreads / 32], warp_u[kMostThreads / 32];
  int warp_count[kMostThreads / 32];
};
template <>
struct ScoreShared<true> : ScoreShared<false> {
  u64 list[kListCap];
  u64 top[kMaxTop];                // this CTA's largest, in order
  u64 tops[kMaxRanks * kMaxTop];   // in the first CTA: every CTA's, n each, 0 behind the last
  uint16_t hot[kMostThreads];
  int hot_count, list_count, bound;
  uint32_t hist[256];
  u64 prefix;
  int want;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Calls f(x, id) for every logit of the CTA's vectors [begin, end), every thread of every warp at the same
// time (beyond the end with -inf), so that f may use warp votes.
template <class T, class F>
__device__ void for_each_logit(const RowView<T>& row, int begin, int end, F&& f) {
  for (int v0 = begin; v0 < end; v0 += static_cast<int>(blockDim.x)) {
    const int v = v0 + static_cast<int>(threadIdx.x);
    float x[RowView<T>::kN];
    if (v < end) row.load(v, x);
#pragma unroll
    for (int j = 0; j < RowView<T>::kN; ++j) f(v < end ? x[j] : -INFINITY, row.id(v) + j);
  }
}

// The CTA's n largest logits (of those above -inf) into s.list and their number into s.list_count, whatever
// their ties: a radix selection of the n-th largest rank key, eight bits at a time from the top, then what
// reaches it.  Slow (nine more reads of the slice) and rare.
template <class T>
__device__ __noinline__ void select_exactly(ScoreShared<true>& s, const RowView<T>& row, int begin, int end, int n) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  if (tid == 0) {
    s.prefix = 0;
    s.want = n;
  }
  for (int shift = 56; shift >= 0; shift -= 8) {
    __syncthreads();
    if (tid < 256) s.hist[tid] = 0;
    __syncthreads();
    const u64 prefix = s.prefix;
    for_each_logit(row, begin, end, [&](float x, int id) {
      const u64 key = rank_key(x, id);
      const bool in = x > -INFINITY && (shift == 56 || (key >> (shift + 8)) == (prefix >> (shift + 8)));
      const int digit = in ? static_cast<int>(key >> shift) & 255 : -1;
      // ties fall into one bin: lanes that agree add together
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&s.hist[digit], static_cast<uint32_t>(__popc(same)));
    });
    __syncthreads();
    if (tid == 0) {
      int left = s.want, digit = 255;
      for (; digit > 0 && static_cast<int>(s.hist[digit]) < left; --digit) left -= static_cast<int>(s.hist[digit]);
      s.want = left;
      s.prefix = prefix | (static_cast<u64>(digit) << shift);
    }
  }
  if (tid == 0) s.list_count = 0;
  __syncthreads();
  const u64 least = s.prefix;
  for_each_logit(row, begin, end, [&](float x, int id) {
    if (x > -INFINITY && rank_key(x, id) >= least) {
      const int at = atomicAdd(&s.list_count, 1);
      if (at < kListCap) s.list[at] = rank_key(x, id);
    }
  });
  __syncthreads();
}

// Calls f(key, place) in one thread for each of the list's n keys, with its place in descending order.  A key is
// compared with the others by as many lanes (a power of two) as the block has for each.
template <int kThreads, class F>
__device__ __forceinline__ void rank_list(const u64* list, int n, F&& f) {
  int lanes = 1;
  while (lanes < 32 && n * lanes * 2 <= kThreads) lanes *= 2;
  const int part = static_cast<int>(threadIdx.x) & (lanes - 1), step = kThreads / lanes;
  for (int q0 = 0; q0 < n; q0 += step) {
    const int q = q0 + static_cast<int>(threadIdx.x) / lanes;
    const u64 key = list[min(q, n - 1)];
    int larger = 0;
#pragma unroll 8
    for (int j = part; j < n; j += lanes) larger += list[j] > key ? 1 : 0;
    for (int o = lanes / 2; o > 0; o >>= 1) larger += __shfl_xor_sync(0xffffffffu, larger, o);
    if (part == 0 && q < n) f(key, larger);
  }
}

// The CTA's n largest logits, in order, into s.top, and their number: see the head of this file.  `mine` is
// the thread's largest logit, `largest` the CTA's.
template <class T, int kThreads>
__device__ __forceinline__ int select_top(ScoreShared<true>& s, const RowView<T>& row, int begin, int end, int from,
                                          int to, int n, float mine, float largest) {
  constexpr int kN = RowView<T>::kN;
  static_assert(kInFlight * kN <= 32, "a bit for each logit in flight");
  const int tid = static_cast<int>(threadIdx.x);
  // The largest 16-bit bound that n threads reach.  It mostly lies within 255 of the CTA's largest (two binary
  // orders of a logit): a histogram of the distances, which the first warp adds up.  Where fewer than n threads
  // lie so near, a search by bits.
  const uint32_t key = order_bits(mine) >> 16, most = order_bits(largest) >> 16;
  if (most - key < 256u) atomicAdd(&s.hist[most - key], 1u);
  __syncthreads();
  if (tid < 32) {
    uint32_t bins[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += bins[i] = s.hist[tid * 8 + i];
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (tid >= o) upto += y;
    }
    const unsigned reached = __ballot_sync(0xffffffffu, upto >= static_cast<uint32_t>(n));
    if (reached == 0) {
      if (tid == 0) s.bound = -1;
    } else if (tid == __ffs(reached) - 1) {
      uint32_t before = upto - sum;
      int i = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (i == k && before + bins[k] < static_cast<uint32_t>(n)) {
          before += bins[k];
          ++i;
        }
      }
      s.bound = static_cast<int>(most) - (tid * 8 + i);
    }
  }
  __syncthreads();
  uint32_t bound = static_cast<uint32_t>(max(s.bound, 0));
  if (s.bound < 0) {
    bound = 0u;
#pragma unroll 1
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t next = bound + (1u << bit);
      if (__syncthreads_count(key >= next) >= n) bound = next;
    }
  }
  const bool is_hot = key >= bound && mine > -INFINITY;
  if (is_hot) s.hot[atomicAdd(&s.hot_count, 1)] = static_cast<uint16_t>(tid);
  __syncthreads();
  // as a logit: every logit (-inf is none) where fewer than n threads have one
  const float least = fmaxf(bound <= 0x007fu ? -FLT_MAX : order_value(bound << 16), -FLT_MAX);
  const int each = (to - from + kThreads - 1) / kThreads;  // vectors of a thread's share
  const int items = to > from ? s.hot_count * each : 0;
  for (int i0 = tid; i0 < items; i0 += kInFlight * kThreads) {
    uint4 raw[kInFlight] = {};
    int vec[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int i = i0 + k * kThreads;
      vec[k] = to;
      if (i < items) {
        const int h = i / each;
        vec[k] = from + s.hot[h] + (i - h * each) * kThreads;
      }
      if (vec[k] < to) raw[k] = *reinterpret_cast<const uint4*>(row.x + row.id(vec[k]));
    }
    // one addition to the list's length for all that this thread has found
    uint32_t found = 0;
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      float x[kN];
      unpack16<T>(raw[k], x);
#pragma unroll
      for (int j = 0; j < kN; ++j) found |= vec[k] < to && x[j] >= least ? 1u << (k * kN + j) : 0u;
    }
    int at = found != 0 ? atomicAdd(&s.list_count, __popc(found)) : 0;
    for (; found != 0; found &= found - 1, ++at) {  // one or two of them: the logit is read once more, from L1
      const int bit = __ffs(found) - 1;
      int v = vec[0];
#pragma unroll
      for (int k = 1; k < kInFlight; ++k) v = bit / kN == k ? vec[k] : v;
      const int id = row.id(v) + bit % kN;
      if (at < kListCap) s.list[at] = rank_key(to_float(row.x[id]), id);
    }
  }
  if (tid == 0 && is_hot && begin < end) {  // the first thread also had the vectors that the row starts and ends in
    auto offer = [&](int v) {
      float x[kN];
      row.load(v, x);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        if (x[j] >= least) {
          const int at = atomicAdd(&s.list_count, 1);
          if (at < kListCap) s.list[at] = rank_key(x[j], row.id(v) + j);
        }
      }
    };
    if (begin < from) offer(begin);
    if (end > to && end - 1 >= from) offer(end - 1);
  }
  __syncthreads();
  if (s.list_count > kListCap) {
    __syncthreads();  // every thread has read the count
    select_exactly(s, row, begin, end, n);
  }
  const int count = s.list_count;
  rank_list<kThreads>(s.list, count, [&](u64 key, int place) {
    if (place < n) s.top[place] = key;
  });
  __syncthreads();
  return count < n ? count : n;
}

template <class T, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) score_kernel(const ScoreArgs g) {
  constexpr int kWarps = kThreads / 32;
  __shared__ ScoreShared<kTop> s;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int ranks = cluster_size();
  const int rank = static_cast<int>(cluster_ctarank());
  const int64_t b = static_cast<int64_t>(blockIdx.x) / ranks;  // every CTA of a cluster has the same row
  const int n = kTop ? g.top_n : 0;
  const bool on = g.mask == nullptr || g.mask[b] != 0;
  const float temp = g.temperature_rows != nullptr ? g.temperature_rows[b] : g.temperature;
  const float inv = 1.f / temp, sc = kLog2e * inv;
  const bool scaled = sc > 0.f && sc < INFINITY;
  if (!on || !scaled) {  // nothing of the row is read
    if (rank == 0) {
      const float none = on ? NAN : 0.f;
      if (tid == 0) {
        g.logprob[b] = none;
        g.entropy[b] = none;
        if (g.stats != nullptr) g.stats[2 * b] = g.stats[2 * b + 1] = none;
      }
      for (int i = tid; i < n; i += kThreads) {
        g.top_ids[b * n + i] = -1;
        g.top_logprobs[b * n + i] = on ? NAN : -INFINITY;
      }
    }
    return;
  }
  if (ranks > 1) cluster_arrive();  // this CTA runs: its shared memory may be written from now on
  if constexpr (kTop) {
    if (tid == 0) s.hot_count = s.list_count = 0;  // seen after the barriers of the sums
    if (tid < 256) s.hist[tid] = 0;
  }
  const float lead = 8.f / sc;
  const RowView<T> row(static_cast<const T*>(g.logits) + b * g.ld, g.V);
  const int begin = min(rank * g.slice, row.count), end = min(begin + g.slice, row.count);
  const int from = max(begin, row.first), to = min(end, row.last);
  float token_x = NAN;  // the token's logit, fetched beside the rest
  int tok = -1;
  if (rank == 0 && tid == 0) {
    tok = g.tokens.get(b, g.V);
    if (tok >= 0) token_x = to_float(row.x[tok]);
  }

  RowSum r;
  {  // one batch of vectors is in flight while the other is added up
    const int batch = kInFlight * kThreads;
    uint4 a[kInFlight], c[kInFlight];
    auto fetch = [&](uint4 (&raw)[kInFlight], int v0) {
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) raw[k] = v0 + k * kThreads < to ? row.raw(v0 + k * kThreads) : none_vec<T>();
    };
    auto add = [&](const uint4 (&raw)[kInFlight]) {
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        float x[RowView<T>::kN];
        unpack16<T>(raw[k], x);
        r.add(x, sc, lead);
      }
    };
    int v0 = from + tid;
    fetch(a, v0);
    while (v0 < to) {
      fetch(c, v0 + batch);
      add(a);
      v0 += batch;
      if (v0 >= to) break;
      fetch(a, v0 + batch);
      add(c);
      v0 += batch;
    }
  }
  if (tid == 0) {
    float x[RowView<T>::kN];
    if (begin < from && begin < end) {
      row.load(begin, x);
      r.add(x, sc, lead);
    }
    if (end > to && end - 1 >= from) {
      row.load(end - 1, x);
      r.add(x, sc, lead);
    }
  }

  // the CTA's largest logit and the sums at it
  const float wm = warp_max(r.largest);
  if (lane == 0) s.warp_max[warp] = wm;
  __syncthreads();
  const float largest = warp_max(s.warp_max[lane % kWarps]);
  r.move_to(largest, sc);
  const float wl = warp_sum(r.l.x + r.l.y), wu = warp_sum(r.u.x + r.u.y);
  if (lane == 0) {
    s.warp_l[warp] = wl;
    s.warp_u[warp] = wu;
  }
  if (largest == INFINITY) {  // the +inf logits share the probability
    int c = 0;
    for_each_logit(row, begin, end, [&](float x, int) { c += x == INFINITY ? 1 : 0; });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (lane == 0) s.warp_count[warp] = c;
  }
  int listed = 0;
  if constexpr (kTop) {
    listed = select_top<T, kThreads>(s, row, begin, end, from, to, n, r.largest, largest);
  } else {
    __syncthreads();
  }
  if (ranks > 1) cluster_wait();  // the first CTA runs
  if (warp == 0) {
    const float l = warp_sum(lane < kWarps ? s.warp_l[lane] : 0.f), u = warp_sum(lane < kWarps ? s.warp_u[lane] : 0.f);
    int c = largest == INFINITY && lane < kWarps ? s.warp_count[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (lane == 0) *peer(&s.part[rank], 0) = Part{largest, l, u, c, listed};
  }
  if constexpr (kTop) {
    u64* tops = peer(&s.tops[rank * n], 0);
    for (int i = tid; i < n; i += kThreads) tops[i] = i < listed ? s.top[i] : 0ull;
    if (tid == 0) s.list_count = 0;  // read by all before select_top's last barrier
  }
  if (ranks > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // a lane per CTA (the lanes beyond repeat the first's sums with weight 0)
  const Part p = s.part[lane < ranks ? lane : 0];
  const float M = warp_max(p.largest);
  const float a = M < INFINITY && p.largest > -INFINITY ? fmaxf((p.largest - M) * sc, -1000.f) : 0.f;
  const float f = lane < ranks && p.largest > -INFINITY ? ex2_approx(a) : 0.f;
  const float L = warp_sum(M == INFINITY ? (lane < ranks ? static_cast<float>(p.infinite) : 0.f) : f > 0.f ? f * p.l : 0.f);
  const float U = warp_sum(M == INFINITY || !(f > 0.f) ? 0.f : f * fmaf(a, p.l, p.u));
  const int total = __reduce_add_sync(0xffffffffu, lane < ranks ? p.listed : 0);
  const float log_sum = M > -INFINITY ? logf(L) : NAN;
  auto logprob_of = [&](float x) {  // NaN where the row has nothing to produce
    if (M == INFINITY) return x == INFINITY ? -log_sum : -INFINITY;
    return (x > -INFINITY ? (x - M) * inv : -INFINITY) - log_sum;
  };
  if (tid == 0) {
    g.logprob[b] = tok >= 0 ? logprob_of(token_x) : NAN;
    g.entropy[b] = M > -INFINITY ? log_sum - kLn2 * U / L : NAN;
    if (g.stats != nullptr) {
      g.stats[2 * b] = M;
      g.stats[2 * b + 1] = log_sum;
    }
  }
  if constexpr (kTop) {
    int32_t* ids = g.top_ids + b * n;
    float* logs = g.top_logprobs + b * n;
    if (ranks == 1) {
      for (int i = tid; i < total; i += kThreads) {
        ids[i] = key_id(s.tops[i]);
        logs[i] = logprob_of(key_logit(s.tops[i]));
      }
    } else {
      // Every list has n / ranks keys (rounded up) that reach the least of those places: n keys do in all, and
      // not many more where the lists are alike.
      const int each = (n + ranks - 1) / ranks;
      u64 least = ~0ull;
      for (int c = 0; c < ranks; ++c) least = min(least, s.tops[c * n + each - 1]);
      for (int i = tid; i < ranks * n; i += kThreads) {
        const u64 key = s.tops[i];
        if (key != 0ull && key >= least) s.list[atomicAdd(&s.list_count, 1)] = key;
      }
      __syncthreads();
      rank_list<kThreads>(s.list, s.list_count, [&](u64 key, int place) {
        if (place < n) {
          ids[place] = key_id(key);
          logs[place] = logprob_of(key_logit(key));
        }
      });
    }
    for (int i = total + tid; i < n; i += kThreads) {
      ids[i] = -1;
      logs[i] = M > -INFINITY ? -INFINITY : NAN;
    }
  }
}

// ---------------------------------------------------------------- gradient
struct GradArgs {
  const void* logits;
  int64_t B, ld;
  int V;
  TokenIds tokens;
  const uint8_t* mask;
  float temperature;
  const float* temperature_rows;
  const float *stats, *entropy, *grad_logprob, *grad_entropy;
  void* dlogits;
  int64_t ldd;
  int piece;  // vectors of a row that one CTA takes
};

constexpr int kGradThreads = 256;
constexpr int kGradInFlight = 4;
constexpr int kGradBatches = 2;  // of kGradInFlight vectors a thread, in a CTA's piece of a row

// What one row's gradient is made of.
struct RowGrad {
  float m, sc, log2_sum, c0, c1;
  __device__ __forceinline__ float2 at(float2 x) const {
    float2 a = ffma2(fadd2(x, make_float2(-m, -m)), make_float2(sc, sc), make_float2(-log2_sum, -log2_sum));
    a = make_float2(fmaxf(a.x, kFloor), fmaxf(a.y, kFloor));
    const float2 q = make_float2(ex2_approx(a.x), ex2_approx(a.y));
    return fmul2(q, ffma2(make_float2(c1, c1), a, make_float2(c0, c0)));
  }
};

template <class T>
__device__ __forceinline__ uint4 pack16(const float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

// A CTA per piece of a row (blockIdx.x), rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <class T>
__global__ void __launch_bounds__(kGradThreads, 4) score_grad_kernel(const GradArgs g) {
  constexpr int N = RowView<T>::kN;
  const int tid = static_cast<int>(threadIdx.x);
  for (int64_t b = blockIdx.y; b < g.B; b += gridDim.y) {
    const RowView<T> row(static_cast<const T*>(g.logits) + b * g.ld, g.V);
    T* out = static_cast<T*>(g.dlogits) + b * g.ldd;
    const int begin = min(static_cast<int>(blockIdx.x) * g.piece, row.count), end = min(begin + g.piece, row.count);
    const bool vectors = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.x)) & 15) == 0;
    const int from = vectors ? max(begin, row.first) : end, to = vectors ? min(end, row.last) : end;

    // The row's values, fetched together: a row left out has zeros, whatever they are.
    const bool on = g.mask == nullptr || g.mask[b] != 0;
    const int given = g.tokens.get(b, g.V);
    const float ga = g.grad_logprob != nullptr ? g.grad_logprob[b] : 0.f;
    const float gb = g.grad_entropy != nullptr ? g.grad_entropy[b] : 0.f;
    const float largest = g.stats[2 * b], log_sum = g.stats[2 * b + 1], entropy = g.entropy[b];
    const float temp = g.temperature_rows != nullptr ? g.temperature_rows[b] : g.temperature;
    const float inv = 1.f / temp;
    const int tok = on ? given : -1;
    // NaN rows: a token outside the row, and what the forward found NaN (no logit, a bad temperature: log_sum is NaN)
    const float scale = given >= 0 ? inv + 0.f * log_sum : NAN;
    const RowGrad r{largest, kLog2e * inv, kLog2e * log_sum, -(gb != 0.f ? fmaf(gb, entropy, ga) : ga) * scale,
                    -gb * kLn2 * scale};
    const float at_token = ga * scale;
    const bool plain = on && r.c0 == r.c0 && largest < INFINITY;
    auto value = [&](float x, int id) {  // of one logit, in any row
      if (!on) return 0.f;
      if (!(r.c0 == r.c0)) return NAN;
      // +inf logits share the probability: log q + entropy is 0 there
      const float y = largest < INFINITY ? r.at(make_float2(x, x)).x : x == INFINITY ? -ga * expf(-log_sum) * scale : 0.f;
      return y + (id == tok ? at_token : 0.f);
    };

    if (plain) {
      const int tok_vec = (tok + row.skip) / N;
      for (int v0 = from + tid; v0 < to; v0 += kGradInFlight * kGradThreads) {
        uint4 raw[kGradInFlight];
#pragma unroll
        for (int k = 0; k < kGradInFlight; ++k)
          raw[k] = v0 + k * kGradThreads < to ? row.raw(v0 + k * kGradThreads) : none_vec<T>();
#pragma unroll
        for (int k = 0; k < kGradInFlight; ++k) {
          const int v = v0 + k * kGradThreads;
          float x[N];
          unpack16<T>(raw[k], x);
#pragma unroll
          for (int j = 0; j < N; j += 2) {
            const float2 y = r.at(make_float2(x[j], x[j + 1]));
            x[j] = y.x;
            x[j + 1] = y.y;
          }
          if (v == tok_vec) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] += row.id(v) + j == tok ? at_token : 0.f;
          }
          if (v < to) __stcs(reinterpret_cast<uint4*>(out + row.id(v)), pack16<T>(x));
        }
      }
    } else {
      for (int v = from + tid; v < to; v += kGradThreads) {
        float x[N];
        row.load(v, x);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = value(x[j], row.id(v) + j);
        *reinterpret_cast<uint4*>(out + row.id(v)) = pack16<T>(x);
      }
    }
    // what is not a whole vector of both, element by element
    auto singly = [&](int lo, int hi) {
      for (int i = max(lo, 0) + tid; i < min(hi, g.V); i += kGradThreads) out[i] = from_float<T>(value(to_float(row.x[i]), i));
    };
    if (!vectors) {
      singly(row.id(begin), row.id(end));
    } else {
      if (begin < from) singly(row.id(begin), row.id(min(from, end)));
      if (end > to && to >= begin) singly(row.id(max(to, from)), row.id(end));
    }
  }
}

fkl_status score_fail(fkl_status st, const char* msg) {
  set_last_error_message(msg);
  return st;
}

// CTAs per row: as many as keep the rows' clusters on the device at once (1024 threads to an SM), no slice
// shorter than kMinSlice logits.
constexpr int64_t kMinSlice = 4096;
int score_ranks(int64_t B, int64_t V, int slots) {
  int ranks = 1;
  while (ranks < kMaxRanks && V >= 2 * kMinSlice * ranks && B * ranks * 2 <= slots) ranks *= 2;
  return ranks;
}

template <class T, bool kTop, int kThreads>
cudaError_t launch_score(ScoreArgs& g, int64_t B, int sms, cudaStream_t st) {
  constexpr int N = RowView<T>::kN;
  const int ranks = score_ranks(B, g.V, sms * (1024 / kThreads));
  const int vecs = (g.V + N - 1) / N + 1;  // a row that starts inside a vector may have one more
  g.slice = (vecs + ranks - 1) / ranks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ranks);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, score_kernel<T, kTop, kThreads>, g);
}

// Blocks of 256 threads, four to an SM, spread many rows more evenly; 512 read a single row sooner, and a
// thread's share of a row, which is read again for each alternative, is half as long.  Forward on the device with
// 0, 5, 8, 12, 20 and 100 alternatives, 256 threads and then 512, in us (behind a write of 256 MB, so above the figures at the
// head of this file): 512 x 151936 bf16 33, 41, 43, 47, 52, 72 and 36, 45, 46, 47, 48, 67; 512 x 201088 fp32 70, 82, 89, 97,
// 111, 158 and 70, 80, 83, 88, 97, 136; 1000 x 32000 bf16 18, 26, 26, 26, 27, 41 and 22, 34, 34, 34, 35, 41.  Few rows:
// 1 x 201088 fp32 8.1, 11, 11, 11, 11, 15 and 6.4, 9.4, 9.4, 9.5, 9.6, 12; 203 x 50261 fp16 9.9, 15, 15, 15, 16, 21 and 10, 14,
// 14, 14, 15, 17.
constexpr int kFewTop = 8;
template <class T>
cudaError_t launch_score(ScoreArgs& g, int64_t B, int sms, cudaStream_t st) {
  const bool narrow = B > sms && g.top_n <= kFewTop;
  if (g.top_n > 0) return narrow ? launch_score<T, true, 256>(g, B, sms, st) : launch_score<T, true, 512>(g, B, sms, st);
  return narrow ? launch_score<T, false, 256>(g, B, sms, st) : launch_score<T, false, 512>(g, B, sms, st);
}

// The checks that both directions share.
fkl_status check_rows(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld, const void* tokens,
                      int32_t token_bytes, const float* temperature_rows, float temperature) {
  if (!type_ok(type)) return score_fail(FKL_ERR_INVALID_ARG, "type must be one of FKL_TYPE_*");
  if (B < 0 || B > INT32_MAX || V < 1 || V > kMaxV || ld < V)
    return score_fail(FKL_ERR_INVALID_ARG, "need 0 <= B < 2^31, 1 <= V <= 2^22 and ld >= V");
  if (token_bytes != 4 && token_bytes != 8) return score_fail(FKL_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
  if (B > 0 && (logits == nullptr || tokens == nullptr)) return score_fail(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (temperature_rows == nullptr && !(temperature > 0.f && temperature < INFINITY && kLog2e * (1.f / temperature) < INFINITY))
    return score_fail(FKL_ERR_INVALID_ARG, "temperature must be finite and > 0, and its inverse too (4.25e-39 and more)");
  if (reinterpret_cast<uintptr_t>(logits) % type_bytes(type) != 0 ||
      reinterpret_cast<uintptr_t>(tokens) % token_bytes != 0 || reinterpret_cast<uintptr_t>(temperature_rows) % 4 != 0)
    return score_fail(FKL_ERR_ALIGNMENT, "logits and tokens must be aligned to their types, temperature_rows to 4 bytes");
  return FKL_OK;
}

bool four(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

}  // namespace
}  // namespace fkl

using namespace fkl;

extern "C" fkl_status fkl_token_logprobs(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld,
                                         const void* tokens, int32_t token_bytes, const uint8_t* mask,
                                         float temperature, const float* temperature_rows, int32_t top_n,
                                         float* logprob, float* entropy, float* stats, int32_t* top_ids,
                                         float* top_logprobs, void* stream) {
  set_last_error_message("");
  fkl_status s = check_rows(logits, type, B, V, ld, tokens, token_bytes, temperature_rows, temperature);
  if (s != FKL_OK) return s;
  if (top_n < 0 || top_n > kMaxTop || top_n > V) return score_fail(FKL_ERR_INVALID_ARG, "need 0 <= top_n <= min(V, 128)");
  if (B > 0 && (logprob == nullptr || entropy == nullptr || (top_n > 0 && (top_ids == nullptr || top_logprobs == nullptr))))
    return score_fail(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!four(logprob) || !four(entropy) || !four(stats) || !four(top_ids) || !four(top_logprobs))
    return score_fail(FKL_ERR_ALIGNMENT, "outputs must be 4-byte aligned");
  int sms = 0;
  if (const int e = require_device(&sms); e != FKL_OK) return static_cast<fkl_status>(e);
  if (B == 0) return FKL_OK;
  const NamedPtr ptrs[] = {{logits, "logits"}, {tokens, "tokens"}, {mask, "mask"},
                           {temperature_rows, "temperature_rows"}, {logprob, "logprob"}, {entropy, "entropy"},
                           {stats, "stats"}, {top_n > 0 ? top_ids : nullptr, "top_ids"},
                           {top_n > 0 ? top_logprobs : nullptr, "top_logprobs"}};
  if (const int e = check_device_memory(ptrs); e != FKL_OK) return static_cast<fkl_status>(e);
  ScoreArgs g{logits, ld, static_cast<int>(V), 0, TokenIds{tokens, token_bytes}, mask, temperature, temperature_rows,
              top_n, logprob, entropy, stats, top_ids, top_logprobs};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = with_type(type, [&](auto t) {
    using T = decltype(t);
    return launch_score<T>(g, B, sms, st);
  });
  if (e != cudaSuccess) {
    cudaGetLastError();
    return score_fail(FKL_ERR_CUDA, cudaGetErrorString(e));
  }
  return FKL_OK;
}

extern "C" fkl_status fkl_token_logprobs_backward(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld,
                                                  const void* tokens, int32_t token_bytes, const uint8_t* mask,
                                                  float temperature, const float* temperature_rows, const float* stats,
                                                  const float* entropy, const float* grad_logprob,
                                                  const float* grad_entropy, void* dlogits, int64_t ldd, void* stream) {
  set_last_error_message("");
  fkl_status s = check_rows(logits, type, B, V, ld, tokens, token_bytes, temperature_rows, temperature);
  if (s != FKL_OK) return s;
  if (ldd < V) return score_fail(FKL_ERR_INVALID_ARG, "need ldd >= V");
  if (B > 0 && (stats == nullptr || entropy == nullptr || dlogits == nullptr))
    return score_fail(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!four(stats) || !four(entropy) || !four(grad_logprob) || !four(grad_entropy) ||
      reinterpret_cast<uintptr_t>(dlogits) % type_bytes(type) != 0)
    return score_fail(FKL_ERR_ALIGNMENT, "dlogits must be aligned to its type, everything else to 4 bytes");
  int sms = 0;
  if (const int e = require_device(&sms); e != FKL_OK) return static_cast<fkl_status>(e);
  if (B == 0) return FKL_OK;
  const NamedPtr ptrs[] = {{logits, "logits"}, {tokens, "tokens"}, {mask, "mask"},
                           {temperature_rows, "temperature_rows"}, {stats, "stats"}, {entropy, "entropy"},
                           {grad_logprob, "grad_logprob"}, {grad_entropy, "grad_entropy"}, {dlogits, "dlogits"}};
  if (const int e = check_device_memory(ptrs); e != FKL_OK) return static_cast<fkl_status>(e);
  GradArgs g{logits, B, ld, static_cast<int>(V), TokenIds{tokens, token_bytes}, mask, temperature, temperature_rows,
             stats, entropy, grad_logprob, grad_entropy, dlogits, ldd, 1};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = with_type(type, [&](auto t) {
    using T = decltype(t);
    constexpr int kBatch = kGradThreads * kGradInFlight;
    const int vecs = static_cast<int>(V / RowView<T>::kN) + 2;  // of a row that starts inside a vector
    g.piece = kGradBatches * kBatch;
    const dim3 grid(static_cast<unsigned>((vecs + g.piece - 1) / g.piece), static_cast<unsigned>(B < 65535 ? B : 65535));
    score_grad_kernel<T><<<grid, kGradThreads, 0, st>>>(g);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return score_fail(FKL_ERR_CUDA, cudaGetErrorString(e));
  return FKL_OK;
}
