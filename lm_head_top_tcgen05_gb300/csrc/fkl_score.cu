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
// logits that do: not many more than top_n of the CTA's 512.  Only their shares are read again, by a warp
// each, and what reaches the bound is ranked by counting.  Where that is more than the list holds (many
// ties), the boundary is found by a radix selection over (logit, id) instead.
//
// A row is split over a cluster of CTAs where there are few rows; the first CTA merges sums and lists
// through distributed shared memory.
//
// Backward.  dx_v = ( q_v (c0 + c1 log2 q_v) + a 1[v = v*] ) / T with c0 = -(a + b entropy), c1 = -b ln 2,
// q_v = 2^((x_v - M) log2(e) / T - log2 L), one pass that reads the logits and writes their gradient.
#include <cfloat>
#include <climits>
#include <cmath>

#include "../../include/fkl_score.h"
#include "fkl_generate.cuh"
#include "fkl_score.cuh"
#include "fkl_types.cuh"

namespace fkl {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRanks = 8;      // CTAs of a row
constexpr int kMaxTop = 128;
constexpr int kListCap = 1024;    // more than (kMaxTop - 1) vectors of 8: a bound that no thread sets cannot fill it
constexpr int kInFlight = 4;      // vectors that a thread loads before it uses the first
constexpr float kFloor = -200.f;  // exponents below it are 0: 2^-200 is below fp32, and 0 * -200 is 0 (0 * -inf is not)
constexpr int64_t kMaxV = int64_t{1} << 22;
static_assert(kListCap >= kMaxTop * 8 && kListCap >= kMaxRanks * kMaxTop, "lists of every CTA fit the first one's");

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

// A row as 16-byte vectors.  The row may start inside a vector and end inside one: those two
// (`skip` > 0, `tail` > 0) are read element by element, the others lie in [first, last).
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

struct ScoreShared {
  u64 list[kListCap];
  u64 top[kMaxTop];  // this CTA's largest, in order
  int top_count;
  float largest, l, u;  // exchanged: this CTA's largest logit and its sums at it
  int infinite;         // exchanged: its +inf logits
  // this CTA only
  float warp_max[kWarps], warp_l[kWarps], warp_u[kWarps];
  int warp_count[kWarps];
  uint16_t hot[kThreads];
  int hot_count, list_count;
  uint32_t hist[256];
  u64 prefix;
  int want;
};

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
// Barrier of the cluster's threads: shared memory written before it is seen by every CTA after.
__device__ __forceinline__ void meet() {
  __syncwarp();
  cluster_sync();
}
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
// time (with valid = false beyond the end), so that f may use warp votes.
template <class T, class F>
__device__ void for_each_logit(const RowView<T>& row, int begin, int end, F&& f) {
  for (int v0 = begin; v0 < end; v0 += kThreads) {
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
__device__ __noinline__ void select_exactly(ScoreShared& s, const RowView<T>& row, int begin, int end, int n) {
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

// The CTA's top_n largest logits, in order, into s.top: see the head of this file.  `largest` is the thread's.
template <class T>
__device__ __forceinline__ void select_top(ScoreShared& s, const RowView<T>& row, int begin, int end, int from, int to,
                                           int n, float largest) {
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const uint32_t mine = order_bits(largest) >> 16;
  uint32_t bound = 0;
#pragma unroll 1
  for (int bit = 15; bit >= 0; --bit) {
    const uint32_t next = bound | (1u << bit);
    if (__syncthreads_count(mine >= next) >= n) bound = next;
  }
  if (mine >= bound && largest > -INFINITY) s.hot[atomicAdd(&s.hot_count, 1)] = static_cast<uint16_t>(tid);
  __syncthreads();
  const uint32_t least = bound << 16;
  auto offer = [&](const float (&x)[RowView<T>::kN], int id) {
#pragma unroll
    for (int j = 0; j < RowView<T>::kN; ++j) {
      if (order_bits(x[j]) >= least && x[j] > -INFINITY) {
        const int at = atomicAdd(&s.list_count, 1);
        if (at < kListCap) s.list[at] = rank_key(x[j], id + j);
      }
    }
  };
  const int hot = s.hot_count;
  for (int h = warp; h < hot; h += kWarps) {
    const int t = s.hot[h];
    for (int v = from + t + lane * kThreads; v < to; v += 32 * kThreads) {
      float x[RowView<T>::kN];
      row.load(v, x);
      offer(x, row.id(v));
    }
    if (t == 0 && lane < 2) {  // the first thread also had the vectors that the row starts and ends in
      const int v = lane == 0 ? begin : end - 1;
      if (begin < end && (lane == 0 ? begin < from : end > to && v >= from)) {
        float x[RowView<T>::kN];
        row.load(v, x);
        offer(x, row.id(v));
      }
    }
  }
  __syncthreads();
  if (s.list_count > kListCap) {
    __syncthreads();  // every thread has read the count
    select_exactly(s, row, begin, end, n);
  }
  const int count = s.list_count;
  for (int i = tid; i < count; i += kThreads) {
    const u64 key = s.list[i];
    int r = 0;
    for (int j = 0; j < count; ++j) r += s.list[j] > key ? 1 : 0;
    if (r < n) s.top[r] = key;
  }
  if (tid == 0) s.top_count = count < n ? count : n;
  __syncthreads();
}

// Keys of the descending list that are larger than `key`.
__device__ __forceinline__ int larger(const u64* list, int n, u64 key) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (list[mid] > key) lo = mid + 1; else hi = mid;
  }
  return lo;
}

template <class T, bool kTop>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const ScoreArgs g) {
  __shared__ ScoreShared s;
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
  if (tid == 0) s.hot_count = s.list_count = s.top_count = 0;
  const float lead = 8.f / sc;
  const RowView<T> row(static_cast<const T*>(g.logits) + b * g.ld, g.V);
  const int begin = min(rank * g.slice, row.count), end = min(begin + g.slice, row.count);
  const int from = max(begin, row.first), to = min(end, row.last);

  RowSum r;
  for (int v0 = from + tid; v0 < to; v0 += kInFlight * kThreads) {
    uint4 raw[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (v0 + k * kThreads < to) raw[k] = row.raw(v0 + k * kThreads);
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      if (v0 + k * kThreads < to) {
        float x[RowView<T>::kN];
        unpack16<T>(raw[k], x);
        r.add(x, sc, lead);
      }
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
  float largest = s.warp_max[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) largest = fmaxf(largest, s.warp_max[w]);
  r.move_to(largest, sc);
  const float wl = warp_sum(r.l.x + r.l.y), wu = warp_sum(r.u.x + r.u.y);
  if (lane == 0) {
    s.warp_l[warp] = wl;
    s.warp_u[warp] = wu;
  }
  int infinite = 0;
  if (largest == INFINITY) {  // the +inf logits share the probability
    for_each_logit(row, begin, end, [&](float x, int) { infinite += x == INFINITY ? 1 : 0; });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) infinite += __shfl_xor_sync(0xffffffffu, infinite, o);
    if (lane == 0) s.warp_count[warp] = infinite;
  }
  __syncthreads();
  if (tid == 0) {
    float l = 0.f, u = 0.f;
    infinite = 0;
    for (int w = 0; w < kWarps; ++w) {
      l += s.warp_l[w];
      u += s.warp_u[w];
      if (largest == INFINITY) infinite += s.warp_count[w];
    }
    s.largest = largest;
    s.l = l;
    s.u = u;
    s.infinite = infinite;
  }
  if (kTop) select_top(s, row, begin, end, from, to, n, r.largest);
  if (ranks > 1) meet();

  if (rank == 0) {
    __syncthreads();
    float M = -INFINITY;
    for (int c = 0; c < ranks; ++c) M = fmaxf(M, peer(&s, c)->largest);
    float L = 0.f, U = 0.f;
    for (int c = 0; c < ranks; ++c) {
      const ScoreShared* p = peer(&s, c);
      if (M == INFINITY) {
        L += static_cast<float>(p->infinite);
      } else if (p->largest > -INFINITY) {
        const float a = fmaxf((p->largest - M) * sc, -1000.f), f = ex2_approx(a);
        L = fmaf(p->l, f, L);
        U = fmaf(fmaf(a, p->l, p->u), f, U);
      }
    }
    const float log_sum = M > -INFINITY ? logf(L) : NAN;
    const float T_inv = inv;
    auto logprob_of = [&](float x) {  // NaN where the row has nothing to produce
      if (M == INFINITY) return x == INFINITY ? -log_sum : -INFINITY;
      return (x > -INFINITY ? (x - M) * T_inv : -INFINITY) - log_sum;
    };
    if (tid == 0) {
      const int tok = g.tokens.get(b, g.V);
      const float x = tok >= 0 ? to_float(row.x[tok]) : 0.f;
      g.logprob[b] = tok >= 0 ? logprob_of(x) : NAN;
      g.entropy[b] = M > -INFINITY ? log_sum - kLn2 * U / L : NAN;
      if (g.stats != nullptr) {
        g.stats[2 * b] = M;
        g.stats[2 * b + 1] = log_sum;
      }
    }
    if constexpr (kTop) {
      int total = 0;
      for (int c = 0; c < ranks; ++c) {
        const ScoreShared* p = peer(&s, c);
        const int have = p->top_count;
        for (int i = tid; i < have; i += kThreads) s.list[c * n + i] = p->top[i];
        total += have;
      }
      __syncthreads();
      int32_t* ids = g.top_ids + b * n;
      float* logs = g.top_logprobs + b * n;
      for (int k = tid; k < ranks * n; k += kThreads) {
        const int c = k / n, i = k - c * n;
        if (i >= peer(&s, c)->top_count) continue;
        const u64 key = s.list[k];
        int place = i;
        for (int o = 0; o < ranks; ++o)
          if (o != c) place += larger(s.list + o * n, peer(&s, o)->top_count, key);
        if (place < n) {
          ids[place] = key_id(key);
          logs[place] = logprob_of(key_logit(key));
        }
      }
      for (int i = total + tid; i < n; i += kThreads) {
        ids[i] = -1;
        logs[i] = M > -INFINITY ? -INFINITY : NAN;
      }
    }
  }
  if (ranks > 1) meet();  // the first CTA has read the others' shared memory
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
  int pieces;  // CTAs' pieces of a row
};

constexpr int kGradThreads = 256;
constexpr int kGradInFlight = 4;

// What one row's gradient is made of.
struct RowGrad {
  float m, sc, log2_sum, c0, c1;
  bool infinite;
  float share;  // of a +inf logit
  __device__ __forceinline__ float at(float x) const {
    if (infinite) return x == INFINITY ? share : 0.f;
    const float a = fmaxf(fmaf(x - m, sc, -log2_sum), kFloor);
    return ex2_approx(a) * fmaf(c1, a, c0);
  }
  __device__ __forceinline__ float2 at(float2 x) const {
    if (infinite) return make_float2(at(x.x), at(x.y));
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

template <class T>
__global__ void __launch_bounds__(kGradThreads) score_grad_kernel(const GradArgs g) {
  constexpr int N = RowView<T>::kN;
  const int64_t items = g.B * g.pieces;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t b = item / g.pieces;
    const int piece = static_cast<int>(item - b * g.pieces);
    const RowView<T> row(static_cast<const T*>(g.logits) + b * g.ld, g.V);
    T* out = static_cast<T*>(g.dlogits) + b * g.ldd;
    const int per = (row.count + g.pieces - 1) / g.pieces;
    const int begin = min(piece * per, row.count), end = min(begin + per, row.count);

    const bool on = g.mask == nullptr || g.mask[b] != 0;
    const int tok = on ? g.tokens.get(b, g.V) : -1;
    RowGrad r{};
    float at_token = 0.f;
    if (on) {
      const float temp = g.temperature_rows != nullptr ? g.temperature_rows[b] : g.temperature;
      const float inv = 1.f / temp;
      const float ga = g.grad_logprob != nullptr ? g.grad_logprob[b] : 0.f;
      const float gb = g.grad_entropy != nullptr ? g.grad_entropy[b] : 0.f;
      const float log_sum = g.stats[2 * b + 1];
      r.m = g.stats[2 * b];
      r.infinite = r.m == INFINITY;
      r.sc = kLog2e * inv;
      r.log2_sum = kLog2e * log_sum;
      // NaN rows: a token outside the row, and what the forward found NaN (no logit, a bad temperature: log_sum is NaN)
      const float scale = tok >= 0 ? inv + 0.f * log_sum : NAN;
      r.c0 = -(gb != 0.f ? fmaf(gb, g.entropy[b], ga) : ga) * scale;
      r.c1 = -gb * kLn2 * scale;
      r.share = -ga * expf(-log_sum) * scale;  // log q + entropy is 0 there
      at_token = ga * scale;
    }
    const bool clean = !on || r.c0 == r.c0;
    auto value = [&](float x, int id) { return !on ? 0.f : !clean ? NAN : r.at(x) + (id == tok ? at_token : 0.f); };
    const bool vectors = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.x)) & 15) == 0;
    const int from = vectors ? max(begin, row.first) : end, to = vectors ? min(end, row.last) : end;
    for (int v0 = from + static_cast<int>(threadIdx.x); v0 < to; v0 += kGradInFlight * kGradThreads) {
      uint4 raw[kGradInFlight];
      if (on) {
#pragma unroll
        for (int k = 0; k < kGradInFlight; ++k)
          if (v0 + k * kGradThreads < to) raw[k] = row.raw(v0 + k * kGradThreads);
      }
#pragma unroll
      for (int k = 0; k < kGradInFlight; ++k) {
        const int v = v0 + k * kGradThreads;
        if (v >= to) continue;
        float x[N];
        if (on && clean) {
          unpack16<T>(raw[k], x);
#pragma unroll
          for (int j = 0; j < N; j += 2) {
            const float2 y = r.at(make_float2(x[j], x[j + 1]));
            x[j] = y.x;
            x[j + 1] = y.y;
          }
          const int k0 = tok - row.id(v);
          if (k0 >= 0 && k0 < N) {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] += j == k0 ? at_token : 0.f;
          }
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) x[j] = on ? NAN : 0.f;
        }
        *reinterpret_cast<uint4*>(out + row.id(v)) = pack16<T>(x);
      }
    }
    // what is not a whole vector of both, element by element
    auto singly = [&](int lo, int hi) {
      for (int i = max(lo, 0) + static_cast<int>(threadIdx.x); i < min(hi, g.V); i += kGradThreads)
        out[i] = from_float<T>(value(on ? to_float(row.x[i]) : 0.f, i));
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

// CTAs per row: as many as keep the rows' clusters on the device at once (two CTAs to an SM), no slice
// shorter than kMinSlice logits.
constexpr int64_t kMinSlice = 4096;
int score_ranks(int64_t B, int64_t V, int sms) {
  int ranks = 1;
  while (ranks < kMaxRanks && V >= 2 * kMinSlice * ranks && B * ranks * 2 <= 2 * sms) ranks *= 2;
  return ranks;
}

template <class T, bool kTop>
cudaError_t launch_score(ScoreArgs& g, int64_t B, int sms, cudaStream_t st) {
  constexpr int N = RowView<T>::kN;
  const int ranks = score_ranks(B, g.V, sms);
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
  return cudaLaunchKernelEx(&cfg, score_kernel<T, kTop>, g);
}

// The checks that both directions share.
fkl_status check_rows(const void* logits, int32_t type, int64_t B, int64_t V, int64_t ld, const void* tokens,
                      int32_t token_bytes, const float* temperature_rows, float temperature) {
  if (!type_ok(type)) return score_fail(FKL_ERR_INVALID_ARG, "type must be one of FKL_TYPE_*");
  if (B < 0 || B > INT32_MAX || V < 1 || V > kMaxV || ld < V)
    return score_fail(FKL_ERR_INVALID_ARG, "need 0 <= B < 2^31, 1 <= V <= 2^22 and ld >= V");
  if (token_bytes != 4 && token_bytes != 8) return score_fail(FKL_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
  if (B > 0 && (logits == nullptr || tokens == nullptr)) return score_fail(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (temperature_rows == nullptr && !(temperature > 0.f && temperature < INFINITY))
    return score_fail(FKL_ERR_INVALID_ARG, "temperature must be finite and > 0");
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
    return top_n > 0 ? launch_score<T, true>(g, B, sms, st) : launch_score<T, false>(g, B, sms, st);
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
    const int64_t piece = static_cast<int64_t>(kGradThreads) * kGradInFlight * RowView<T>::kN;
    g.pieces = static_cast<int>((V + piece - 1) / piece);
    const int64_t items = B * g.pieces, most = static_cast<int64_t>(sms) * 8 * 64;
    score_grad_kernel<T><<<static_cast<unsigned>(items < most ? items : most), kGradThreads, 0, st>>>(g);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return score_fail(FKL_ERR_CUDA, cudaGetErrorString(e));
  return FKL_OK;
}
