// The sampler of a generation step (fkl_sample): temperature, top-k, top-p, min-p and the
// draw, from given random numbers.
//
// Every sum is one of whole numbers, w_v = floor(2^40 exp(z_v)), so it is exact and does not
// depend on how the row is split.  Nothing is sorted: the logits that a filter keeps are the
// ones before a boundary in the order (logit descending, id ascending), and a boundary is found
// digit by digit on the logits' bits, from histograms of counts and weights; the draw then
// walks the ids in their own order.
#include <cmath>

#include "fkl_internal.h"
#include "fkl_types.cuh"

namespace fkl {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int64_t kMaxSampleV = int64_t{1} << 22;  // 2^22 weights of 2^40 stay below 2^63

using u64 = unsigned long long;

// Order-preserving bits of a logit (-0 and +0 are the same logit).
__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <class T>
__device__ __forceinline__ float logit_at(const T* row, int v) {
  const float x = to_float(row[v]);
  return isnan(x) ? -INFINITY : x;
}

// Settings of one row and its scale.
struct RowScale {
  float m, inv_t;
  __device__ __forceinline__ float z(float x) const { return x == m ? 0.f : (x - m) * inv_t; }
  // floor(2^40 exp(z)); 0 for -inf (and where infinities leave no number)
  __device__ __forceinline__ u64 weight(float x) const {
    const float e = x > -INFINITY ? expf(z(x)) : 0.f;
    return e > 0.f ? static_cast<u64>(e * 1099511627776.f) : 0ull;
  }
};

// A boundary in the order (logit descending, id ascending).
struct Boundary {
  uint32_t key;
  int id;
  __device__ __forceinline__ bool keeps(uint32_t k, int v) const { return k > key || (k == key && v <= id); }
};

struct SampleShared {
  u64 mass[256];
  uint32_t count[256];
  u64 warp_sum[kSampleWarps];
  float warp_max[kSampleWarps];
  u64 total;
  uint32_t digit;
  u64 before_count, before_mass, tie_count, tie_weight;
  int id;
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ u64 block_sum(u64 v, SampleShared& s) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
  for (int w = 0; w < kSampleWarps; ++w) t += s.warp_sum[w];
  return t;
}

// The first id, in the order of ids, at which the running sum of f exceeds r (-1: none).
template <class F>
__device__ int first_past(int V, u64 r, SampleShared& s, F f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (V + kSampleWarps - 1) / kSampleWarps;
  const int b = min(V, warp * per), e = min(V, b + per);
  u64 sum = 0;
  for (int v = b + lane; v < e; v += 32) sum += f(v);
  sum = warp_sum(sum);
  __syncthreads();
  if (lane == 0) s.warp_sum[warp] = sum;
  if (threadIdx.x == 0) s.id = -1;
  __syncthreads();
  u64 before = 0;
  for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
  if (before <= r && r < before + sum) {
    for (int v0 = b; v0 < e; v0 += 32) {
      const u64 x = v0 + lane < e ? f(v0 + lane) : 0ull;
      u64 run = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + run > r);
      if (hit) {
        if (lane == 0) s.id = v0 + __ffs(hit) - 1;
        break;
      }
      before += __shfl_sync(0xffffffffu, run, 31);
    }
  }
  __syncthreads();
  const int id = s.id;
  __syncthreads();
  return id;
}

// The boundary after which `want_count` logits (by_mass false) or a weight of at least
// `want_mass` (by_mass true) have been kept, among those that `keeps`.  Both are at least 1 and
// at most what there is.
template <class T>
__device__ Boundary find_boundary(const T* row, int V, const RowScale& rs, const Boundary& keeps, bool by_mass,
                                  u64 want, SampleShared& s) {
  uint32_t prefix = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSampleThreads) {
      s.mass[i] = 0;
      s.count[i] = 0;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < V; v += kSampleThreads) {
      const float x = logit_at(row, v);
      const uint32_t k = logit_key(x);
      if (shift < 24 && (k >> (shift + 8)) != (prefix >> (shift + 8))) continue;
      if (!keeps.keeps(k, v)) continue;
      const u64 w = rs.weight(x);
      if (w == 0) continue;
      atomicAdd(&s.mass[(k >> shift) & 255], w);
      atomicAdd(&s.count[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int d = 255;
      for (; d > 0; --d) {
        const u64 have = by_mass ? s.mass[d] : s.count[d];
        if (have >= want) break;
        want -= have;
      }
      s.digit = d;
      s.before_mass = want;
      s.tie_count = s.count[d];
      s.tie_weight = s.count[d] ? s.mass[d] / s.count[d] : 1;  // equal weights once the key is whole
    }
    __syncthreads();
    prefix |= s.digit << shift;
    want = s.before_mass;
    __syncthreads();
  }
  // the logits of this value that are still wanted, by ascending id
  const u64 tie_weight = s.tie_weight;
  const u64 ties = by_mass ? (want + tie_weight - 1) / tie_weight : want;
  const int id = first_past(V, ties - 1, s, [&](int v) -> u64 { return logit_key(logit_at(row, v)) == prefix; });
  return Boundary{prefix, id < 0 ? INT32_MAX : id};
}

template <class T>
__global__ void __launch_bounds__(kSampleThreads)
    sample_kernel(const T* __restrict__ logits, int V, int64_t ld, const float* __restrict__ u,
                  const fkl_sample_params p, int32_t* __restrict__ token, float* __restrict__ logprob) {
  __shared__ SampleShared s;
  const int64_t b = blockIdx.x;
  const T* row = logits + b * ld;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int v = threadIdx.x; v < V; v += kSampleThreads) m = fmaxf(m, logit_at(row, v));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s.warp_max[warp] = m;
  __syncthreads();
  for (int w = 0; w < kSampleWarps; ++w) m = fmaxf(m, s.warp_max[w]);
  if (!(m > -INFINITY)) {
    if (threadIdx.x == 0) {
      token[b] = -1;
      if (logprob != nullptr) logprob[b] = NAN;
    }
    return;
  }
  const float t = p.temperature_rows != nullptr ? p.temperature_rows[b] : p.temperature;
  int k = p.top_k_rows != nullptr ? p.top_k_rows[b] : p.top_k;
  const float top_p = p.top_p_rows != nullptr ? p.top_p_rows[b] : p.top_p;
  const float min_p = p.min_p_rows != nullptr ? p.min_p_rows[b] : p.min_p;
  const bool greedy = !(t > 0.f);
  if (greedy) k = 1;
  if (k <= 0 || k > V) k = V;
  const RowScale rs{m, greedy ? 1.f : 1.f / t};

  u64 total = 0, live = 0;
  for (int v = threadIdx.x; v < V; v += kSampleThreads) {
    const u64 w = rs.weight(logit_at(row, v));
    total += w;
    live += w != 0;
  }
  total = block_sum(total, s);
  live = block_sum(live, s);
  Boundary bound{0u, INT32_MAX};
  if (static_cast<u64>(k) < live) {
    bound = find_boundary(row, V, rs, bound, false, static_cast<u64>(k), s);
    total = 0;
    for (int v = threadIdx.x; v < V; v += kSampleThreads) {
      const float x = logit_at(row, v);
      if (bound.keeps(logit_key(x), v)) total += rs.weight(x);
    }
    total = block_sum(total, s);
  }
  if (!(top_p >= 1.f)) {
    const double lim = ceil(static_cast<double>(top_p) * static_cast<double>(total));
    const u64 want = lim >= 1.0 ? static_cast<u64>(lim) : 1ull;  // NaN and p <= 0 keep the largest
    bound = find_boundary(row, V, rs, bound, true, want, s);
  }
  auto kept = [&](int v) -> u64 {
    const float x = logit_at(row, v);
    if (!bound.keeps(logit_key(x), v)) return 0;
    if (!(x == m) && !(expf(rs.z(x)) >= min_p)) return 0;
    return rs.weight(x);
  };
  total = 0;
  for (int v = threadIdx.x; v < V; v += kSampleThreads) total += kept(v);
  total = block_sum(total, s);
  const double rd = static_cast<double>(u[b]) * static_cast<double>(total);
  u64 r = rd >= 1.0 ? static_cast<u64>(rd) : 0ull;  // NaN draws the first kept id
  if (r > total - 1) r = total - 1;
  const int id = first_past(V, r, s, kept);
  if (threadIdx.x == 0) {
    token[b] = id;
    if (logprob != nullptr)
      logprob[b] = rs.z(logit_at(row, id)) - logf(static_cast<float>(total) * 9.094947017729282e-13f);
  }
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
    sample_kernel<T><<<static_cast<unsigned>(B), kSampleThreads, 0, st>>>(static_cast<const T*>(logits),
                                                                        static_cast<int>(V), ld, u, *params, token,
                                                                        logprob);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? FKL_OK : sample_fail(FKL_ERR_CUDA, "sampler launch failed");
}
