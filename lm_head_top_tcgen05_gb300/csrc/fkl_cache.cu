// The teacher cache in few bits: fkl_cache_pack and fkl_cache_unpack (format in include/fkl_cache.h).
//
// A warp per row, a lane per slot of the 32 that share a scale: the group's largest and smallest logit are
// warp reductions, and a part's words are put together from the lanes by shuffles.  Both directions read and
// write each byte once; HBM bounds them.
#include <climits>
#include <cmath>

#include "../../include/fkl_cache.h"
#include "fkl_generate.cuh"

namespace fkl {
namespace {

constexpr int kGroup = 32;        // slots that share a scale
constexpr int kMaxK = 1024;
constexpr float kSpan = 4096.f;   // a logit further below its row's largest is stored as -inf
constexpr int kWarps = 8;

struct Format {
  int K, V, bits, id_bits, groups, code_words, id_words, words;
};

bool make_format(int64_t K, int64_t V, int32_t bits, Format* f) {
  if (K < 1 || K > kMaxK || V < 1 || V > (int64_t{1} << 30) || (bits != 4 && bits != 8)) return false;
  f->K = static_cast<int>(K);
  f->V = static_cast<int>(V);
  f->bits = bits;
  f->id_bits = 1;
  while ((int64_t{1} << f->id_bits) <= V) ++f->id_bits;  // at most 31
  f->groups = static_cast<int>((K + kGroup - 1) / kGroup);
  f->code_words = static_cast<int>((K * bits + 31) / 32);
  f->id_words = static_cast<int>((K * f->id_bits + 31) / 32);
  f->words = 2 * f->groups + f->code_words + f->id_words;
  return true;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_min(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Word `lane` of the 32 lanes' values of `width` bits (1 to 31) laid one after the other: the values
// that overlap bits [32 lane, 32 lane + 32).
__device__ __forceinline__ uint32_t gather_bits(uint32_t value, int width, int lane) {
  const int first = 32 * lane / width;  // the value that holds the word's first bit
  uint32_t word = 0;
  for (int k = 0, n = 31 / width + 2; k < n; ++k) {
    const int from = first + k;
    const uint32_t v = __shfl_sync(0xffffffffu, value, from & 31);
    const int at = from * width - 32 * lane;  // its first bit in the word
    if (from < 32 && at < 32) word |= at >= 0 ? v << at : v >> -at;
  }
  return word;
}

// The lane's value of `width` bits (1 to 31) of words that lie one to a lane.
__device__ __forceinline__ uint32_t spread_bits(uint32_t word, int width, int lane) {
  const int at = lane * width;
  const uint32_t lo = __shfl_sync(0xffffffffu, word, at >> 5), hi = __shfl_sync(0xffffffffu, word, ((at >> 5) + 1) & 31);
  return __funnelshift_r(lo, hi, at) & ((1u << width) - 1u);
}

// round((top - z) levels / (top - low)), a tie to the even one.  In fp32 the quotient is off by less than 2^-14
// of a level (four roundings of at most 254); only where that leaves the nearest level open, or per_level =
// levels / (top - low) is no number, is it taken again in fp64: there the product is exact, and so is a tie.
__device__ __forceinline__ uint32_t level_of(float top, float z, float low, float levels, float per_level) {
  const float t = (top - z) * per_level;
  float r = rintf(t);
  if (!(per_level < INFINITY) || fabsf(fabsf(t - r) - 0.5f) < 0x1p-10f) {
    const double down = static_cast<double>(top) - z, span = static_cast<double>(top) - low;
    r = static_cast<float>(rint(down * levels / span));
  }
  return static_cast<uint32_t>(fminf(fmaxf(r, 0.f), levels));
}

__global__ void __launch_bounds__(kWarps * 32)
    pack_kernel(const int32_t* __restrict__ idx, const float* __restrict__ logits, int64_t T, const Format f,
                uint32_t* __restrict__ records) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;  // uniform per warp
  const int32_t* ri = idx + t * f.K;
  const float* rz = logits + t * f.K;
  uint32_t* out = records + t * f.words;
  const float levels = static_cast<float>((1 << f.bits) - 2);
  const uint32_t none = (1u << f.bits) - 1u, no_id = (1u << f.id_bits) - 1u;

  float row_max = -INFINITY;
  bool bad = false;
  for (int k = lane; k < f.K; k += 32) {
    const float z = rz[k];
    row_max = fmaxf(row_max, z);
    bad |= !(z < INFINITY);  // NaN, +inf
  }
  row_max = warp_max(row_max);
  bad = __any_sync(0xffffffffu, bad);
  const float least = row_max - kSpan;

  for (int g = 0; g < f.groups; ++g) {
    const int k = g * kGroup + lane, slots = min(kGroup, f.K - g * kGroup);
    const bool in = lane < slots;
    const float z = in ? rz[k] : -INFINITY;
    const int id = in ? ri[k] : 0;
    const bool has = z >= least && z > -INFINITY && !bad;
    const float top = warp_max(has ? z : -INFINITY), low = warp_min(has ? z : INFINITY);
    const bool some = top > -INFINITY;
    const float span = some ? top - low : 0.f;
    if (lane == 0) {
      out[2 * g] = __float_as_uint(bad ? NAN : some ? top : 0.f);
      out[2 * g + 1] = __float_as_uint(__fdiv_rn(span, levels));
    }
    uint32_t code = none;
    if (has) code = span > 0.f ? level_of(top, z, low, levels, levels / span) : 0u;
    const uint32_t codes = gather_bits(in ? code : 0u, f.bits, lane);
    const int cw = (slots * f.bits + 31) / 32, iw = (slots * f.id_bits + 31) / 32;
    if (lane < cw) out[2 * f.groups + g * f.bits + lane] = codes;
    const uint32_t stored = id >= 0 && id < f.V ? static_cast<uint32_t>(id) : no_id;
    const uint32_t ids = gather_bits(in ? stored : 0u, f.id_bits, lane);
    if (lane < iw) out[2 * f.groups + f.code_words + g * f.id_bits + lane] = ids;
  }
}

__global__ void __launch_bounds__(kWarps * 32)
    unpack_kernel(const uint32_t* __restrict__ records, int64_t T, const Format f, int32_t* __restrict__ idx,
                  float* __restrict__ logits) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;  // uniform per warp
  const uint32_t* in = records + t * f.words;
  const uint32_t none = (1u << f.bits) - 1u;
  for (int g = 0; g < f.groups; ++g) {
    const int k = g * kGroup + lane, slots = min(kGroup, f.K - g * kGroup);
    const int cw = (slots * f.bits + 31) / 32, iw = (slots * f.id_bits + 31) / 32;
    const float top = __uint_as_float(in[2 * g]), step = __uint_as_float(in[2 * g + 1]);
    const uint32_t cword = lane < cw ? in[2 * f.groups + g * f.bits + lane] : 0u;
    const uint32_t iword = lane < iw ? in[2 * f.groups + f.code_words + g * f.id_bits + lane] : 0u;
    const uint32_t code = spread_bits(cword, f.bits, lane), id = spread_bits(iword, f.id_bits, lane);
    if (lane < slots) {
      const float z = __fsub_rn(top, __fmul_rn(static_cast<float>(code), step));
      logits[t * f.K + k] = code == none && top == top ? -INFINITY : z;
      idx[t * f.K + k] = id < static_cast<uint32_t>(f.V) ? static_cast<int32_t>(id) : -1;
    }
  }
}

fkl_status cache_fail(fkl_status st, const char* msg) {
  set_last_error_message(msg);
  return st;
}

// The checks of both directions.
fkl_status check_cache(const void* records, const void* idx, const void* logits, int64_t T, int64_t K, int64_t V,
                       int32_t bits, Format* f) {
  if (!make_format(K, V, bits, f))
    return cache_fail(FKL_ERR_INVALID_ARG, "need 1 <= K <= 1024, 1 <= V <= 2^30 and bits 4 or 8");
  if (T < 0 || T > INT32_MAX) return cache_fail(FKL_ERR_INVALID_ARG, "need 0 <= T < 2^31");
  if (T > 0 && (records == nullptr || idx == nullptr || logits == nullptr))
    return cache_fail(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((reinterpret_cast<uintptr_t>(records) | reinterpret_cast<uintptr_t>(idx) | reinterpret_cast<uintptr_t>(logits)) % 4 != 0)
    return cache_fail(FKL_ERR_ALIGNMENT, "records, topk_idx and topk_logits must be 4-byte aligned");
  int sms = 0;
  if (const int e = require_device(&sms); e != FKL_OK) return static_cast<fkl_status>(e);
  const NamedPtr ptrs[] = {{T > 0 ? records : nullptr, "records"}, {T > 0 ? idx : nullptr, "topk_idx"},
                           {T > 0 ? logits : nullptr, "topk_logits"}};
  return static_cast<fkl_status>(check_device_memory(ptrs));
}

unsigned cache_blocks(int64_t T) { return static_cast<unsigned>((T + kWarps - 1) / kWarps); }

fkl_status cache_done() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FKL_OK : cache_fail(FKL_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace
}  // namespace fkl

using namespace fkl;

extern "C" int32_t fkl_cache_words(int64_t K, int64_t V, int32_t bits) {
  Format f;
  return make_format(K, V, bits, &f) ? f.words : 0;
}

extern "C" fkl_status fkl_cache_pack(const int32_t* topk_idx, const float* topk_logits, int64_t T, int64_t K, int64_t V,
                                     int32_t bits, uint32_t* records, void* stream) {
  set_last_error_message("");
  Format f;
  const fkl_status s = check_cache(records, topk_idx, topk_logits, T, K, V, bits, &f);
  if (s != FKL_OK || T == 0) return s;
  pack_kernel<<<cache_blocks(T), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(topk_idx, topk_logits, T, f, records);
  return cache_done();
}

extern "C" fkl_status fkl_cache_unpack(const uint32_t* records, int64_t T, int64_t K, int64_t V, int32_t bits,
                                       int32_t* topk_idx, float* topk_logits, void* stream) {
  set_last_error_message("");
  Format f;
  const fkl_status s = check_cache(records, topk_idx, topk_logits, T, K, V, bits, &f);
  if (s != FKL_OK || T == 0) return s;
  unpack_kernel<<<cache_blocks(T), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(records, T, f, topk_idx, topk_logits);
  return cache_done();
}
