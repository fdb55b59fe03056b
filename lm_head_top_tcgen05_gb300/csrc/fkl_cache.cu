// The teacher cache in few bits: fkl_cache_pack and fkl_cache_unpack (format in include/fkl_cache.h).
//
// A thread per group of 32 slots: it has the group's logits in registers, so largest, smallest and codes are
// its own, and it puts words together bit by bit, at positions that are the same in every thread of the warp.  Rows
// pass through shared memory, the slots of a group 36 words from the next group's: four words at a time, eight
// threads that walk their groups together then touch all 32 banks once.  A block's rows, and its records, are
// one stretch of memory each, moved 16 bytes a thread where K and the pointers allow it, else 4.
// A lane per slot, with warp reductions for a group's range and shuffles to assemble words, was the first form: 250
// instructions to 32 slots against about 50 here, and the instructions were what it took its time for.  They
// still are (63 % of issue slots): 262144 x 100 slots in 8 bits take 62 us to write (4.9 TB/s) and 56 to read (5.4).
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/fkl_cache.h"
#include "fkl_generate.cuh"

namespace fkl {
namespace {

constexpr int kGroup = 32;        // slots that share a scale
constexpr int kMaxK = 1024;
constexpr float kSpan = 4096.f;   // a logit further below its row's largest is stored as -inf
constexpr int kThreads = 128;     // groups of a block's rows (one row at least: up to 32 groups)
constexpr int kStride = kGroup + 4;

struct Format {
  int K, V, bits, id_bits, groups, code_words, id_words, words;
  int full;  // groups of a row with all of their slots
  int rows;  // of a block: kThreads groups, and records that fit their slots' shared memory
};

bool make_format(int64_t K, int64_t V, int32_t bits, Format* f) {
  if (K < 1 || K > kMaxK || V < 1 || V > (int64_t{1} << 30) || (bits != 4 && bits != 8)) return false;
  f->K = static_cast<int>(K);
  f->V = static_cast<int>(V);
  f->bits = bits;
  f->id_bits = 1;
  while ((int64_t{1} << f->id_bits) <= V) ++f->id_bits;  // at most 31
  f->groups = static_cast<int>((K + kGroup - 1) / kGroup);
  f->full = static_cast<int>(K / kGroup);
  f->code_words = static_cast<int>((K * bits + 31) / 32);
  f->id_words = static_cast<int>((K * f->id_bits + 31) / 32);
  f->words = 2 * f->groups + f->code_words + f->id_words;
  f->rows = kThreads / f->groups;
  if (f->rows * f->words > kThreads * kStride) f->rows = kThreads * kStride / f->words;
  if (f->rows > 4) f->rows = f->rows / 4 * 4;  // whole 16-byte units of records
  return true;
}

// 4 bytes from global to shared memory by the calling thread (see copy_async_wait).
__device__ __forceinline__ void copy4_async(void* dst_smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst_smem)), "l"(src) : "memory");
}

// The level nearest to z, from the definition: in fp64 the product is exact, and so is a tie.
__device__ __noinline__ uint32_t exact_level(float top, float z, float low, float levels) {
  const double down = static_cast<double>(top) - z, span = static_cast<double>(top) - low;
  return static_cast<uint32_t>(rint(down * levels / span));
}

// A block's groups in the order of its threads: the full groups of its rows, then each row's last, shorter one, so that
// whole warps have the short ones and stop early.
struct Task {
  int r, g, slots;
  __device__ __forceinline__ Task(const Format& f, int rows) {
    const int tid = static_cast<int>(threadIdx.x), fulls = f.rows * f.full;
    r = tid < fulls ? tid / f.full : tid - fulls;
    g = tid < fulls ? tid - r * f.full : f.full;
    slots = r < rows ? max(min(kGroup, f.K - g * kGroup), 0) : 0;
  }
};
__device__ __forceinline__ int task_of(const Format& f, int r, int g) { return g < f.full ? r * f.full + g : f.rows * f.full + r; }

// Calls f(unit, place) for the thread's share of a block's slots, which are one stretch of memory: units of kUnit
// slots, and where the unit lies among the groups in shared memory.
template <int kUnit, class F>
__device__ __forceinline__ void for_slots(const Format& f, int rows, F&& fn) {
  const int per_row = f.K / kUnit, units = rows * per_row;
  const int rows_on = kThreads / per_row, on = kThreads - rows_on * per_row;  // what a step of kThreads units moves
  int r = static_cast<int>(threadIdx.x) / per_row, k = static_cast<int>(threadIdx.x) - r * per_row;
  for (int u = static_cast<int>(threadIdx.x); u < units; u += kThreads) {
    const int slot = k * kUnit;
    fn(u * kUnit, task_of(f, r, slot / kGroup) * kStride + slot % kGroup);
    r += rows_on;
    k += on;
    if (k >= per_row) {
      k -= per_row;
      ++r;
    }
  }
}

// kVec: K, the pointers and a block's records are whole 16-byte units (`whole_units` below).
template <int kBits, bool kVec>
__global__ void __launch_bounds__(kThreads, 6)
    pack_kernel(const int32_t* __restrict__ idx, const float* __restrict__ logits, int64_t T, const Format f,
                uint32_t* __restrict__ records) {
  __shared__ __align__(16) float z_part[kThreads * kStride];  // logits by group, then the records
  __shared__ __align__(16) int32_t id_part[kThreads * kStride];
  __shared__ float group_max[kThreads];
  constexpr float kLevels = static_cast<float>((1 << kBits) - 2);
  constexpr uint32_t kNone = (1u << kBits) - 1u;
  constexpr int kPerWord = 32 / kBits;
  const int tid = static_cast<int>(threadIdx.x);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * f.rows;
  const int rows = static_cast<int>(T - t0 < f.rows ? T - t0 : f.rows);
  const Task task(f, rows);
  const int r = task.r, g = task.g, slots = task.slots, quads = (slots + 3) / 4;
  const bool on = slots > 0;
  const float* zr = logits + t0 * f.K;
  const int32_t* ir = idx + t0 * f.K;
  for_slots<kVec ? 4 : 1>(f, rows, [&](int i, int at) {
    if (kVec) {
      copy16_async(z_part + at, zr + i);
      copy16_async(id_part + at, ir + i);
    } else {
      copy4_async(z_part + at, zr + i);
      copy4_async(id_part + at, ir + i);
    }
  });
  for (int j = slots; j < 4 * quads; ++j) z_part[tid * kStride + j] = -INFINITY;  // behind the row's last slot
  copy_async_wait();
  __syncthreads();

  const float4* mine = reinterpret_cast<const float4*>(&z_part[tid * kStride]);
  // Calls fn(j, slots 4 j to 4 j + 3), straight through in a warp of full groups.
  const bool fulls = __all_sync(0xffffffffu, quads == kGroup / 4);
  auto for_quads = [&](auto&& fn) {
    if (fulls) {
#pragma unroll
      for (int j = 0; j < kGroup / 4; ++j) fn(j, mine[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kGroup / 4; ++j) {
        if (j >= quads) break;
        fn(j, mine[j]);
      }
    }
  };
  float largest = -INFINITY;
  for_quads([&](int, const float4& v) { largest = max_nan(max_nan(largest, max_nan(v.x, v.y)), max_nan(v.z, v.w)); });
  group_max[tid] = largest;
  __syncthreads();
  float row_max = -INFINITY;
  if (on)
    for (int i = 0; i < f.groups; ++i) row_max = max_nan(row_max, group_max[task_of(f, r, i)]);
  const bool bad = !(row_max < INFINITY);                               // a NaN or +inf
  const float least = fmaxf(row_max - kSpan, -3.40282347e38f);          // -inf does not reach it
  const bool some = !bad && largest >= least;
  float low = INFINITY;
  for_quads([&](int, const float4& v) {
    low = fminf(fminf(low, v.x >= least ? v.x : INFINITY), v.y >= least ? v.y : INFINITY);
    low = fminf(fminf(low, v.z >= least ? v.z : INFINITY), v.w >= least ? v.w : INFINITY);
  });
  const float top = some ? largest : 0.f, span = some ? top - low : 0.f;
  const float floor = some ? least : NAN;  // no slot reaches it where there is none
  const float per_level = span > 0.f ? kLevels / span : 0.f;
  // Nearest levels: adding 1.5 2^23 leaves the whole number in a float's low bits, and the words are sums of
  // those floats' bits in their places, less the bits of 1.5 2^23.  In fp32 the quotient is off by less
  // than four roundings of at most kLevels; the slots (`open`) that this leaves between two levels, and all where
  // levels / span is no number, are decided in fp64.
  constexpr float kRound = 12582912.f;
  constexpr uint32_t kRoundBits = 0x4B400000u;
  constexpr float kNear = 0.5f - kLevels * 0x1p-21f;
  auto level = [&](float x, float& t) {  // each operation rounded by itself: both calls give the same bits
    t = __fmul_rn(__fsub_rn(top, x), per_level);
    return __fadd_rn(t, kRound);
  };
  uint32_t codes[kBits], open = 0;
#pragma unroll
  for (int w = 0; w < kBits; ++w) codes[w] = 0;
  for_quads([&](int quad, const float4& v) {
    const float x[4] = {v.x, v.y, v.z, v.w};
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t;
      const float n = level(x[i], t);
      const bool has = x[i] >= floor;
      if (has && !(fabsf(t - (n - kRound)) < kNear)) open |= 1u << (quad * 4 + i);
      word += ((has ? __float_as_uint(n) : kRoundBits + kNone) - kRoundBits) << (i * kBits);
    }
    codes[quad * 4 / kPerWord] += word << (quad * 4 % kPerWord * kBits);
  });
  while (open != 0) {
    const int j = __ffs(open) - 1;
    open &= open - 1;
    const float x = z_part[tid * kStride + j];
    float t;
    const uint32_t fix = (exact_level(top, x, low, kLevels) - (__float_as_uint(level(x, t)) - kRoundBits)) << (j % kPerWord * kBits);
#pragma unroll
    for (int w = 0; w < kBits; ++w) codes[w] += w == j / kPerWord ? fix : 0u;
  }
  __syncthreads();  // the logits are read: their memory is free for the records
  if (on) {
    uint32_t* out = reinterpret_cast<uint32_t*>(z_part) + r * f.words;
    out[2 * g] = __float_as_uint(bad ? NAN : top);
    out[2 * g + 1] = __float_as_uint(__fdiv_rn(span, kLevels));
#pragma unroll
    for (int w = 0; w < kBits; ++w) {
      const int bits = slots * kBits - w * 32;  // of the word that slots have
      if (bits > 0) out[2 * f.groups + g * kBits + w] = bits < 32 ? codes[w] & ((1u << bits) - 1u) : codes[w];
    }
    const uint32_t no_id = (1u << f.id_bits) - 1u, V = static_cast<uint32_t>(f.V);
    uint32_t* to = out + 2 * f.groups + f.code_words + g * f.id_bits;
    uint64_t held = 0;
    int fill = 0;
    auto put = [&](uint32_t id) {
      held += static_cast<uint64_t>(id < V ? id : no_id) * (1u << fill);
      fill += f.id_bits;
      if (fill >= 32) {
        *to++ = static_cast<uint32_t>(held);
        held >>= 32;
        fill -= 32;
      }
    };
    const int32_t* from = &id_part[tid * kStride];
    int j = 0;
    for (; j + 4 <= slots; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(from + j);
      put(v.x);
      put(v.y);
      put(v.z);
      put(v.w);
    }
    for (; j < slots; ++j) put(static_cast<uint32_t>(from[j]));
    if (fill > 0) *to = static_cast<uint32_t>(held);
  }
  __syncthreads();
  uint32_t* record = records + t0 * f.words;
  const int total = rows * f.words;
  int done = 0;
  if (kVec) {
    done = total / 4 * 4;
    for (int i = tid * 4; i < done; i += kThreads * 4)
      *reinterpret_cast<uint4*>(record + i) = *reinterpret_cast<const uint4*>(z_part + i);
  }
  for (int i = done + tid; i < total; i += kThreads) record[i] = __float_as_uint(z_part[i]);
}

template <int kBits, bool kVec>
__global__ void __launch_bounds__(kThreads, 6)
    unpack_kernel(const uint32_t* __restrict__ records, int64_t T, const Format f, int32_t* __restrict__ idx,
                  float* __restrict__ logits) {
  __shared__ __align__(16) uint32_t part[kThreads * kStride];  // the records, then the logits by group
  __shared__ __align__(16) int32_t id_part[kThreads * kStride];
  constexpr uint32_t kNone = (1u << kBits) - 1u;
  constexpr int kPerWord = 32 / kBits;
  const int tid = static_cast<int>(threadIdx.x);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * f.rows;
  const int rows = static_cast<int>(T - t0 < f.rows ? T - t0 : f.rows);
  const uint32_t* record = records + t0 * f.words;
  const int total = rows * f.words;
  int done = 0;
  if (kVec) {
    done = total / 4 * 4;
    for (int i = tid * 4; i < done; i += kThreads * 4) copy16_async(part + i, record + i);
  }
  for (int i = done + tid; i < total; i += kThreads) copy4_async(part + i, record + i);
  copy_async_wait();
  __syncthreads();

  const Task task(f, rows);
  const int r = task.r, g = task.g, slots = task.slots;
  float top = 0.f, step = 0.f;
  uint32_t codes[kBits];
  if (slots > 0) {
    const uint32_t* in = part + r * f.words;
    top = __uint_as_float(in[2 * g]);
    step = __uint_as_float(in[2 * g + 1]);
#pragma unroll
    for (int w = 0; w < kBits; ++w) codes[w] = w * 32 < slots * kBits ? in[2 * f.groups + g * kBits + w] : 0u;
    const uint32_t* from = in + 2 * f.groups + f.code_words + g * f.id_bits;
    const uint32_t mask = (1u << f.id_bits) - 1u, V = static_cast<uint32_t>(f.V);
    uint64_t held = 0;
    int fill = 0;
    auto take = [&]() {
      if (fill < f.id_bits) {
        held += static_cast<uint64_t>(*from++) * (1u << fill);
        fill += 32;
      }
      const uint32_t id = static_cast<uint32_t>(held) & mask;
      held >>= f.id_bits;
      fill -= f.id_bits;
      return id < V ? static_cast<int32_t>(id) : -1;
    };
    int32_t* to = &id_part[tid * kStride];
    int j = 0;
    for (; j + 4 <= slots; j += 4) {
      int4 v;
      v.x = take();
      v.y = take();
      v.z = take();
      v.w = take();
      *reinterpret_cast<int4*>(to + j) = v;
    }
    for (; j < slots; ++j) to[j] = take();
  }
  __syncthreads();  // every record is read: its memory is free for the logits
  if (slots > 0) {
    float* z = reinterpret_cast<float*>(part) + tid * kStride;
    const float none = top == top ? -INFINITY : NAN;
#pragma unroll
    for (int j = 0; j < kGroup; j += 4) {
      if (j >= slots) break;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t code = codes[(j + i) / kPerWord] >> ((j + i) % kPerWord * kBits) & kNone;
        // 2^23 + code has the code in its low bits: a subtraction instead of a conversion
        const float level = __uint_as_float(0x4B000000u | code) - 8388608.f;
        v[i] = code == kNone ? none : __fsub_rn(top, __fmul_rn(level, step));
      }
      *reinterpret_cast<float4*>(z + j) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  __syncthreads();
  float* zr = logits + t0 * f.K;
  int32_t* ir = idx + t0 * f.K;
  for_slots<kVec ? 4 : 1>(f, rows, [&](int i, int at) {
    if (kVec) {
      *reinterpret_cast<uint4*>(zr + i) = *reinterpret_cast<const uint4*>(part + at);
      *reinterpret_cast<int4*>(ir + i) = *reinterpret_cast<const int4*>(id_part + at);
    } else {
      zr[i] = __uint_as_float(part[at]);
      ir[i] = id_part[at];
    }
  });
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

unsigned cache_blocks(int64_t T, const Format& f) { return static_cast<unsigned>((T + f.rows - 1) / f.rows); }

// Whether rows of slots and the blocks' records start and end at 16-byte units.
bool whole_units(const Format& f, const void* records, const void* idx, const void* logits) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(records) | reinterpret_cast<uintptr_t>(idx) | reinterpret_cast<uintptr_t>(logits);
  return all % 16 == 0 && f.K % 4 == 0 && f.rows * f.words % 4 == 0;
}

// Calls fn with the two template arguments of a kernel as constants.
template <class F>
void with_variant(const Format& f, bool vec, F&& fn) {
  using yes = std::true_type;
  using no = std::false_type;
  if (f.bits == 8) {
    if (vec) fn(std::integral_constant<int, 8>{}, yes{}); else fn(std::integral_constant<int, 8>{}, no{});
  } else {
    if (vec) fn(std::integral_constant<int, 4>{}, yes{}); else fn(std::integral_constant<int, 4>{}, no{});
  }
}

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
  with_variant(f, whole_units(f, records, topk_idx, topk_logits), [&](auto b, auto vec) {
    pack_kernel<decltype(b)::value, decltype(vec)::value>
        <<<cache_blocks(T, f), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(topk_idx, topk_logits, T, f, records);
  });
  return cache_done();
}

extern "C" fkl_status fkl_cache_unpack(const uint32_t* records, int64_t T, int64_t K, int64_t V, int32_t bits,
                                       int32_t* topk_idx, float* topk_logits, void* stream) {
  set_last_error_message("");
  Format f;
  const fkl_status s = check_cache(records, topk_idx, topk_logits, T, K, V, bits, &f);
  if (s != FKL_OK || T == 0) return s;
  with_variant(f, whole_units(f, records, topk_idx, topk_logits), [&](auto b, auto vec) {
    unpack_kernel<decltype(b)::value, decltype(vec)::value>
        <<<cache_blocks(T, f), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(records, T, f, topk_idx, topk_logits);
  });
  return cache_done();
}
