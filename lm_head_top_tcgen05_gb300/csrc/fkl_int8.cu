// The 8-bit product of a generation step (fkl_quantize_int8, fkl_int8_matmul,
// fkl_int8_linear).
//
//     s_m = max_k |x_mk| * fl(1/127),  q_mk = rint(x_mk / s_m)
//     y_mn = (sum_k q_mk w_nk) * s_m * t_n
//
// Up to 4 tokens run on the kernel below, which streams W through registers; more, or tokens
// too long for shared memory, on the tensor cores (fkl_int8_gemm.cu).  W 201088 x 2880 on a GB300:
// 1 token 84 us (86 us is W at the measured copy bandwidth), 4 tokens 90 us; with 8 tokens the
// streaming kernel took 123 us, bound by its reads of the tokens from shared memory, and the
// tensor cores take 103 to 106 us.
#include <climits>

#include "../../include/fkl_testing.h"
#include "fkl_gemm.cuh"
#include "fkl_generate.cuh"
#include "fkl_int8.h"
#include "fkl_types.cuh"

namespace fkl {

constexpr int64_t kMaxInt8K = 131072;
// Largest M and N: a tile of 256 tokens or channels more stays an int.
constexpr int64_t kMaxInt8Extent = INT32_MAX - 511;

// ---------------------------------------------------------------- quantisation
constexpr uint32_t kInfBits = 0x7f800000u;

// Scale of a row whose largest magnitude has the bits amax; NaN when the row holds a NaN or an
// infinity (their bits exceed every finite magnitude's).
__device__ __forceinline__ float row_scale(uint32_t amax) {
  return amax >= kInfBits ? __uint_as_float(0x7fc00000u) : __uint_as_float(amax) * (1.0f / 127.0f);
}
// The scale of a row and how its values are rounded.  The definition divides (IEEE) and rounds to
// nearest even; a product with 1/s is within 2^-23 of the quotient, relative, at most 1.6e-5 for
// quotients up to 127.  So the rounded product is the answer unless it lies within 1e-4 of a
// tie; only then (and for scales whose reciprocal is not an ordinary number) is the division
// made.  8192 x 4096 values took 40 us with divisions alone.
struct RowQuant {
  float s, inv;
  bool plain;
  __device__ explicit RowQuant(float scale)
      : s(scale), inv(1.0f / scale), plain(scale > 7.8886e-31f && scale < 1.2676e30f) {}  // 2^-100 .. 2^100
  // A whole number in [-127, 127]; 0 for s = 0 (a row of zeros, or of values whose scale underflows)
  // and s = NaN.
  __device__ __forceinline__ float operator()(float x) const {
    const float t = x * inv;
    float q = (t + 12582912.f) - 12582912.f;  // 1.5 * 2^23: rounds to nearest even
    if (!plain || fabsf(t - q) > 0.4999f) q = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f) : 0.f;
    return q;
  }
};

// Four whole numbers in [-128, 127] as bytes, or (for the tensor cores) as fp16.
__device__ __forceinline__ void put4(int8_t* o, const float (&q)[4]) {
  uint32_t w[4];  // the low byte of 1.5 * 2^23 + q
#pragma unroll
  for (int b = 0; b < 4; ++b) w[b] = __float_as_uint(q[b] + 12582912.f);
  *reinterpret_cast<uint32_t*>(o) = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}
__device__ __forceinline__ void put4(__half* o, const float (&q)[4]) {
  *reinterpret_cast<uint2*>(o) = make_uint2(pack2<__half>(q[0], q[1]), pack2<__half>(q[2], q[3]));
}

// One block per row.  A thread's first kHeld vectors (16 bytes) stay in registers between the
// two passes; the rest of a longer row is read twice, the second time from cache.  The IEEE
// division keeps the integers equal to the definition's.  Block 0 zeroes `hdr`, if there is one.
template <class T, class Q, bool kVec, int kQuantThreads>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_kernel(const T* __restrict__ x, int64_t cols, int64_t ldx, Q* __restrict__ q, float* __restrict__ scale,
                    uint4* __restrict__ hdr) {
  constexpr int E = 16 / sizeof(T), kHeld = 4;
  __shared__ uint32_t warp_max[kQuantThreads / 32];
  if (hdr != nullptr) launch_dependents();  // the product follows
  const T* row = x + static_cast<int64_t>(blockIdx.x) * ldx;
  const uint4* rowv = reinterpret_cast<const uint4*>(row);
  Q* out = q + static_cast<int64_t>(blockIdx.x) * cols;
  const int64_t vecs = kVec ? cols / E : 0;
  uint32_t amax = 0;
  uint4 held[kHeld];
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int64_t i = threadIdx.x + h * kQuantThreads;
    held[h] = i < vecs ? rowv[i] : make_uint4(0, 0, 0, 0);
  }
  if (hdr != nullptr && blockIdx.x == 0)
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(Int8Header) / 16); i += kQuantThreads)
      hdr[i] = make_uint4(0, 0, 0, 0);
  auto largest = [&](const uint4& raw) {
    float v[E];
    unpack16<T>(raw, v);
#pragma unroll
    for (int j = 0; j < E; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) largest(held[h]);
  for (int64_t i = threadIdx.x + kHeld * kQuantThreads; i < vecs; i += kQuantThreads) largest(rowv[i]);
  if (!kVec)
    for (int64_t i = threadIdx.x; i < cols; i += kQuantThreads)
      amax = max(amax, __float_as_uint(to_float(row[i])) & 0x7fffffffu);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = 0;
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) amax = max(amax, warp_max[w]);
  const RowQuant quantize(row_scale(amax));
  if (threadIdx.x == 0) scale[blockIdx.x] = quantize.s;
  auto put = [&](const uint4& raw, int64_t i) {
    float v[E];
    unpack16<T>(raw, v);
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
      float w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) w[b] = quantize(v[4 * j + b]);
      put4(out + i * E + 4 * j, w);
    }
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int64_t i = threadIdx.x + h * kQuantThreads;
    if (i < vecs) put(held[h], i);
  }
  for (int64_t i = threadIdx.x + kHeld * kQuantThreads; i < vecs; i += kQuantThreads) put(rowv[i], i);
  if (!kVec)
    for (int64_t i = threadIdx.x; i < cols; i += kQuantThreads)
      out[i] = static_cast<Q>(quantize(to_float(row[i])));
}

template <class Q>
static cudaError_t launch_quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ldx, Q* q,
                                   float* scale, Int8Header* hdr, cudaStream_t st) {
  return with_type(type, [&](auto t) {
    using T = decltype(t);
    const T* p = static_cast<const T*>(x);
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * sizeof(T) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(q) % (4 * sizeof(Q)) == 0 && cols % 16 == 0;
    uint4* h = reinterpret_cast<uint4*>(hdr);
    const unsigned n = static_cast<unsigned>(rows);
    // Many rows: small blocks keep more bytes in flight per SM (8192 x 4096: 27 us against 35).  Few
    // rows: larger blocks finish a row sooner (9 x 2880: 3.5 us against 5.2).
    if (rows >= 2048) {
      if (vec)
        quantize_kernel<T, Q, true, 128><<<n, 128, 0, st>>>(p, cols, ldx, q, scale, h);
      else
        quantize_kernel<T, Q, false, 128><<<n, 128, 0, st>>>(p, cols, ldx, q, scale, h);
    } else {
      if (vec)
        quantize_kernel<T, Q, true, 256><<<n, 256, 0, st>>>(p, cols, ldx, q, scale, h);
      else
        quantize_kernel<T, Q, false, 256><<<n, 256, 0, st>>>(p, cols, ldx, q, scale, h);
    }
    return cudaGetLastError();
  });
}

// Tokens that are in 8 bits already, as fp16 for the tensor cores, and an aligned copy of their
// scales; zeroes `hdr`.
__global__ void __launch_bounds__(256)
    widen_kernel(const uint32_t* __restrict__ xq, int64_t words, uint2* __restrict__ x16,
                 const float* __restrict__ x_scale, int M, float* __restrict__ scale, uint4* __restrict__ hdr) {
  launch_dependents();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t i = i0; i < M; i += static_cast<int64_t>(gridDim.x) * 256) scale[i] = x_scale[i];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(Int8Header) / 16); i += 256) hdr[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = i0; i < words; i += static_cast<int64_t>(gridDim.x) * 256) {
    const uint32_t w = xq[i];
    float q[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) q[b] = static_cast<float>(static_cast<int8_t>(w >> (8 * b)));
    put4(reinterpret_cast<__half*>(x16 + i), q);
  }
}

// Test hook: holds the product's tokens back for `ns` while the product runs (fkl_testing.h).
__global__ void late_kernel(uint64_t ns) {
  launch_dependents();
  const uint64_t t0 = global_timer_ns();
  for (int i = 0; i < (1 << 21) && global_timer_ns() - t0 < ns; ++i) __nanosleep(1000);
}

// ---------------------------------------------------------------- few tokens: dp4a
// Each warp streams rows of W through registers, 16 bytes a lane, against the tokens' integers in
// shared memory; the sums are exact int32.  Bound by reading W, so what counts is bytes in flight:
// 2 rows x 3 pieces per lane (96 KB per SM) took 85.0 us for one token, 4 rows x 1 piece 89.5 us
// (201088 x 2880).  Every block brings the tokens to 8 bits for itself (they come from L2), so a
// call is one launch; the first rows' pieces are under way meanwhile.
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int64_t kFewTokens = 4;
constexpr int64_t kFewSmem = 96 * 1024;  // two blocks to an SM
static_assert(128 * 128 * kFewSmem <= INT32_MAX, "the int32 sums of K <= kFewSmem products do not overflow");

// V values per lane, summed over the lanes: lane l gets the sum of value l * V / 32 (V < 32: of
// the value whose 32 / V lanes it is one of).
template <int V>
__device__ __forceinline__ int reduce_over_lanes(int (&v)[V], int lane) {
  static_assert(V <= 32 && (V & (V - 1)) == 0, "a power of two up to 32");
  int n = V;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (i < n) {
          const int give = up ? v[i] : v[i + n];
          const int keep = up ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return v[0];
}

struct FewParams {
  const void* x;  // float types of x_type with rows ldx apart, or (x_scale given) int8 [M][K]
  const float* x_scale;
  int64_t ldx;
  int x_type, vec;
  const int8_t* wq;
  const float* w_scale;
  void* out;
  int64_t ldo;
  int out_type;
  int M, N, K;
  uint4* hdr;
};

// The tokens' integers into shared memory: kFewWarps / MT warps per token.  A thread's first
// kHeld vectors stay in registers between the two passes.
template <int MT, class T>
__device__ void few_quantize(const FewParams& p, int8_t* sq, float* ss, uint32_t* warp_max) {
  constexpr int W = kFewWarps / MT, E = 16 / sizeof(T), kHeld = 2;
  const int warp = threadIdx.x >> 5, m = warp / W;
  const int at = threadIdx.x - m * W * 32;
  const T* row = static_cast<const T*>(p.x) + static_cast<int64_t>(m) * p.ldx;
  const bool live = m < p.M;
  const int vecs = live && p.vec ? p.K / E : 0;
  uint32_t amax = 0;
  uint4 held[kHeld];
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    held[h] = at + h * W * 32 < vecs ? reinterpret_cast<const uint4*>(row)[at + h * W * 32] : make_uint4(0, 0, 0, 0);
  auto largest = [&](const uint4& raw) {
    float v[E];
    unpack16<T>(raw, v);
#pragma unroll
    for (int j = 0; j < E; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) largest(held[h]);
  for (int i = at + kHeld * W * 32; i < vecs; i += W * 32) largest(reinterpret_cast<const uint4*>(row)[i]);
  if (live && !p.vec)
    for (int i = at; i < p.K; i += W * 32) amax = max(amax, __float_as_uint(to_float(row[i])) & 0x7fffffffu);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) warp_max[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) amax = max(amax, warp_max[m * W + w]);
  const RowQuant quantize(live ? row_scale(amax) : 0.f);
  if (at == 0) ss[m] = quantize.s;
  int8_t* out = sq + static_cast<int64_t>(m) * p.K;
  auto put = [&](const uint4& raw, int i) {
    float v[E];
    unpack16<T>(raw, v);
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
      float q[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) q[b] = quantize(v[4 * j + b]);
      put4(out + i * E + 4 * j, q);
    }
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (at + h * W * 32 < vecs) put(held[h], at + h * W * 32);
  for (int i = at + kHeld * W * 32; i < vecs; i += W * 32) put(reinterpret_cast<const uint4*>(row)[i], i);
  if (!live || !p.vec)
    for (int i = at; i < p.K; i += W * 32) out[i] = live ? static_cast<int8_t>(quantize(to_float(row[i]))) : 0;
}

template <class T>
__device__ __forceinline__ void few_store(const FewParams& p, int m, int n, float y) {
  static_cast<T*>(p.out)[static_cast<int64_t>(m) * p.ldo + n] = from_float<T>(y);
}

template <int MT, int R>
__device__ __forceinline__ void few_dot(int (&acc)[MT * R], const uint4 (&wv)[R], const uint4* xs, int chunks, int c) {
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const uint4 xv = xs[m * chunks + c];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int a = acc[m * R + r];
      a = __dp4a(static_cast<int>(wv[r].x), static_cast<int>(xv.x), a);
      a = __dp4a(static_cast<int>(wv[r].y), static_cast<int>(xv.y), a);
      a = __dp4a(static_cast<int>(wv[r].z), static_cast<int>(xv.z), a);
      acc[m * R + r] = __dp4a(static_cast<int>(wv[r].w), static_cast<int>(xv.w), a);
    }
  }
}

// MT tokens (those past M are zero), R rows of W per warp at a time, H 16-byte pieces of each row
// in flight per lane.  The first rows' pieces are loaded before the tokens are brought to 8 bits.
template <int MT, int R, int H>
__global__ void __launch_bounds__(kFewThreads, 2) few_tokens_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(16) int8_t sq[];  // [MT][K]
  __shared__ float ss[MT];
  __shared__ uint32_t warp_max[kFewWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.N + R - 1) / R, step = static_cast<int>(gridDim.x) * kFewWarps;
  const int chunks = p.K / 16;
  int g = static_cast<int>(blockIdx.x) * kFewWarps + warp;
  uint4 held[H][R];
  auto load = [&](int c0) {  // rows past N read the last one; their sums are not stored
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int c = c0 + 32 * h;
#pragma unroll
      for (int r = 0; r < R; ++r)
        held[h][r] = c < chunks
                         ? __ldcs(reinterpret_cast<const uint4*>(p.wq + static_cast<int64_t>(min(g * R + r, p.N - 1)) * p.K) + c)
                         : make_uint4(0, 0, 0, 0);
    }
  };
  if (g < groups) load(lane);
  if (blockIdx.x == 0 && threadIdx.x < 16) p.hdr[threadIdx.x] = make_uint4(0, 0, 0, 0);
  if (p.x_scale != nullptr) {
    const uint4* src = static_cast<const uint4*>(p.x);
    for (int i = threadIdx.x; i < MT * chunks; i += kFewThreads)
      reinterpret_cast<uint4*>(sq)[i] = i < p.M * chunks ? src[i] : make_uint4(0, 0, 0, 0);
    if (threadIdx.x < MT) ss[threadIdx.x] = static_cast<int>(threadIdx.x) < p.M ? p.x_scale[threadIdx.x] : 0.f;
  } else if (p.x_type == FKL_TYPE_F32) {
    few_quantize<MT, float>(p, sq, ss, warp_max);
  } else if (p.x_type == FKL_TYPE_BF16) {
    few_quantize<MT, __nv_bfloat16>(p, sq, ss, warp_max);
  } else {
    few_quantize<MT, __half>(p, sq, ss, warp_max);
  }
  __syncthreads();

  const uint4* xs = reinterpret_cast<const uint4*>(sq);
  while (g < groups) {
    int acc[MT * R] = {};
    const int row0 = g * R;
    for (int c0 = lane;;) {
#pragma unroll
      for (int h = 0; h < H; ++h) few_dot<MT, R>(acc, held[h], xs, chunks, min(c0 + 32 * h, chunks - 1));
      c0 += 32 * H;
      if (c0 - lane >= chunks) break;
      load(c0);
    }
    g += step;
    if (g < groups) load(lane);  // the next rows' pieces, while this group's sums are finished
    const int sum = reduce_over_lanes<MT * R>(acc, lane);
    constexpr int kLanes = 32 / (MT * R);  // lanes that hold the same sum
    const int i = lane / kLanes, m = i / R, n = row0 + i % R;
    if (lane % kLanes == 0 && m < p.M && n < p.N) {
      const float y = static_cast<float>(sum) * ss[m] * p.w_scale[n];
      if (p.out_type == FKL_TYPE_F32)
        few_store<float>(p, m, n, y);
      else if (p.out_type == FKL_TYPE_BF16)
        few_store<__nv_bfloat16>(p, m, n, y);
      else
        few_store<__half>(p, m, n, y);
    }
  }
}

template <int MT, int R, int H>
static cudaError_t launch_few_t(const FewParams& p, int sms, cudaStream_t st) {
  static bool done[128];
  const size_t smem = static_cast<size_t>(MT) * p.K;
  const cudaError_t e = smem_limit_once(few_tokens_kernel<MT, R, H>, kFewSmem, done);
  if (e != cudaSuccess) return e;
  const int blocks = ((p.N + R - 1) / R + kFewWarps - 1) / kFewWarps;
  few_tokens_kernel<MT, R, H><<<blocks < 2 * sms ? blocks : 2 * sms, kFewThreads, smem, st>>>(p);
  return cudaGetLastError();
}

// Two rows of W per warp share each read of the tokens; with fewer rows than keep every warp busy
// four times over, one row per warp with more of its pieces in flight.
template <int MT>
static cudaError_t launch_few_m(const FewParams& p, int sms, cudaStream_t st) {
  return p.N < 4 * 2 * kFewWarps * sms ? launch_few_t<MT, 1, MT == 4 ? 4 : 6>(p, sms, st)
                                       : launch_few_t<MT, 2, 3>(p, sms, st);
}

static int few_rounded(int64_t M) { return M <= 1 ? 1 : M <= 2 ? 2 : 4; }

static bool few_tokens(int64_t M, int64_t K) { return M <= kFewTokens && few_rounded(M) * K <= kFewSmem; }

static cudaError_t launch_few(const FewParams& p, int sms, cudaStream_t st) {
  switch (few_rounded(p.M)) {
    case 1: return launch_few_m<1>(p, sms, st);
    case 2: return launch_few_m<2>(p, sms, st);
    default: return launch_few_m<4>(p, sms, st);
  }
}

// ---------------------------------------------------------------- host side
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Int8Plan {
  bool few;
  Int8GemmPlan gemm;
  size_t off_x16, off_scale, off_part, total;
};

// The workspace for a device of `sms` SMs.
static bool make_int8_plan(int64_t M, int64_t N, int64_t K, int sms, Int8Plan* p) {
  if (M < 0 || M > kMaxInt8Extent || N < 1 || N > kMaxInt8Extent || K < 16 || K % 16 != 0 || K > kMaxInt8K) return false;
  if ((M + 127) / 128 * ((N + 255) / 256) > INT32_MAX) return false;  // tiles
  p->few = few_tokens(M, K);
  size_t off = p->few ? 256 : up256(sizeof(Int8Header));  // few tokens: the status word's 256 bytes
  p->off_x16 = p->off_scale = p->off_part = off;
  if (!p->few) {
    p->gemm = plan_int8_gemm(M, N, K, sms);
    off = up256(off + static_cast<size_t>(M) * K * 2);
    p->off_scale = off;
    off = up256(off + static_cast<size_t>(M) * 4);
    p->off_part = off;
    off = up256(off + p->gemm.part_bytes);
  }
  p->total = off;
  return true;
}

// Bytes on the current device (the partial sums grow with the number of its SMs; a GB300's 152
// are assumed when no device is visible).
static size_t int8_workspace(int64_t M, int64_t N, int64_t K) {
  int sms = 0;
  if (require_device(&sms) != FKL_OK) {
    sms = 152;
    set_last_error_message("");
  }
  Int8Plan p;
  return make_int8_plan(M, N, K, sms, &p) ? p.total : 0;
}

static fkl_status bad(fkl_status s, const char* msg) {
  set_last_error_message(msg);
  return s;
}

static bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace fkl

using namespace fkl;

extern "C" fkl_status fkl_quantize_int8(const void* x, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                                        int8_t* q, float* scale, void* stream) {
  set_last_error_message("");
  if (!type_ok(x_type)) return bad(FKL_ERR_INVALID_ARG, "x_type must be one of FKL_TYPE_*");
  if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > INT32_MAX || ldx < cols)
    return bad(FKL_ERR_INVALID_ARG, "need 0 <= rows < 2^31, 1 <= cols < 2^31 and ldx >= cols");
  if (rows > 0 && (x == nullptr || q == nullptr || scale == nullptr))
    return bad(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (misaligned(x, type_bytes(x_type)) || misaligned(scale, 4))
    return bad(FKL_ERR_ALIGNMENT, "x and scale must be aligned to their elements");
  int sms = 0;
  if (const int s = require_device(&sms); s != FKL_OK) return static_cast<fkl_status>(s);
  if (rows == 0) return FKL_OK;
  const NamedPtr ptrs[] = {{x, "x"}, {q, "q"}, {scale, "scale"}};
  if (const int s = check_device_memory(ptrs); s != FKL_OK) return static_cast<fkl_status>(s);
  if (launch_quantize(x, x_type, rows, cols, ldx, q, scale, nullptr, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return bad(FKL_ERR_CUDA, "quantisation launch failed");
  return FKL_OK;
}

extern "C" size_t fkl_int8_matmul_workspace_size(int64_t M, int64_t N, int64_t K) { return int8_workspace(M, N, K); }

extern "C" size_t fkl_int8_linear_workspace_size(int64_t M, int64_t N, int64_t K) { return int8_workspace(M, N, K); }

namespace fkl {

// Both products; x_type < 0: x is int8 [M][K] with the scales x_scale.  limit_ns: of each wait of the
// tensor-core kernel; late_ns: what a test holds the tokens back.
static fkl_status int8_product(const char* x_name, const void* x, int32_t x_type, int64_t ldx, const float* x_scale,
                               const int8_t* wq, const float* w_scale, const Int8Shape& g, int32_t out_type, void* out,
                               void* workspace, size_t ws_bytes, void* stream, uint64_t limit_ns = kWaitLimitNs,
                               uint64_t late_ns = 0) {
  const bool given = x_type < 0;
  if (!type_ok(out_type)) return bad(FKL_ERR_INVALID_ARG, "out_type must be one of FKL_TYPE_*");
  const size_t need = int8_workspace(g.M, g.N, g.K);
  if (need == 0)
    return bad(FKL_ERR_INVALID_ARG, "unsupported shape (need K % 16 == 0, 16 <= K <= 131072, 0 <= M <= 2^31 - 512, 1 <= N <= 2^31 - 512)");
  if (g.ldo < g.N) return bad(FKL_ERR_INVALID_ARG, "ldo must be at least N");
  if (wq == nullptr || w_scale == nullptr ||
      (g.M > 0 && (x == nullptr || out == nullptr || (given && x_scale == nullptr))))
    return bad(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (misaligned(wq, 16) || misaligned(x, given ? 16 : type_bytes(x_type)) || misaligned(x_scale, 4) ||
      misaligned(w_scale, 4) || misaligned(out, type_bytes(out_type)))
    return bad(FKL_ERR_ALIGNMENT, "8-bit operands need 16-byte alignment, everything else its element's");
  if (workspace == nullptr || ws_bytes < need) return bad(FKL_ERR_WORKSPACE, "workspace missing or too small");
  if (misaligned(workspace, 256)) return bad(FKL_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  int sms = 0;
  if (const int s = require_device(&sms); s != FKL_OK) return static_cast<fkl_status>(s);
  const NamedPtr ptrs[] = {{x, x_name}, {x_scale, "x_scale"}, {wq, "wq"}, {w_scale, "w_scale"}, {out, "out"},
                           {workspace, "workspace"}};
  if (const int s = check_device_memory(ptrs); s != FKL_OK) return static_cast<fkl_status>(s);

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Int8Header* hdr = reinterpret_cast<Int8Header*>(ws);
  if (g.M == 0)
    return cudaMemsetAsync(ws, 0, 256, st) == cudaSuccess ? FKL_OK : bad(FKL_ERR_CUDA, "cudaMemsetAsync failed");
  Int8Plan pl;
  make_int8_plan(g.M, g.N, g.K, sms, &pl);
  if (pl.few) {
    FewParams p;
    p.x = x;
    p.x_scale = given ? x_scale : nullptr;
    p.ldx = ldx;
    p.x_type = x_type;
    p.vec = !given && !misaligned(x, 16) && ldx * type_bytes(x_type) % 16 == 0;
    p.wq = wq;
    p.w_scale = w_scale;
    p.out = out;
    p.ldo = g.ldo;
    p.out_type = out_type;
    p.M = static_cast<int>(g.M);
    p.N = static_cast<int>(g.N);
    p.K = static_cast<int>(g.K);
    p.hdr = reinterpret_cast<uint4*>(hdr);
    return launch_few(p, sms, st) == cudaSuccess ? FKL_OK : bad(FKL_ERR_CUDA, "8-bit product launch failed");
  }
  __half* x16 = reinterpret_cast<__half*>(ws + pl.off_x16);
  float* scale = reinterpret_cast<float*>(ws + pl.off_scale);
  cudaError_t e;
  if (given) {
    const int64_t words = g.M * g.K / 4, blocks = (words + 255) / 256;
    widen_kernel<<<static_cast<unsigned>(blocks < 16 * sms ? blocks : 16 * sms), 256, 0, st>>>(
        static_cast<const uint32_t*>(x), words, reinterpret_cast<uint2*>(x16), x_scale, static_cast<int>(g.M), scale,
        reinterpret_cast<uint4*>(hdr));
    e = cudaGetLastError();
  } else {
    e = launch_quantize(x, x_type, g.M, g.K, ldx, x16, scale, hdr, st);
  }
  if (e == cudaSuccess && late_ns > 0) {
    // with its SM's memory split as the product needs it, so that every pair starts beside it
    e = cudaFuncSetAttribute(late_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) late_kernel<<<1, 1, 0, st>>>(late_ns);
    if (e == cudaSuccess) e = cudaGetLastError();
  }
  if (e != cudaSuccess) return bad(FKL_ERR_CUDA, "launch of the tokens' kernel failed");
  e = launch_int8_gemm(reinterpret_cast<const uint16_t*>(x16), scale, wq, w_scale, g, out_type, out,
                       pl.gemm, reinterpret_cast<float*>(ws + pl.off_part), hdr, limit_ns, st);
  return e == cudaSuccess ? FKL_OK : bad(FKL_ERR_CUDA, "8-bit product launch failed");
}

}  // namespace fkl

extern "C" fkl_status fkl_int8_matmul(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                                      int64_t M, int64_t N, int64_t K, int32_t out_type, void* out, int64_t ldo,
                                      void* workspace, size_t ws_bytes, void* stream) {
  set_last_error_message("");
  return int8_product("xq", xq, -1, K, x_scale, wq, w_scale, Int8Shape{M, N, K, ldo}, out_type, out, workspace, ws_bytes,
                      stream);
}

extern "C" fkl_status fkl_int8_linear(const void* x, int32_t x_type, int64_t ldx, const int8_t* wq,
                                      const float* w_scale, int64_t M, int64_t N, int64_t K, int32_t out_type,
                                      void* out, int64_t ldo, void* workspace, size_t ws_bytes, void* stream) {
  set_last_error_message("");
  if (!type_ok(x_type)) return bad(FKL_ERR_INVALID_ARG, "x_type must be one of FKL_TYPE_*");
  if (ldx < K) return bad(FKL_ERR_INVALID_ARG, "ldx must be at least K");
  return int8_product("x", x, x_type, ldx, nullptr, wq, w_scale, Int8Shape{M, N, K, ldo}, out_type, out, workspace,
                      ws_bytes, stream);
}

extern "C" fkl_status fkl_test_int8_matmul_late(const int8_t* xq, const float* x_scale, const int8_t* wq,
                                                const float* w_scale, int64_t M, int64_t N, int64_t K, int32_t out_type,
                                                void* out, int64_t ldo, uint64_t limit_ns, uint64_t late_ns,
                                                void* workspace, size_t ws_bytes, void* stream) {
  set_last_error_message("");
  constexpr uint64_t kMs = 1000000;
  if (M < 1 || few_tokens(M, K)) return bad(FKL_ERR_INVALID_ARG, "the shape must run on the tensor cores");
  if (limit_ns < kMs || limit_ns > 1000 * kMs || late_ns < kMs || late_ns > 1000 * kMs)
    return bad(FKL_ERR_INVALID_ARG, "limit_ns and late_ns must be 1 ms to 1 s");
  return int8_product("xq", xq, -1, K, x_scale, wq, w_scale, Int8Shape{M, N, K, ldo}, out_type, out, workspace, ws_bytes,
                      stream, limit_ns, late_ns);
}
