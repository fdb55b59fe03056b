// The 8-bit product of a generation step (fkl_quantize_int8, fkl_int8_matmul,
// fkl_int8_linear).
//
//     s_m = max_k |x_mk| * fl(1/127),  q_mk = rint(x_mk / s_m)
//     y_mn = (sum_k q_mk w_nk) * s_m * t_n
#include <climits>

#include "fkl_internal.h"
#include "fkl_types.cuh"

namespace fkl {

constexpr int64_t kMaxInt8K = 131072;  // 128 * 128 * K stays within an int32 sum

// ---------------------------------------------------------------- quantisation
constexpr int kQuantThreads = 256;
constexpr uint32_t kInfBits = 0x7f800000u;

// Scale of a row whose largest magnitude has the bits amax; NaN when the row holds a NaN or an
// infinity (their bits exceed every finite magnitude's).
__device__ __forceinline__ float row_scale(uint32_t amax) {
  return amax >= kInfBits ? __uint_as_float(0x7fc00000u) : __uint_as_float(amax) * (1.0f / 127.0f);
}
// s = 0 (a row of zeros, or of values whose scale underflows) and s = NaN give 0.
__device__ __forceinline__ int quantize(float x, float s) {
  if (!(s > 0.f)) return 0;
  return static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f));
}

// One block per row, two reads of it (the second from cache).  The IEEE division keeps the
// integers equal to the definition's.
template <class T, bool kVec>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_kernel(const T* __restrict__ x, int64_t cols, int64_t ldx, int8_t* __restrict__ q,
                    float* __restrict__ scale) {
  constexpr int E = 16 / sizeof(T);
  __shared__ uint32_t warp_max[kQuantThreads / 32];
  const T* row = x + static_cast<int64_t>(blockIdx.x) * ldx;
  int8_t* out = q + static_cast<int64_t>(blockIdx.x) * cols;
  uint32_t amax = 0;
  if (kVec) {
    for (int64_t i = threadIdx.x; i < cols / E; i += kQuantThreads) {
      float v[E];
      unpack16<T>(reinterpret_cast<const uint4*>(row)[i], v);
#pragma unroll
      for (int j = 0; j < E; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
    }
  } else {
    for (int64_t i = threadIdx.x; i < cols; i += kQuantThreads)
      amax = max(amax, __float_as_uint(to_float(row[i])) & 0x7fffffffu);
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = 0;
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) amax = max(amax, warp_max[w]);
  const float s = row_scale(amax);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
  if (kVec) {
    for (int64_t i = threadIdx.x; i < cols / E; i += kQuantThreads) {
      float v[E];
      unpack16<T>(reinterpret_cast<const uint4*>(row)[i], v);
      uint32_t w[E / 4];
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        w[j] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) w[j] |= (static_cast<uint32_t>(quantize(v[4 * j + b], s)) & 0xffu) << (8 * b);
      }
#pragma unroll
      for (int j = 0; j < E / 4; ++j) reinterpret_cast<uint32_t*>(out)[i * (E / 4) + j] = w[j];
    }
  } else {
    for (int64_t i = threadIdx.x; i < cols; i += kQuantThreads)
      out[i] = static_cast<int8_t>(quantize(to_float(row[i]), s));
  }
}

static cudaError_t launch_quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                                   float* scale, cudaStream_t st) {
  return with_type(type, [&](auto t) {
    using T = decltype(t);
    const T* p = static_cast<const T*>(x);
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * sizeof(T) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(q) % 4 == 0 && cols % 16 == 0;
    if (vec)
      quantize_kernel<T, true><<<static_cast<unsigned>(rows), kQuantThreads, 0, st>>>(p, cols, ldx, q, scale);
    else
      quantize_kernel<T, false><<<static_cast<unsigned>(rows), kQuantThreads, 0, st>>>(p, cols, ldx, q, scale);
    return cudaGetLastError();
  });
}

// ---------------------------------------------------------------- product
struct Int8Shape {
  int64_t M, N, K, ldo;
};

constexpr int kTile = 64;  // outputs per block along M and along N
constexpr int kTileK = 64;

// 64 x 64 outputs per block of 256 threads, 4 x 4 per thread, by dp4a.
template <class T>
__global__ void __launch_bounds__(256)
    int8_tile_kernel(const int8_t* __restrict__ xq, const float* __restrict__ xs, const int8_t* __restrict__ wq,
                     const float* __restrict__ ws, const Int8Shape g, T* __restrict__ out) {
  __shared__ int sx[kTile][kTileK / 4 + 1], sw[kTile][kTileK / 4 + 1];
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile, m0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  const int lr = threadIdx.x >> 2, lc = threadIdx.x & 3;  // row and 16-byte chunk this thread loads
  for (int64_t k0 = 0; k0 < g.K; k0 += kTileK) {
    const int64_t k = k0 + 16 * lc;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 a = m0 + lr < g.M && k < g.K ? *reinterpret_cast<const uint4*>(xq + (m0 + lr) * g.K + k) : zero;
    const uint4 b = n0 + lr < g.N && k < g.K ? *reinterpret_cast<const uint4*>(wq + (n0 + lr) * g.K + k) : zero;
    __syncthreads();
    sx[lr][4 * lc] = a.x; sx[lr][4 * lc + 1] = a.y; sx[lr][4 * lc + 2] = a.z; sx[lr][4 * lc + 3] = a.w;
    sw[lr][4 * lc] = b.x; sw[lr][4 * lc + 1] = b.y; sw[lr][4 * lc + 2] = b.z; sw[lr][4 * lc + 3] = b.w;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kTileK / 4; ++c) {
      int av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) av[i] = sx[ty * 4 + i][c];
#pragma unroll
      for (int j = 0; j < 4; ++j) bv[j] = sw[tx + 16 * j][c];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(av[i], bv[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= g.M) continue;
    const float s = xs[m];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx + 16 * j;
      if (n < g.N) out[m * g.ldo + n] = from_float<T>(static_cast<float>(acc[i][j]) * s * ws[n]);
    }
  }
}

static cudaError_t launch_product(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                                  const Int8Shape& g, int32_t type, void* out, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((g.N + kTile - 1) / kTile), static_cast<unsigned>((g.M + kTile - 1) / kTile));
  return with_type(type, [&](auto t) {
    using T = decltype(t);
    int8_tile_kernel<T><<<grid, 256, 0, st>>>(xq, xs, wq, ws, g, static_cast<T*>(out));
    return cudaGetLastError();
  });
}

// ---------------------------------------------------------------- host side
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Int8Plan {
  size_t off_q, off_scale, total;
};

static bool make_int8_plan(int64_t M, int64_t N, int64_t K, bool quantize, Int8Plan* p) {
  if (M < 0 || M > INT32_MAX || N < 1 || N > INT32_MAX || K < 16 || K % 16 != 0 || K > kMaxInt8K) return false;
  size_t off = 256;  // status header
  p->off_q = off;
  if (quantize) off = up256(off + static_cast<size_t>(M) * K);
  p->off_scale = off;
  if (quantize) off = up256(off + static_cast<size_t>(M) * 4);
  p->total = off;
  return true;
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
  if (launch_quantize(x, x_type, rows, cols, ldx, q, scale, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return bad(FKL_ERR_CUDA, "quantisation launch failed");
  return FKL_OK;
}

extern "C" size_t fkl_int8_matmul_workspace_size(int64_t M, int64_t N, int64_t K) {
  Int8Plan p;
  return make_int8_plan(M, N, K, false, &p) ? p.total : 0;
}

extern "C" size_t fkl_int8_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
  Int8Plan p;
  return make_int8_plan(M, N, K, true, &p) ? p.total : 0;
}

namespace fkl {

// Checks shared by the two products; `x` is the tokens (of x_align-byte alignment).
static fkl_status check_product(bool quantize, const void* x, size_t x_align, const float* x_scale, const int8_t* wq,
                                const float* w_scale, const Int8Shape& g, int32_t out_type, const void* out,
                                const void* workspace, size_t ws_bytes, Int8Plan* pl, int* sms) {
  if (!type_ok(out_type)) return bad(FKL_ERR_INVALID_ARG, "out_type must be one of FKL_TYPE_*");
  if (!make_int8_plan(g.M, g.N, g.K, quantize, pl))
    return bad(FKL_ERR_INVALID_ARG, "unsupported shape (need K % 16 == 0, 16 <= K <= 131072, 0 <= M < 2^31, 1 <= N < 2^31)");
  if (g.ldo < g.N) return bad(FKL_ERR_INVALID_ARG, "ldo must be at least N");
  if (wq == nullptr || w_scale == nullptr ||
      (g.M > 0 && (x == nullptr || out == nullptr || (!quantize && x_scale == nullptr))))
    return bad(FKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (misaligned(wq, 16) || misaligned(x, x_align) || misaligned(x_scale, 4) || misaligned(w_scale, 4) ||
      misaligned(out, type_bytes(out_type)))
    return bad(FKL_ERR_ALIGNMENT, "8-bit operands need 16-byte alignment, everything else its element's");
  if (workspace == nullptr || ws_bytes < pl->total) return bad(FKL_ERR_WORKSPACE, "workspace missing or too small");
  if (misaligned(workspace, 256)) return bad(FKL_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if (const int s = require_device(sms); s != FKL_OK) return static_cast<fkl_status>(s);
  const NamedPtr ptrs[] = {{x, quantize ? "x" : "xq"}, {x_scale, "x_scale"}, {wq, "wq"}, {w_scale, "w_scale"},
                           {out, "out"}, {workspace, "workspace"}};
  return static_cast<fkl_status>(check_device_memory(ptrs));
}

}  // namespace fkl

extern "C" fkl_status fkl_int8_matmul(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                                      int64_t M, int64_t N, int64_t K, int32_t out_type, void* out, int64_t ldo,
                                      void* workspace, size_t ws_bytes, void* stream) {
  set_last_error_message("");
  const Int8Shape g{M, N, K, ldo};
  Int8Plan pl;
  int sms = 0;
  const fkl_status s =
      check_product(false, xq, 16, x_scale, wq, w_scale, g, out_type, out, workspace, ws_bytes, &pl, &sms);
  if (s != FKL_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 256, st) != cudaSuccess) return bad(FKL_ERR_CUDA, "cudaMemsetAsync failed");
  if (M == 0) return FKL_OK;
  if (launch_product(xq, x_scale, wq, w_scale, g, out_type, out, st) != cudaSuccess)
    return bad(FKL_ERR_CUDA, "8-bit product launch failed");
  return FKL_OK;
}

extern "C" fkl_status fkl_int8_linear(const void* x, int32_t x_type, int64_t ldx, const int8_t* wq,
                                      const float* w_scale, int64_t M, int64_t N, int64_t K, int32_t out_type,
                                      void* out, int64_t ldo, void* workspace, size_t ws_bytes, void* stream) {
  set_last_error_message("");
  if (!type_ok(x_type)) return bad(FKL_ERR_INVALID_ARG, "x_type must be one of FKL_TYPE_*");
  if (ldx < K) return bad(FKL_ERR_INVALID_ARG, "ldx must be at least K");
  const Int8Shape g{M, N, K, ldo};
  Int8Plan pl;
  int sms = 0;
  const fkl_status s = check_product(true, x, type_bytes(x_type), nullptr, wq, w_scale, g, out_type, out, workspace,
                                     ws_bytes, &pl, &sms);
  if (s != FKL_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 256, st) != cudaSuccess) return bad(FKL_ERR_CUDA, "cudaMemsetAsync failed");
  if (M == 0) return FKL_OK;
  uint8_t* w8 = static_cast<uint8_t*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(w8 + pl.off_q);
  float* xs = reinterpret_cast<float*>(w8 + pl.off_scale);
  if (launch_quantize(x, x_type, M, K, ldx, xq, xs, st) != cudaSuccess)
    return bad(FKL_ERR_CUDA, "quantisation launch failed");
  if (launch_product(xq, xs, wq, w_scale, g, out_type, out, st) != cudaSuccess)
    return bad(FKL_ERR_CUDA, "8-bit product launch failed");
  return FKL_OK;
}
