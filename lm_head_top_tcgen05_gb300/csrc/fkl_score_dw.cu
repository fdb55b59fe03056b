// dW (+)= dS^T H of the scores from hidden states (fkl_score_fused.cu), on the two-SM product of fkl_gemm2.cuh.
//
// Its epilogue adds, in fp32 and in the order of tokens, what the rounding of dS took from the tokens' own
// entries, and rounds once; rows that more than kMaxTargets tokens share it leaves in fp32 for the kernel behind it
// (reading a sum made beforehand cost a warp a load's latency for each 32 columns: 64 tokens, 20 of one row, 279 us
// without and 310 with it).  A lane has a row of the tile, so each of its stores is a separate line: 32-byte
// stores move the bf16 tile in half the instructions of 16-byte ones, which is what a short batch's
// product waits for (64 x 201088 x 2880: 466 us with 16-byte stores, 335 with these, 300 with four tiles to a unit; a
// plain fill of dW takes 287, as HBM takes writes alone at 4.0 TB/s).  Boxes of 32 rows in shared memory that leave
// by TMA stores took 340: they leave room for 128-wide tiles only, and A is read again for each.
#include "fkl_score_dw.cuh"

#include "fkl_gemm2.cuh"

namespace fkl {
namespace {

template <bool kBf16>
struct EpiDw {
  using Params = DwParams;
  const Params& p;
  bool row_ok;
  float* rowp;
  uint16_t* rowp16;
  int n;
  int token[kMaxTargets];
  float rest[kMaxTargets];
  float* held;  // where a shared row's fp32 values go in place of bf16, or NULL

  __device__ explicit EpiDw(const Params& prm) : p(prm) {}

  __device__ __forceinline__ void begin_unit(int row0, int, int, int row) {
    const int r = row0 + row;
    row_ok = r < p.to.M;
    const size_t rr = static_cast<size_t>(row_ok ? r : 0);
    rowp = p.to.out != nullptr ? p.to.out + rr * p.to.ldo : nullptr;
    rowp16 = kBf16 ? p.to.out16 + rr * p.to.ldo16 : nullptr;
    n = row_ok && p.count != nullptr ? p.count[rr] : 0;
    held = nullptr;
    if (n > kMaxTargets) {
      if (kBf16) held = p.held + static_cast<size_t>(p.slot_of[rr]) * p.to.N;
      n = 0;
    }
#pragma unroll
    for (int k = 0; k < kMaxTargets; ++k) token[k] = k < n ? p.token_of[rr * kMaxTargets + k] : INT_MAX;
    // the tokens came in any order; a fixed one gives the same sums every time
    auto order = [&](int a, int b) {
      const int lo = min(token[a], token[b]), hi = max(token[a], token[b]);
      token[a] = lo;
      token[b] = hi;
    };
    static_assert(kMaxTargets == 4, "a sorting network of four");
    order(0, 1);
    order(2, 3);
    order(0, 2);
    order(1, 3);
    order(1, 2);
#pragma unroll
    for (int k = 0; k < kMaxTargets; ++k) rest[k] = k < n ? p.rest[token[k]] : 0.f;
  }

  template <int BN>
  __device__ __forceinline__ void tile(uint32_t taddr, int tile_n, int) {
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      const int col0 = tile_n * BN + c * 32, left = p.to.N - col0;  // columns from here on, a multiple of 8
      if (left <= 0) break;  // same for the whole warp
      float v[32];
      tmem_ld32(taddr + c * 32, v);
      tmem_ld_wait(v);
      if (!row_ok) continue;
      if (p.to.accumulate) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (8 * j < left) {
            const float4* from = reinterpret_cast<const float4*>(rowp + col0 + 8 * j);
            const float4 lo = from[0], hi = from[1];
            v[8 * j] += lo.x; v[8 * j + 1] += lo.y; v[8 * j + 2] += lo.z; v[8 * j + 3] += lo.w;
            v[8 * j + 4] += hi.x; v[8 * j + 5] += hi.y; v[8 * j + 6] += hi.z; v[8 * j + 7] += hi.w;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kMaxTargets; ++k) {
        if (k < n) {
          const uint4* h = reinterpret_cast<const uint4*>(p.H + static_cast<size_t>(token[k]) * p.to.N + col0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (8 * j < left) {
              const uint4 w = h[j];
              add_bf16x2(v[8 * j], v[8 * j + 1], w.x, rest[k]);
              add_bf16x2(v[8 * j + 2], v[8 * j + 3], w.y, rest[k]);
              add_bf16x2(v[8 * j + 4], v[8 * j + 5], w.z, rest[k]);
              add_bf16x2(v[8 * j + 6], v[8 * j + 7], w.w, rest[k]);
            }
          }
        }
      }
      if (kBf16 && held != nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (8 * j < left)
            st_v8(held + col0 + 8 * j, __float_as_uint(v[8 * j]), __float_as_uint(v[8 * j + 1]), __float_as_uint(v[8 * j + 2]),
                  __float_as_uint(v[8 * j + 3]), __float_as_uint(v[8 * j + 4]), __float_as_uint(v[8 * j + 5]),
                  __float_as_uint(v[8 * j + 6]), __float_as_uint(v[8 * j + 7]));
        }
      } else if (kBf16) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        uint16_t* o = rowp16 + col0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (p.wide16 && 16 * j + 16 <= left) {
            st_v8(o + 16 * j, w[8 * j], w[8 * j + 1], w[8 * j + 2], w[8 * j + 3], w[8 * j + 4], w[8 * j + 5], w[8 * j + 6],
                  w[8 * j + 7]);
          } else {
            uint4* o4 = reinterpret_cast<uint4*>(o + 16 * j);
            if (16 * j < left) o4[0] = make_uint4(w[8 * j], w[8 * j + 1], w[8 * j + 2], w[8 * j + 3]);
            if (16 * j + 8 < left) o4[1] = make_uint4(w[8 * j + 4], w[8 * j + 5], w[8 * j + 6], w[8 * j + 7]);
          }
        }
      } else {
        float* o = rowp + col0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (8 * j >= left) continue;
          if (p.to.vec_ok) {
            st_v8(o + 8 * j, __float_as_uint(v[8 * j]), __float_as_uint(v[8 * j + 1]), __float_as_uint(v[8 * j + 2]),
                  __float_as_uint(v[8 * j + 3]), __float_as_uint(v[8 * j + 4]), __float_as_uint(v[8 * j + 5]),
                  __float_as_uint(v[8 * j + 6]), __float_as_uint(v[8 * j + 7]));
          } else {
            float4* o4 = reinterpret_cast<float4*>(o + 8 * j);
            o4[0] = make_float4(v[8 * j], v[8 * j + 1], v[8 * j + 2], v[8 * j + 3]);
            o4[1] = make_float4(v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]);
          }
        }
      }
    }
  }

  __device__ __forceinline__ void end_unit(int, int) {}
};

}  // namespace

cudaError_t launch_score_dw(int bn, const CUtensorMap& a, const CUtensorMap& b, const GemmShape& g, const DwParams& p,
                            int sms, cudaStream_t st) {
  const bool bf16 = p.to.out16 != nullptr;
  switch (bn) {
    case 256:
      return bf16 ? launch_gemm2_t<256, true, true, EpiDw<true>>(a, b, g, p, sms, st)
                  : launch_gemm2_t<256, true, true, EpiDw<false>>(a, b, g, p, sms, st);
    case 192:
      return bf16 ? launch_gemm2_t<192, true, true, EpiDw<true>>(a, b, g, p, sms, st)
                  : launch_gemm2_t<192, true, true, EpiDw<false>>(a, b, g, p, sms, st);
    default:
      return bf16 ? launch_gemm2_t<128, true, true, EpiDw<true>>(a, b, g, p, sms, st)
                  : launch_gemm2_t<128, true, true, EpiDw<false>>(a, b, g, p, sms, st);
  }
}

}  // namespace fkl
