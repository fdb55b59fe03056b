// The head's gradient of the scores from hidden states: parameters and launch of its product.
#pragma once

#include "fkl_internal.h"

namespace fkl {

// What rounding took from the tokens' entries is added back to dW's rows: by the product's epilogue in rows of at
// most this many tokens, by a kernel behind it in rows that more tokens share.  It does not average out there: tokens of
// one weight and a small q have entries that round alike (500 tokens, a = 1 / 3001: 0.2 % of their sum).
constexpr int kMaxTargets = 4;

// Tile of dW (+)= dS^T H: F32Params, the row's tokens (up to kMaxTargets, in any order) and what
// rounding took from each of their entries in dS.
struct DwParams {
  F32Params to;
  int wide16;           // out16 and its row stride allow 32-byte vectors
  const int* count;     // tokens of each row, or NULL: nothing to add
  const int* token_of;  // [row][kMaxTargets]
  const int* slot_of;   // [row], where there are more than kMaxTargets tokens
  float* held;          // [slot][N]: such a row of a bf16 gradient, not rounded yet
  const float* rest;    // by token
  const uint16_t* H;    // [T][N]
};

cudaError_t launch_score_dw(int bn, const CUtensorMap& a, const CUtensorMap& b, const GemmShape& g, const DwParams& p,
                            int sms, cudaStream_t st);

// lo += r * w's low bf16, hi += r * its high one.
__device__ __forceinline__ void add_bf16x2(float& lo, float& hi, uint32_t w, float r) {
  lo = fmaf(r, __uint_as_float(w << 16), lo);
  hi = fmaf(r, __uint_as_float(w & 0xffff0000u), hi);
}

}  // namespace fkl
