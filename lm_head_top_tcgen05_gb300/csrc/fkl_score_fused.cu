// Scores given tokens from hidden states (fkl_logprob_forward) and the gradients in the hidden states and
// the LM head (fkl_logprob_backward), on the two-SM tensor-core product of fkl_gemm2.cuh.
//
// Forward: the logits s = H W^T live in tensor memory, a tile at a time.  Each (row, vocabulary split) keeps
// a reference logit m, l = sum of 2^a and u = sum of 2^a a with a = (s - m) log2(e) / tau, and the split that holds
// the row's token stores its logit.  A kernel over the rows then joins the splits: with c = log2(e) / tau,
// logprob = ln 2 (c (s_token - M) - log2 L), entropy = ln 2 (log2 L - U / L), lse = ln 2 (c M + log2 L).  The reference is
// a logit and not, as in the loss, its product with c: that product's rounding grows with 1 / tau, and would be
// what a row's likeliest token scores at a low temperature (4e-3 above 0 at tau = 1e-4).  It takes an addition and a
// product where one multiply-add would do: 2 % of the time at d = 128 to 512, 1 % at 1024, none beyond.
//
// Backward: log2 q_tv = c (s_tv - M_t) - log2 L_t with the forward's reference and sum (statistics of a row; from
// lse, their rounded sum, q would be off by 2^-24 lse of itself, 2 % for a logit of 30 at tau = 1e-4), and
// dS_tv = q_tv (c0_t + c1_t log2 q_tv) + k_t [v = v*_t] with c0 = -(a + b entropy) / tau,
// c1 = -b ln 2 / tau, k = a / tau, rounded to bf16 and written block by block (tokens x a vocabulary slab),
// then dW[slab] += dS^T H and dH[block] += dS W[slab] in fp32, in a fixed order: the blocks are those of the
// loss's backward, planned by the same functions.  The bf16 of dS (half a step is 2^-8 of each value) is what
// the tensor cores multiply; sums stay fp32.  A row's largest entry mostly is the one of its token, so what
// rounding takes from that one, r_t, is not lost: dH's sums start at r_t W[v*_t], and dW's rows add r_t H_t, of
// however many tokens, before they are rounded (fkl_score_dw.cu).  Without, both gradients were 1.4 times as far from
// exact ones as their own rounding to bf16 makes them.
//
// The tensor pipe bounds both: 2 T V d operations forward, 6 T V d backward.  4096 x 201088 x 2880: 2.7 ms forward
// (1750 TFLOP/s), 8.8 ms backward (1615), as the loss of the same shape.  Few tokens wait for the head's bytes: 64
// tokens 202 us forward (5.7 TB/s) and 707 backward, of which reading the head twice and filling its gradient are 627.
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/fkl_score.h"
#include "fkl_gemm2.cuh"
#include "fkl_generate.cuh"
#include "fkl_score.cuh"
#include "fkl_score_dw.cuh"

namespace fkl {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool on_boundary(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr float kFloor = -200.f;  // exponents below it are 0: 2^-200 is below fp32

// ---------------------------------------------------------------- forward epilogue
struct ScoreFwdParams {
  TokenIds tokens;
  const uint8_t* mask;
  float* part;       // [3][nsplit][T]: reference logit, sum, weighted sum
  float* token_s;    // [T]: the token's logit
  int T, V, nsplit;
  float scale2;      // log2(e) / tau
};

struct EpiScore {
  using Params = ScoreFwdParams;
  const Params& p;
  int t, tok;
  bool row_ok;
  float m, l, u;

  __device__ explicit EpiScore(const Params& prm) : p(prm) {}

  __device__ __forceinline__ void begin_unit(int row0, int, int, int row) {
    t = row0 + row;
    row_ok = t < p.T;
    tok = row_ok && (p.mask == nullptr || p.mask[t] != 0) ? p.tokens.get(t, p.V) : -1;
    m = -INFINITY;
    l = u = 0.f;
  }

  // The sum of the chunk's weights at reference `ref`, and their weighted sum.  kGuard: a logit of -inf, whose
  // exponent is -inf too, has weight 0 in both (0 * -inf would be NaN); NaN stays.
  template <bool kGuard>
  __device__ __forceinline__ float sums(const float (&v)[32], float ref, float& weighted) const {
    const float2 sc = make_float2(p.scale2, p.scale2), om = make_float2(-ref, -ref);
    auto exponent = [&](float x, float y) {
      const float2 a = fmul2(fadd2(make_float2(x, y), om), sc);
      return kGuard ? make_float2(max_nan(a.x, kFloor), max_nan(a.y, kFloor)) : a;
    };
    float2 t0 = make_float2(0.f, 0.f), t1 = t0, w0 = t0, w1 = t0;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float2 a0 = exponent(v[j], v[j + 1]), a1 = exponent(v[j + 2], v[j + 3]);
      const float2 e0 = make_float2(ex2_approx(a0.x), ex2_approx(a0.y)), e1 = make_float2(ex2_approx(a1.x), ex2_approx(a1.y));
      t0 = fadd2(t0, e0);
      t1 = fadd2(t1, e1);
      w0 = ffma2(e0, a0, w0);
      w1 = ffma2(e1, a1, w1);
    }
    weighted = (w0.x + w0.y) + (w1.x + w1.y);
    return (t0.x + t0.y) + (t1.x + t1.y);
  }

  __device__ __forceinline__ void chunk(float (&v)[32], int col0) {
    if (col0 >= p.V) return;
    if (tok >= col0 && tok < col0 + 32) p.token_s[t] = pick(v, tok - col0);
    const bool whole = col0 + 32 <= p.V;
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col0 + j >= p.V) v[j] = -INFINITY;
    }
    float weighted;
    if (whole && m != -INFINITY) {
      // A reference 2^10 below a term would cost the entropy 10 binary orders of its last digits: log2 L
      // and U / L then cancel.  It moves before that.  A weighted sum of NaN has a logit of -inf, or NaN, in it.
      const float sum = sums<false>(v, m, weighted);
      if (sum < 1024.f && weighted == weighted) {
        l += sum;
        u += weighted;
        return;
      }
    }
    float c0 = fmax3(v[0], v[1], v[2]), c1 = fmax3(v[3], v[4], v[5]);
#pragma unroll
    for (int j = 6; j < 30; j += 4) {
      c0 = fmax3(c0, v[j], v[j + 1]);
      c1 = fmax3(c1, v[j + 2], v[j + 3]);
    }
    const float to = fmaxf(m, fmax3(c0, c1, fmaxf(v[30], v[31])));
    const float ref = to > -INFINITY ? to : 0.f;  // no logit yet: sums of 0, or NaN, which stays
    const float sum = sums<true>(v, ref, weighted);
    const float r = fmaxf((m - ref) * p.scale2, -1000.f), f = ex2_approx(r);
    u = fmaf(fmaf(r, l, u), f, weighted);
    l = fmaf(l, f, sum);
    m = to;
  }

  template <int BN>
  __device__ __forceinline__ void tile(uint32_t taddr, int n, int) {
#pragma unroll 1
    for (int c = 0; c < BN / 32; c += 2) {
      float v0[32], v1[32];
      tmem_ld32(taddr + c * 32, v0);
      tmem_ld32(taddr + c * 32 + 32, v1);
      tmem_wait_ld();
      pin(v0);
      pin(v1);
      chunk(v0, n * BN + c * 32);
      chunk(v1, n * BN + c * 32 + 32);
    }
  }

  __device__ __forceinline__ void end_unit(int split, int) {
    if (!row_ok) return;
    const size_t plane = static_cast<size_t>(p.nsplit) * p.T, i = static_cast<size_t>(split) * p.T + t;
    p.part[i] = m;
    p.part[plane + i] = l;
    p.part[2 * plane + i] = u;
  }
};

// ---------------------------------------------------------------- backward epilogue
struct ScoreDsParams {
  TokenIds tokens;            // of all tokens: row t of the block is token r0 + t
  int64_t r0;
  const float *c0, *c1;       // of the block's tokens; a row left out has zeros
  const float* hit;           // the token's entry, rounded (0 in a row left out)
  const float2* ref;          // reference logit and log2 of the sum of the weights at it
  uint16_t* ds;
  int64_t ld_ds;
  int T, V, v0, slab_w;
  float scale2;
};

struct EpiScoreDs {
  using Params = ScoreDsParams;
  const Params& p;
  bool row_ok, off;
  int tok;
  float c0, c1, hit;
  float2 ref;
  uint16_t* dst;

  __device__ explicit EpiScoreDs(const Params& prm) : p(prm) {}

  __device__ __forceinline__ void begin_unit(int row0, int, int, int row) {
    const int t = row0 + row;
    row_ok = t < p.T;
    off = true;
    tok = -1;
    c0 = c1 = hit = 0.f;
    ref = make_float2(0.f, 0.f);
    dst = nullptr;
    if (row_ok) {
      c0 = p.c0[t];
      c1 = p.c1[t];
      hit = p.hit[t];
      off = c0 == 0.f && c1 == 0.f && hit == 0.f;
      ref = p.ref[t];
      if (!off) tok = p.tokens.get(p.r0 + t, p.V);
      dst = p.ds + static_cast<size_t>(t) * p.ld_ds;
    }
  }

  __device__ __forceinline__ void chunk(float (&v)[32], int cl0) {
    if (!row_ok) return;
    uint16_t* o = dst + cl0;
    if (off) {
#pragma unroll
      for (int j = 0; j < 2; ++j) st_v8(o + 16 * j, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u);
      return;
    }
    {
      const float2 sc = make_float2(p.scale2, p.scale2);
      const float2 nm = make_float2(-ref.x, -ref.x), sh = make_float2(-ref.y, -ref.y);
      const float2 k0 = make_float2(c0, c0), k1 = make_float2(c1, c1);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float2 a = ffma2(fadd2(make_float2(v[j], v[j + 1]), nm), sc, sh);  // log2 q
        a = make_float2(max_nan(a.x, kFloor), max_nan(a.y, kFloor));       // 0 * -inf would be NaN
        const float2 y = fmul2(make_float2(ex2_approx(a.x), ex2_approx(a.y)), ffma2(k1, a, k0));
        v[j] = y.x;
        v[j + 1] = y.y;
      }
    }
    const int jt = tok - (p.v0 + cl0);
    if (jt >= 0 && jt < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = j == jt ? hit : v[j];
    }
    if (cl0 + 32 > p.slab_w) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (cl0 + j >= p.slab_w) v[j] = 0.f;
    }
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      st_v8(o + 16 * j, w[8 * j], w[8 * j + 1], w[8 * j + 2], w[8 * j + 3], w[8 * j + 4], w[8 * j + 5], w[8 * j + 6],
            w[8 * j + 7]);
  }

  template <int BN>
  __device__ __forceinline__ void tile(uint32_t taddr, int n, int) {
#pragma unroll 1
    for (int c = 0; c < BN / 32; c += 2) {
      float v0[32], v1[32];
      tmem_ld32(taddr + c * 32, v0);
      tmem_ld32(taddr + c * 32 + 32, v1);
      tmem_wait_ld();
      pin(v0);
      pin(v1);
      chunk(v0, n * BN + c * 32);
      chunk(v1, n * BN + c * 32 + 32);
    }
  }

  __device__ __forceinline__ void end_unit(int, int) {}
};

// ---------------------------------------------------------------- kernels over the rows
constexpr int kRowThreads = 256;

// Joins the splits of 32 rows, a row to a lane, a share of the splits to a warp.  The weights between splits are
// fp32, the same for L and U; the sums and the two terms of the entropy, which may cancel, are fp64.  Every
// term has the weights' own constant, so that what rounds in it scales the distances between logits and no more.  What
// rounding leaves beyond the scores' range (log q <= 0 <= entropy) is cut off.
__global__ void __launch_bounds__(kRowThreads)
    score_rows_kernel(const float* __restrict__ part, int nsplit, const float* __restrict__ token_s, TokenIds tokens,
                      const uint8_t* __restrict__ mask, int64_t T, int V, float scale2, uint32_t* status,
                      float* __restrict__ logprob, float* __restrict__ entropy, float* __restrict__ lse,
                      float* __restrict__ stats) {
  constexpr int kWarps = kRowThreads / 32;
  __shared__ float warp_m[kWarps][32];
  __shared__ double warp_l[kWarps][32], warp_u[kWarps][32];
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const size_t plane = static_cast<size_t>(nsplit) * T;
  float M = -INFINITY;
  if (t < T)
    for (int s = warp; s < nsplit; s += kWarps) M = fmaxf(M, part[static_cast<size_t>(s) * T + t]);
  warp_m[warp][lane] = M;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, warp_m[w][lane]);
  double L = 0.0, U = 0.0;
  if (t < T) {
    for (int s = warp; s < nsplit; s += kWarps) {
      const size_t i = static_cast<size_t>(s) * T + t;
      const float a = fmaxf((part[i] - M) * scale2, -1000.f);
      const double f = exp2f(a), l = part[plane + i];
      L += f * l;
      U += f * (part[2 * plane + i] + a * l);
    }
  }
  warp_l[warp][lane] = L;
  warp_u[warp][lane] = U;
  __syncthreads();
  if (warp != 0 || t >= T) return;
  for (int w = 1; w < kWarps; ++w) {
    L += warp_l[w][lane];
    U += warp_u[w][lane];
  }
  const double ln2 = 0.69314718055994530942, log2_sum = log2(L);
  const bool late = (*reinterpret_cast<const volatile uint32_t*>(status) & kStatusTimeoutBit) != 0;
  if (lse != nullptr) lse[t] = late ? NAN : static_cast<float>((static_cast<double>(M) * scale2 + log2_sum) * ln2);
  if (stats != nullptr) {
    stats[2 * t] = late ? NAN : M;
    stats[2 * t + 1] = late ? NAN : static_cast<float>(log2_sum * ln2);
  }
  if (mask != nullptr && mask[t] == 0) {
    logprob[t] = late ? NAN : 0.f;
    entropy[t] = late ? NAN : 0.f;
    return;
  }
  const int tok = tokens.get(t, V);
  if (tok < 0) atomicOr(status, kStatusBadIdBit);
  const double lp = late || tok < 0 ? NAN : ((static_cast<double>(token_s[t]) - M) * scale2 - log2_sum) * ln2;
  const double ent = late ? NAN : (log2_sum - U / L) * ln2;
  logprob[t] = lp > 0.0 ? 0.f : static_cast<float>(lp);  // NaN stays
  entropy[t] = ent < 0.0 ? 0.f : static_cast<float>(ent);
}

// Without the rows' statistics log q is a logit less lse, off by 2^-24 lse.  Above this lse that passes half a step of
// dS's bf16 (2^-9 to 2^-8 of a value), and the row is NaN.
constexpr float kMaxLse = 32768.f;

// The tokens of each vocabulary row: what the head's gradient adds back to it.  A row that more than kMaxTargets
// tokens have is shared; one of more than kMostFew is long.
constexpr int kMostFew = 64;
struct TargetRows {
  int* count;     // [V]: tokens of each row; then the counters below, zero at the start like it
  int* token_of;  // [V][kMaxTargets]
  int* slot_of;   // [V]: place among the shared rows
  int* shared;    // [T / (kMaxTargets + 1)]: the shared rows
  int* base_of;   // [T / (kMaxTargets + 1)]: where a shared row's tokens start in the list
  int* longs;     // [T / (kMostFew + 1)]: slots of the long rows
  int* row_of;    // [T]: the row of each token that takes part, or -1
  int* order;     // [T]: how many of its row's tokens were counted before it
  int* list;      // [T]: the shared rows' tokens
  int V;
  __device__ __forceinline__ int* counter(int i) const { return count + V + i; }
};
constexpr int kShared = 0, kLong = 1, kListed = 2, kBlocksDone = 3, kCounters = 4;

// The factors of each token's dS, its entry at the token with what rounding takes from it, where its log q is counted
// from, and the tokens of each vocabulary row; a token outside the vocabulary is recorded.  Slots, places in the list and the
// order within a row come from atomics, in any order: no sum depends on them (finish_few sorts, finish_long looks through
// the tokens in order).
__global__ void __launch_bounds__(kRowThreads)
    score_factors_kernel(TokenIds tokens, const uint8_t* __restrict__ mask, const float* __restrict__ logprob,
                         const float* __restrict__ entropy, const float* __restrict__ lse,
                         const float* __restrict__ stats, const float* __restrict__ grad_logprob,
                         const float* __restrict__ grad_entropy, int64_t T, int V, float inv_tau,
                         uint32_t* __restrict__ status, float* __restrict__ c0, float* __restrict__ c1,
                         float* __restrict__ hit, float* __restrict__ rest, float2* __restrict__ ref,
                         const TargetRows rows) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (t < T) {
    float a = 0.f, b = 0.f, h = 0.f, log2_q = 0.f;
    int tok = -1;
    if (mask == nullptr || mask[t] != 0) {
      tok = tokens.get(t, V);
      if (tok < 0) atomicOr(status, kStatusBadIdBit);
      if (grad_logprob != nullptr) a = grad_logprob[t];
      if (grad_entropy != nullptr) b = grad_entropy[t];
      if (b != 0.f) h = entropy[t];
      log2_q = fmaxf(logprob[t], -1000.f) * kLog2e;  // below that q is 0, and 0 * -inf would be none
    }
    const float f0 = -fmaf(b, h, a) * inv_tau, f1 = -b * kLn2 * inv_tau;
    const float2 from = stats != nullptr ? make_float2(stats[2 * t], stats[2 * t + 1] * kLog2e)
                                         : make_float2(0.f, fabsf(lse[t]) <= kMaxLse ? lse[t] * kLog2e : NAN);
    const bool target = tok >= 0 && (f0 != 0.f || f1 != 0.f);
    float entry = fmaf(exp2f(log2_q), fmaf(f1, log2_q, f0), a * inv_tau);
    if (target && !(from.y == from.y)) entry = NAN;  // as the rest of its row
    const float rounded = __uint_as_float(pack_bf16x2(entry, 0.f) << 16);
    c0[t] = f0;
    c1[t] = f1;
    hit[t] = rounded;
    rest[t] = entry - rounded;
    ref[t] = from;
    rows.row_of[t] = target ? tok : -1;
    if (target) {
      const int n = atomicAdd(&rows.count[tok], 1);
      rows.order[t] = n;
      if (n < kMaxTargets) rows.token_of[static_cast<size_t>(tok) * kMaxTargets + n] = static_cast<int>(t);
      if (n == kMaxTargets) {
        const int slot = atomicAdd(rows.counter(kShared), 1);
        rows.shared[slot] = tok;
        rows.slot_of[tok] = slot;
      }
    }
  }
  // the last block to come here gives each shared row its part of the list
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(rows.counter(kBlocksDone), 1) == static_cast<int>(gridDim.x) - 1 ? 1 : 0;
  __syncthreads();
  if (last == 0) return;
  __threadfence();
  const int shared = __ldcg(rows.counter(kShared));
  for (int i = static_cast<int>(threadIdx.x); i < shared; i += kRowThreads) {
    const int n = __ldcg(&rows.count[__ldcg(&rows.shared[i])]);
    rows.base_of[i] = atomicAdd(rows.counter(kListed), n);
    if (n > kMostFew) rows.longs[atomicAdd(rows.counter(kLong), 1)] = i;
  }
}

// A product of few rows loads the same few lines for every tile: such rows are padded with zeros to kLeastRows (one
// token against a 201088 x 2880 head took 282 us, 64 tokens 199).
constexpr int kLeastRows = 64;

// What is laid out for a block of tokens before its products; each part is left out where its destination is NULL.
struct RowJobs {
  const uint4* H;        // [rows][per_row], 8 values each
  const uint8_t* mask;   // of these rows, or NULL
  int64_t rows;
  int per_row;
  uint4* few;            // [kLeastRows][per_row]: H, padded
  // [rows][per_row]: H for dW, with zeros in the rows that the mask leaves out: their dS is 0, but 0 times
  // the NaN or infinity that such a row may hold would be none
  uint4* clean;
  // [rows][per_row] fp32: where dH's sums start, rest_t W[v*_t] (added to what is there where `add`)
  float4* start;
  const uint4* W;
  TokenIds tokens;       // of all tokens: row t is token r0 + t
  int64_t r0;
  const float* rest;     // of these rows
  int V, add;
  TargetRows list;       // the list of the shared rows' tokens is filled in, where `listed` is not 0
  int64_t listed;        // tokens of the batch
};

__global__ void __launch_bounds__(kRowThreads) row_jobs_kernel(const RowJobs p) {
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; t < p.listed;
       t += static_cast<int64_t>(gridDim.x) * kRowThreads) {
    const int row = p.list.row_of[t];
    if (row >= 0 && p.list.count[row] > kMaxTargets)
      p.list.list[p.list.base_of[p.list.slot_of[row]] + p.list.order[t]] = static_cast<int>(t);
  }
  if (p.few == nullptr && p.clean == nullptr && p.start == nullptr) return;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int64_t all = p.few != nullptr && p.rows < kLeastRows ? kLeastRows : p.rows;
  for (int64_t t = blockIdx.x; t < all; t += gridDim.x) {
    const bool in = t < p.rows, on = in && (p.mask == nullptr || p.mask[t] != 0);
    const float r = p.start != nullptr && in ? p.rest[t] : 0.f;
    const int tok = r != 0.f ? p.tokens.get(p.r0 + t, p.V) : -1;
    for (int i = static_cast<int>(threadIdx.x); i < p.per_row; i += kRowThreads) {
      const int64_t at = t * p.per_row + i;
      if (p.few != nullptr) p.few[at] = in ? p.H[at] : zero;
      if (!in) continue;
      if (p.clean != nullptr) p.clean[at] = on ? p.H[at] : zero;
      if (p.start != nullptr) {
        float4* o = p.start + at * 2;
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        if (p.add) {
          lo = o[0];
          hi = o[1];
        }
        if (tok >= 0) {
          const uint4 w = p.W[static_cast<int64_t>(tok) * p.per_row + i];
          add_bf16x2(lo.x, lo.y, w.x, r);
          add_bf16x2(lo.z, lo.w, w.y, r);
          add_bf16x2(hi.x, hi.y, w.z, r);
          add_bf16x2(hi.z, hi.w, w.w, r);
        }
        o[0] = lo;
        o[1] = hi;
      }
    }
  }
}

cudaError_t launch_row_jobs(const RowJobs& p, int sms, cudaStream_t st) {
  if (p.few == nullptr && p.clean == nullptr && p.start == nullptr && p.listed == 0) return cudaSuccess;
  const int64_t rows = p.rows < kLeastRows ? kLeastRows : p.rows;
  row_jobs_kernel<<<static_cast<unsigned>(rows < 8 * sms ? rows : 8 * sms), kRowThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- behind the products
struct FinishJobs {
  const uint32_t* status;
  void *dH, *dW;          // either may be NULL
  int64_t nh, nw;         // their values
  TargetRows targets;
  const uint4* H;         // [T][per_row]
  const float* rest;      // [T]
  const float4* held;     // [shared row][per_row] fp32: such rows of a bf16 dW (DwParams)
  int64_t T;
  int per_row;
};

// What rounding took from the tokens of a shared row, sum_t rest_t H_t in the order of tokens, is added to dW by a CTA
// (finish_few) or, for a long row, a cluster of them (finish_long).  A thread has up to two vectors of 8 columns; where a
// row has fewer vectors than the CTA threads, groups of threads take equal parts of the list.  The groups' sums, then the
// CTAs', are added in order, so that the bits are always the same.
//
// What bounds it is the latency of a few dependent reads for each row, and of a row's tokens one batch of 8 after another,
// for which two CTAs of 128 registers are left to an SM.  With tokens drawn by 1 / rank: 16384 of a 50257 x 2880
// head 67 us of 8.9 ms; 8192 of a 1000 x 2880 one, the longest row 1100 of them, 48 (a CTA to a row 99, a cluster to
// every row 154).  No shared row: 3 us, as the check for errors takes alone.
constexpr int kScan = 4 * kRowThreads;
constexpr int kLongCluster = 8;

struct FinishShared {
  int list[kScan];
  float taken[kScan];  // rest of the listed tokens
  int raw[kMostFew];
  int warp_found[kRowThreads / 32];
  float4 part[2][kRowThreads][2];
};

// How a CTA's threads share a row's vectors.
struct Columns {
  int width, groups, group, c, span;  // vectors of a group; this thread's group and place in it; vectors at a time
  __device__ __forceinline__ explicit Columns(int per_row) {
    width = 32;
    while (width < per_row && width < kRowThreads) width *= 2;
    groups = kRowThreads / width;
    group = static_cast<int>(threadIdx.x) / width;
    c = static_cast<int>(threadIdx.x) - group * width;
    span = groups == 1 ? 2 * kRowThreads : width;
  }
};

__device__ __forceinline__ void add4(float4& s, const float4& v) {
  s.x += v.x;
  s.y += v.y;
  s.z += v.z;
  s.w += v.w;
}

// Adds the group's part of a list of n tokens: the columns of vector `at` and, where `two`, of at + kRowThreads.
__device__ __forceinline__ void add_listed(const FinishJobs& p, const FinishShared& s, const Columns& col, int n, int at,
                                           bool two, float4 (&v)[4]) {
  const int to = n * (col.group + 1) / col.groups;
#pragma unroll 8
  for (int i = n * col.group / col.groups; i < to; ++i) {
    const uint4* h = p.H + static_cast<int64_t>(s.list[i]) * p.per_row + at;
    const float f = s.taken[i];
    const uint4 x = h[0], y = two ? h[kRowThreads] : make_uint4(0u, 0u, 0u, 0u);
    add_bf16x2(v[0].x, v[0].y, x.x, f);
    add_bf16x2(v[0].z, v[0].w, x.y, f);
    add_bf16x2(v[1].x, v[1].y, x.z, f);
    add_bf16x2(v[1].z, v[1].w, x.w, f);
    add_bf16x2(v[2].x, v[2].y, y.x, f);
    add_bf16x2(v[2].z, v[2].w, y.y, f);
    add_bf16x2(v[3].x, v[3].y, y.z, f);
    add_bf16x2(v[3].z, v[3].w, y.w, f);
  }
}

// The groups' sums in the first one's places of s.part (a single group's too); a barrier has to follow.
__device__ __forceinline__ void join_groups(FinishShared& s, const Columns& col, float4 (&v)[4]) {
  const int tid = static_cast<int>(threadIdx.x);
#pragma unroll
  for (int k = 0; k < 4; ++k) s.part[k / 2][tid][k % 2] = v[k];
  if (col.groups == 1) return;
  __syncthreads();
  if (tid >= col.width) return;
  for (int g = 1; g < col.groups; ++g) {
    add4(v[0], s.part[0][g * col.width + tid][0]);
    add4(v[1], s.part[0][g * col.width + tid][1]);
  }
  s.part[0][tid][0] = v[0];  // this thread alone has read it
  s.part[0][tid][1] = v[1];
}

template <bool kBf16>
__device__ __forceinline__ void add_to_row(const FinishJobs& p, int slot, int row, int vec, float4 lo, float4 hi) {
  const int64_t at = static_cast<int64_t>(row) * p.per_row + vec;
  if constexpr (kBf16) {
    const float4* from = p.held + (static_cast<int64_t>(slot) * p.per_row + vec) * 2;
    add4(lo, from[0]);
    add4(hi, from[1]);
    static_cast<uint4*>(p.dW)[at] = make_uint4(pack_bf16x2(lo.x, lo.y), pack_bf16x2(lo.z, lo.w), pack_bf16x2(hi.x, hi.y),
                                               pack_bf16x2(hi.z, hi.w));
  } else {
    float4* o = static_cast<float4*>(p.dW) + 2 * at;
    add4(lo, o[0]);
    add4(hi, o[1]);
    o[0] = lo;
    o[1] = hi;
  }
}

// The shared rows that are not long, one to a CTA: their part of the list, sorted.
template <bool kBf16>
__device__ __forceinline__ void finish_few(const FinishJobs& p, FinishShared& s) {
  const Columns col(p.per_row);
  const int tid = static_cast<int>(threadIdx.x), shared = *p.targets.counter(kShared);
  for (int slot = static_cast<int>(blockIdx.x); slot < shared; slot += static_cast<int>(gridDim.x)) {
    const int row = p.targets.shared[slot], n = p.targets.count[row];
    if (n > kMostFew) continue;
    const int token = tid < n ? p.targets.list[p.targets.base_of[slot] + tid] : INT_MAX;
    const float rest = tid < n ? p.rest[token] : 0.f;
    __syncthreads();  // the row before is done with the shared memory
    if (tid < n) s.raw[tid] = token;
    __syncthreads();
    if (tid < n) {
      int place = 0;
      for (int j = 0; j < n; ++j) place += s.raw[j] < token ? 1 : 0;
      s.list[place] = token;
      s.taken[place] = rest;
    }
    __syncthreads();
    for (int first = 0; first < p.per_row; first += col.span) {  // once, where there are several groups
      const int at = first + col.c;
      const bool two = col.groups == 1 && at + kRowThreads < p.per_row;
      float4 v[4] = {};
      if (at < p.per_row) add_listed(p, s, col, n, at, two, v);
      if (col.groups > 1) join_groups(s, col, v);
      if (col.group == 0 && at < p.per_row) add_to_row<kBf16>(p, slot, row, at, v[0], v[1]);
      if (two) add_to_row<kBf16>(p, slot, row, at + kRowThreads, v[2], v[3]);
    }
  }
}

// The long rows, one to a cluster: each CTA looks through its share of all tokens, kScan at a time, and lists those of the
// row in order.
template <bool kBf16>
__device__ __forceinline__ void finish_long(const FinishJobs& p, FinishShared& s) {
  constexpr int kWarps = kRowThreads / 32;
  const Columns col(p.per_row);
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int ranks = cluster_size(), rank = static_cast<int>(cluster_ctarank());
  const int pieces = (p.per_row + col.span - 1) / col.span;
  const int64_t items = static_cast<int64_t>(*p.targets.counter(kLong)) * pieces;
  const int64_t share = (p.T + 4 * ranks - 1) / (4 * ranks) * 4, begin = rank * share;
  const int64_t end = begin + share < p.T ? begin + share : p.T;
  for (int64_t item = blockIdx.x / ranks; item < items; item += gridDim.x / ranks) {
    const int slot = p.targets.longs[item / pieces], first = static_cast<int>(item % pieces) * col.span;
    const int row = p.targets.shared[slot], at = first + col.c;
    const bool two = col.groups == 1 && at + kRowThreads < p.per_row;
    float4 v[4] = {};
    for (int64_t t0 = begin; t0 < end; t0 += kScan) {
      const int64_t t = t0 + tid * 4;
      int4 r = make_int4(-1, -1, -1, -1);
      if (t + 4 <= end) {
        r = *reinterpret_cast<const int4*>(p.targets.row_of + t);
      } else {
        if (t < end) r.x = p.targets.row_of[t];
        if (t + 1 < end) r.y = p.targets.row_of[t + 1];
        if (t + 2 < end) r.z = p.targets.row_of[t + 2];
      }
      const uint32_t found = (r.x == row ? 1u : 0u) | (r.y == row ? 2u : 0u) | (r.z == row ? 4u : 0u) | (r.w == row ? 8u : 0u);
      if (__syncthreads_count(found != 0) == 0) continue;  // also: the list before is read
      int upto = __popc(found);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) s.warp_found[warp] = upto;
      __syncthreads();
      int place = upto - __popc(found), n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) place += s.warp_found[w];
        n += s.warp_found[w];
      }
      for (uint32_t left = found; left != 0; left &= left - 1, ++place) {
        const int64_t token = t + (__ffs(left) - 1);
        s.list[place] = static_cast<int>(token);
        s.taken[place] = p.rest[token];
      }
      __syncthreads();
      if (at < p.per_row) add_listed(p, s, col, n, at, two, v);
    }
    join_groups(s, col, v);
    cluster_arrive();
    cluster_wait();
    const int q = tid * ranks + rank;  // every CTA adds up its share of the columns
    if (q < col.span && first + q < p.per_row) {
      const float4* mine = s.part[q / kRowThreads][q % kRowThreads];
      float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
#pragma unroll 8
      for (int k = 0; k < ranks; ++k) {
        const float4* theirs = peer(mine, k);
        add4(lo, theirs[0]);
        add4(hi, theirs[1]);
      }
      add_to_row<kBf16>(p, slot, row, first + q, lo, hi);
    }
    cluster_arrive();  // the sums are read: their memory may be written, or the CTA end
    cluster_wait();
  }
}

// The last launch of the backward: NaN in both gradients where the device recorded an error, else the shared rows.
template <bool kBf16>
__global__ void __launch_bounds__(kRowThreads, 2) finish_kernel(const FinishJobs p) {
  if (*reinterpret_cast<const volatile uint32_t*>(p.status) != 0u) {
    using T = std::conditional_t<kBf16, uint16_t, float>;
    T nan;
    if constexpr (kBf16) nan = 0x7FC0u; else nan = NAN;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRowThreads;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
    for (int64_t i = at; i < p.nh; i += stride) static_cast<T*>(p.dH)[i] = nan;
    for (int64_t i = at; i < p.nw; i += stride) static_cast<T*>(p.dW)[i] = nan;
    return;
  }
  if (p.nw == 0) return;
  __shared__ FinishShared s;
  finish_long<kBf16>(p, s);
  finish_few<kBf16>(p, s);
}

cudaError_t launch_finish(const FinishJobs& p, bool bf16, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * sms) / kLongCluster * kLongCluster);
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kLongCluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, finish_kernel<true>, p) : cudaLaunchKernelEx(&cfg, finish_kernel<false>, p);
}

unsigned row_blocks(int64_t T) { return static_cast<unsigned>((T + kRowThreads - 1) / kRowThreads); }

// ---------------------------------------------------------------- planning
// The loss's plan of the backward's blocks (with one pair a row, whose area is not used here).  It rounds slabs
// down to whole tiles; a batch that `chunk` takes at once has the whole vocabulary in one slab, rounded up,
// for the few columns that are left would cost a slab's launches of their own (54 us of 830 for 64 tokens).
bool score_plan(int64_t T, int64_t d, int64_t V, int64_t chunk, bool bf16, Plan* p) {
  if (!make_plan(T, d, V, 1, chunk, p, bf16)) return false;
  if (T > 0 && T <= chunk && p->nt == 1) {
    p->Vmax = p->Vc = ceil_div(V, kVocabTile) * kVocabTile;
    p->nslabs = 1;
  }
  return true;
}

// Partial tiles that dH's units may be cut into.
constexpr int kPieces = 160;

// The backward's workspace.
struct Areas {
  size_t c0, c1, hit, rest;   // float [T]: the factors of dS, its entry at the token and what rounding takes from it
  size_t ref;                 // float2 [T]: reference logit and log2 of the sum
  size_t count, token_of, slot_of, shared, base_of, longs, row_of, order, list;  // int: TargetRows
  size_t held;                // bf16 gradients: fp32 [T / (kMaxTargets + 1)][d], the shared rows of dW
  size_t few;                 // bf16 [kLeastRows][d]: see kLeastRows
  size_t clean;               // bf16 [Ct][d]: a block's hidden states without the rows that a mask leaves out
  size_t ds;                  // bf16 [Ct][Vmax]
  size_t pieces;              // fp32 [kPieces][256][256]
  size_t hsum, wsum;          // bf16 gradients: fp32 sums of dH over slabs and of dW over token blocks (see Plan)
  size_t total;
};
Areas backward_areas(const Plan& p, bool bf16) {
  size_t off = 256;  // status
  auto take = [&](int64_t elements, size_t bytes) {
    const size_t at = off;
    off = (off + static_cast<size_t>(elements) * bytes + 255) / 256 * 256;
    return at;
  };
  const bool sums = bf16 && p.T > 0;
  Areas a;
  a.count = take(p.V + kCounters, 4);  // zeroed with the status before it
  a.c0 = take(p.T, 4);
  a.c1 = take(p.T, 4);
  a.hit = take(p.T, 4);
  a.rest = take(p.T, 4);
  a.ref = take(p.T, 8);
  a.token_of = take(p.V * kMaxTargets, 4);
  a.slot_of = take(p.V, 4);
  a.shared = take(p.T / (kMaxTargets + 1), 4);
  a.base_of = take(p.T / (kMaxTargets + 1), 4);
  a.longs = take(p.T / (kMostFew + 1), 4);
  a.row_of = take(p.T, 4);
  a.order = take(p.T, 4);
  a.list = take(p.T, 4);
  a.held = take(sums ? p.T / (kMaxTargets + 1) * p.d : 0, 4);
  a.few = take(p.T > 0 ? kLeastRows * p.d : 0, 2);
  a.clean = take(p.Ct * p.d, 2);
  a.ds = take(p.Ct * p.Vmax, 2);
  a.pieces = take(p.T > 0 ? int64_t{kPieces} * 256 * 256 : 0, 4);
  a.hsum = take(sums ? (p.slab_outer ? p.T : p.Ct) * p.d : 0, 4);
  a.wsum = take(sums && p.nt > 1 ? (p.slab_outer ? p.Vmax : p.V) * p.d : 0, 4);
  a.total = off;
  return a;
}

// Cuts dH's units along K.  Where there are more units than CTA pairs, the last wave's, as in the loss.  Else all of
// them, into the number of pieces with the least time by this count: a wave's 64-deep steps at 645 cycles with 2500
// for a tile's start and end, and a pass that adds the pieces up.  Whole and in pieces, on the device, with the
// pass: 64 tokens of 201088 x 2880 836 and 191 us, 256 tokens 836 and 211, 1024 tokens (48 units on 76 pairs)
// 867 and 720; 512 of 32000 x 512 145 and 33, 1024 of 50257 x 512 220 and 49.
void plan_pieces(GemmShape* g, int pairs, float* pieces) {
  if (g->num_units >= pairs) {
    plan_ksplit(g, pairs, pieces, kKsplitSlots);
    return;
  }
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= 64 && s * g->num_units <= kPieces && (s == 1 || s * kKsplitMinBlocks <= g->k_blocks); ++s) {
    const double waves = static_cast<double>(ceil_div(static_cast<int64_t>(g->num_units) * s, pairs));
    const double time = waves * (ceil_div(g->k_blocks, s) * 645.0 + 2500.0) + (s > 1 ? 8000.0 + 1900.0 * s : 0.0);
    if (time < least) {
      least = time;
      best = s;
    }
  }
  if (best == 1) return;
  g->split_from = 0;
  g->ksplit = best;
  g->kpart = pieces;
}

// Splits of a row block's vocabulary for the forward.  Up to four row blocks have a unit to each CTA pair and
// block: the loss's rule, made for many blocks, leaves pairs idle there (1024 x 201088 x 2880: 724 us with its 64
// splits, 681 with 76; 300 tokens 376 and 350).
constexpr int kFewBlocks = 4, kFewSplits = 80;
int split_room(int64_t T) { return ceil_div(T, 256) <= kFewBlocks ? kFewSplits : kMaxSplit; }
int forward_splits(int m_tiles, int n_tiles, int pairs) {
  if (m_tiles > kFewBlocks) return dynamic_splits(m_tiles, n_tiles, pairs);
  const int s = pairs < kFewSplits ? pairs : kFewSplits;
  return s < n_tiles ? s : n_tiles;
}

// Splits of the logits' recompute in the backward, whose units are dealt round-robin: the loss's, at most 32,
// unless that is less than a unit to a pair.
int recompute_splits(int m_tiles, int n_tiles, int pairs) {
  const int s = plan_splits(m_tiles, n_tiles, pairs, group_rows(m_tiles));
  if (m_tiles * s >= pairs) return s;
  const int all = (pairs + m_tiles - 1) / m_tiles;
  return all < n_tiles ? all : n_tiles;
}

// Tile width along d of dW and dH: the one with the least time, by columns (padded ones too) and the measured
// time per column of each width.  256-wide tiles read the fewest operand bytes per product, so narrower ones
// (1.23 and 1.3 times the time a column) pay only where 256 pads far more.
int tile_width(int64_t d) {
  int best = 256;
  double least = 1e300;
  const struct { int bn; double cost; } widths[] = {{256, 1.0}, {192, 1.23}, {128, 1.3}};
  for (const auto& w : widths) {
    const double time = static_cast<double>(ceil_div(d, w.bn) * w.bn) * w.cost;
    if (time < least) {
      least = time;
      best = w.bn;
    }
  }
  return best;
}

// Map of an operand whose contiguous axis is the product's N (H for dW, the W slab for dH), half a tile
// wide: one 3-D box where the extent allows, 2-D boxes elsewhere; 64-byte swizzle for 96-wide halves.
bool map_columns(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, int bn, bool* box3d) {
  const bool narrow = (bn / 2) % 64 != 0;
  *box3d = narrow ? encode_map_mn3d_sw64(map, base, cols, rows, cols * 2, bn / 2)
                  : encode_map_mn3d(map, base, cols, rows, cols * 2, bn / 2);
  if (*box3d) return true;
  return narrow ? encode_map_bf16_sw64(map, base, cols, rows, cols * 2)
                : encode_map_bf16(map, base, cols, rows, cols * 2, 64, 64);
}

fkl_status fused_fail(fkl_status st, const char* msg) {
  set_last_error_message(msg);
  return st;
}
fkl_status fused_cuda(cudaError_t e) { return fused_fail(FKL_ERR_CUDA, cudaGetErrorString(e)); }

// Destination of a product that is summed over `count` blocks, of which this is number `at`: the caller's
// fp32 gradient, or fp32 sums in the workspace that the last block rounds to bf16.  accumulate: the first adds too.
F32Params destination(int64_t rows, int64_t d, int64_t at, int64_t count, float* out32, uint16_t* out16, float* sums,
                      bool accumulate) {
  F32Params p;
  p.ldo = d;
  p.M = static_cast<int>(rows);
  p.N = static_cast<int>(d);
  p.out = out16 == nullptr ? out32 : sums;
  p.accumulate = at > 0 || accumulate ? 1 : 0;
  p.vec_ok = on_boundary(p.out, 32) && d % 8 == 0 ? 1 : 0;
  if (out16 != nullptr && at == count - 1) {
    p.out16 = out16;
    p.ldo16 = d;
    p.vec16_ok = on_boundary(out16, 16) ? 1 : 0;
  }
  return p;
}

struct Backward {
  const uint16_t *H, *W;
  TokenIds tokens;
  const uint8_t* mask;
  int64_t T, d, V;
  float tau;
  int accumulate;
  bool bf16;
  void *dH, *dW;
  uint8_t* ws;
  int sms;
  cudaStream_t st;
  Plan pl;
  Areas at;
  template <class P>
  P* area(size_t off) const { return reinterpret_cast<P*>(ws + off); }
  TargetRows targets() const {
    return TargetRows{area<int>(at.count),  area<int>(at.token_of), area<int>(at.slot_of),
                      area<int>(at.shared), area<int>(at.base_of),  area<int>(at.longs),
                      area<int>(at.row_of), area<int>(at.order),    area<int>(at.list), static_cast<int>(V)};
  }
};

// One block: tokens [b Ct, ...) x vocabulary columns [j Vc, ...).
fkl_status score_block(const Backward& c, int64_t b, int64_t j) {
  const Plan& pl = c.pl;
  const int64_t d = c.d, Vc = pl.Vc, r0 = b * pl.Ct, v0 = j * Vc;
  const int64_t rows = c.T - r0 < pl.Ct ? c.T - r0 : pl.Ct, w = c.V - v0 < Vc ? c.V - v0 : Vc;
  const uint16_t *Hb = c.H + r0 * d, *Wj = c.W + v0 * d;
  uint16_t* ds = c.area<uint16_t>(c.at.ds);
  uint32_t* status = reinterpret_cast<uint32_t*>(c.ws);
  float* pieces = c.area<float>(c.at.pieces);
  const int bn = tile_width(d), pairs = c.sms / 2;
  const bool padded = rows < kLeastRows, cleaned = c.mask != nullptr && c.dW != nullptr;
  // slabs outer: the areas of a token block may hold another block's rows by now
  const bool again = pl.slab_outer && pl.nt > 1;
  const F32Params ph = destination(rows, d, j, pl.nslabs, static_cast<float*>(c.dH) + (c.bf16 ? 0 : r0 * d),
                                   c.bf16 ? static_cast<uint16_t*>(c.dH) + r0 * d : nullptr,
                                   c.area<float>(c.at.hsum) + (pl.slab_outer ? r0 * d : 0), true);
  RowJobs jobs{};
  jobs.H = reinterpret_cast<const uint4*>(Hb);
  jobs.mask = c.mask != nullptr ? c.mask + r0 : nullptr;
  jobs.rows = rows;
  jobs.per_row = static_cast<int>(d / 8);
  jobs.few = padded && (j == 0 || again) ? c.area<uint4>(c.at.few) : nullptr;
  jobs.clean = cleaned && (j == 0 || again) ? c.area<uint4>(c.at.clean) : nullptr;
  jobs.start = c.dH != nullptr && j == 0 ? reinterpret_cast<float4*>(ph.out) : nullptr;
  jobs.W = reinterpret_cast<const uint4*>(c.W);
  jobs.tokens = c.tokens;
  jobs.r0 = r0;
  jobs.rest = c.area<const float>(c.at.rest) + r0;
  jobs.V = static_cast<int>(c.V);
  jobs.list = c.targets();
  jobs.listed = c.dW != nullptr && b == 0 && j == 0 ? c.T : 0;  // the first block of either order
  jobs.add = !c.bf16 && (c.accumulate & FKL_ACCUMULATE_DH) != 0 ? 1 : 0;
  cudaError_t e = launch_row_jobs(jobs, c.sms, c.st);
  if (e != cudaSuccess) return fused_cuda(e);
  const uint16_t *Ha = padded ? c.area<const uint16_t>(c.at.few) : Hb, *Hw = cleaned ? c.area<const uint16_t>(c.at.clean) : Hb;
  CUtensorMap h_rows, h_cols, w_rows, w_cols, ds_cols, ds_rows;
  bool h3d = false, w3d = false;
  // dS has zeros in the columns [w, round_up(w, 256)) of every row, so its 3-D view may span round_up(w, 64)
  const bool ds3d = encode_map_mn3d(&ds_cols, ds, ceil_div(w, 64) * 64, rows, Vc * 2, 128);
  if (!encode_map_bf16(&h_rows, Ha, d, padded ? kLeastRows : rows, d * 2, 64, 128) || !map_columns(&h_cols, Hw, d, rows, bn, &h3d) ||
      !encode_map_bf16(&w_rows, Wj, d, w, d * 2, 64, kVocabTile / 2) || !map_columns(&w_cols, Wj, d, w, bn, &w3d) ||
      (!ds3d && !encode_map_bf16(&ds_cols, ds, w, rows, Vc * 2, 64, 64)) ||
      !encode_map_bf16(&ds_rows, ds, w, rows, Vc * 2, 64, 128))
    return fused_fail(FKL_ERR_CUDA, "cuTensorMapEncodeTiled failed");

  const int m_tiles = static_cast<int>(ceil_div(rows, 256)), n_tiles = static_cast<int>(ceil_div(w, kVocabTile));
  GemmShape g = make_shape(rows, w, d, kVocabTile, recompute_splits(m_tiles, n_tiles, pairs), status, 256);
  g.group_m = group_rows(m_tiles);
  ScoreDsParams p;
  p.tokens = c.tokens;
  p.r0 = r0;
  p.c0 = c.area<const float>(c.at.c0) + r0;
  p.c1 = c.area<const float>(c.at.c1) + r0;
  p.hit = c.area<const float>(c.at.hit) + r0;
  p.ref = c.area<const float2>(c.at.ref) + r0;
  p.ds = ds;
  p.ld_ds = Vc;
  p.T = static_cast<int>(rows);
  p.V = static_cast<int>(c.V);
  p.v0 = static_cast<int>(v0);
  p.slab_w = static_cast<int>(w);
  p.scale2 = kLog2e / c.tau;
  if ((e = launch_gemm2_t<kVocabTile, false, false, EpiScoreDs>(h_rows, w_rows, g, p, c.sms, c.st)) != cudaSuccess)
    return fused_cuda(e);

  if (c.dW != nullptr) {  // dW[slab] (+)= dS[block]^T H[block], token blocks in order
    float* wsum = c.area<float>(c.at.wsum) + (pl.slab_outer ? 0 : v0 * d);
    // Few tokens' tiles are short: four to a unit share its start (64 tokens, dW alone 557 -> 502 us; beyond
    // 256 tokens a unit of one tile balances better, 512 tokens 798 against 833).
    const int64_t d_tiles = ceil_div(d, bn);
    GemmShape gw = make_shape(w, d, rows, bn, static_cast<int>(rows <= 256 ? ceil_div(d_tiles, 4) : d_tiles), status, 256);
    gw.a_box3d = ds3d ? 1 : 0;
    gw.b_box3d = h3d ? 1 : 0;
    DwParams pw;
    pw.to = destination(w, d, b, pl.nt, static_cast<float*>(c.dW) + (c.bf16 ? 0 : v0 * d),
                        c.bf16 ? static_cast<uint16_t*>(c.dW) + v0 * d : nullptr, wsum,
                        !c.bf16 && (c.accumulate & FKL_ACCUMULATE_DW) != 0);
    pw.wide16 = on_boundary(pw.to.out16, 32) && d % 16 == 0 ? 1 : 0;
    pw.H = c.H;
    pw.rest = c.area<const float>(c.at.rest);
    // what rounding took is added with the last block's sums
    pw.count = b == pl.nt - 1 ? c.area<const int>(c.at.count) + v0 : nullptr;
    pw.token_of = c.area<const int>(c.at.token_of) + v0 * kMaxTargets;
    pw.slot_of = c.area<const int>(c.at.slot_of) + v0;
    pw.held = c.area<float>(c.at.held);
    if ((e = launch_score_dw(bn, ds_cols, h_cols, gw, pw, c.sms, c.st)) != cudaSuccess) return fused_cuda(e);
  }
  if (c.dH == nullptr) return FKL_OK;

  // dH[block] (what rounding took from the tokens' entries, above) += dS[block] W[slab], slabs in order
  GemmShape gh = make_shape(rows, d, w, bn, static_cast<int>(ceil_div(d, bn)), status, 256);
  gh.b_box3d = w3d ? 1 : 0;
  plan_pieces(&gh, pairs, pieces);
  if ((e = launch_gemm2_f32(bn, false, true, ds_rows, w_cols, gh, ph, c.sms, c.st)) != cudaSuccess ||
      (e = launch_ksplit_fixup(bn, gh, ph, c.st)) != cudaSuccess)
    return fused_cuda(e);
  return FKL_OK;
}

// What both directions check.
fkl_status check_fused(const uint16_t* H, const uint16_t* W, const void* tokens, int32_t token_bytes, int64_t T,
                       float tau, const void* ws, size_t ws_bytes, size_t need) {
  if (!(tau > 0.f) || !std::isfinite(tau) || !std::isfinite(kLog2e / tau))
    return fused_fail(FKL_ERR_INVALID_ARG, "tau must be finite and > 0, and its inverse too (4.25e-39 and more)");
  if (token_bytes != 4 && token_bytes != 8) return fused_fail(FKL_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
  if (W == nullptr || (T > 0 && (H == nullptr || tokens == nullptr)))
    return fused_fail(FKL_ERR_INVALID_ARG, "H, W and tokens must not be NULL");
  if (!on_boundary(H, 16) || !on_boundary(W, 16)) return fused_fail(FKL_ERR_ALIGNMENT, "H and W must be 16-byte aligned");
  if (!on_boundary(tokens, token_bytes)) return fused_fail(FKL_ERR_ALIGNMENT, "tokens must be aligned to their type");
  if (ws == nullptr || ws_bytes < need) return fused_fail(FKL_ERR_WORKSPACE, "workspace missing or too small");
  if (!on_boundary(ws, 256)) return fused_fail(FKL_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return FKL_OK;
}
constexpr char kShapeRule[] = "unsupported shape (need 0 <= T < 2^31, d % 8 == 0, 8 <= d < 2^20, 1 <= V <= 2^30, chunk >= 1)";

// Workspace of the forward: the status, the partials of the splits and the tokens' logits.
struct ForwardPlan {
  size_t part, token_s, few, total;
};
bool forward_plan(int64_t T, int64_t d, int64_t V, ForwardPlan* p) {
  Plan pl;
  if (!score_plan(T, d, V, 1, false, &pl)) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p->part = 256;
  p->token_s = up(p->part + static_cast<size_t>(T) * 3 * split_room(T) * 4);
  p->few = up(p->token_s + static_cast<size_t>(T) * 4);
  p->total = up(p->few + (T > 0 ? static_cast<size_t>(kLeastRows) * d * 2 : 0));
  return true;
}

}  // namespace
}  // namespace fkl

using namespace fkl;

extern "C" size_t fkl_logprob_workspace_size(int64_t T, int64_t d, int64_t V) {
  ForwardPlan p;
  return forward_plan(T, d, V, &p) ? p.total : 0;
}

extern "C" size_t fkl_logprob_backward_workspace_size(int64_t T, int64_t d, int64_t V, int64_t chunk, int32_t grad_bf16) {
  Plan p;
  return score_plan(T, d, V, chunk, grad_bf16 != 0, &p) ? backward_areas(p, grad_bf16 != 0).total : 0;
}

extern "C" fkl_status fkl_logprob_forward_ex(const uint16_t* H, const uint16_t* W, const void* tokens,
                                             int32_t token_bytes, const uint8_t* mask, int64_t T, int64_t d, int64_t V,
                                             float tau, float* logprob, float* entropy, float* lse, float* stats,
                                             void* workspace, size_t ws_bytes, void* stream) {
  set_last_error_message("");
  ForwardPlan pl;
  if (!forward_plan(T, d, V, &pl)) return fused_fail(FKL_ERR_INVALID_ARG, kShapeRule);
  fkl_status s = check_fused(H, W, tokens, token_bytes, T, tau, workspace, ws_bytes, pl.total);
  if (s != FKL_OK) return s;
  if (T > 0 && (logprob == nullptr || entropy == nullptr))
    return fused_fail(FKL_ERR_INVALID_ARG, "logprob and entropy must not be NULL");
  if (!on_boundary(logprob, 4) || !on_boundary(entropy, 4) || !on_boundary(lse, 4) || !on_boundary(stats, 4))
    return fused_fail(FKL_ERR_ALIGNMENT, "logprob, entropy, lse and stats must be 4-byte aligned");
  int sms = 0;
  if (const int e = require_device(&sms); e != FKL_OK) return static_cast<fkl_status>(e);
  const NamedPtr ptrs[] = {{H, "H"}, {W, "W"}, {tokens, "tokens"}, {mask, "mask"}, {logprob, "logprob"},
                           {entropy, "entropy"}, {lse, "lse"}, {stats, "stats"}, {workspace, "workspace"}};
  if (const int e = check_device_memory(ptrs); e != FKL_OK) return static_cast<fkl_status>(e);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws);
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return fused_cuda(e);
  if (T == 0) return FKL_OK;
  CUtensorMap mH, mW;
  RowJobs jobs{};
  jobs.H = reinterpret_cast<const uint4*>(H);
  jobs.rows = T;
  jobs.per_row = static_cast<int>(d / 8);
  jobs.few = T < kLeastRows ? reinterpret_cast<uint4*>(ws + pl.few) : nullptr;
  if ((e = launch_row_jobs(jobs, sms, st)) != cudaSuccess) return fused_cuda(e);
  if (!encode_map_bf16(&mH, jobs.few != nullptr ? reinterpret_cast<const uint16_t*>(jobs.few) : H, d,
                       jobs.few != nullptr ? kLeastRows : T, d * 2, 64, 128) ||
      !encode_map_bf16(&mW, W, d, V, d * 2, 64, kVocabTile / 2))
    return fused_fail(FKL_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  const int m_tiles = static_cast<int>(ceil_div(T, 256)), n_tiles = static_cast<int>(ceil_div(V, kVocabTile));
  GemmShape g = make_shape(T, V, d, kVocabTile, forward_splits(m_tiles, n_tiles, sms / 2), &hdr->status, 256);
  g.group_m = fwd_group_rows(m_tiles, sms / 2);
  g.sched = &hdr->items_taken;
  ScoreFwdParams p;
  p.tokens = TokenIds{tokens, token_bytes};
  p.mask = mask;
  p.part = reinterpret_cast<float*>(ws + pl.part);
  p.token_s = reinterpret_cast<float*>(ws + pl.token_s);
  p.T = static_cast<int>(T);
  p.V = static_cast<int>(V);
  p.nsplit = g.nsplit;
  p.scale2 = kLog2e / tau;
  if ((e = launch_gemm2_t<kVocabTile, false, false, EpiScore>(mH, mW, g, p, sms, st)) != cudaSuccess) return fused_cuda(e);
  score_rows_kernel<<<static_cast<unsigned>(ceil_div(T, 32)), kRowThreads, 0, st>>>(
      p.part, p.nsplit, p.token_s, p.tokens, mask, T, p.V, p.scale2, &hdr->status, logprob, entropy, lse, stats);
  if ((e = cudaGetLastError()) != cudaSuccess) return fused_cuda(e);
  return FKL_OK;
}

extern "C" fkl_status fkl_logprob_forward(const uint16_t* H, const uint16_t* W, const void* tokens, int32_t token_bytes,
                                          const uint8_t* mask, int64_t T, int64_t d, int64_t V, float tau,
                                          float* logprob, float* entropy, float* lse, void* workspace, size_t ws_bytes,
                                          void* stream) {
  if (T > 0 && lse == nullptr) return fused_fail(FKL_ERR_INVALID_ARG, "lse must not be NULL");
  return fkl_logprob_forward_ex(H, W, tokens, token_bytes, mask, T, d, V, tau, logprob, entropy, lse, nullptr, workspace,
                                ws_bytes, stream);
}

extern "C" fkl_status fkl_logprob_backward_ex(const uint16_t* H, const uint16_t* W, const void* tokens,
                                              int32_t token_bytes, const uint8_t* mask, const float* logprob,
                                              const float* entropy, const float* lse, const float* stats,
                                              const float* grad_logprob, const float* grad_entropy, int64_t T, int64_t d,
                                              int64_t V, float tau, int64_t chunk, int32_t grad_bf16, int32_t accumulate,
                                              void* dH, void* dW, void* workspace, size_t ws_bytes, void* stream) {
  set_last_error_message("");
  if (grad_bf16 != 0 && grad_bf16 != 1) return fused_fail(FKL_ERR_INVALID_ARG, "grad_bf16 must be 0 or 1");
  Backward c{H, W, TokenIds{tokens, token_bytes}, mask, T, d, V, tau, accumulate, grad_bf16 == 1, dH, dW,
             static_cast<uint8_t*>(workspace), 0, static_cast<cudaStream_t>(stream), Plan{}, Areas{}};
  if (!score_plan(T, d, V, chunk, c.bf16, &c.pl)) return fused_fail(FKL_ERR_INVALID_ARG, kShapeRule);
  c.at = backward_areas(c.pl, c.bf16);
  fkl_status s = check_fused(H, W, tokens, token_bytes, T, tau, workspace, ws_bytes, c.at.total);
  if (s != FKL_OK) return s;
  if (accumulate < 0 || accumulate > 3) return fused_fail(FKL_ERR_INVALID_ARG, "bad accumulate");
  if (c.bf16 && accumulate != 0) return fused_fail(FKL_ERR_INVALID_ARG, "bf16 gradients do not accumulate");
  if ((dW == nullptr && dH == nullptr) ||
      (T > 0 && (logprob == nullptr || entropy == nullptr || (lse == nullptr && stats == nullptr))))
    return fused_fail(FKL_ERR_INVALID_ARG, "logprob, entropy, one of lse and stats and one of dH and dW must not be NULL");
  if (!on_boundary(dH, 16) || !on_boundary(dW, 16)) return fused_fail(FKL_ERR_ALIGNMENT, "dH and dW must be 16-byte aligned");
  if (!on_boundary(logprob, 4) || !on_boundary(lse, 4) || !on_boundary(stats, 4) || !on_boundary(entropy, 4) ||
      !on_boundary(grad_logprob, 4) || !on_boundary(grad_entropy, 4))
    return fused_fail(FKL_ERR_ALIGNMENT, "logprob, entropy, lse, stats and the gradients must be 4-byte aligned");
  if (const int e = require_device(&c.sms); e != FKL_OK) return static_cast<fkl_status>(e);
  const NamedPtr ptrs[] = {{H, "H"}, {W, "W"}, {tokens, "tokens"}, {mask, "mask"}, {logprob, "logprob"},
                           {lse, "lse"}, {stats, "stats"}, {entropy, "entropy"}, {grad_logprob, "grad_logprob"}, {grad_entropy, "grad_entropy"}, {dH, "dH"}, {dW, "dW"},
                           {workspace, "workspace"}};
  if (const int e = check_device_memory(ptrs); e != FKL_OK) return static_cast<fkl_status>(e);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(c.ws);
  cudaError_t e = cudaMemsetAsync(c.ws, 0, T > 0 ? c.at.count + static_cast<size_t>(V + kCounters) * 4 : 256, c.st);
  if (e != cudaSuccess) return fused_cuda(e);
  if (T == 0) {
    if (dW != nullptr && !(accumulate & FKL_ACCUMULATE_DW) &&
        (e = cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * d * (c.bf16 ? 2 : 4), c.st)) != cudaSuccess)
      return fused_cuda(e);
    return FKL_OK;
  }
  choose_slab_width(&c.pl, c.sms / 2);
  score_factors_kernel<<<row_blocks(T), kRowThreads, 0, c.st>>>(
      c.tokens, mask, logprob, entropy, lse, stats, grad_logprob, grad_entropy, T, static_cast<int>(V), 1.f / tau,
      &hdr->status, c.area<float>(c.at.c0), c.area<float>(c.at.c1), c.area<float>(c.at.hit), c.area<float>(c.at.rest),
      c.area<float2>(c.at.ref), c.targets());
  if ((e = cudaGetLastError()) != cudaSuccess) return fused_cuda(e);
  const Plan& pl = c.pl;
  for (int64_t o = 0; o < (pl.slab_outer ? pl.nslabs : pl.nt); ++o)
    for (int64_t i = 0; i < (pl.slab_outer ? pl.nt : pl.nslabs); ++i)
      if ((s = score_block(c, pl.slab_outer ? i : o, pl.slab_outer ? o : i)) != FKL_OK) return s;
  FinishJobs jobs{};
  jobs.status = &hdr->status;
  jobs.dH = dH;
  jobs.dW = dW;
  jobs.nh = dH != nullptr ? T * d : 0;
  jobs.nw = dW != nullptr ? V * d : 0;
  jobs.targets = c.targets();
  jobs.H = reinterpret_cast<const uint4*>(H);
  jobs.rest = c.area<const float>(c.at.rest);
  jobs.held = c.area<const float4>(c.at.held);
  jobs.T = T;
  jobs.per_row = static_cast<int>(d / 8);
  e = launch_finish(jobs, c.bf16, c.sms, c.st);
  if (e != cudaSuccess) return fused_cuda(e);
  return FKL_OK;
}

extern "C" fkl_status fkl_logprob_backward(const uint16_t* H, const uint16_t* W, const void* tokens, int32_t token_bytes,
                                           const uint8_t* mask, const float* logprob, const float* entropy,
                                           const float* lse, const float* grad_logprob, const float* grad_entropy,
                                           int64_t T, int64_t d, int64_t V, float tau, int64_t chunk, int32_t grad_bf16,
                                           int32_t accumulate, void* dH, void* dW, void* workspace, size_t ws_bytes,
                                           void* stream) {
  return fkl_logprob_backward_ex(H, W, tokens, token_bytes, mask, logprob, entropy, lse, nullptr, grad_logprob,
                                 grad_entropy, T, d, V, tau, chunk, grad_bf16, accumulate, dH, dW, workspace, ws_bytes,
                                 stream);
}
