// The 8-bit product on the tensor cores, for more tokens than the dp4a kernel takes.
//
//     y[m][n] = (sum_k q_mk w_nk) * s_m * t_n
//
// sm_103a's fast tensor formats do not include 8-bit integers, but fp16 holds every int8 value
// exactly and the products of two (at most 2^14) add up exactly in fp32 up to 2^24.  So the
// weights stay in 8 bits in HBM, where reading them is what a generation step costs, and are
// turned into fp16 on the way to the tensor cores:
//
//   HBM --TMA--> shared memory (int8) --8 warps--> TMEM (fp16 A operand) --tcgen05.mma--> TMEM
//
// The weights are the A operand (256 rows of W per CTA pair, 128 per CTA), read from TMEM, so
// their fp16 form costs no shared-memory traffic; the tokens, quantised to fp16 integers by a
// kernel before, are the B operand in shared memory (up to 256 per tile, half per CTA).
//
// What bounds it (GB300, W 201088 x 2880): up to about 128 tokens the HBM reads of W, 579 MB, 86 us at
// the measured 6.78 TB/s: 16 tokens take 102 us on the device, 128 tokens 124 us with 103 MB of
// output.  Beyond, the tensor pipe: 4096 tokens 2.54 to 2.70 ms, as the clock under the power cap
// allows, 1760 to 1870 TFLOP/s (a bf16 library product: 1932 in a burst, 1704 sustained); a tile of
// more than 128 tokens has one accumulator, so its epilogue (about 1 us of 13) is not hidden.
//
// Roles per CTA (20 warps):
//   warps 0..7   convert: 128 rows x 128 k of int8 to fp16 in a TMEM slot; warps 0..3 take the
//                lower 64 k, warps 4..7 the upper (a warp reaches the 32 TMEM lanes of its
//                number modulo 4);
//   warps 8..15  epilogue: accumulator * s_m * t_n, rounded and stored; lane = row of W = n,
//                warps 8..11 and 12..15 take alternate groups of 32 tokens;
//   warp 16      TMA producer of W, warp 17 of the tokens;
//   warp 18      (even CTA) issues the MMAs.
// The work is tiles of 256 rows of W x one tile of tokens, walked in blocks of 128 or 256 k.  Tiles
// are dealt round-robin to the pairs.  Those that would leave many pairs idle in the last wave
// (or the only one) are a line of blocks cut into equal parts, one for each pair that shares it.  A
// tile that is cut has its fp32 partial sums in the workspace; the last of its parts to finish (per
// warp of the epilogue) adds them in the order of the parts, so the result does not depend on which
// one that is.  The cut tiles come first, so that adding them up overlaps the whole ones.
//
// The kernel starts while the tokens are still being quantised (programmatic launch): W's first
// blocks are loaded and converted meanwhile, and only what reads the tokens, their scales or the
// workspace's header waits.
#include <algorithm>

#include "fkl_gemm.cuh"
#include "fkl_generate.cuh"
#include "fkl_int8.h"
#include "fkl_types.cuh"

namespace fkl {

constexpr int kI8Threads = 640;
constexpr int kI8K = 128;  // k per 128-byte row of a W box: a block is p.sub of them
constexpr uint32_t kI8WBytes = 128 * kI8K;
constexpr int kI8MaxSlots = 7, kI8MaxStages = 10;
constexpr uint32_t kI8Ring = 224 * 1024;  // shared memory of both rings
constexpr size_t kI8Smem = kI8Ring + 1024 + 512;
constexpr uint32_t kI8ConvertWarps = 8, kI8EpiWarps = 8;

struct I8Params {
  int M, N, K;
  int nt;        // tokens per tile, a multiple of 16 up to 256
  int m_tiles, k_blocks;
  // TMEM: accs accumulators acc_cols columns apart (2 for tiles of up to 128 tokens, so that a
  // tile's epilogue runs beside the next tile's MMAs), then slots of 64 columns for W's fp16
  // blocks, with as many token blocks in shared memory; the rest of that holds int8 blocks of W.
  int accs, acc_cols, slots, w_stages;
  int tiles, rounds;     // tiles in all; whole tiles of a pair, at most
  long long cut_blocks;  // blocks of the cut tiles
  int cut_pairs;         // pairs that share them, each at least one
  const float* x_scale;
  const float* w_scale;
  void* out;
  int64_t ldo;
  int out_type, paired;  // paired: two adjacent 16-bit outputs share an aligned word
  float* part;   // [2 * cut_pairs][nt][256], where tiles are cut
  int* arrived;  // [pairs][16]
  uint32_t* status;
  uint64_t limit_ns;
};

// This pair's items: its part of the line of cut tiles, tile by tile, then its whole tiles.
struct I8Seq {
  long long at, end;  // in the line
  int round, tile, kb0, kb1;
  const int pair, pairs;
  __device__ I8Seq(const I8Params& p, int pair_, int pairs_) : pair(pair_), pairs(pairs_) {
    at = p.cut_blocks * min(pair, p.cut_pairs) / p.cut_pairs;
    end = p.cut_blocks * min(pair + 1, p.cut_pairs) / p.cut_pairs;
    round = 0;
    set(p);
  }
  __device__ __forceinline__ void set(const I8Params& p) {
    if (at < end) {
      const int t = static_cast<int>(at / p.k_blocks);
      tile = p.rounds * pairs + t;
      kb0 = static_cast<int>(at - static_cast<long long>(t) * p.k_blocks);
      kb1 = static_cast<int>(min(static_cast<long long>(p.k_blocks), kb0 + (end - at)));
    } else {
      tile = round * pairs + pair;
      kb0 = 0;
      kb1 = p.k_blocks;
    }
  }
  __device__ __forceinline__ bool more(const I8Params& p) const {
    return at < end || (round < p.rounds && tile < p.tiles);
  }
  __device__ __forceinline__ void next(const I8Params& p) {
    if (at < end)
      at += kb1 - kb0;
    else
      ++round;
    set(p);
  }
};

struct I8Ctx {
  uint32_t rank;
  bool even;
  int pair, pairs;
  uint32_t w0, x0, x_bytes;  // shared-memory rings; bytes of a token block (this CTA's half)
  uint32_t tmem_a;           // first column of the A slots
  uint32_t wfull0, wempty0, xfull0, afull0, empty0, tfull0, tempty0, drain;
  uint32_t tmem;
  WaitCtl ctl;
};

// Four int8 values as two pairs of fp16: with the sign bit flipped a byte u = v + 128 is the
// low byte of the fp16 number 1024 + u.
__device__ __forceinline__ void int8x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// A wait of a whole warp, with one answer for all of its lanes.  Each lane polls for itself, so when a
// wait runs out some may have given up while others saw the barrier complete; lanes that went on by
// their own answers would part for good and wait for each other without a limit at the next
// warp or block barrier.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl) {
  return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, ctl));
}
// The same for two barriers in the same phase, with one vote.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t then, uint32_t parity, const WaitCtl& ctl) {
  return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, ctl) && mbar_wait_cluster(then, parity, ctl));
}

template <int SUB>
__device__ void i8_w_producer(const CUtensorMap* tm, const I8Params& p, const I8Ctx& c) {
  int stage = 0;
  uint32_t phase = 0, issued = 0, issued_par = 0;
  bool ok = true;
  for (I8Seq q(p, c.pair, c.pairs); ok && q.more(p); q.next(p)) {
    const int row = (q.tile / p.m_tiles) * 256 + static_cast<int>(c.rank) * 128;
    for (int kb = q.kb0; kb < q.kb1; ++kb) {
      if (!mbar_wait(c.wempty0 + 8 * stage, phase ^ 1u, c.ctl)) { ok = false; break; }
      mbar_arrive_expect_tx(c.wfull0 + 8 * stage, SUB * kI8WBytes);
#pragma unroll
      for (int j = 0; j < SUB; ++j)
        tma_load_2d(c.w0 + (stage * SUB + j) * kI8WBytes, tm, c.wfull0 + 8 * stage, (kb * SUB + j) * kI8K, row);
      issued |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == p.w_stages) { stage = 0; phase ^= 1u; }
    }
  }
  for (int s = 0; s < p.w_stages; ++s)
    if ((issued >> s) & 1u) mbar_wait_drain(c.wfull0 + 8 * s, (issued_par >> s) & 1u, p.limit_ns);
}

template <int SUB>
__device__ void i8_x_producer(const CUtensorMap* tm, const I8Params& p, const I8Ctx& c) {
  int slot = 0;
  uint32_t phase = 0, issued = 0, issued_par = 0;
  bool ok = true;
  grid_dependency_wait();
  const uint32_t even_full = map_to_rank(c.xfull0, 0);
  const uint32_t half_bytes = static_cast<uint32_t>(p.nt / 2) * 128;  // 64 k of this CTA's tokens
  for (I8Seq q(p, c.pair, c.pairs); ok && q.more(p); q.next(p)) {
    const int row = (q.tile % p.m_tiles) * p.nt + static_cast<int>(c.rank) * (p.nt / 2);
    for (int kb = q.kb0; kb < q.kb1; ++kb) {
      if (!mbar_wait_cluster(c.empty0 + 8 * slot, phase ^ 1u, c.ctl)) { ok = false; break; }
      if (c.even) mbar_arrive_expect_tx(c.xfull0 + 8 * slot, 4 * SUB * half_bytes);
      const uint32_t to = c.x0 + slot * c.x_bytes;
#pragma unroll
      for (int j = 0; j < 2 * SUB; ++j)
        tma_load_2d_pair(to + j * half_bytes, tm, even_full + 8 * slot, kb * SUB * kI8K + 64 * j, row);
      issued |= 1u << slot;
      issued_par = (issued_par & ~(1u << slot)) | (phase << slot);
      if (++slot == p.slots) { slot = 0; phase ^= 1u; }
    }
  }
  if (c.even)  // the even CTA's phases count the copies of both
    for (int s = 0; s < p.slots; ++s)
      if ((issued >> s) & 1u) mbar_wait_drain(c.xfull0 + 8 * s, (issued_par >> s) & 1u, p.limit_ns);
}

// Convert warps: lane = row of W.  A row's 128 bytes lie in 16-byte pieces permuted by the
// TMA's swizzle (piece j of row r at j ^ (r & 7)), which spreads a warp's reads over all banks.
template <int SUB>
__device__ void i8_convert(const I8Params& p, const I8Ctx& c, int warp, int lane) {
  const int row = (warp & 3) * 32 + lane;
  const int upper = warp >> 2;  // which 64 of the block's 128 k
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t even_afull = map_to_rank(c.afull0, 0);
  int stage = 0, slot = 0;
  uint32_t wphase = 0, phase = 0;
  for (I8Seq q(p, c.pair, c.pairs); q.more(p); q.next(p)) {
    for (int kb = q.kb0; kb < q.kb1; ++kb) {
      if (!warp_wait(c.wfull0 + 8 * stage, wphase, c.ctl)) return;
      const uint32_t to = c.tmem_a + lanes + static_cast<uint32_t>(slot * (64 * SUB) + upper * 32);
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        const uint32_t base = c.w0 + (stage * SUB + j) * kI8WBytes + static_cast<uint32_t>(row) * 128;
        uint32_t h[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = ld_shared_v4(base + static_cast<uint32_t>(((upper * 4 + i) ^ (row & 7)) * 16));
          int8x4_to_half(v.x, h[8 * i + 0], h[8 * i + 1]);
          int8x4_to_half(v.y, h[8 * i + 2], h[8 * i + 3]);
          int8x4_to_half(v.z, h[8 * i + 4], h[8 * i + 5]);
          int8x4_to_half(v.w, h[8 * i + 6], h[8 * i + 7]);
        }
        if (j == SUB - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(c.wempty0 + 8 * stage);
        }
        if (j == 0) {
          if (!warp_wait(c.empty0 + 8 * slot, phase ^ 1u, c.ctl)) return;
          tc_fence_after();
        }
        tmem_st32(to + static_cast<uint32_t>(j * 64), h);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(even_afull + 8 * slot);
      if (++stage == p.w_stages) { stage = 0; wphase ^= 1u; }
      if (++slot == p.slots) { slot = 0; phase ^= 1u; }
    }
  }
}

// One thread issues, but the whole warp walks the loop: its operands are then the same for the
// warp as the compiler sees it and stay in uniform registers.  (With the loop inside the one
// thread's branch each MMA took about 50 cycles to issue, more than a tile of few tokens takes
// to execute.)
template <int SUB>
__device__ void i8_mma(const I8Params& p, const I8Ctx& c) {
  const uint32_t idesc = instr_desc_f16(256, p.nt);
  const uint32_t half_step = (static_cast<uint32_t>(p.nt / 2) * 128) >> 4;
  const uint64_t b_desc0 = smem_desc_sw128(c.x0, 16, 1024);
  const bool issuer = elect_one();
  int slot = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool ok = true;
  for (I8Seq q(p, c.pair, c.pairs); ok && q.more(p); q.next(p)) {
    if (!warp_wait(c.tempty0 + 8 * acc, acc_phase ^ 1u, c.ctl)) { ok = false; break; }
    tc_fence_after();
    const uint32_t d = c.tmem + static_cast<uint32_t>(acc * p.acc_cols);
    for (int kb = q.kb0; kb < q.kb1; ++kb) {
      if (!warp_wait(c.xfull0 + 8 * slot, c.afull0 + 8 * slot, phase, c.ctl)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t b0 = b_desc0 + ((static_cast<uint32_t>(slot) * c.x_bytes) >> 4);
      const uint32_t a0 = c.tmem_a + static_cast<uint32_t>(slot * (64 * SUB));
      const int slices = min(kI8K * SUB, p.K - kb * (kI8K * SUB)) / 16;
      const uint32_t first = kb == q.kb0 ? 0u : 1u;
      if (slices == 8 * SUB) {
        if (issuer) {
#pragma unroll
          for (int k = 0; k < 8 * SUB; ++k)
            tc_mma_f16_pair_ta(d, a0 + static_cast<uint32_t>(8 * k), b0 + ((k >> 2) * half_step + (k & 3) * 2), idesc,
                               k != 0 ? 1u : first);
        }
      } else {
        for (int k = 0; k < slices; ++k) {
          const uint64_t bk = b0 + ((k >> 2) * half_step + (k & 3) * 2);
          if (issuer) tc_mma_f16_pair_ta(d, a0 + static_cast<uint32_t>(8 * k), bk, idesc, k != 0 ? 1u : first);
        }
      }
      if (issuer) tc_commit_pair_mc(c.empty0 + 8 * slot, 0x3);
      __syncwarp();
      if (++slot == p.slots) { slot = 0; phase ^= 1u; }
    }
    if (!ok) break;
    if (issuer) tc_commit_pair_mc(c.tfull0 + 8 * acc, 0x3);
    __syncwarp();
    if (++acc == p.accs) { acc = 0; acc_phase ^= 1u; }
  }
  if (issuer) {
    tc_commit_pair(c.drain);
    mbar_wait_drain(c.drain, 0u, p.limit_ns);
  }
  __syncwarp();
}

// C tokens from m0 on of this lane's column n: scaled, rounded and stored.  A warp has one
// instruction stream, so this is counted in instructions: a whole group takes about 4 per
// value.  16-bit outputs: lanes 2i and 2i + 1 hold two adjacent columns; the even lane stores
// both of one token, the odd lane both of the next (p.paired).  The kernel starts before the tokens'
// scales are written, so they are not read as constant data (__ldg); ordinary loads stay behind the
// stores that may alias them, so a group's are all made before its first store (between the
// stores, 4096 x 201088 x 2880 took 2.86 ms, not 2.54).
template <class T, int C>
__device__ __forceinline__ void i8_store(const I8Params& p, const float (&v)[C], int m0, int m_end, int n, float ws,
                                         int lane) {
  T* out = static_cast<T*>(p.out);
  const int64_t ldo = p.ldo;
  const float2 ws2 = make_float2(ws, ws);
  const bool odd = lane & 1;
  const bool whole = m0 + C <= m_end && (n | 31) < p.N;  // the same for the whole warp
  if (whole && (sizeof(T) == 4 || p.paired)) {
    const float4* xs = reinterpret_cast<const float4*>(p.x_scale + m0);  // m0 is a multiple of 16
    T* o = sizeof(T) == 4 ? out + static_cast<int64_t>(m0) * ldo + n
                          : out + static_cast<int64_t>(m0 + (odd ? 1 : 0)) * ldo + (n & ~1);
    float4 scales[C / 4];
#pragma unroll
    for (int j = 0; j < C / 4; ++j) scales[j] = xs[j];
#pragma unroll
    for (int j = 0; j < C; j += 4) {
      const float4 s = scales[j / 4];
      const float2 a = fmul2(fmul2(make_float2(v[j], v[j + 1]), make_float2(s.x, s.y)), ws2);
      const float2 b = fmul2(fmul2(make_float2(v[j + 2], v[j + 3]), make_float2(s.z, s.w)), ws2);
      if constexpr (sizeof(T) == 4) {
        o[0] = a.x;
        o[ldo] = a.y;
        o[2 * ldo] = b.x;
        o[3 * ldo] = b.y;
      } else {
        const float oa = __shfl_xor_sync(0xffffffffu, odd ? a.x : a.y, 1);
        const float ob = __shfl_xor_sync(0xffffffffu, odd ? b.x : b.y, 1);
        *reinterpret_cast<uint32_t*>(o) = pack2<T>(odd ? oa : a.x, odd ? a.y : oa);
        *reinterpret_cast<uint32_t*>(o + 2 * ldo) = pack2<T>(odd ? ob : b.x, odd ? b.y : ob);
      }
      o += 4 * ldo;
    }
    return;
  }
  if (n >= p.N) return;
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (m0 + j < m_end)
      out[static_cast<int64_t>(m0 + j) * ldo + n] = from_float<T>(v[j] * p.x_scale[m0 + j] * ws);
}

template <int C>
__device__ __forceinline__ void i8_store_any(const I8Params& p, const float (&v)[C], int m0, int m_end, int n, float ws,
                                             int lane) {
  if (p.out_type == FKL_TYPE_F32)
    i8_store<float, C>(p, v, m0, m_end, n, ws, lane);
  else if (p.out_type == FKL_TYPE_BF16)
    i8_store<__nv_bfloat16, C>(p, v, m0, m_end, n, ws, lane);
  else
    i8_store<__half, C>(p, v, m0, m_end, n, ws, lane);
}

// When a wait has run out: NaN in place of what this warp of the epilogue has not stored, so that a
// failed launch cannot pass for a result.  A tile that is cut gets it too: its parts are added up by
// the last warp to arrive, and this one does not.
__device__ __noinline__ void i8_unfinished(const I8Params& p, I8Seq q, int row, int half) {
  for (; q.more(p); q.next(p)) {
    const int n = (q.tile / p.m_tiles) * 256 + row;
    const int m0 = (q.tile % p.m_tiles) * p.nt;
    const int m_end = min(p.M, m0 + p.nt);
    if (n >= p.N) continue;
    for (int col = 32 * half; m0 + col < m_end; col += 64)
      for (int m = m0 + col; m < min(m_end, m0 + col + 32); ++m) {
        const int64_t at = static_cast<int64_t>(m) * p.ldo + n;
        if (p.out_type == FKL_TYPE_F32)
          static_cast<uint32_t*>(p.out)[at] = 0x7fffffffu;
        else
          static_cast<uint16_t*>(p.out)[at] = 0x7fffu;  // NaN in both 16-bit types
      }
  }
}

// The pair whose part of the line of cut tiles holds block x.
__device__ __forceinline__ int i8_owner(const I8Params& p, long long x) {
  return static_cast<int>(((x + 1) * p.cut_pairs - 1) / p.cut_blocks);
}

__device__ void i8_epilogue(const I8Params& p, const I8Ctx& c, int warp, int lane) {
  const int strip = warp & 3, half = (warp >> 2) & 1;
  const int row = static_cast<int>(c.rank) * 128 + strip * 32 + lane;  // of the pair's 256
  const uint32_t lanes = static_cast<uint32_t>(strip * 32) << 16;
  const uint32_t even_tempty = map_to_rank(c.tempty0, 0);
  int acc = 0;
  uint32_t acc_phase = 0;
  grid_dependency_wait();
  for (I8Seq q(p, c.pair, c.pairs); q.more(p); q.next(p)) {
    const int n = (q.tile / p.m_tiles) * 256 + row;
    const int m0 = (q.tile % p.m_tiles) * p.nt;
    const int m_end = min(p.M, m0 + p.nt);
    const float ws = n < p.N ? p.w_scale[n] : 0.f;
    const bool whole = q.kb1 - q.kb0 == p.k_blocks;
    float* part = p.part + static_cast<size_t>(2 * c.pair + (q.kb0 == 0 ? 1 : 0)) * p.nt * 256 + row;
    if (!warp_wait(c.tfull0 + 8 * acc, acc_phase, c.ctl)) {
      i8_unfinished(p, q, row, half);
      return;
    }
    tc_fence_after();
    const uint32_t t = c.tmem + lanes + static_cast<uint32_t>(acc * p.acc_cols);
#pragma unroll 1
    for (int col = 32 * half; m0 + col < m_end; col += 64) {
      float v[32];
      tmem_ld32(t + col, v);
      tmem_ld_wait(v);
      if (whole) {
        i8_store_any(p, v, m0 + col, m_end, n, ws, lane);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (m0 + col + j < m_end) part[static_cast<size_t>(col + j) * 256] = v[j];
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(even_tempty + 8 * acc);
    if (++acc == p.accs) { acc = 0; acc_phase ^= 1u; }
    if (whole) continue;
    // a cut tile: the last part to arrive adds them all up, in their order
    const long long first = static_cast<long long>(q.tile - p.rounds * c.pairs) * p.k_blocks;
    const int p0 = i8_owner(p, first), p1 = i8_owner(p, first + p.k_blocks - 1);
    __threadfence();
    __syncwarp();
    int before = 0;
    if (lane == 0) before = atomicAdd(p.arrived + p0 * 16 + static_cast<int>(c.rank) * 8 + half * 4 + strip, 1);
    before = __shfl_sync(0xffffffffu, before, 0);
    if (before != p1 - p0) continue;
    __threadfence();
#pragma unroll 1
    for (int col = 32 * half; m0 + col < m_end; col += col % 32 ? 48 : 16) {
      // Two parts' loads are in flight at once.  Columns past m_end are read, not stored.
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
      // the tile's first part is the last of its pair, the others the first of theirs
      const size_t part_step = static_cast<size_t>(p.nt) * 256;
      const float* src = p.part + (2 * p0 + 1) * part_step + static_cast<size_t>(col) * 256 + row;
      for (int r = p0; r <= p1; r += 2) {
        float u[2][16];
        const float* from = r == p0 ? src : src + (2 * (r - p0) - 1) * part_step;
        const float* then = r < p1 ? src + (2 * (r + 1 - p0) - 1) * part_step : from;
#pragma unroll
        for (int j = 0; j < 16; ++j) u[0][j] = __ldcg(from + j * 256);
#pragma unroll
        for (int j = 0; j < 16; ++j) u[1][j] = __ldcg(then + j * 256);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += u[0][j];
        if (r < p1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += u[1][j];
        }
      }
      i8_store_any(p, v, m0 + col, m_end, n, ws, lane);
    }
  }
}

// SUB: 128-k pieces per block.
template <int SUB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ I8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kI8Ring);
  constexpr int kBars = 2 * kI8MaxStages + 3 * kI8MaxSlots + 5;
  static_assert(kBars * 8 + 8 <= 512, "barriers and words fit in their 512 bytes");
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + kBars);  // [0] TMEM base, [1] abort
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  I8Ctx c;
  c.rank = cluster_ctarank();
  c.even = c.rank == 0;
  c.pair = static_cast<int>(blockIdx.x >> 1);
  c.pairs = static_cast<int>(gridDim.x >> 1);
  c.w0 = smem_addr(smem);
  c.x0 = c.w0 + static_cast<uint32_t>(p.w_stages * SUB) * kI8WBytes;
  c.x_bytes = static_cast<uint32_t>(p.nt / 2) * (kI8K * 2 * SUB);
  c.wfull0 = smem_addr(bars);
  c.wempty0 = c.wfull0 + 8 * kI8MaxStages;
  c.xfull0 = c.wempty0 + 8 * kI8MaxStages;
  c.afull0 = c.xfull0 + 8 * kI8MaxSlots;
  c.empty0 = c.afull0 + 8 * kI8MaxSlots;
  c.tfull0 = c.empty0 + 8 * kI8MaxSlots;
  c.tempty0 = c.tfull0 + 16;
  c.drain = c.tempty0 + 16;
  c.ctl = WaitCtl{reinterpret_cast<volatile uint32_t*>(&misc[1]), p.status, p.limit_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.w_stages; ++s) {
      mbar_init(c.wfull0 + 8 * s, 1);
      mbar_init(c.wempty0 + 8 * s, kI8ConvertWarps);
    }
    for (int s = 0; s < p.slots; ++s) {
      mbar_init(c.xfull0 + 8 * s, 1);
      mbar_init(c.afull0 + 8 * s, 2 * kI8ConvertWarps);
      mbar_init(c.empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(c.tfull0 + 8 * b, 1);
      mbar_init(c.tempty0 + 8 * b, 2 * kI8EpiWarps);
    }
    mbar_init(c.drain, 1);
    misc[1] = 0u;
    fence_barrier_init();
  }
  if (warp == 16 && lane == 0) tma_prefetch_desc(&tmW);
  if (warp == 17 && lane == 0) tma_prefetch_desc(&tmX);
  if (warp == 18) {
    tmem_alloc_pair(smem_addr(&misc[0]), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  c.tmem = misc[0];
  c.tmem_a = c.tmem + static_cast<uint32_t>(p.accs * p.acc_cols);

  if (warp < 8) {
    i8_convert<SUB>(p, c, warp, lane);
  } else if (warp < 16) {
    i8_epilogue(p, c, warp, lane);
  } else if (warp == 18) {
    if (c.even) i8_mma<SUB>(p, c);
  } else if (lane == 0) {
    if (warp == 16) i8_w_producer<SUB>(&tmW, p, c);
    if (warp == 17) i8_x_producer<SUB>(&tmX, p, c);
  }

  grid_dependency_wait();  // every thread: the launch's order holds for what follows it, too
  __syncwarp();
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 18) tmem_dealloc_pair(c.tmem, kTmemCols);
}

// ---------------------------------------------------------------- host side
Int8GemmPlan plan_int8_gemm(int64_t M, int64_t N, int64_t K, int sms) {
  Int8GemmPlan g;
  // Measured: a block of 128 k takes a pair 0.36 us (W from HBM) or nt / 256 * 0.55 us (MMAs).
  const auto tile_time = [&](int64_t nt) { return static_cast<double>(K) / kI8K * std::max(0.36, nt / 256.0 * 0.55); };
  // Tiles of up to 256 tokens, or of up to 128 with a second accumulator that hides the epilogue: a
  // wave of tiles then costs about 2 us beyond its blocks, not 5, but there are more waves, and each
  // converts W once more.  256 against 128 tokens, in us on the device: 512 x 4096 x 4096 27.2, 21.5;
  // 512 x 50261 x 1456 94.2, 74.8; 350 x 65536 x 640 44.5, 38.8; 1024 x 4096 x 4096 30.3, 37.0;
  // 203 x 151936 x 4096 177, 225; 640 x 20000 x 5120 98.0, 108.7.  It misses where a tile has somewhat
  // more than 200 tokens and few blocks: 700 x 50261 x 1456 gets 256 (121.4, 105.0).
  const int64_t n_tiles = (N + 255) / 256, most_pairs = std::min(sms / 2, kMaxPairs);
  const auto waves_time = [&](int64_t m_tiles) {
    const int64_t nt = (M + m_tiles - 1) / m_tiles;
    return static_cast<double>((n_tiles * m_tiles + most_pairs - 1) / most_pairs) * (tile_time(nt) + (nt > 128 ? 5.0 : 2.0));
  };
  const int64_t large = (M + 255) / 256, small = (M + 127) / 128;
  g.m_tiles = static_cast<int>(waves_time(small) < waves_time(large) ? small : large);
  const int64_t even = (M + g.m_tiles - 1) / g.m_tiles;
  g.nt = static_cast<int>((even + 15) / 16 * 16);
  // TMEM: the accumulators, then the slots.  Blocks of 256 k (half as many hand-offs) where at
  // least 3 such slots fit.
  g.accs = g.nt <= 128 ? 2 : 1;
  g.acc_cols = (g.nt + 31) / 32 * 32;
  const int cols = static_cast<int>(kTmemCols) - g.accs * g.acc_cols;
  g.sub = cols >= 3 * 128 ? 2 : 1;
  g.slots = std::min(kI8MaxSlots, cols / (64 * g.sub));
  g.w_stages = std::min<int>(kI8MaxStages, (static_cast<int>(kI8Ring) - g.slots * g.sub * g.nt * kI8K) / static_cast<int>(g.sub * kI8WBytes));
  g.k_blocks = static_cast<int>((K + kI8K * g.sub - 1) / (kI8K * g.sub));
  const int64_t tiles = n_tiles * g.m_tiles;
  g.pairs = static_cast<int>(std::min<int64_t>(most_pairs, tiles * g.k_blocks));
  // Tiles beyond whole waves of pairs either leave pairs idle for part of a tile's time or are cut,
  // which costs the fences and sums of their parts at the end: measured about 5 us + nt * 0.06 us with
  // up to 4 parts to a tile, and more with more, which pays where each part keeps 16 blocks or so.
  // 140 x 19500 x 8000 in 4, 8, 16 and 63 parts: 48, 57, 81 and 232 us; 16 x 256 x 40000 in 4, 16 and 76:
  // 36, 28 and 47 us.  Whole against cut, in us on the device: 9 x 4096 x 2880 12.4, 11.3;
  // 16 x 4096 x 8192 22.2, 13.6; 140 x 19500 x 8000 67.9, 47.9; 64 x 25600 x 4096 29.3, 31.4;
  // 203 x 50261 x 1456 40.9, 57.9.
  g.rounds = static_cast<int>(tiles / g.pairs);
  const int64_t rest = tiles - static_cast<int64_t>(g.rounds) * g.pairs;
  const int64_t parts = std::min<int64_t>(std::max<int64_t>(4, K / 2048), g.k_blocks);
  const int64_t sharing = std::max<int64_t>(1, std::min<int64_t>(g.pairs, rest * parts));
  const double tile_us = tile_time(g.nt);
  const bool cut = rest * tile_us / sharing + 5.0 + 0.06 * g.nt < tile_us;
  if (rest > 0 && !cut) ++g.rounds;
  g.tiles = static_cast<int>(tiles);
  g.cut_blocks = cut ? rest * g.k_blocks : 0;
  // a pair without a block would be a part that the tile's last one waits for in vain
  g.cut_pairs = static_cast<int>(sharing);
  // two parts of each pair that shares the line: the end of one tile, the start of the next
  g.part_bytes = g.cut_blocks > 0 ? static_cast<size_t>(2 * g.cut_pairs) * g.nt * 256 * 4 : 0;
  return g;
}

template <int SUB>
static cudaError_t launch_int8_gemm_t(const CUtensorMap& mw, const CUtensorMap& mx, const I8Params& p, int pairs,
                                      cudaStream_t st) {
  static bool done[128];
  const cudaError_t e = smem_limit_once(int8_gemm_kernel<SUB>, kI8Smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = kI8Smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int8_gemm_kernel<SUB>, mw, mx, p);
}

cudaError_t launch_int8_gemm(const uint16_t* x16, const float* x_scale, const int8_t* wq, const float* w_scale,
                             const Int8Shape& s, int32_t out_type, void* out, const Int8GemmPlan& g, float* part,
                             Int8Header* hdr, uint64_t limit_ns, cudaStream_t st) {
  CUtensorMap mw, mx;
  if (!encode_map_bytes(&mw, wq, s.K, s.N, s.K, kI8K, 128) ||
      !encode_map_f16(&mx, x16, s.K, s.M, s.K * 2, 64, static_cast<uint32_t>(g.nt / 2)))
    return cudaErrorInvalidValue;
  I8Params p;
  p.M = static_cast<int>(s.M);
  p.N = static_cast<int>(s.N);
  p.K = static_cast<int>(s.K);
  p.nt = g.nt;
  p.m_tiles = g.m_tiles;
  p.k_blocks = g.k_blocks;
  p.accs = g.accs;
  p.acc_cols = g.acc_cols;
  p.slots = g.slots;
  p.w_stages = g.w_stages;
  p.tiles = g.tiles;
  p.rounds = g.rounds;
  p.cut_blocks = g.cut_blocks;
  p.cut_pairs = g.cut_pairs;
  p.x_scale = x_scale;
  p.w_scale = w_scale;
  p.out = out;
  p.ldo = s.ldo;
  p.out_type = out_type;
  p.paired = reinterpret_cast<uintptr_t>(out) % 4 == 0 && s.ldo % 2 == 0;
  p.part = part;
  p.arrived = hdr->arrived;
  p.status = &hdr->status;
  p.limit_ns = limit_ns;
  return g.sub == 2 ? launch_int8_gemm_t<2>(mw, mx, p, g.pairs, st) : launch_int8_gemm_t<1>(mw, mx, p, g.pairs, st);
}

}  // namespace fkl
