// Declarations shared by the translation units of the 8-bit product.
#pragma once

#include "fkl_internal.h"

namespace fkl {

struct Int8Shape {
  int64_t M, N, K, ldo;
};

constexpr int kMaxPairs = 128;  // most CTA pairs of a launch

// Head of the workspace, zeroed by the kernel that prepares the tokens.
struct Int8Header {
  uint32_t status;
  uint32_t pad[63];
  int arrived[kMaxPairs * 16];  // parts of a cut tile that are done, per epilogue warp
};

// How the tensor-core product is cut (fkl_int8_gemm.cu): tiles of 256 channels x nt tokens,
// blocks of 128 * sub k.
struct Int8GemmPlan {
  int m_tiles, nt, sub, k_blocks, pairs;
  int accs, acc_cols, slots, w_stages;  // TMEM and shared memory
  int tiles, rounds;                    // tiles in all; whole tiles of a pair, at most
  int64_t cut_blocks;                   // blocks of the tiles that are cut
  int cut_pairs;                        // pairs that share them
  size_t part_bytes;                    // their partial sums
};
Int8GemmPlan plan_int8_gemm(int64_t M, int64_t N, int64_t K, int sms);
// x16: the tokens' integers as fp16 [M][K]; x_scale: 16-byte aligned; hdr zeroed before on the
// stream.  Each wait of the kernel is limited to limit_ns.
cudaError_t launch_int8_gemm(const uint16_t* x16, const float* x_scale, const int8_t* wq, const float* w_scale,
                             const Int8Shape& s, int32_t out_type, void* out, const Int8GemmPlan& g, float* part,
                             Int8Header* hdr, uint64_t limit_ns, cudaStream_t st);

}  // namespace fkl
