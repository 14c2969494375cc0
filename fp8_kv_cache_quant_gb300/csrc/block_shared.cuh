// The decode for sequences that share a prefix: its parameters and launch.
#pragma once
#include "block_common.cuh"

namespace fkv {

// A group of sequences, as planned on the GPU.
struct SharedGroup {
  int first, members;
  int keys, lo;        // shared keys (0: it shares nothing), the first that any sharing member sees
  int base, shares;    // place of its first piece, pieces that each (row tile, KV head)'s keys are cut into
  int row;             // the sequence whose blocks are read
};

struct SharedParams {
  int B, Hq, Hkv, D, max_blocks, window, num_groups, num_sms;
  int tok;                                    // members of a row tile
  int most_pieces;
  const int32_t* ctx;                         // [B]
  const int32_t* starts;                      // [num_groups + 1]
  const int32_t* lens;                        // [num_groups]
  __nv_bfloat16* out;                         // [B][Hq][D]
  int32_t* fault;
  const float *lse_part, *o_part;             // of the decode's own pieces
  // the workspace's parts
  SharedGroup* groups;
  unsigned long long* least;                  // [num_groups] of the sharing members the shortest: context, then the sequence
  int* pieces;                                // their number
  int4* info;                                 // [B], see BlockDecodeParams::shared
  int2* units;
  float* piece_lse;                           // [pieces][128]
  float4* piece_o;                            // [pieces][D / 4][128]
};

// The decode dp (its workspace as for launch_block_decode) on `ctas` CTAs with its groups; workspace: of block_shared_workspace bytes.
size_t block_shared_workspace(int B, int Hq, int Hkv, int D, int num_groups, int num_sms);
cudaError_t launch_block_shared(BlockDecodeParams dp, int D, int ctas, const int32_t* starts, const int32_t* lens, int num_groups, void* workspace,
                                int num_sms, cudaStream_t s);

}  // namespace fkv
