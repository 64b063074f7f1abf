// Host interfaces of the language-model operators beside the linears: the
// softmax cross entropy's reductions, rotary positions and attention.
#pragma once

#include "common.cuh"

namespace qat {

// ---- cross entropy: joins the partial softmax statistics of each token
// (slots x T pairs, see CeArgs) into lse and loss; with `mean`, also the mean
// loss over the tokens that have a target and 1 / their count (0, 0 if none).
struct CeJoin {
  const float2* stats;
  const float* tlogit;
  const int64_t* targets;
  float* loss;
  float* lse;
  float* mean;  // [2], nullable
  void* parts;  // ce_parts_bytes(T), 16-byte aligned (only with mean)
  int64_t T;
  int slots, vocab;
};
int64_t ce_parts_bytes(int64_t T);
int launch_ce_join(const CeJoin& j, cudaStream_t stream);

// ---- cross entropy, few tokens: dZ = bf16(sum of the product's slabs + rem *
// the target's row of the operand)
struct CeDz {
  const float* slabs;  // [count][rows][d]
  int count;
  int64_t rows;
  const int64_t* targets;  // [n]
  const float* rem;        // [n], read where the row has a target
  const __nv_bfloat16* words;  // [vocab, d]
  __nv_bfloat16* dZ;           // [n, d]
  int64_t n;
  int d, vocab;
};
int launch_ce_dz_join(const CeDz& j, cudaStream_t stream);

// ---- cross entropy, small heads: dW (+)= the sum of the product's slabs, in order
struct CeDw {
  const float* slabs;  // [count][stride]
  int count;
  int64_t stride;
  float* dW;  // [n], n a multiple of 4
  int64_t n;
  bool add;
};
int launch_ce_dw_join(const CeDw& j, cudaStream_t stream);

// ---- rotary positions (row strides in elements; Y may equal X)
struct RopeArgs {
  const void* X;
  void* Y;
  int64_t ldx, ldy, T;
  const int64_t* positions;  // [T], or null: the row's number modulo seq_len (0: not wrapped)
  int64_t seq_len;
  const double* freqs;       // [rotary / 2] turns per position
  float scale;
  int heads, head_dim, rotary, interleaved, inverse;
  int copy_rest;             // Y is another tensor: the unrotated dimensions are copied
};
int launch_rope(const RopeArgs& r, bool bf16, cudaStream_t stream);

// ---- attention over packed or equal-length sequences.  Q, O, dO, dQ rows hold
// `heads` heads of hd, K, V, dK, dV rows heads / group; strides in elements.
struct AttnArgs {
  int64_t Tq, Tk;
  const int32_t* cu_q;  // [batch + 1] first rows, or null: sequences of max_q rows
  const int32_t* cu_k;
  int batch, max_q, max_k;
  int heads, group, hd, causal, window;
  int rows;  // forward of short queries: rows of a tile per head (0: tiles of one head)
  float scale;
  const void *Q, *K, *V, *dO;
  void* O;
  float* lse;    // [heads][Tq]
  float* delta;  // [heads][Tq], backward: rowsum(dO * O)
  void *dQ, *dK, *dV;
  int64_t ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;
  int* err;
};
int launch_attn_fwd(AttnArgs a, cudaStream_t stream);
int launch_attn_bwd(AttnArgs a, cudaStream_t stream);

}  // namespace qat
