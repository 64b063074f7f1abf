// Host interface of the tcgen05 GEMM used by every linear of the library.
#pragma once

#include "common.cuh"

namespace qat {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (null when the driver has none).
EncodeFn get_encode();

// Epilogue applied to the fp32 accumulator tile.
enum Epi : int {
  EPI_BF16 = 0,        // D = bf16(acc)
  EPI_BF16_RESID = 1,  // D = bf16(acc + R)
  EPI_RELU2 = 2,       // D = bf16(acc) (optional), D2 = bf16(relu(acc)^2)
  EPI_DRELU2 = 3,      // D = bf16(acc * 2*relu(R))     (R = saved pre-activation)
  EPI_F32 = 4,         // D = acc (+ D if accumulate), single writer per element
  EPI_F32_ATOMIC = 5,  // D += acc with atomics (split-K partial sums)
  EPI_LRELU2 = 6,      // D = bf16(acc) (optional), D2 = bf16(leaky_relu(acc, 0.5)^2)
  EPI_DLRELU2 = 7,     // D = bf16(acc * g(R)), g = 2R for R > 0 else R/2 (its derivative)
  EPI_CE_STATS = 8,    // no D: per-row softmax statistics of the acc tile and the target's acc
  EPI_CE_GRAD = 9,     // g = (exp(acc - lse) - [target]) * scale: D = bf16(g), D2 = bf16(g - D)
  EPI_CE_DZ = 10,      // D = bf16(acc + rem[m] * B[target[m]])  (rem as EPI_CE_GRAD left it)
};

// Epilogues that read a bf16 tile R, and those that write the activation pair.
constexpr bool epi_reads_r(int e) {
  return e == EPI_BF16_RESID || e == EPI_DRELU2 || e == EPI_DLRELU2;
}
constexpr bool epi_act_fwd(int e) { return e == EPI_RELU2 || e == EPI_LRELU2; }
constexpr bool epi_ce(int e) { return e == EPI_CE_STATS || e == EPI_CE_GRAD || e == EPI_CE_DZ; }

// Per-row inputs and outputs of the cross-entropy epilogues (row m of A is a
// token; in STATS and GRAD column n of the product is the logit of word n).
struct CeArgs {
  const int64_t* targets = nullptr;  // [M]; outside [0, vocab): the row has no target
  int vocab = 0;
  const float* lse = nullptr;        // GRAD: [M] log-sum-exp of the logits
  const float* dloss = nullptr;      // GRAD: [M] upstream gradient (null: 1)
  const float* gscale = nullptr;     // GRAD: one factor of every row (null: 1)
  float2* stats = nullptr;           // STATS: [ce_slots(M, N)][M] (max, sum of exp(logit - max))
  float* tlogit = nullptr;           // STATS: [M], written where the row has a target
  // GRAD writes, DZ reads, where the row has a target: what bf16 rounding left
  // of g at the target.  That element is the row's largest, and with the mean's
  // 1 / count in it nearly the same for all rows, so its rounding error is
  // common to them instead of averaging out: dZ of a 50,257-word head was
  // 2e-3 to 3.5e-3 off without the remainder.
  float* rem = nullptr;              // [M]
  const __nv_bfloat16* words = nullptr;  // DZ: the operand [vocab, N], rows N apart
};

// D[M,N] = A[M,K] . B[N,K]^T with bf16 operands and fp32 accumulation.
// A is K-major (row m contiguous along K, row stride lda) unless a_mn, in which
// case it is stored [K][lda] with M contiguous (the transpose of a row-major
// [K,M] tensor).  Likewise B.  All strides are in elements.
struct GemmDesc {
  const void* A = nullptr;
  int64_t lda = 0;
  bool a_mn = false;
  const void* B = nullptr;
  int64_t ldb = 0;
  bool b_mn = false;
  int64_t M = 0, N = 0, K = 0;
  int epi = EPI_BF16;
  void* D = nullptr;
  int64_t ldd = 0;
  void* D2 = nullptr;
  int64_t ldd2 = 0;
  const void* R = nullptr;
  int64_t ldr = 0;
  bool accumulate = false;  // fp32 epilogues: add into D instead of overwriting
  // fp32 epilogues: longest run of K that one accumulator sums (0: no limit).
  // The tensor core's fp32 accumulation truncates at every step, so a sum over
  // very long K drifts; runs are added to D in 32 bits, rounded to nearest.
  int64_t k_run = 0;
  // fp32 epilogues of MN-major operands: a second A of the same shape and stride,
  // multiplied with the same B into the same accumulators, D = A^T B + A2^T B.
  const void* A2 = nullptr;
  // EPI_F32: the reduction is split as f32_slabs() says and D holds the partial products,
  // slab s at row s * rows (added up by the caller's next kernel, in order).
  bool slabs = false;
  // Fused quantizing B producer: when set, B / ldb are ignored and the kernel
  // builds the bf16 operand bf16(fl32(c * s)) of this fp32 weight [N,K]
  // (row-major, ld = K) on the grid `bits` in shared memory -- the quantized
  // weight never reaches global memory.  Forward epilogues, M >= 256 and
  // fused_b_supported() only.
  const float* Wraw = nullptr;
  int bits = 0;
  CeArgs ce;  // cross-entropy epilogues
};

// Partial statistics per row that EPI_CE_STATS writes for an M x N product.
int64_t ce_slots(int64_t M, int64_t N);

// Slabs that the product of `slabs` writes: count (1: the output's tiles alone occupy
// half the CTAs or pairs, a split would not pay) and rows of each.  A slab is the sum of
// up to `runs` of the `splits` parts of the reduction, `per` k-blocks each.
struct Slabs {
  int count;
  int64_t rows;
  int runs, splits, per;
};
Slabs f32_slabs(const GemmDesc& g);

// Whether launch_gemm can quantize B inside the GEMM for this shape / epilogue.
bool fused_b_supported(int64_t M, int64_t N, int64_t K, int epi);


// Validates, encodes the tensor maps and launches.  Returns a QAT_* code.
int launch_gemm(const GemmDesc& g, cudaStream_t stream);

}  // namespace qat
