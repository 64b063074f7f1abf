// Reductions of the softmax cross entropy.  The logits themselves only ever
// exist as accumulator tiles of the GEMM (its EPI_CE_STATS and EPI_CE_GRAD
// epilogues); what reaches global memory is one (max, sum) pair per token and
// 128 columns (64 where the narrow tile is chosen: two warps share a tile's
// columns), joined here.
#include <algorithm>

#include "lm_ops.cuh"

namespace qat {

namespace {

constexpr int kJoinRows = 32;   // tokens of a block: one per lane, so the pairs load coalesced
constexpr int kJoinWarps = 32;  // most warps of a block; slots are dealt to them in turn

// Up to this many tokens a block joins a single one, its lanes taking the slots: a
// block of 32 tokens would leave most of the GPU idle and walk the slots one after
// another (loss and gradients of one token of 50,000 words, d = 512: 103 -> 89 us with
// the slabs' join by parts; 130 tokens of 1,024 words: 42.6 -> 40 us).
constexpr int64_t kJoinSingle = 1024;

// (sum of losses, counted tokens) of a block's tokens.
struct alignas(16) CePart {
  double sum;
  int64_t count;
};

// (m, s) <- the statistics of both halves: s = sum of exp(l - m) over both.
// m = -inf: no logit above -inf; s is then 0, or NaN where logits are (fmaxf passes them
// over, so the sum carries them).
__device__ __forceinline__ void merge_stats(float& m, float& s, float m2, float s2) {
  const float t = fmaxf(m, m2);
  if (t == -INFINITY) {
    s += s2;
    return;
  }
  s = s * expf(m - t) + s2 * expf(m2 - t);
  m = t;
}

// lse = m + log s, loss = lse - logit of the target (0 without one).  Bound by
// reading slots * T pairs: 33.5 MB for 65,536 tokens of 8,192 words.
__global__ void __launch_bounds__(kJoinRows* kJoinWarps) ce_join_kernel(const CeJoin j) {
  const int warps = blockDim.x >> 5;
  __shared__ float2 part[kJoinWarps][kJoinRows];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kJoinRows + lane;
  float m = -INFINITY, s = 0.0f;
  if (t < j.T) {
#pragma unroll 4
    for (int i = w; i < j.slots; i += warps) {
      const float2 v = j.stats[static_cast<int64_t>(i) * j.T + t];
      merge_stats(m, s, v.x, v.y);
    }
  }
  part[w][lane] = make_float2(m, s);
  __syncthreads();
  if (w != 0) return;
  for (int i = 1; i < warps; ++i) merge_stats(m, s, part[i][lane].x, part[i][lane].y);
  double sum = 0.0;
  int count = 0;
  if (t < j.T) {
    const float lse = m + logf(s);
    const int64_t y = j.targets[t];
    float loss = 0.0f;
    if (y >= 0 && y < j.vocab) {
      loss = lse - j.tlogit[t];
      sum = loss;
      count = 1;
    }
    j.lse[t] = lse;
    j.loss[t] = loss;
  }
  if (!j.mean) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  if (lane == 0) static_cast<CePart*>(j.parts)[blockIdx.x] = CePart{sum, count};
}

// The same for one token per block, a lane taking every blockDim.x-th slot.
__global__ void __launch_bounds__(256) ce_join_single_kernel(const CeJoin j) {
  __shared__ float2 part[8];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t t = blockIdx.x;
  float m = -INFINITY, s = 0.0f;
  for (int i = threadIdx.x; i < j.slots; i += blockDim.x) {
    const float2 v = j.stats[i * j.T + t];
    merge_stats(m, s, v.x, v.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_down_sync(0xffffffffu, m, o), s2 = __shfl_down_sync(0xffffffffu, s, o);
    merge_stats(m, s, m2, s2);
  }
  if (lane == 0) part[w] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < warps; ++i) merge_stats(m, s, part[i].x, part[i].y);
  const float lse = m + logf(s);
  const int64_t y = j.targets[t];
  const bool counted = y >= 0 && y < j.vocab;
  const float loss = counted ? lse - j.tlogit[t] : 0.0f;
  j.lse[t] = lse;
  j.loss[t] = loss;
  if (j.mean) static_cast<CePart*>(j.parts)[t] = CePart{loss, counted};
}

// Mean loss over the counted tokens: the blocks' sums in 64 bits and in a fixed
// order, so the same inputs always give the same bits.
__global__ void __launch_bounds__(1024) ce_mean_kernel(const CePart* parts, int64_t n, float* mean) {
  __shared__ double ssum[32];
  __shared__ int64_t scnt[32];
  double sum = 0.0;
  int64_t count = 0;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    sum += parts[i].sum;
    count += parts[i].count;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  if (lane == 0) {
    ssum[w] = sum;
    scnt[w] = count;
  }
  __syncthreads();
  if (w != 0) return;
  const int warps = blockDim.x >> 5;
  sum = lane < warps ? ssum[lane] : 0.0;
  count = lane < warps ? scnt[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  if (lane == 0) {
    mean[0] = count ? static_cast<float>(sum / static_cast<double>(count)) : 0.0f;
    mean[1] = count ? static_cast<float>(1.0 / static_cast<double>(count)) : 0.0f;
  }
}

// The slabs of dZ: a block takes 128 columns of a token, four a thread; blockDim.y
// threads share a column's slabs and the first adds their sums in order.  Bound by
// reading count * n * d floats, which the product has just left in L2 (one output tile
// per CTA or pair, under 20 MB, or the few that fill its waves better).
constexpr int kDzParts = 8;
__global__ void __launch_bounds__(32 * kDzParts) ce_dz_join_kernel(const CeDz j) {
  __shared__ float4 part[kDzParts][32];
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * 32 + threadIdx.x) * 4;
  const bool live = c < j.d;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4& v) {
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  };
  if (live) {
    const float* p = j.slabs + t * j.d + c;
    const int64_t step = j.rows * j.d;
#pragma unroll 8
    for (int s = threadIdx.y; s < j.count; s += blockDim.y) add(*reinterpret_cast<const float4*>(p + s * step));
  }
  part[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y != 0 || !live) return;
  for (int i = 1; i < static_cast<int>(blockDim.y); ++i) add(part[i][threadIdx.x]);
  const int64_t y = j.targets[t];
  if (y >= 0 && y < j.vocab) {
    const float r = j.rem[t];
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(j.words + y * j.d + c);
    const float2 u = __bfloat1622float2(w[0]), v = __bfloat1622float2(w[1]);
    a = make_float4(fmaf(r, u.x, a.x), fmaf(r, u.y, a.y), fmaf(r, v.x, a.z), fmaf(r, v.y, a.w));
  }
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(j.dZ + t * j.d + c);
  o[0] = __floats2bfloat162_rn(a.x, a.y);
  o[1] = __floats2bfloat162_rn(a.z, a.w);
}

// The slabs of dW, four columns a thread.  Bound by reading count * n floats that the
// product has just left in L2 (heads whose tiles fill less than half the GPU: under 10 MB a
// slab, and about as many tiles in all slabs together as CTAs or pairs).
constexpr int kDwThreads = 256;
__global__ void __launch_bounds__(kDwThreads) ce_dw_join_kernel(const CeDw j) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kDwThreads + threadIdx.x) * 4;
  if (i >= j.n) return;
  float4 a = j.add ? *reinterpret_cast<const float4*>(j.dW + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int s = 0; s < j.count; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(j.slabs + s * j.stride + i);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  *reinterpret_cast<float4*>(j.dW + i) = a;
}

int64_t join_blocks(int64_t T) { return T <= kJoinSingle ? T : (T + kJoinRows - 1) / kJoinRows; }

}  // namespace

// (never less than fewer tokens need: a workspace of the longest batch serves the others)
int64_t ce_parts_bytes(int64_t T) {
  return std::max(join_blocks(T), std::min(T, kJoinSingle)) * static_cast<int64_t>(sizeof(CePart));
}

int launch_ce_dz_join(const CeDz& j, cudaStream_t stream) {
  const int64_t columns = (j.d + 127) / 128;
  if (j.n > (1ll << 31) - 1 || columns > 65535) return QAT_ERR_SHAPE;
  const int parts = std::min(kDzParts, (j.count + 3) / 4);  // four slabs a thread or more
  ce_dz_join_kernel<<<dim3(static_cast<unsigned>(j.n), static_cast<unsigned>(columns)), dim3(32, parts), 0, stream>>>(j);
  count_launch();
  return cuda_status(cudaGetLastError());
}

int launch_ce_dw_join(const CeDw& j, cudaStream_t stream) {
  const int64_t blocks = (j.n / 4 + kDwThreads - 1) / kDwThreads;
  ce_dw_join_kernel<<<static_cast<unsigned>(blocks), kDwThreads, 0, stream>>>(j);
  count_launch();
  return cuda_status(cudaGetLastError());
}

int launch_ce_join(const CeJoin& j, cudaStream_t stream) {
  const int64_t blocks = join_blocks(j.T);
  // about 8 slots a warp: 64 slots (8,192 words) 8 warps, 394 (50,257 words) 32, where 8
  // warps took 25 us for 4,099 tokens
  const int warps = std::min(kJoinWarps, std::max(1, (j.slots + 7) / 8));
  if (j.T <= kJoinSingle)
    ce_join_single_kernel<<<static_cast<unsigned>(blocks), std::min(256, (j.slots + 31) / 32 * 32), 0, stream>>>(j);
  else
    ce_join_kernel<<<static_cast<unsigned>(blocks), kJoinRows * warps, 0, stream>>>(j);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return QAT_ERR_CUDA;
  if (!j.mean) return QAT_OK;
  const int threads = static_cast<int>(std::min<int64_t>(1024, (blocks + 31) / 32 * 32));
  ce_mean_kernel<<<1, threads, 0, stream>>>(static_cast<const CePart*>(j.parts), blocks, j.mean);
  count_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace qat
