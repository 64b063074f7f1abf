// Rotary positions: each pair (a, b) of a head's first `rotary` dimensions is
// turned by 2 pi * position * freqs[i] and scaled by m,
//   a' = m (a cos - b sin),  b' = m (a sin + b cos)   (inverse: -sin),
// the rest of the head is copied.  Bound by reading and writing the rows once.
//
// The angle is the same for all heads of a token, so a block computes the
// sines of its tokens once into shared memory and then streams the rows.  Only
// the fraction of a turn is kept: the whole turns, from the product position *
// freqs in 64 bits, are taken off its exact value by a multiply-add, so what is
// left is off by 2^-54 at any position (one radian a position: the rounded
// product's own fraction is 1e-4 radians off at 2^40, an fp32 product's a whole
// turn at two million).
#include <algorithm>
#include <type_traits>

#include "lm_ops.cuh"

namespace qat {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;       // rotary <= 1024
constexpr int kTablePairs = 2048;    // (cos, sin) pairs of a block: 16 KiB

template <class T>
__device__ __forceinline__ float to_f(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else return __bfloat162float(v);
}
template <class T>
__device__ __forceinline__ T from_f(float v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else return __float2bfloat16_rn(v);
}

// 16 bytes of a row, moved at once.
template <class T>
struct alignas(16) Pack {
  T v[16 / sizeof(T)];
};
template <class T>
__device__ __forceinline__ Pack<T> load(const T* p) {
  Pack<T> r;
  *reinterpret_cast<uint4*>(r.v) = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <class T>
__device__ __forceinline__ void store(T* p, const Pack<T>& r) {
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.v);
}

// n / d for 0 <= n < 2^31 by a multiply-high and a shift (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994: m = floor(2^32 (2^l - d)
// / d) + 1 with 2^(l-1) < d <= 2^l): two divisions a pack were most of the kernel's
// instructions.
struct FastDiv {
  uint32_t m, l, d;
  explicit FastDiv(uint32_t div) : d(div) {
    l = 0;
    while ((uint64_t{1} << l) < div) ++l;
    m = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << l) - div)) / div + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> l);
  }
};

// How a head's rotated dimensions lie in its 16-byte packs of W elements.
//   kPairs  interleaved: a pack holds whole pairs, wherever `rotary` ends
//   kHalves pairs (i, i + rotary/2), rotary/2 a multiple of W: a thread takes both packs
//   kAcross any other rotary/2: a pack's partners lie across two packs, so the packs
//           of whole heads go through shared memory first (which in-place calls need
//           as well: every partner is read before a pack is written)
// The pack in which `rotary` ends also copies what lies behind it; the packs behind
// are copied, unless Y is X.
//
// Measured, 12 heads: 65,536 tokens of 64 bf16, halves 34.2 us (5.9 TB/s), interleaved
// 40.3; 16,383 tokens of 64 fp32, 16 dims interleaved 19.1 us (5.3 TB/s).  Where a part
// ends off a pack, against loads and stores of single elements: 65,536 tokens of 72,
// 30 dims in halves 245 -> 58 us, 40,000 of 80, 20 dims interleaved 88 -> 32 us.  More
// packs of a thread in flight gave nothing (halves, 2 to 8) or lost (interleaved, 2:
// 40.3 -> 44.4 us).
enum Layout : int { kPairs, kHalves, kAcross };

template <class T, Layout L>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs r, int tokens_per_block, const FastDiv by_token,
                                                        const FastDiv by_head) {
  constexpr int W = 16 / sizeof(T);
  __shared__ alignas(16) float2 table[kTablePairs];  // rows of an even number of pairs: two are read at once
  __shared__ Pack<T> staged[L == kAcross ? kThreads : 1];
  const int pairs = r.rotary >> 1, stride = (pairs + 1) & ~1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), r.T - t0));
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, k = i - t * pairs;
    const int64_t pos = r.positions ? r.positions[t0 + t] : (r.seq_len > 0 ? (t0 + t) % r.seq_len : t0 + t);
    const double n = static_cast<double>(pos), freq = r.freqs[k];
    float s, c;
    sincospif(2.0f * static_cast<float>(fma(n, freq, -rint(n * freq))), &s, &c);
    table[t * stride + k] = make_float2(c * r.scale, (r.inverse ? -s : s) * r.scale);
  }
  __syncthreads();
  const int units = static_cast<int>(by_head.d), per_token = static_cast<int>(by_token.d);
  const T* X = static_cast<const T*>(r.X) + t0 * r.ldx;
  T* Y = static_cast<T*>(r.Y) + t0 * r.ldy;
  const int rot_units = L == kHalves ? pairs / W : (r.rotary + W - 1) / W;
  // kAcross: as many whole heads' rotated packs at a time as the block has threads
  const int step = L == kAcross ? kThreads / units * units : kThreads;
  for (int first = 0; first < nt * per_token; first += step) {
    const int i = first + threadIdx.x;
    const bool live = i < nt * per_token && static_cast<int>(threadIdx.x) < step;
    if (L != kAcross && !live) break;
    const int t = by_token.div(i), j = i - t * per_token;
    const int h = by_head.div(j), u = j - h * units;
    const int64_t at = static_cast<int64_t>(h) * r.head_dim;
    const T* x = X + t * r.ldx + at;
    T* y = Y + t * r.ldy + at;
    const float2* tab = table + t * stride;
    if constexpr (L == kPairs) {
      Pack<T> a = load(x + u * W);
#pragma unroll
      for (int e = 0; e < W; e += 4) {
        const int k = (u * W + e) >> 1;
        if (k < pairs) {
          const float4 cs = *reinterpret_cast<const float4*>(tab + k);
          float p = to_f(a.v[e]), q = to_f(a.v[e + 1]);
          a.v[e] = from_f<T>(p * cs.x - q * cs.y);
          a.v[e + 1] = from_f<T>(p * cs.y + q * cs.x);
          if (k + 1 < pairs) {
            p = to_f(a.v[e + 2]);
            q = to_f(a.v[e + 3]);
            a.v[e + 2] = from_f<T>(p * cs.z - q * cs.w);
            a.v[e + 3] = from_f<T>(p * cs.w + q * cs.z);
          }
        }
      }
      store(y + u * W, a);
    } else if constexpr (L == kHalves) {
      if (u >= rot_units) {
        const int d = r.rotary + (u - rot_units) * W;
        store(y + d, load(x + d));
        continue;
      }
      Pack<T> a = load(x + u * W), b = load(x + pairs + u * W);
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const float4 cs = *reinterpret_cast<const float4*>(tab + u * W + e);
        const float p = to_f(a.v[e]), q = to_f(b.v[e]), v = to_f(a.v[e + 1]), w = to_f(b.v[e + 1]);
        a.v[e] = from_f<T>(p * cs.x - q * cs.y);
        b.v[e] = from_f<T>(p * cs.y + q * cs.x);
        a.v[e + 1] = from_f<T>(v * cs.z - w * cs.w);
        b.v[e + 1] = from_f<T>(v * cs.w + w * cs.z);
      }
      store(y + u * W, a);
      store(y + pairs + u * W, b);
    } else {
      Pack<T> a;
      if (live) staged[threadIdx.x] = a = load(x + u * W);
      __syncthreads();
      if (live) {
        const T* head = reinterpret_cast<const T*>(staged) + (static_cast<int>(threadIdx.x) - u) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int d = u * W + e;
          if (d < r.rotary) {
            const bool second = d >= pairs;
            const float2 cs = tab[second ? d - pairs : d];
            const float p = to_f(a.v[e]), q = to_f(head[second ? d - pairs : d + pairs]);
            a.v[e] = from_f<T>(second ? q * cs.y + p * cs.x : p * cs.x - q * cs.y);
          }
        }
        store(y + u * W, a);
      }
      __syncthreads();
    }
  }
  if constexpr (L == kAcross) {  // the packs behind
    const int rest = r.copy_rest ? r.head_dim / W - units : 0, n = rest * r.heads;
    for (int i = threadIdx.x; i < nt * n; i += kThreads) {
      const int t = i / n, j = i - t * n, h = j / rest;
      const int64_t at = static_cast<int64_t>(h) * r.head_dim + (units + j - h * rest) * W;
      store(Y + t * r.ldy + at, load(X + t * r.ldx + at));
    }
  }
}

template <class T, Layout L>
int launch(const RopeArgs& r, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int pairs = r.rotary / 2;
  // enough rows for a few packs per thread, a table that fits, and blocks for every SM
  const int64_t row_units = static_cast<int64_t>(r.heads) * r.head_dim / W;
  int64_t tok = std::max<int64_t>(1, 4 * kThreads / std::max<int64_t>(1, row_units));
  tok = std::min<int64_t>(tok, std::max(1, kTablePairs / (pairs + 1)));
  const int64_t blocks = (r.T + tok - 1) / tok;
  if (blocks > (1ll << 31) - 1) return QAT_ERR_SHAPE;
  const int rotated = (r.rotary + W - 1) / W;
  const int units = L == kAcross   ? rotated
                    : L == kHalves ? pairs / W + (r.copy_rest ? (r.head_dim - r.rotary) / W : 0)
                                   : (r.copy_rest ? r.head_dim / W : rotated);
  rope_kernel<T, L><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      r, static_cast<int>(tok), FastDiv(static_cast<uint32_t>(units) * r.heads), FastDiv(units));
  count_launch();
  return cuda_status(cudaGetLastError());
}

// Rows and heads start on a pack's boundary: head_dim and the row strides are
// multiples of 8 elements.
template <class T>
int dispatch(const RopeArgs& r, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  if (r.interleaved) return launch<T, kPairs>(r, s);
  if (r.rotary / 2 % W == 0) return launch<T, kHalves>(r, s);
  return launch<T, kAcross>(r, s);
}

}  // namespace

int launch_rope(const RopeArgs& r, bool bf16, cudaStream_t stream) {
  if (r.rotary / 2 > kMaxPairs) return QAT_ERR_SHAPE;
  return bf16 ? dispatch<__nv_bfloat16>(r, stream) : dispatch<float>(r, stream);
}

}  // namespace qat
