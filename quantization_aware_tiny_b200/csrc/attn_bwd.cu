// Attention backward on tcgen05.  With P recomputed from Q, K and the forward's
// lse, and delta = rowsum(dO * O):
//   dP = dO V^T,  dS = P * (dP - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Two kernels, each with its sums in tensor memory from first to last:
//   attn_dq_kernel   a CTA owns 2 x 128 queries of a head and walks the keys
//   attn_dkv_kernel  a CTA owns 128 keys of a key head and walks the queries of
//                    all heads of its group (their gradients meet in the sum)
// S and dP are thus formed twice, 7 products instead of 5; in return no partial
// sum ever leaves a CTA: no fp32 copy of dQ in memory, no atomics, and the same
// inputs give the same bits.
//
// P and dS are rounded to bf16 for the second products.  In both kernels they
// replace S and dP in tensor memory and are read from there as operand A; the
// keys go in blocks of 64 (dq) and the queries too (dkv), so that two blocks are
// in flight: the tensor core works on one while the other is turned into dS.
#include <algorithm>
#include <atomic>

#include "attn_maps.cuh"
#include "attn_sm100.cuh"

namespace qat {

namespace {

constexpr int BT = 128;  // rows of a stationary tile
constexpr int BS = 64;   // rows of a streamed block

template <int NC>
struct Cfg {
  static constexpr int THREADS = 384;
  // registers per thread: 168 at launch, 72 + 216 + 216 = 3 * 168 after the split
  static constexpr int REGS_ISSUE = 72, REGS_MATH = 216;
  static constexpr int TILE = tile_bytes(BT, NC), BLOCK = tile_bytes(BS, NC);
  static constexpr int DQ_ST = NC == 1 ? 4 : 3;   // stages (K and V block each)
  static constexpr int DQ_SMEM = 4 * TILE + DQ_ST * 2 * BLOCK + 1024 + 256;
  static constexpr int KV_ST = 4;                 // stages (Q and dO block each)
  static constexpr int ROWS_BYTES = 8 * 2 * BS * 4;  // lse and delta of a block, per warp
  static constexpr int KV_SMEM = 2 * TILE + KV_ST * 2 * BLOCK + ROWS_BYTES + 1024 + 256;
  static constexpr int COLS = 64 * NC;            // tensor-memory columns of an accumulator
};

// bf16(a * f) of one accumulator row of hd columns, from tensor memory to global.
__device__ __forceinline__ void store_row(__nv_bfloat16* out, uint32_t t, int hd, float f, bool any,
                                          bool write) {
  for (int c = 0; c < (hd + 31) / 32; ++c) {
    uint32_t o[32];
    if (any) {
      tmem_ld32(t + c * 32, o);
      tmem_ld_wait();
    }
    if (!write) continue;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = any ? __uint_as_float(o[g * 8 + k]) * f : 0.0f;
      if (c * 32 + g * 8 < hd)
        *reinterpret_cast<uint4*>(out + c * 32 + g * 8) =
            make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    }
  }
}

// ------------------------------------------------------------------------ dQ

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::THREADS, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const AttnArgs p) {
  using C = Cfg<NC>;
  constexpr int ST = C::DQ_ST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sdO = sQ + 2 * C::TILE;
  uint8_t* sKV = sdO + 2 * C::TILE;  // stage: K block, V block
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + ST * 2 * C::BLOCK);
  uint64_t* q_full = bars;
  uint64_t* kv_full = q_full + 1;
  uint64_t* kv_empty = kv_full + ST;
  uint64_t* s_full = kv_empty + ST;  // [2] S and dP of a tile are in tensor memory
  uint64_t* ds_full = s_full + 2;    // [2] dS of a tile is
  uint64_t* acc_full = ds_full + 2;  // [2] dQ of a tile is complete
  uint64_t* mma_done = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((1 + 2 * ST + 7) * 8 + 8 <= 256, "barrier block overflow");
  constexpr uint32_t PER_TILE = 2 * BS + C::COLS;  // tensor memory of a tile: S, dP, dQ
  static_assert(2 * PER_TILE <= 512, "tensor memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = static_cast<int>(blockIdx.x % p.heads);
  const Seq sq = seq_of(p, static_cast<int>(blockIdx.x / p.heads));
  const int i0 = static_cast<int>(gridDim.y - 1 - blockIdx.y) * 2 * BT;  // longest rows first
  if (i0 >= sq.nq) return;
  int b0[2], b1[2], j0, j1;
  key_blocks<BT, BS>(p, sq, i0, b0, b1, j0, j1);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&ds_full[i], 4);
      mbar_init(&acc_full[i], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmdO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int kv_head = head / p.group;

  if (warp < 4) {
    set_regs_dec<C::REGS_ISSUE>();
    if (warp == 0 && lane == 0 && j1 > j0) {
      // ------------------------------------------------ TMA producer
      const int tiles = i0 + BT < sq.nq ? 2 : 1;
      mbar_arrive_expect_tx(q_full, 2 * tiles * C::TILE);
      for (int w = 0; w < tiles; ++w)
        for (int c = 0; c < NC; ++c) {
          const int at = w * C::TILE + c * BT * 128, row = static_cast<int>(sq.q0) + i0 + w * BT;
          tma_load_3d(&tmQ, q_full, sQ + at, c * 64, head, row);
          tma_load_3d(&tmdO, q_full, sdO + at, c * 64, head, row);
        }
      int issued = 0;
      for (int j = j0; j < j1; ++j, ++issued) {
        const int st = issued % ST;
        if (!mbar_wait(&kv_empty[st], ((issued / ST) & 1) ^ 1, abort_flag, p.err)) break;
        mbar_arrive_expect_tx(&kv_full[st], 2 * C::BLOCK);
        const int row = static_cast<int>(sq.k0) + j * BS;
        for (int c = 0; c < NC; ++c) {
          uint8_t* dst = sKV + st * 2 * C::BLOCK + c * BS * 128;
          tma_load_3d(&tmK, &kv_full[st], dst, c * 64, kv_head, row);
          tma_load_3d(&tmV, &kv_full[st], dst + C::BLOCK, c * 64, kv_head, row);
        }
      }
      // every copy has landed before the block may exit (at once, unless a wait ran out)
      mbar_drain(q_full, 0);
      for (int n = max(0, issued - ST); n < issued; ++n) mbar_drain(&kv_full[n % ST], (n / ST) & 1);
    } else if (warp == 1 && j1 > j0) {
      // ------------------------------------------------ MMA issuer
      const int ks = (p.hd + 15) / 16;
      const uint32_t id_s = idesc_bf16(BT, BS, false, false);
      const uint32_t id_q = idesc_bf16(BT, ks * 16, false, true);
      bool ok = warp_wait(q_full, 0, abort_flag, p.err);
      uint32_t dph[2] = {0, 0};
      for (int j = j0; ok && j <= j1; ++j) {
        const int n = j - j0, st = n % ST, pst = (n + ST - 1) % ST;
        uint8_t* kb = sKV + st * 2 * C::BLOCK;
        if (j < j1) {
          ok = warp_wait(&kv_full[st], (n / ST) & 1, abort_flag, p.err);
          if (!ok) break;
          const int rows = sq.nk - j * BS;
          if (rows < BS) {
            clear_rows<NC>(kb, BS, rows, lane);
            clear_rows<NC>(kb + C::BLOCK, BS, rows, lane);
          }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t t = tmem + w * PER_TILE;
          if (j > j0 && j - 1 >= b0[w] && j - 1 < b1[w]) {  // dQ += dS K of block j - 1
            ok = warp_wait(&ds_full[w], dph[w], abort_flag, p.err);
            dph[w] ^= 1u;
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
              const uint32_t more = j - 1 > b0[w];
#pragma unroll
              for (int kk = 0; kk < BS / 16; ++kk)
                umma_bf16_ts(t + 2 * BS, t + kk * 8, rows_desc(sKV + pst * 2 * C::BLOCK, BS, kk), id_q,
                             (kk > 0) | more);
              if (j == b1[w]) umma_commit(&acc_full[w]);
            }
          }
          if (j < j1 && j >= b0[w] && j < b1[w]) {  // S = Q K^T, dP = dO V^T of block j
            tc_fence_after();
            if (lane == 0) {
              for (int kk = 0; kk < ks; ++kk)
                umma_bf16(t, kmajor_desc(sQ + w * C::TILE, BT, kk), kmajor_desc(kb, BS, kk), id_s, kk > 0);
              for (int kk = 0; kk < ks; ++kk)
                umma_bf16(t + BS, kmajor_desc(sdO + w * C::TILE, BT, kk),
                          kmajor_desc(kb + C::BLOCK, BS, kk), id_s, kk > 0);
              umma_commit(&s_full[w]);
            }
          }
        }
        if (ok && j > j0 && lane == 0) umma_commit(&kv_empty[pst]);
      }
      if (lane == 0) umma_commit(mma_done);
      warp_wait(mma_done, 0, abort_flag, p.err);  // before tensor memory is freed
    }
  } else {
    set_regs_inc<C::REGS_MATH>();
    // ------------------------------------------------ dS, a query row per thread
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int first = i0 + w * BT;
    const int i = first + quarter * 32 + lane;
    const uint32_t t = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + w * PER_TILE;
    const float c2 = p.scale * kAttnLog2e;
    const int64_t at = sq.q0 + i;
    int lo, hi;
    keys_of(p, sq, i, lo, hi);
    int full0 = 0, full1 = 0;  // keys that every row of the tile sees
    if (first < sq.nq) {
      int a, b;
      keys_of(p, sq, first, a, b);
      full1 = b;
      keys_of(p, sq, first + BT - 1, a, b);
      full0 = a;
    }
    float lse2 = 0.0f, delta = 0.0f;
    if (i < sq.nq) {
      lse2 = p.lse[head * p.Tq + at] * kAttnLog2e;
      const uint4* o = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.O) + at * p.ldo + head * p.hd);
      const uint4* d = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dO) + at * p.lddo + head * p.hd);
      float part[2] = {0.0f, 0.0f};
#pragma unroll 4
      for (int c = 0; c < p.hd / 8; ++c) {
        const uint4 x = __ldg(o + c), y = __ldg(d + c);
        const __nv_bfloat162* a = reinterpret_cast<const __nv_bfloat162*>(&x);
        const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = __bfloat1622float2(a[k]), v = __bfloat1622float2(b[k]);
          part[0] = fmaf(u.x, v.x, part[0]);
          part[1] = fmaf(u.y, v.y, part[1]);
        }
      }
      delta = part[0] + part[1];
      p.delta[head * p.Tq + at] = delta;  // for the other kernel
    }
    uint32_t ph = 0;
    bool ok = true;
    for (int j = b0[w]; j < b1[w]; ++j) {
      if (!warp_wait(&s_full[w], ph, abort_flag, p.err)) { ok = false; break; }
      ph ^= 1u;
      tc_fence_after();
      uint32_t s[2][32], g[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tmem_ld32(t + c * 32, s[c]);
        tmem_ld32(t + BS + c * 32, g[c]);
      }
      tmem_ld_wait();
      const int key0 = j * BS;
      const bool masked = key0 < full0 || key0 + BS > full1;
      uint32_t pk[32];
      const float2 cc = make_float2(c2, c2), nl = make_float2(-lse2, -lse2), nd = make_float2(-delta, -delta);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float2 x = fma2(make_float2(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])), cc, nl);
          const float2 y = add2(make_float2(__uint_as_float(g[c][k]), __uint_as_float(g[c][k + 1])), nd);
          float2 ds = mul2(make_float2(attn_exp2(x.x), attn_exp2(x.y)), y);
          if (masked) {
            const uint32_t n = static_cast<uint32_t>(hi - lo);
            const int a = key0 + c * 32 + k - lo;
            if (static_cast<uint32_t>(a) >= n) ds.x = 0.0f;
            if (static_cast<uint32_t>(a + 1) >= n) ds.y = 0.0f;
          }
          pk[c * 16 + k / 2] = pack2(ds.x, ds.y);
        }
      tmem_st32(t, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full[w]);
    }
    const bool any = b1[w] > b0[w];
    if (ok && any) ok = warp_wait(&acc_full[w], 0, abort_flag, p.err);
    tc_fence_after();
    if (ok && first < sq.nq)
      store_row(static_cast<__nv_bfloat16*>(p.dQ) + at * p.lddq + head * p.hd, t + 2 * BS, p.hd, p.scale,
                any, i < sq.nq);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------------- dK, dV

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::THREADS, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const AttnArgs p) {
  using C = Cfg<NC>;
  constexpr int ST = C::KV_ST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::TILE;
  uint8_t* sQ = sV + C::TILE;  // stage: Q block, dO block
  float* rows = reinterpret_cast<float*>(sQ + ST * 2 * C::BLOCK);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(rows) + C::ROWS_BYTES);
  uint64_t* k_full = bars;
  uint64_t* q_full = k_full + 1;
  uint64_t* q_empty = q_full + ST;
  uint64_t* s_full = q_empty + ST;  // [2] S^T and dP^T of a buffer are in tensor memory
  uint64_t* ds_full = s_full + 2;   // [2] P^T and dS^T of a buffer are
  uint64_t* acc_full = ds_full + 2;
  uint64_t* mma_done = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((1 + 2 * ST + 6) * 8 + 8 <= 256, "barrier block overflow");
  constexpr uint32_t ACC = 4 * BS;  // dV, then dK, behind two buffers of S^T and dP^T
  static_assert(ACC + 2 * C::COLS <= 512, "tensor memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv_heads = p.heads / p.group;
  const int kv_head = static_cast<int>(blockIdx.x % kv_heads);
  const Seq sq = seq_of(p, static_cast<int>(blockIdx.x / kv_heads));
  const int key0 = static_cast<int>(blockIdx.y) * BT;  // early keys are seen by most queries: first
  if (key0 >= sq.nk) return;
  // Queries that see some key of this tile, and their blocks.
  int qa, qb, ra, rb;
  queries_of(p, sq, key0, qa, rb);
  queries_of(p, sq, min(key0 + BT, sq.nk) - 1, ra, qb);
  const int j0 = qa / BS, nb = qb > qa ? (qb + BS - 1) / BS - j0 : 0;
  const int steps = nb * p.group;  // step n: head n / nb of the group, block j0 + n % nb

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&ds_full[i], 4);
    }
    mbar_init(acc_full, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmdO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    set_regs_dec<C::REGS_ISSUE>();
    if (warp == 0 && lane == 0 && steps > 0) {
      // ------------------------------------------------ TMA producer
      mbar_arrive_expect_tx(k_full, 2 * C::TILE);
      for (int c = 0; c < NC; ++c) {
        const int row = static_cast<int>(sq.k0) + key0;
        tma_load_3d(&tmK, k_full, sK + c * BT * 128, c * 64, kv_head, row);
        tma_load_3d(&tmV, k_full, sV + c * BT * 128, c * 64, kv_head, row);
      }
      int n = 0;
      for (; n < steps; ++n) {
        const int st = n % ST;
        if (!mbar_wait(&q_empty[st], ((n / ST) & 1) ^ 1, abort_flag, p.err)) break;
        mbar_arrive_expect_tx(&q_full[st], 2 * C::BLOCK);
        const int head = kv_head * p.group + n / nb;
        const int row = static_cast<int>(sq.q0) + (j0 + n % nb) * BS;
        for (int c = 0; c < NC; ++c) {
          uint8_t* dst = sQ + st * 2 * C::BLOCK + c * BS * 128;
          tma_load_3d(&tmQ, &q_full[st], dst, c * 64, head, row);
          tma_load_3d(&tmdO, &q_full[st], dst + C::BLOCK, c * 64, head, row);
        }
      }
      mbar_drain(k_full, 0);
      for (int m = max(0, n - ST); m < n; ++m) mbar_drain(&q_full[m % ST], (m / ST) & 1);
    } else if (warp == 1 && steps > 0) {
      // ------------------------------------------------ MMA issuer
      const int ks = (p.hd + 15) / 16;
      const uint32_t id_s = idesc_bf16(BT, BS, false, false);
      const uint32_t id_a = idesc_bf16(BT, ks * 16, false, true);
      bool ok = warp_wait(k_full, 0, abort_flag, p.err);
      for (int n = 0; ok && n <= steps; ++n) {
        if (n < steps) {  // S^T = K Q^T, dP^T = V dO^T of step n
          const int st = n % ST;
          ok = warp_wait(&q_full[st], (n / ST) & 1, abort_flag, p.err);
          if (!ok) break;
          uint8_t* q = sQ + st * 2 * C::BLOCK;
          const int live = sq.nq - (j0 + n % nb) * BS;
          if (live < BS) {
            clear_rows<NC>(q, BS, live, lane);
            clear_rows<NC>(q + C::BLOCK, BS, live, lane);
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t t = tmem + (n & 1) * 2 * BS;
            for (int kk = 0; kk < ks; ++kk)
              umma_bf16(t, kmajor_desc(sK, BT, kk), kmajor_desc(q, BS, kk), id_s, kk > 0);
            for (int kk = 0; kk < ks; ++kk)
              umma_bf16(t + BS, kmajor_desc(sV, BT, kk), kmajor_desc(q + C::BLOCK, BS, kk), id_s, kk > 0);
            umma_commit(&s_full[n & 1]);
          }
        }
        if (n > 0) {  // dV += P^T dO, dK += dS^T Q of step n - 1
          const int m = n - 1, st = m % ST;
          ok = warp_wait(&ds_full[m & 1], (m >> 1) & 1, abort_flag, p.err);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint8_t* q = sQ + st * 2 * C::BLOCK;
            const uint32_t t = tmem + (m & 1) * 2 * BS;
#pragma unroll
            for (int kk = 0; kk < BS / 16; ++kk)
              umma_bf16_ts(tmem + ACC, t + kk * 8, rows_desc(q + C::BLOCK, BS, kk), id_a, (kk > 0) | (m > 0));
#pragma unroll
            for (int kk = 0; kk < BS / 16; ++kk)
              umma_bf16_ts(tmem + ACC + C::COLS, t + BS + kk * 8, rows_desc(q, BS, kk), id_a,
                           (kk > 0) | (m > 0));
            umma_commit(&q_empty[st]);
            if (n == steps) umma_commit(acc_full);
          }
        }
      }
      if (lane == 0) umma_commit(mma_done);
      warp_wait(mma_done, 0, abort_flag, p.err);  // before tensor memory is freed
    }
  } else {
    set_regs_inc<C::REGS_MATH>();
    // ------------------------------------------------ P^T and dS^T, a key per thread
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t = tmem + lanes + w * 2 * BS;
    const float c2 = p.scale * kAttnLog2e;
    int lo, hi;  // queries that see this thread's key
    queries_of(p, sq, key0 + r, lo, hi);
    // Queries that see every key of the tile: blocks inside need no mask.
    const int full0 = ra, full1 = rb;
    // lse and delta of a block, a copy per warp: warps wait for nothing but their barriers
    float* buf = rows + (warp - 4) * 2 * BS;
    bool ok = true;
    for (int n = w; n < steps; n += 2) {
      const int head = kv_head * p.group + n / nb, i0 = (j0 + n % nb) * BS;
      __syncwarp();  // the previous block's values are read
#pragma unroll
      for (int e = 0; e < BS / 32; ++e) {
        const int k = e * 32 + lane;
        const bool live = i0 + k < sq.nq;
        const int64_t at = head * p.Tq + sq.q0 + i0 + k;
        buf[k] = live ? -p.lse[at] * kAttnLog2e : 0.0f;
        buf[BS + k] = live ? -p.delta[at] : 0.0f;
      }
      __syncwarp();
      if (!warp_wait(&s_full[w], (n >> 1) & 1, abort_flag, p.err)) { ok = false; break; }
      tc_fence_after();
      const bool masked = i0 < full0 || i0 + BS > full1;
      const float2 cc = make_float2(c2, c2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t s[32], g[32], pp[16], pd[16];
        tmem_ld32(t + c * 32, s);
        tmem_ld32(t + BS + c * 32, g);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const float4 nl = *reinterpret_cast<const float4*>(buf + c * 32 + k);
          const float4 nd = *reinterpret_cast<const float4*>(buf + BS + c * 32 + k);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 x = fma2(make_float2(__uint_as_float(s[k + e]), __uint_as_float(s[k + e + 1])), cc,
                                  e ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y));
            const float2 y = add2(make_float2(__uint_as_float(g[k + e]), __uint_as_float(g[k + e + 1])),
                                  e ? make_float2(nd.z, nd.w) : make_float2(nd.x, nd.y));
            float2 pr = make_float2(attn_exp2(x.x), attn_exp2(x.y));
            float2 ds = mul2(pr, y);
            if (masked) {
              const uint32_t cnt = static_cast<uint32_t>(hi - lo);
              const int a = i0 + c * 32 + k + e - lo;
              if (static_cast<uint32_t>(a) >= cnt) pr.x = ds.x = 0.0f;
              if (static_cast<uint32_t>(a + 1) >= cnt) pr.y = ds.y = 0.0f;
            }
            pp[(k + e) / 2] = pack2(pr.x, pr.y);
            pd[(k + e) / 2] = pack2(ds.x, ds.y);
          }
        }
        // columns 16 c .. 16 c + 15: read already (the halves go in order)
        tmem_st16(t + c * 16, pp);
        tmem_st16(t + BS + c * 16, pd);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full[w]);
    }
    if (ok && steps > 0) ok = warp_wait(acc_full, 0, abort_flag, p.err);
    tc_fence_after();
    if (ok) {  // the first warpgroup writes dV, the second dK
      const int64_t at = sq.k0 + key0 + r;
      const bool write = key0 + r < sq.nk;
      if (w == 0)
        store_row(static_cast<__nv_bfloat16*>(p.dV) + at * p.lddv + kv_head * p.hd, tmem + lanes + ACC, p.hd,
                  1.0f, steps > 0, write);
      else
        store_row(static_cast<__nv_bfloat16*>(p.dK) + at * p.lddk + kv_head * p.hd,
                  tmem + lanes + ACC + C::COLS, p.hd, p.scale, steps > 0, write);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int NC>
int launch(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<NC>;
  const int kv_heads = a.heads / a.group;
  static std::atomic<uint64_t> dq_done{0}, dkv_done{0};
  int rc = allow_smem(reinterpret_cast<const void*>(attn_dq_kernel<NC>), C::DQ_SMEM, dq_done);
  if (!rc) rc = allow_smem(reinterpret_cast<const void*>(attn_dkv_kernel<NC>), C::KV_SMEM, dkv_done);
  if (rc) return rc;
  CUtensorMap mq, mo, mk, mv;
  const int64_t lists = static_cast<int64_t>(a.heads) * a.batch;
  const int64_t qb = (static_cast<int64_t>(a.max_q) + 2 * BT - 1) / (2 * BT);
  const int64_t kb = (static_cast<int64_t>(a.max_k) + BT - 1) / BT;
  if (qb > 65535 || kb > 65535 || lists > (1ll << 31) - 1) return QAT_ERR_SHAPE;
  if (a.Tq > 0 && qb > 0) {
    if ((rc = make_head_map(&mq, a.Q, a.hd, a.heads, a.Tq, a.ldq, BT))) return rc;
    if ((rc = make_head_map(&mo, a.dO, a.hd, a.heads, a.Tq, a.lddo, BT))) return rc;
    if ((rc = make_head_map(&mk, a.K, a.hd, kv_heads, std::max<int64_t>(a.Tk, 1), a.ldk, BS))) return rc;
    if ((rc = make_head_map(&mv, a.V, a.hd, kv_heads, std::max<int64_t>(a.Tk, 1), a.ldv, BS))) return rc;
    attn_dq_kernel<NC><<<dim3(static_cast<unsigned>(lists), static_cast<unsigned>(qb)), C::THREADS,
                         C::DQ_SMEM, s>>>(mq, mo, mk, mv, a);
    count_launch();
    if (cudaGetLastError() != cudaSuccess) return QAT_ERR_CUDA;
  }
  if (a.Tk > 0 && kb > 0) {
    if ((rc = make_head_map(&mq, a.Q, a.hd, a.heads, std::max<int64_t>(a.Tq, 1), a.ldq, BS))) return rc;
    if ((rc = make_head_map(&mo, a.dO, a.hd, a.heads, std::max<int64_t>(a.Tq, 1), a.lddo, BS))) return rc;
    if ((rc = make_head_map(&mk, a.K, a.hd, kv_heads, a.Tk, a.ldk, BT))) return rc;
    if ((rc = make_head_map(&mv, a.V, a.hd, kv_heads, a.Tk, a.ldv, BT))) return rc;
    attn_dkv_kernel<NC><<<dim3(static_cast<unsigned>(lists / a.group), static_cast<unsigned>(kb)), C::THREADS,
                          C::KV_SMEM, s>>>(mq, mo, mk, mv, a);
    count_launch();
    if (cudaGetLastError() != cudaSuccess) return QAT_ERR_CUDA;
  }
  return QAT_OK;
}

}  // namespace

int launch_attn_bwd(AttnArgs a, cudaStream_t stream) {
  a.err = device_error_ptr();
  return a.hd <= 64 ? launch<1>(a, stream) : launch<2>(a, stream);
}

}  // namespace qat
