// Attention forward on tcgen05: O = softmax(scale Q K^T + mask) V in one pass
// over the keys with a running maximum and sum.
//
// A CTA owns two tiles of 128 queries of one head and walks the keys in blocks
// of 128, so every staged K and V block serves 256 queries, and the tensor core
// works on one tile while the other's softmax runs:
//   warp 0      TMA producer: Q once, then K and V blocks through a ring
//   warp 1      TMEM owner and MMA issuer: S = Q K^T, then O += P V with P read
//               as operand A straight from tensor memory
//   warps 4-7   softmax of tile 0, a thread per query row (warps 8-11: tile 1)
// (warps 2 and 3 only complete the first warpgroup, which hands most of its
// registers to the others: a softmax thread holds a whole row of S)
// Tensor memory: S of both tiles (128 columns each; P replaces it in place as
// bf16) and both O accumulators (64 or 128 columns each).
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the
// last time: probabilities then stay below 2^8, which fp32 sums and bf16
// operands hold as precisely as values below one.
#include <algorithm>
#include <atomic>

#include "attn_sm100.cuh"
#include "attn_maps.cuh"

namespace qat {

namespace {

constexpr int BQ = 128;  // queries of a tile
constexpr int BKV = 128;

template <int NC>
struct Cfg {
  static constexpr int THREADS = 384;
  // registers per thread: 168 at launch (65,536 / 384), 72 + 216 + 216 = 3 * 168 after the split
  static constexpr int REGS_ISSUE = 72, REGS_SOFTMAX = 216;
  static constexpr int TILE = tile_bytes(128, NC);
  static constexpr int ST = NC == 1 ? 4 : 2;  // stages of the K ring and of the V ring
  static constexpr int SMEM = 2 * TILE + 2 * ST * TILE + 1024 + 256;
  static constexpr int O_COLS = 64 * NC;
  static constexpr float RESCALE = 8.0f;
};

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::THREADS, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const AttnArgs p) {
  using C = Cfg<NC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * C::TILE;
  uint8_t* sV = sK + C::ST * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + C::ST * C::TILE);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + C::ST;
  uint64_t* v_full = k_empty + C::ST;
  uint64_t* v_empty = v_full + C::ST;
  uint64_t* s_full = v_empty + C::ST;  // [2] S of a tile is in tensor memory
  uint64_t* p_full = s_full + 2;       // [2] P of a tile is
  uint64_t* o_full = p_full + 2;       // [2] O of a tile is complete
  uint64_t* mma_done = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((1 + 4 * C::ST + 7) * 8 + 8 <= 256, "barrier block overflow");

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int head = static_cast<int>(blockIdx.x % p.heads);
  const Seq sq = seq_of(p, static_cast<int>(blockIdx.x / p.heads));
  // late query blocks see most keys under a causal mask: they start first
  const int i0 = static_cast<int>(gridDim.y - 1 - blockIdx.y) * 2 * BQ;
  if (i0 >= sq.nq) return;
  int b0[2], b1[2], j0, j1;
  key_blocks<BQ, BKV>(p, sq, i0, b0[0], b1[0]);
  key_blocks<BQ, BKV>(p, sq, i0 + BQ, b0[1], b1[1]);
  j0 = b1[0] > b0[0] ? b0[0] : b0[1];
  if (b1[1] > b0[1]) j0 = min(j0, b0[1]);
  j1 = max(max(b1[0], b1[1]), j0);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
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
  if (warp == 0) {
    if (lane == 0 && j1 > j0) {
      // ------------------------------------------------ TMA producer
      const int tiles = i0 + BQ < sq.nq ? 2 : 1;
      mbar_arrive_expect_tx(q_full, tiles * C::TILE);
      for (int w = 0; w < tiles; ++w)
        for (int c = 0; c < NC; ++c)
          tma_load_3d(&tmQ, q_full, sQ + w * C::TILE + c * BQ * 128, c * 64, head,
                      static_cast<int>(sq.q0) + i0 + w * BQ);
      int st = 0;
      uint32_t ph = 0;
      int issued = 0;
      for (int j = j0; j < j1; ++j) {
        const int row = static_cast<int>(sq.k0) + j * BKV;
        if (!mbar_wait(&k_empty[st], ph ^ 1u, abort_flag, p.err)) break;
        mbar_arrive_expect_tx(&k_full[st], C::TILE);
        for (int c = 0; c < NC; ++c)
          tma_load_3d(&tmK, &k_full[st], sK + st * C::TILE + c * BKV * 128, c * 64, kv_head, row);
        // (a K block without its V block is landed below as well)
        const bool ok = mbar_wait(&v_empty[st], ph ^ 1u, abort_flag, p.err);
        if (!ok) {
          mbar_drain(&k_full[st], ph);
          break;
        }
        mbar_arrive_expect_tx(&v_full[st], C::TILE);
        for (int c = 0; c < NC; ++c)
          tma_load_3d(&tmV, &v_full[st], sV + st * C::TILE + c * BKV * 128, c * 64, kv_head, row);
        ++issued;
        if (++st == C::ST) { st = 0; ph ^= 1u; }
      }
      // every copy has landed before the block may exit (at once, unless a wait ran out)
      mbar_drain(q_full, 0);
      for (int n = max(0, issued - C::ST); n < issued; ++n) {
        mbar_drain(&k_full[n % C::ST], (n / C::ST) & 1);
        mbar_drain(&v_full[n % C::ST], (n / C::ST) & 1);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------- MMA issuer
    if (j1 > j0) {
      const int ks = (p.hd + 15) / 16;
      const uint32_t id_s = idesc_bf16(BQ, BKV, false, false);
      const uint32_t id_o = idesc_bf16(BQ, ks * 16, false, true);
      const uint32_t issue = elect_lane();
      const uint64_t dq = kmajor_desc<BQ>(sQ), dk = kmajor_desc<BKV>(sK), dv = rows_desc<BKV>(sV);
      constexpr uint32_t STAGE = C::TILE >> 4;
      bool ok = warp_wait(q_full, 0, abort_flag, p.err);
      uint32_t pph[2] = {0, 0};
      for (int j = j0; ok && j <= j1; ++j) {
        const int n = j - j0, st = n % C::ST, pst = (n + C::ST - 1) % C::ST;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (ok && j > j0 && j - 1 >= b0[w] && j - 1 < b1[w]) {  // O += P V of block j - 1
            ok = warp_wait(&v_full[pst], ((n - 1) / C::ST) & 1, abort_flag, p.err) &&
                 warp_wait(&p_full[w], pph[w], abort_flag, p.err);
            pph[w] ^= 1u;
            if (!ok) break;
            tc_fence_after();
            const int rows = sq.nk - (j - 1) * BKV;
            if (rows < BKV) clear_rows<NC>(sV + pst * C::TILE, BKV, rows, lane);
            const uint32_t more = j - 1 > b0[w];
#pragma unroll
            for (int kk = 0; kk < BKV / 16; ++kk)
              mma_ts(tmem + 256 + w * C::O_COLS, tmem + w * 128 + kk * 8, dv + pst * STAGE + rows_step(kk),
                     id_o, (kk > 0) | more, issue);
            if (j == b1[w]) mma_commit(&o_full[w], issue);
          }
          if (ok && j < j1 && j >= b0[w] && j < b1[w]) {  // S = Q K^T of block j
            ok = warp_wait(&k_full[st], (n / C::ST) & 1, abort_flag, p.err);
            if (!ok) break;
            tc_fence_after();
            product<NC, BQ>(tmem + w * 128, dq + w * STAGE, dk + st * STAGE, id_s, ks, issue);
            mma_commit(&s_full[w], issue);
          }
        }
        if (ok && j < j1) mma_commit(&k_empty[st], issue);
        if (ok && j > j0) mma_commit(&v_empty[pst], issue);
      }
      mma_commit(mma_done, issue);
      mbar_wait(mma_done, 0, abort_flag, p.err);  // before tensor memory is freed
    }
  }
  } else {
    set_regs_inc<C::REGS_SOFTMAX>();
    // ------------------------------------------------ softmax, a row per thread
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;  // tensor-memory lanes this warp may access
    const int row = quarter * 32 + lane;
    const int i = i0 + w * BQ + row;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + w * 128, t_o = tmem + lanes + 256 + w * C::O_COLS;
    const int ocols = (p.hd + 31) / 32;
    const float c2 = p.scale * kAttnLog2e;
    int lo, hi;
    keys_of(p, sq, i, lo, hi);
    // blocks that need no mask: [full0, full1) keys seen by the tile's first and last row
    int full0 = 0, full1 = 0;
    if (i0 + w * BQ < sq.nq) {
      int a, b;
      keys_of(p, sq, i0 + w * BQ, a, b);
      full1 = b;
      keys_of(p, sq, i0 + w * BQ + BQ - 1, a, b);
      full0 = a;
    }
    float m = -INFINITY, l = 0.0f;
    uint32_t ph = 0;
    bool ok = true;
    for (int j = b0[w]; j < b1[w]; ++j) {
      if (!warp_wait(&s_full[w], ph, abort_flag, p.err)) { ok = false; break; }
      ph ^= 1u;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, s[c]);
      tmem_ld_wait();
      const int key0 = j * BKV;
      if (key0 < full0 || key0 + BKV > full1) {
        const int a = lo - key0;
        const uint32_t n = static_cast<uint32_t>(hi - lo);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (static_cast<uint32_t>(c * 32 + k - a) >= n) s[c][k] = 0xff800000u;  // -inf
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
        for (int k = 2; k < 32; k += 2) mx[c] = max3(mx[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
      }
      const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const bool grow = (mb - m) * c2 > C::RESCALE || m == -INFINITY;
      const float mn = grow ? fmaxf(m, mb) : m;
      if (j > b0[w] && __any_sync(0xffffffffu, mn > m && m != -INFINITY)) {
        // S complete implies every earlier product is: O may be read and written
        const float f = mn > m ? attn_exp2((m - mn) * c2) : 1.0f;
        l *= f;
        for (int c = 0; c < (p.hd + 15) / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(t_o + c * 16, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          tmem_st16(t_o + c * 16, o);
        }
        tmem_st_wait();
      }
      m = mn;
      const float mc = m == -INFINITY ? 0.0f : m * c2;
      const float2 cc = make_float2(c2, c2), nm = make_float2(-mc, -mc);
      float2 sum[4] = {};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float2 x = fma2(make_float2(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])), cc, nm);
          x = make_float2(attn_exp2(x.x), attn_exp2(x.y));
          sum[c] = add2(sum[c], x);
          pk[k / 2] = pack2(x.x, x.y);
        }
        tmem_st16(t_s + c * 16, pk);
      }
      const float2 both = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
      l += both.x + both.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[w]);
    }
    const bool any = b1[w] > b0[w];
    if (ok && any) ok = warp_wait(&o_full[w], 0, abort_flag, p.err);
    // (the row's way out is Q's place: a tile that sees nothing still has its Q on the way)
    if (ok && j1 > j0) ok = warp_wait(q_full, 0, abort_flag, p.err);
    tc_fence_after();
    if (ok && i0 + w * BQ < sq.nq) {  // the same for all rows of the tile
      const bool none = l == 0.0f;  // the mask leaves the row no key
      const float inv = none ? 0.0f : 1.0f / l;
      const int r0 = i0 + w * BQ + quarter * 32;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.O) + (sq.q0 + r0) * p.ldo + head * p.hd;
      const uint32_t stage = smem_u32(sQ) + w * C::TILE + quarter * 2048;  // (Q has been multiplied)
      for (int c = 0; c < ocols; ++c) {
        uint32_t o[32] = {};
        if (any) {
          tmem_ld32(t_o + c * 32, o);
          tmem_ld_wait();
          if (none) {  // (0 * NaN of a place that the mask leaves out)
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
        }
        store_piece(out + c * 32, p.ldo, o, inv, p.hd - c * 32, sq.nq - r0, stage, lane);
      }
      if (i < sq.nq)
        p.lse[head * p.Tq + sq.q0 + i] = none ? -INFINITY : fmaf(m, p.scale, logf(l));
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
  static std::atomic<uint64_t> done{0};
  int rc = allow_smem(reinterpret_cast<const void*>(attn_fwd_kernel<NC>), C::SMEM, done);
  if (rc) return rc;
  CUtensorMap mq, mk, mv;
  if ((rc = make_head_map(&mq, a.Q, a.hd, a.heads, a.Tq, a.ldq, BQ))) return rc;
  if ((rc = make_head_map(&mk, a.K, a.hd, a.heads / a.group, a.Tk, a.ldk, BKV))) return rc;
  if ((rc = make_head_map(&mv, a.V, a.hd, a.heads / a.group, a.Tk, a.ldv, BKV))) return rc;
  const int64_t blocks = (static_cast<int64_t>(a.max_q) + 2 * BQ - 1) / (2 * BQ);
  const int64_t lists = static_cast<int64_t>(a.heads) * a.batch;
  if (blocks > 65535 || lists > (1ll << 31) - 1) return QAT_ERR_SHAPE;
  attn_fwd_kernel<NC><<<dim3(static_cast<unsigned>(lists), static_cast<unsigned>(blocks)), C::THREADS,
                        C::SMEM, s>>>(mq, mk, mv, a);
  count_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_attn_fwd(AttnArgs a, cudaStream_t stream) {
  a.err = device_error_ptr();
  return a.hd <= 64 ? launch<1>(a, stream) : launch<2>(a, stream);
}

}  // namespace qat
