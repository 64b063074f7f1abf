// Attention forward on tcgen05: O = softmax(scale Q K^T + mask) V in one pass
// over the keys with a running maximum and sum.
//
// A piece of work is two tiles of 128 queries, of two heads of a group or of one
// head, walked over the keys in blocks of 128, so that every staged K and V block
// serves both and the tensor core works on one tile while the other's softmax runs:
//   warp 0      TMA producer: Q, then K and V blocks through a ring
//   warp 1      MMA issuer: S = Q K^T, then O += P V with P read as operand A
//               straight from tensor memory
//   warps 4-7   softmax of tile 0, a thread per query row (warps 8-11: tile 1)
// (warps 2 and 3 only complete the first warpgroup, which hands most of its
// registers to the others: a softmax thread holds a whole row of S)
// Tensor memory: S of both tiles (128 columns each; P replaces it in place as
// bf16) and both O accumulators (64 or 128 columns each).
//
// Short queries (at most 128 per sequence: evaluation of a window's last tokens,
// single tokens) leave no second tile.  Both tiles then hold the same queries and
// take every other key block; their sums are joined at the end.  Where several
// query heads share a key head, the tile's rows are those of up to 4 heads, so K
// and V are read once for all of them (256 windows of 64 queries and 1,024 keys, 8
// heads of 64 over 4: 259 us with a piece per head and one tile, 104 us so).
//
// Measured (causal): 8,192 tokens, 8 heads of 128: 128 us, 1,070 TFLOP/s; 16
// sequences of 1,024, 8 heads of 80: 52 us, 415 TFLOP/s, where a piece has 1 to 8
// blocks a tile and loading Q, the first scores and writing O show; 64 windows of
// one token and 4,096 keys, 32 heads of 128 over 8: 194 us, 5.5 TB/s of K and V.
// A block walks all keys of its piece: fewer pieces than SMs (one token of one
// sequence over 8 key heads: 8) leave the others idle.
//
// P goes to the second product as bf16, the operand type that tensor memory feeds
// at full rate: each is off by at most 2^-8 of itself, and over a row's keys that
// comes to what rounding O to bf16 costs anyway (O 2.0e-3 to 2.3e-3 off in the
// 2-norm, 1.6e-3 to 1.7e-3 from its own rounding alone).  A second half of P would
// halve the second product's rate.  The maximum, the sum, lse and O are fp32; the
// sum takes P as it was before that rounding.
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
  static constexpr int OUT = 8 * 2048;        // the output rows' way out, per softmax warp
  static constexpr int MERGE = BQ * 8;        // short queries: tile 1's maximum and sum
  static constexpr int SMEM = 2 * TILE + 2 * ST * TILE + OUT + MERGE + 1024 + 512;
  static constexpr int O_COLS = 64 * NC;
  static constexpr float RESCALE = 8.0f;
};

// What the two tiles of a piece hold: 256 queries of one head, 128 queries of two
// heads of a group (both tiles then see the same key blocks), or short queries.
enum Mode : int { kRows, kHeads, kShort };

// A piece of work: which rows, which keys.
template <int MODE>
struct Piece {
  static constexpr bool SHORT = MODE == kShort;
  static constexpr bool HEADS = MODE == kHeads;
  Seq sq;
  int head, kv_head;  // first (or only) head
  int heads;          // SHORT: heads in the tile
  int i0;             // first query
  int b0[2], b1[2];   // key blocks of the tiles: b0, b0 + step, ... below b1
  int j0, j1;         // covers both
  bool live;

  __device__ Piece(const AttnArgs& p, const Work& w) {
    static_assert(!(SHORT && HEADS), "one mode");
    if constexpr (SHORT) {
      const int per = BQ / p.rows, chunks = (p.group + per - 1) / per;
      const int kv_heads = p.heads / p.group;
      const int c = w.list % (kv_heads * chunks);
      sq = seq_of(p, w.list / (kv_heads * chunks));
      kv_head = c / chunks;
      head = kv_head * p.group + c % chunks * per;
      heads = min(per, (kv_head + 1) * p.group - head);
      i0 = 0;
      live = sq.nq > 0;
      key_blocks<BQ, BKV>(p, sq, 0, j0, j1);
      b0[0] = j0;
      b0[1] = j0 + 1;
      b1[0] = b1[1] = j1;
    } else {
      const int lists = HEADS ? p.heads / 2 : p.heads;
      head = w.list % lists * (HEADS ? 2 : 1);
      kv_head = head / p.group;
      heads = 1;
      sq = seq_of(p, w.list / lists);
      // late query blocks see most keys under a causal mask: they come first
      i0 = (static_cast<int>(gridDim.y) - 1 - w.block) * (HEADS ? BQ : 2 * BQ);
      live = i0 < sq.nq;
      key_blocks<BQ, BKV>(p, sq, i0, b0[0], b1[0]);
      key_blocks<BQ, BKV>(p, sq, HEADS ? i0 : i0 + BQ, b0[1], b1[1]);
      j0 = b1[0] > b0[0] ? b0[0] : b0[1];
      if (b1[1] > b0[1]) j0 = min(j0, b0[1]);
      j1 = max(max(b1[0], b1[1]), j0);
    }
    if (!live) j1 = j0;
  }
  static constexpr int STEP = SHORT ? 2 : 1;
  __device__ int from(int w) const { return w ? b0[1] : b0[0]; }
  __device__ int to(int w) const { return w ? b1[1] : b1[0]; }
  __device__ bool has(int w, int j) const {
    return j >= from(w) && j < to(w) && (!SHORT || ((j - from(w)) & 1) == 0);
  }
  __device__ bool any(int w) const { return from(w) < to(w); }
  __device__ bool last(int w, int j) const { return j + STEP >= to(w); }
};

template <int NC, int MODE>
__global__ void __launch_bounds__(Cfg<NC>::THREADS, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const AttnArgs p) {
  using C = Cfg<NC>;
  constexpr bool SHORT = MODE == kShort, HEADS = MODE == kHeads;
  constexpr int ST = C::ST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * C::TILE;
  uint8_t* sV = sK + ST * C::TILE;
  uint8_t* sOut = sV + ST * C::TILE;
  float2* merge = reinterpret_cast<float2*>(sOut + C::OUT);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + C::OUT + C::MERGE);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + ST;
  uint64_t* v_full = k_empty + ST;
  uint64_t* v_empty = v_full + ST;
  uint64_t* s_full = v_empty + ST;     // [2] S of a tile is in tensor memory
  uint64_t* p_full = s_full + 2;       // [2] P of a tile is
  uint64_t* o_full = p_full + 2;       // [2] O of a tile is complete
  uint64_t* m_full = o_full + 2;       // tile 1's maximum and sum are in `merge`
  uint64_t* m_empty = m_full + 1;      // and have been read, with its O
  uint64_t* mma_done = m_empty + 1;
  uint64_t* work_bars = mma_done + 1;  // [4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(work_bars + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* answers = reinterpret_cast<uint8_t*>(bars) + 512 - 32;
  static_assert((2 + 4 * ST + 13) * 8 + 8 <= 512 - 32, "barrier block overflow");
  WorkQueue queue{smem_u32(answers), work_bars, work_bars + 2};

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Work work{static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y)};

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < ST; ++i) {
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
    mbar_init(m_full, 4);
    mbar_init(m_empty, 4);
    mbar_init(mma_done, 1);
    queue.init(10);  // producer, MMA, 8 softmax warps
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

  if (warp < 4) {
    set_regs_dec<C::REGS_ISSUE>();
    if (warp == 0) {
      // ------------------------------------------------ TMA producer (lane 0 of a warp
      // that walks together)
      int n = 0, pieces = 0, asked = 0, loads = 0;  // K, V blocks; pieces of work; Q tiles
      bool ok = true;
      for (bool more = true; more; ++pieces) {
        if (lane == 0) {
          const Piece<MODE> x(p, work);
          if (x.j1 > x.j0) {
            ok = loads == 0 || mbar_wait(q_empty, (loads - 1) & 1, abort_flag, p.err);
            if (ok) {
              const int row = static_cast<int>(x.sq.q0) + x.i0;
              if constexpr (SHORT) {
                mbar_arrive_expect_tx(q_full, x.heads * p.rows * 128 * NC);
                for (int h = 0; h < x.heads; ++h)
                  for (int c = 0; c < NC; ++c)
                    tma_load_3d(&tmQ, q_full, sQ + c * BQ * 128 + h * p.rows * 128, c * 64, x.head + h, row);
              } else {
                const int tiles = HEADS || x.i0 + BQ < x.sq.nq ? 2 : 1;
                mbar_arrive_expect_tx(q_full, tiles * C::TILE);
                for (int w = 0; w < tiles; ++w)
                  for (int c = 0; c < NC; ++c)
                    tma_load_3d(&tmQ, q_full, sQ + w * C::TILE + c * BQ * 128, c * 64, x.head + (HEADS ? w : 0),
                                row + (HEADS ? 0 : w * BQ));
              }
              ++loads;
            }
            for (int j = x.j0; ok && j < x.j1; ++j) {
              const int row = static_cast<int>(x.sq.k0) + j * BKV, st = n % ST;
              const uint32_t ph = (n / ST) & 1;
              ok = mbar_wait(&k_empty[st], ph ^ 1u, abort_flag, p.err);
              if (!ok) break;
              mbar_arrive_expect_tx(&k_full[st], C::TILE);
              for (int c = 0; c < NC; ++c)
                tma_load_3d(&tmK, &k_full[st], sK + st * C::TILE + c * BKV * 128, c * 64, x.kv_head, row);
              ok = mbar_wait(&v_empty[st], ph ^ 1u, abort_flag, p.err);
              if (!ok) {
                mbar_drain(&k_full[st], ph);
                break;
              }
              mbar_arrive_expect_tx(&v_full[st], C::TILE);
              for (int c = 0; c < NC; ++c)
                tma_load_3d(&tmV, &v_full[st], sV + st * C::TILE + c * BKV * 128, c * 64, x.kv_head, row);
              ++n;
            }
          }
          // only now: a block that asked early would hold a piece that an idle one could
          // start (8 heads of 8,192 tokens: 176 us asking first, 134 us asking here)
          ok = ok && queue.ask(pieces, abort_flag, p.err);
          asked += ok;
        }
        __syncwarp();
        more = __all_sync(0xffffffffu, ok) && queue.next(pieces, work, lane, abort_flag, p.err);
      }
      if (lane == 0) {
        // every copy has landed before the block may exit (at once, unless a wait ran out)
        if (loads > 0) mbar_drain(q_full, (loads - 1) & 1);
        for (int i = max(0, n - ST); i < n; ++i) {
          mbar_drain(&k_full[i % ST], (i / ST) & 1);
          mbar_drain(&v_full[i % ST], (i / ST) & 1);
        }
        if (asked > 0) mbar_drain(&queue.full[(asked - 1) & 1], ((asked - 1) >> 1) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer
      const int ks = (p.hd + 15) / 16;
      const uint32_t id_s = idesc_bf16(BQ, BKV, false, false);
      const uint32_t id_o = idesc_bf16(BQ, ks * 16, false, true);
      const uint32_t issue = elect_lane();
      const uint64_t dq = kmajor_desc<BQ>(sQ), dk = kmajor_desc<BKV>(sK), dv = rows_desc<BKV>(sV);
      constexpr uint32_t STAGE = C::TILE >> 4;
      uint32_t pph[2] = {0, 0};
      int n = 0, loads = 0;  // K, V blocks; Q tiles
      bool ok = true;
      for (int pieces = 0;; ++pieces) {
        const Piece<MODE> x(p, work);
        if (x.j1 > x.j0) {
          ok = warp_wait(q_full, loads & 1, abort_flag, p.err);
          ++loads;
          for (int j = x.j0; ok && j <= x.j1; ++j, ++n) {
            const int st = n % ST, pst = (n + ST - 1) % ST;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              if (ok && j > x.j0 && x.has(w, j - 1)) {  // O += P V of block j - 1
                ok = warp_wait(&v_full[pst], ((n - 1) / ST) & 1, abort_flag, p.err) &&
                     warp_wait(&p_full[w], pph[w], abort_flag, p.err);
                pph[w] ^= 1u;
                if (!ok) break;
                const int rows = x.sq.nk - (j - 1) * BKV;
                if (rows < BKV) clear_rows<NC>(sV + pst * C::TILE, BKV, rows, lane);
                tc_fence_after();
                const uint32_t more = j - 1 > x.from(w);
#pragma unroll
                for (int kk = 0; kk < BKV / 16; ++kk)
                  mma_ts(tmem + 256 + w * C::O_COLS, tmem + w * 128 + kk * 8,
                         dv + pst * STAGE + rows_step(kk), id_o, (kk > 0) | more, issue);
                if (x.last(w, j - 1)) mma_commit(&o_full[w], issue);
              }
              if (ok && j < x.j1 && x.has(w, j)) {  // S = Q K^T of block j
                ok = warp_wait(&k_full[st], (n / ST) & 1, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after();
                product<NC, BQ>(tmem + w * 128, dq + (SHORT ? 0 : w) * STAGE, dk + st * STAGE, id_s, ks, issue);
                mma_commit(&s_full[w], issue);
              }
            }
            if (!ok) break;
            if (j < x.j1) mma_commit(&k_empty[st], issue);
            if (j + 1 == x.j1) mma_commit(q_empty, issue);
            if (j > x.j0) mma_commit(&v_empty[pst], issue);
          }
          --n;  // (the last turn issued no block)
        }
        if (!ok || !queue.next(pieces, work, lane, abort_flag, p.err)) break;
      }
      mma_commit(mma_done, issue);
      warp_wait(mma_done, 0, abort_flag, p.err);  // before tensor memory is freed
    }
  } else {
    set_regs_inc<C::REGS_SOFTMAX>();
    // ------------------------------------------------ softmax, a row per thread
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;  // tensor-memory lanes this warp may access
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + w * 128, t_o = tmem + lanes + 256;
    const uint32_t stage = smem_u32(sOut) + (warp - 4) * 2048;
    const int ocols = (p.hd + 31) / 32;
    const float c2 = p.scale * kAttnLog2e;
    uint32_t ph = 0, oph = 0, oph1 = 0, mph = 0;  // oph: the own tile's O, oph1: SHORT, tile 1's
    bool ok = true;
    for (int pieces = 0;; ++pieces) {
      const Piece<MODE> x(p, work);
      // this warp's 32 rows are queries i0 + r0 .. of one head; the tile's rows start at query `first`
      const int first = SHORT ? 0 : HEADS ? x.i0 : x.i0 + w * BQ;
      const int h = SHORT ? quarter * 32 / p.rows : HEADS ? w : 0;
      const int r0 = SHORT ? quarter * 32 % p.rows : first + quarter * 32;
      const int i = r0 + lane;
      int lo, hi;
      keys_of(p, x.sq, i, lo, hi);
      // blocks that need no mask: [full0, full1) keys seen by the tile's first and last row
      int full0 = 0, full1 = 0;
      if (first < x.sq.nq) {
        int a, b;
        keys_of(p, x.sq, first, a, b);
        full1 = b;
        keys_of(p, x.sq, first + (SHORT ? p.rows : BQ) - 1, a, b);
        full0 = a;
      }
      float m = -INFINITY, l = 0.0f;
      if (SHORT && w == 1 && pieces > 0) {  // tile 0 has read the sums and the O of the piece before
        ok = warp_wait(m_empty, mph, abort_flag, p.err);
        mph ^= 1u;
      }
      const int from = x.from(w), to = x.to(w);
      for (int j = from; ok && j < to; j += x.STEP) {
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
        if (j > from && __any_sync(0xffffffffu, mn > m && m != -INFINITY)) {
          // S complete implies every earlier product is: O may be read and written
          const float f = mn > m ? attn_exp2((m - mn) * c2) : 1.0f;
          l *= f;
          for (int c = 0; c < (p.hd + 15) / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(t_o + w * C::O_COLS + c * 16, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st16(t_o + w * C::O_COLS + c * 16, o);
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
            float2 e = fma2(make_float2(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])), cc, nm);
            e = make_float2(attn_exp2(e.x), attn_exp2(e.y));
            sum[c] = add2(sum[c], e);
            pk[k / 2] = pack2(e.x, e.y);
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
      bool rows = ok && first < x.sq.nq && (!SHORT || h < x.heads);  // the same for the warp
      float f0 = 1.0f, f1 = 0.0f;  // weights of the tiles' O
      const bool any0 = x.any(SHORT ? 0 : w), any1 = SHORT && x.any(1);
      if constexpr (SHORT) {
        // tile 1 hands its maximum and sum over, tile 0 joins both and writes the rows
        if (w == 1) {
          merge[quarter * 32 + lane] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(m_full);
          rows = false;
        } else {
          if (ok) ok = warp_wait(m_full, mph, abort_flag, p.err);
          mph ^= 1u;
          const float2 other = merge[quarter * 32 + lane];
          const float top = fmaxf(m, other.x);
          f0 = m == -INFINITY ? 0.0f : attn_exp2((m - top) * c2);
          f1 = other.x == -INFINITY ? 0.0f : attn_exp2((other.x - top) * c2);
          l = l * f0 + other.y * f1;
          m = top;
          if (ok && any1) ok = warp_wait(&o_full[1], oph1, abort_flag, p.err);
          if (any1) oph1 ^= 1u;
        }
      }
      if (!SHORT || w == 0) {
        if (ok && any0) ok = warp_wait(&o_full[w], oph, abort_flag, p.err);
        if (any0) oph ^= 1u;
      }
      tc_fence_after();
      if (rows && ok) {
        const bool none = l == 0.0f;  // the mask leaves the row no key
        const float inv = none ? 0.0f : 1.0f / l;
        const int head = x.head + h;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.O) + (x.sq.q0 + r0) * p.ldo + head * p.hd;
        for (int c = 0; c < ocols; ++c) {
          uint32_t o[32] = {};
          if (any0) {
            tmem_ld32(t_o + (SHORT ? 0 : w) * C::O_COLS + c * 32, o);
            tmem_ld_wait();
          }
          if constexpr (SHORT) {
            if (any1) {
              uint32_t q[32];
              tmem_ld32(t_o + C::O_COLS + c * 32, q);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k)
                o[k] = __float_as_uint(fmaf(__uint_as_float(q[k]), f1, __uint_as_float(o[k]) * f0));
            }
          }
          if (none) {  // (0 * NaN of a place that the mask leaves out)
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
          store_piece(out + c * 32, p.ldo, o, inv, p.hd - c * 32, x.sq.nq - r0, stage, lane);
        }
        if (i < x.sq.nq)
          p.lse[head * p.Tq + x.sq.q0 + i] = none ? -INFINITY : fmaf(m, p.scale, logf(l));
      }
      tc_fence_before();
      if (SHORT && w == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(m_empty);  // tile 1 may go on: its sums and its O are read
      }
      if (!ok || !queue.next(pieces, work, lane, abort_flag, p.err)) break;
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int NC, int MODE>
int launch(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<NC>;
  constexpr bool SHORT = MODE == kShort, HEADS = MODE == kHeads;
  static std::atomic<uint64_t> done{0};
  int rc = allow_smem(reinterpret_cast<const void*>(attn_fwd_kernel<NC, MODE>), C::SMEM, done);
  if (rc) return rc;
  CUtensorMap mq, mk, mv;
  const int kv_heads = a.heads / a.group;
  if ((rc = make_head_map(&mq, a.Q, a.hd, a.heads, a.Tq, a.ldq, SHORT ? a.rows : BQ))) return rc;
  if ((rc = make_head_map(&mk, a.K, a.hd, kv_heads, std::max<int64_t>(a.Tk, 1), a.ldk, BKV))) return rc;
  if ((rc = make_head_map(&mv, a.V, a.hd, kv_heads, std::max<int64_t>(a.Tk, 1), a.ldv, BKV))) return rc;
  constexpr int rows = HEADS ? BQ : 2 * BQ;  // queries of a piece
  int64_t blocks = (static_cast<int64_t>(a.max_q) + rows - 1) / rows;
  int64_t lists = static_cast<int64_t>(HEADS ? a.heads / 2 : a.heads) * a.batch;
  if (SHORT) {
    const int per = BQ / a.rows;
    blocks = 1;
    lists = static_cast<int64_t>(kv_heads) * ((a.group + per - 1) / per) * a.batch;
  }
  if (blocks > 65535 || lists > (1ll << 31) - 1) return QAT_ERR_SHAPE;
  attn_fwd_kernel<NC, MODE><<<dim3(static_cast<unsigned>(lists), static_cast<unsigned>(blocks)), C::THREADS,
                               C::SMEM, s>>>(mq, mk, mv, a);
  count_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_attn_fwd(AttnArgs a, cudaStream_t stream) {
  a.err = device_error_ptr();
  if (a.max_q > BQ) {
    // Two heads of a group where it has an even number: both tiles then walk the same
    // blocks.  Against 256 rows of one head (of which the later 128 see one block more):
    // 16 x 1,024 tokens, 8 heads of 64 / 80 / 128: 52.1 -> 47.2, 55.2 -> 51.8, 58.3 ->
    // 55.7 us; 8,192 tokens of 128: 127.9 -> 127.5 us.
    if (a.group % 2 == 0)
      return a.hd <= 64 ? launch<1, kHeads>(a, stream) : launch<2, kHeads>(a, stream);
    return a.hd <= 64 ? launch<1, kRows>(a, stream) : launch<2, kRows>(a, stream);
  }
  // rows per head: as few as hold the queries, but no fewer than the group's heads can fill
  a.rows = BQ;
  while (a.rows > 32 && a.rows / 2 >= a.max_q && BQ / a.rows < a.group) a.rows /= 2;
  return a.hd <= 64 ? launch<1, kShort>(a, stream) : launch<2, kShort>(a, stream);
}

}  // namespace qat
