// cross_attn.cu -- a softmax block's attention to the encoder's states (the
// prompt's, or a source clip's): queries [B, Tq, Hq, D] over keys and values
// [B, S, Hk, D] of another length, a mask over the keys of each batch row, Hq a
// multiple G of Hk (query head h reads key head h / G).
//
//   s = scale q.k over the seen keys, lse = log sum e^s, out = sum e^(s - lse) v
//
// in one pass over the keys with a running maximum m and sum l per query row;
// a row that sees no key gives out 0 and lse -inf.
//
// Query rows.  The G query heads of one key head and Tq tokens are the rows of
// one product with that head's keys: a tile holds 128 / G tokens of all G heads
// (row = token * G + head), so shared keys and values are loaded once for the
// group and a few tokens still fill a tile.
//
// A CTA takes two such tiles g (one where there is only one) of a (b, key head)
// and walks 128-key tiles; every K and V tile loaded serves both.
//   warp 16        TMA producer: the Q tiles, then K_0 V_0 K_1 V_1 ... through a
//                  ring of four slots (128-byte swizzle: a box row is 128 bytes).
//   warp 17        MMA issue, one lane, g = 0, 1 in turn: S_g = Q_g K_j^T (M 128,
//                  N 128, K D) and O_g += P_g V_j (M 128, N D, K 128), both in
//                  TMEM; P_g is read from TMEM (bf16, over columns of
//                  S_g), which leaves shared memory's bandwidth to K and V: from
//                  shared memory P alone would take 4 KB per 16 keys against V's
//                  2 D bytes x 16, more than the tensor core's time allows.
//   warps 0-15     softmax, eight warps for each g: a row (TMEM lane) by two
//                  threads, 64 keys each: maximum, p = 2^(s c - m), sum, P back to
//                  TMEM.  m moves, and O is rescaled in TMEM, only when a row's
//                  maximum has grown by more than 2^8 (until then p may reach 2^8,
//                  which fp32 sums and bf16 P hold as well as 1), so the halves of a
//                  row only vote in a barrier whether any has, and exchange maxima
//                  if so.  One thread per row left the schedulers idle two cycles in
//                  three.  The product with V starts on the half that is ready.
// P_g,j is used up before S_g,j+1 is written over it because one thread issues
// both and tensor-core operations of one thread complete in order.  That thread
// takes the tiles strictly in turn (P V and the next S of g = 0, then of g = 1),
// which keeps them half a step apart: one's softmax runs under the other's
// products.  With an issuing thread each, the products interleaved, both tiles'
// scores were ready at the same time and their softmaxes ran together, the tensor
// core waiting (7920 keys, 7 x 256 queries, 20 heads of 112: 186 us).
// Masked keys: a CTA first reads its batch row's mask into one bit per key and
// lists the key tiles that have any, so tiles without are never loaded (but for the
// first where there are few: it is on its way before the mask is known, which took
// the chunk's 300 keys under a mask from 18.9 to 18.0 us); in tiles
// with some, scores of masked keys become -inf whatever they were, and the masked
// rows of V are cleared in shared memory, since 0 * NaN would reach the sum.
// Few query tiles and many keys: the key tiles are split over CTAs, each leaves
// its normalised fp32 part and its lse, and gdn_cross_join_kernel joins them.
// 2640 queries over 7920 keys, 20 heads of 112: 203-210 us on fresh inputs (891-920
// TFLOP/s); replayed a few times from a cool start 180 (1040), tensor core 53% and
// special-function unit 46% busy: what is left is the hand-offs between them, and the
// power limit.  Over 300 keys 21.2 us, over 225 of them 17.6-19.4, the chain of a
// CTA's three or two tiles, twice.
// Every wait is bounded; one that gives up sets the error word and the CTA drains
// its copies and MMAs before it frees TMEM.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "cross_attn.cuh"
#include "gdn_internal.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kRows = 128;             // rows of a query tile, keys of a key tile
constexpr int kHalf = kRows / 2;       // keys of a softmax thread
constexpr int kSingleTiles = 16;       // key tiles up to which a CTA takes one query tile
constexpr int kMaskTiles = 1024;       // key tiles that a CTA can list under a mask
template <int NQ>  // query tiles of a CTA
struct Roles {
  static constexpr int softmax_warps = 8 * NQ;  // two groups of four warps per query tile
  static constexpr int producer = softmax_warps, mma = producer + 1;
  static constexpr int threads = 32 * (mma + 1);
  static constexpr int slots = 2 * NQ;          // ring of K and V tiles
};
constexpr uint32_t kTileCols = 256;    // TMEM columns of a tile: S (and P) [0, 128) | O [128, 128 + D)
constexpr uint32_t kBlock = kRows * 128;  // one 64-feature block of a 128-row tile, bytes
constexpr float kRescaleLog2 = 8.f;
constexpr long long kDrainPolls = 1LL << 40;  // drains are bounded by the 2 s timer

template <int NQ>
struct CrossAux {
  uint64_t q_full;
  uint64_t full[Roles<NQ>::slots], empty[Roles<NQ>::slots];
  uint64_t s_full[NQ], p_full[NQ][2], o_full[NQ], drain;
  uint32_t tmem;
  int abort;
  int count;                       // key tiles to walk
  float row[NQ][2][kRows];    // a row's two halves exchange maxima, later sums
  uint16_t list[NQ == 1 ? kSingleTiles : kMaskTiles];  // under a mask: the tiles with any seen key
};

// Shared memory: Q tiles, the ring, the barriers and mask.
template <int NB, int NQ>  // 64-feature blocks of a head, query tiles
struct CrossLayout {
  static constexpr uint32_t tile = NB * kBlock;
  static constexpr uint32_t q = 0;
  static constexpr uint32_t ring = NQ * tile;
  static constexpr uint32_t aux = ring + Roles<NQ>::slots * tile;
  // under a mask: the seen keys of each of the CTA's tiles, one bit each
  static constexpr uint32_t mask = aux + ((uint32_t)sizeof(CrossAux<NQ>) + 15) / 16 * 16;
  static constexpr uint32_t mask_tile = 4 * sizeof(uint32_t);
};

// 32 scores of a row, those of masked keys -inf whatever they were.
__device__ __forceinline__ void scores(uint32_t taddr, uint32_t seen, float (&s)[32]) {
  tmem_ld32(taddr, s);
  tmem_wait_ld();
  if (seen != ~0u) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(seen >> i & 1)) s[i] = -INFINITY;
  }
}

template <int NB, int NQ>
__global__ void __launch_bounds__(Roles<NQ>::threads, 3 - NQ)
gdn_cross_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CrossParams P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int D = P.D;
  constexpr int nb = NB, kSlots = Roles<NQ>::slots;
  constexpr bool kEarly = NQ == 1;  // few tiles: the first is loaded before the mask is known
  using L = CrossLayout<NB, NQ>;
  CrossAux<NQ>& aux = *reinterpret_cast<CrossAux<NQ>*>(smem + L::aux);
  uint32_t* const mask_bits = reinterpret_cast<uint32_t*>(smem + L::mask);
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;  // uniform
  // unit: (b * Hk + hk) * groups + group
  const bool whole = blockIdx.x < P.full;
  const unsigned x = blockIdx.x - P.full;
  const int split = whole ? 0 : x % P.nsplit;
  const unsigned u = whole ? blockIdx.x : P.full + x / P.nsplit;
  const int group = u % P.groups, bh = u / P.groups;
  const int b = bh / P.Hk, hk = bh - b * P.Hk;
  const int tile0 = group * NQ, nq = min(NQ, P.qtiles - tile0);
  const int k0 = split * P.per_split;                               // key tiles k0 .. k0 + kn - 1
  const int kn = whole ? P.ntiles : min(P.per_split, P.ntiles - k0);
  volatile int* abort_flag = &aux.abort;
  // ring item i: K (even i) or V (odd i) of listed tile i / 2
  auto slot_ptr = [&](int i) { return smem + L::ring + (i % kSlots) * L::tile; };
  auto load_item = [&](int i, int tile) {
    uint64_t* bar = &aux.full[i % kSlots];
    mbar_arrive_expect_tx(bar, L::tile);
    for (int c = 0; c < nb; ++c)
      tma_load_5d(slot_ptr(i) + c * kBlock, i & 1 ? &tm_v : &tm_k, bar, c * 64, 0, tile * kRows, hk,
                  b * (i & 1 ? P.vb : P.kb));
  };

  if (warp == Roles<NQ>::producer && lane == 0) {
    prefetch_map(&tm_q);
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
    mbar_init(&aux.q_full, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&aux.full[s], 1);
      mbar_init(&aux.empty[s], 1);
    }
    for (int g = 0; g < NQ; ++g) {
      mbar_init(&aux.s_full[g], 1);
      mbar_init(&aux.p_full[g][0], 4);  // warps of a half
      mbar_init(&aux.p_full[g][1], 4);
      mbar_init(&aux.o_full[g], 1);
    }
    mbar_init(&aux.drain, 1);
    aux.abort = 0;
    aux.count = kn;
    fence_mbar_init();
    pdl_wait();  // inputs may come from the kernel in front
    // the queries are on their way while the CTA sets up and reads its mask
    const uint32_t qbytes = (uint32_t)P.tokens * P.G * 128;  // of one 64-feature block
    mbar_arrive_expect_tx(&aux.q_full, nq * nb * qbytes);
    for (int g = 0; g < nq; ++g)
      for (int c = 0; c < nb; ++c)
        tma_load_5d(smem + L::q + g * L::tile + c * kBlock, &tm_q, &aux.q_full, c * 64, 0,
                    (tile0 + g) * P.tokens, hk, b * P.qb);
    // and so is the first key tile
    if (kEarly && kn > 0) {
      load_item(0, k0);
      load_item(1, k0);
    }
  }
  if (warp == Roles<NQ>::mma) {
    tmem_alloc(&aux.tmem, kTileCols * NQ);
    tmem_relinquish();
  }
  pdl_wait();
  if (P.mask) {
    const uint8_t* mrow = P.mask + b * P.mask_bs;
    for (int w = warp; w < kn * 4; w += Roles<NQ>::softmax_warps) {
      if (warp >= Roles<NQ>::softmax_warps) break;
      const long long key = (long long)(k0 * 4 + w) * 32 + lane;
      const uint32_t bits = __ballot_sync(~0u, key < P.S && mrow[key] != 0);
      if (lane == 0) mask_bits[w] = bits;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // The next kernel's blocks may take their places; they wait for this grid.  Not before
  // this CTA has its tensor memory: a block of theirs on this SM could take the columns
  // first, and would give them back only after this grid.
  pdl_trigger();
  if (P.mask) {
    if (warp == 0) {
      int n = 0;
      bool seen = false;
      for (int t0 = 0; t0 < kn; t0 += 32) {
        const int t = t0 + lane;
        bool any = t < kn && (mask_bits[4 * t] | mask_bits[4 * t + 1] | mask_bits[4 * t + 2] |
                              mask_bits[4 * t + 3]) != 0;
        seen = __any_sync(~0u, any) || seen;
        any = any || (kEarly && t == 0);  // it is there already
        const uint32_t bal = __ballot_sync(~0u, any);
        if (any) aux.list[n + __popc(bal & ((1u << lane) - 1))] = (uint16_t)t;
        n += __popc(bal);
      }
      if (lane == 0) aux.count = seen ? n : 0;
    }
    __syncthreads();
  }
  // two tiles hold all 512 columns, an allocation that starts at the first
  const uint32_t tm = NQ == 2 ? 0u : __reduce_max_sync(~0u, aux.tmem);  // (a reduction's result is uniform)
  const int n = __reduce_max_sync(~0u, aux.count);
  const bool masked = P.mask != nullptr;
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(P.err, kErrTimeout);
  };
  auto wait_full = [&](int i) { return mbar_wait(&aux.full[i % kSlots], (i / kSlots) & 1, P.limit); };

  if (warp == Roles<NQ>::producer) {
    if (lane == 0) {
      int issued = kEarly && kn > 0 ? 2 : 0;
      for (int i = issued; i < 2 * n; ++i) {
        if (*abort_flag) break;
        if (i >= kSlots && !mbar_wait(&aux.empty[i % kSlots], (i / kSlots - 1) & 1, P.limit)) {
          fail();
          break;
        }
        load_item(i, k0 + (masked ? aux.list[i / 2] : i / 2));
        ++issued;
      }
      // every load has landed before shared memory goes
      mbar_wait(&aux.q_full, 0, kDrainPolls);
      for (int i = max(0, issued - kSlots); i < issued; ++i)
        mbar_wait(&aux.full[i % kSlots], (i / kSlots) & 1, kDrainPolls);
    }
  } else if (warp == Roles<NQ>::mma) {
    if (n > 0) {  // the whole warp walks the loop, one elected lane issues
      const uint32_t idS = idesc_bf16(kRows, kRows, 0, 0), idO = idesc_bf16(kRows, D, 0, 1);
      const uint64_t dq = sdesc_sw128(smem_u32(smem + L::q), 16);
      bool ok = __all_sync(~0u, mbar_wait(&aux.q_full, 0, P.limit));
      for (int j = 0; ok && j <= n; ++j) {
        for (int g = 0; g < nq; ++g) {
          const uint32_t tS = tm + g * kTileCols, tO = tS + kRows;
          if (j > 0) {
            // O_g += P_g V, a half of the keys at a time: P in TMEM (8 columns per
            // 16 keys, over the half's own scores), V MN-major
            const int i = 2 * (j - 1) + 1;
            if (g == 0) ok = __all_sync(~0u, wait_full(i));
            const uint64_t dv = sdesc_sw128(smem_u32(slot_ptr(i)), kBlock);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && __all_sync(~0u, mbar_wait(&aux.p_full[g][half], (j - 1) & 1, P.limit));
              if (!ok) break;
              tc_fence_after_sync();
#pragma unroll
              for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                mma_bf16_ts_elect(tO, tS + kHalf * half + (ks & 3) * 8, dv + ks * (2048 >> 4), idO,
                                  j > 1 || ks > 0);
            }
            if (!ok) break;
            if (g == nq - 1) mma_commit_elect(&aux.empty[i % kSlots]);
          }
          if (j < n) {
            // S_g = Q_g K^T: both K-major
            const int i = 2 * j;
            if (g == 0) ok = __all_sync(~0u, wait_full(i));
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t dk = sdesc_sw128(smem_u32(slot_ptr(i)), 16);
            const uint64_t dqg = dq + (g * L::tile >> 4);
#pragma unroll
            for (int ks = 0; ks < 4 * NB; ++ks) {
              const uint32_t at = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
              if (ks < D / 16) mma_bf16_elect(tS, dqg + at, dk + at, idS, ks > 0);
            }
            mma_commit_elect(&aux.s_full[g]);
            if (g == nq - 1) mma_commit_elect(&aux.empty[i % kSlots]);
          } else {
            mma_commit_elect(&aux.o_full[g]);
          }
        }
        if (__any_sync(~0u, *abort_flag != 0)) break;
      }
      // every MMA issued has completed before TMEM and shared memory go
      if (!ok && lane == 0) fail();
      mma_commit_elect(&aux.drain);
      mbar_wait(&aux.drain, 0, kDrainPolls);
      __syncwarp();
    }
  } else if ((warp >> 3) < nq) {
    const int g = warp >> 3, half = (warp >> 2) & 1;  // keys [64 half, 64 half + 64) of each tile
    const int r = tid & (kRows - 1);
    const uint32_t tS = tm + g * kTileCols + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = tS + kRows;
    const int oc0 = half ? (D / 32 + (D / 16) % 2) * 16 : 0;  // this half's columns of O
    const int oc1 = half ? D : (D / 32 + (D / 16) % 2) * 16;
    const int Hq = P.Hk * P.G, tok0 = (tile0 + g) * P.tokens;
    const int t = tok0 + (r * P.gmul >> 16), head = hk * P.G + r - (r * P.gmul >> 16) * P.G;
    const bool row = r < P.tokens * P.G && t < P.Tq;
    __nv_bfloat16* const out0 = P.out + (((long long)b * P.Tq + tok0) * Hq + hk * P.G) * D;
    // half of a thread's scores stay in registers from the maximum to p where a CTA
    // has many tiles (7 x 256 queries, 7920 keys, 20 heads of 64: 115.1 -> 111.4 us; one
    // tile of queries, 1024 keys: 44.5 -> 46.0)
    constexpr bool kKeep = NQ == 2;
    float m_run = kLowest, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      bool got = __all_sync(~0u, *abort_flag == 0 && mbar_wait(&aux.s_full[g], j & 1, P.limit));
      tc_fence_after_sync();
      // the seen keys of this half of the tile
      uint32_t bits[2] = {~0u, ~0u};
      if (masked) {
        const int w = 4 * aux.list[j] + 2 * half;
        bits[0] = mask_bits[w];
        bits[1] = mask_bits[w + 1];
      } else if (j == n - 1) {
        const int left = P.S - (k0 + j) * kRows - kHalf * half;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (left < 32 * (c + 1)) bits[c] = left <= 32 * c ? 0u : (1u << (left - 32 * c)) - 1;
      }
      if (masked && (bits[0] & bits[1]) != ~0u) {  // clear the masked rows of V, a row by two threads
        const int i = 2 * j + 1;
        got = __all_sync(~0u, wait_full(i)) && got;
        const int key = r >> 1, side = r & 1;
        if (got && !(bits[key / 32] >> (key % 32) & 1)) {
          uint8_t* row = slot_ptr(i) + (half * kHalf + key) * 128 + side * 64;
          for (int c = 0; c < nb * 4; ++c)
            *reinterpret_cast<uint4*>(row + (c >> 2) * kBlock + (c & 3) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      // the scores are read for the maximum and for p, 32 at a time: holding all 64
      // between costs more registers than 16 warps can have
      float mx = -INFINITY, s[32];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = kKeep ? 1 - i : i;
        scores(tS + kHalf * half + 32 * c, bits[c], s);
        float acc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmax3_nan(s[e], s[e + 4], s[e + 8]);
#pragma unroll
        for (int x = 12; x + 8 <= 28; x += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fmax3_nan(acc[e], s[x + e], s[x + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmax_nan(acc[e], s[28 + e]);
        mx = fmax_nan(mx, fmax_nan(fmax3_nan(acc[0], acc[1], acc[2]), acc[3]));
      }
      mx *= P.scale_log2;
      // does any row of the tile need a larger maximum (or has a wait given up)?
      // One barrier with a vote; the rows' halves meet in shared memory only then.
      float alpha = 1.f;
      const bool quiet = got && (mx <= m_run + kRescaleLog2 || !row);
      if (!named_barrier_and(1 + g, 2 * kRows, quiet)) {
        aux.row[g][half][r] = mx;
        if (!named_barrier_and(1 + g, 2 * kRows, got)) {
          if (!got) fail();
          ok = false;
          break;
        }
        mx = fmax_nan(mx, aux.row[g][half ^ 1][r]);
        // a score that is no number, or infinite, makes the row's sum and so its result
        // none (exp2_poly2_fine, which takes some of the keys, loses it)
        if (!(mx < INFINITY)) l_run = NAN;
        const bool grow = mx > m_run + kRescaleLog2;
        if (grow) {
          alpha = ex2_approx(m_run - mx);  // 0 on the first tile
          m_run = mx;
        }
        if (j > 0) {  // P V of the tile before is done: S of this one came after it
          if (__any_sync(~0u, grow)) {
            for (int c0 = oc0; c0 < oc1; c0 += 16) {
              float o[16];
              tmem_ld16(tO + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= alpha;
              tmem_st16(tO + c0, o);
            }
            tmem_wait_st();
          }
          tc_fence_before_sync();
        }
        named_barrier(1 + g, 2 * kRows);  // O is whole again before either half's P is handed on
        tc_fence_after_sync();
      }
      // p = 2^(s c - m), two at a time: one pair in eight on the FMA pipe, the
      // rest on the special-function unit (7920 keys, repeated, us: none 219, one in
      // eight 213, in four 217, in two 232); P packed to bf16 into TMEM as it goes,
      // over columns of this half that have been read
      const uint64_t c2 = f2_pack(P.scale_log2, P.scale_log2), nm2 = f2_pack(-m_run, -m_run);
      uint64_t sum2[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!kKeep || c) scores(tS + kHalf * half + 32 * c, bits[c], s);
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint64_t x = f2_fma(f2_pack(s[i], s[i + 1]), c2, nm2);
          uint64_t p2;
          float a, e;
          if ((i & 15) == 14) {
            p2 = exp2_poly2_fine(x);
            f2_unpack(p2, a, e);
          } else {
            f2_unpack(x, a, e);
            a = ex2_approx(a);
            e = ex2_approx(e);
            p2 = f2_pack(a, e);
          }
          sum2[(i >> 1) & 1] = f2_add(sum2[(i >> 1) & 1], p2);
          pk[i >> 1] = pack_bf16x2(a, e);
        }
        tmem_st16u(tS + kHalf * half + 16 * c, pk);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive_warp(&aux.p_full[g][half], lane);
      const uint64_t sa = f2_add(sum2[0], sum2[1]);
      float rs0, rs1;
      f2_unpack(sa, rs0, rs1);
      l_run = l_run * alpha + (rs0 + rs1);
    }
    // the last product, or, with no key tile and so no product that has waited for
    // them, the queries: their copy is started before the mask is known and lands
    // where the rows are staged below
    if (ok && !__all_sync(~0u, mbar_wait(n > 0 ? &aux.o_full[g] : &aux.q_full, 0, P.limit))) {
      fail();
      ok = false;
    }
    aux.row[g][half][r] = l_run;
    ok = named_barrier_and(1 + g, 2 * kRows, ok);  // all rows of the tile agree before it is stored
    if (ok) {
      tc_fence_after_sync();
      l_run += aux.row[g][half ^ 1][r];
      // no key is seen, or every score is -inf (the sum is then what the polynomial gives
      // for 0, 2^-125 each) and none is NaN
      const bool any = n > 0 && !(m_run == kLowest && l_run < 1.f);
      const float lse = any ? (m_run + log2f(l_run)) * 0.6931471805599453f : -INFINITY;
      const float inv = any ? 1.f / l_run : 0.f;
      if (row && half == 0 && P.lse && whole) P.lse[((long long)b * Hq + head) * P.Tq + t] = lse;
      const long long part = ((long long)x * NQ + g) * kRows;  // x: split unit * nsplit + split
      if (half == 0 && !whole) P.part_lse[part + r] = lse;
      // every S MMA has completed, or none was issued and Q has landed: the tile's Q
      // buffer takes its rows, 4 KB a warp
      uint8_t* stage = smem + L::q + g * L::tile + (warp & 7) * (L::tile / 8);
      const int r0 = (warp & 3) * 32;
      for (int c0 = oc0; c0 < oc1; c0 += 32) {
        float o[32];
        const int cols = min(32, oc1 - c0);
        if (n > 0) {
          if (cols == 32)
            tmem_ld32(tO + c0, o);
          else
            tmem_ld16(tO + c0, *reinterpret_cast<float(*)[16]>(o));
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = any ? o[e] * inv : 0.f;
        if (whole) {
          const uint4 v[4] = {pack8_bf16(o), pack8_bf16(o + 8), pack8_bf16(o + 16), pack8_bf16(o + 24)};
          store_rows<4>(stage, lane, v, cols / 8, [&](int i) -> void* {
            const int q = r0 + i, dt = q * P.gmul >> 16, dh = q - dt * P.G;  // row = token * G + head
            return dt < P.tokens && tok0 + dt < P.Tq ? out0 + ((long long)dt * Hq + dh) * D + c0 : nullptr;
          });
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float* f = o + 16 * h + 4 * e;
              v[e] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                __float_as_uint(f[3]));
            }
            if (16 * h < cols)
              store_rows<4>(stage, lane, v, 4,
                            [&](int i) -> void* { return P.part_o + (part + r0 + i) * D + c0 + 16 * h; });
          }
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == Roles<NQ>::mma) {
    tc_fence_after_sync();
    tmem_dealloc(aux.tmem, kTileCols * NQ);
  }
}

// Joins the splits: out = sum_i w_i o_i with w_i = e^(lse_i - lse).  Four features a
// lane; a warp takes two rows of the split units, or, where there are many splits (few
// query rows over many keys), eight warps take one and add up in their order.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kJoinSplits = 8;  // above, eight warps to a row
template <int W>  // warps of a row
__global__ void __launch_bounds__(kJoinThreads)
gdn_cross_join_kernel(const __grid_constant__ CrossParams P, int per, unsigned rows) {
  constexpr int R = W == 1 ? 2 : 1;                   // rows of a warp
  __shared__ float4 sums[W > 1 ? W : 1][33];          // a warp's o of 4 x 32 features, and its weights' sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = W > 1 ? warp % W : 0, f = lane * 4;
  bool on[R];
  long long at[R], to[R], to_lse[R];
  pdl_wait();
#pragma unroll
  for (int e = 0; e < R; ++e) {
    const unsigned i = (blockIdx.x * (kJoinWarps / W) + warp / W) * R + e;
    const unsigned su = i / per, ur = i - su * per, r = ur % kRows;  // per: rows of a unit, in whole tiles or one of few
    const unsigned u = P.full + su, bh = u / P.groups;
    const int tile = ((u - bh * P.groups) * per + ur) / kRows;
    const int b = bh / P.Hk, hk = bh - b * P.Hk, dt = r * P.gmul >> 16;
    const int t = tile * P.tokens + dt, head = hk * P.G + r - dt * P.G, Hq = P.Hk * P.G;
    on[e] = i < rows && r < P.tokens * P.G && t < P.Tq;  // a row
    at[e] = (long long)su * P.nsplit * per + ur;         // of split 0, then every `per`
    to[e] = (((long long)b * P.Tq + t) * Hq + head) * P.D + f;
    to_lse[e] = ((long long)b * Hq + head) * P.Tq + t;
  }
  float top[R], sum[R], o[R][4];
#pragma unroll
  for (int e = 0; e < R; ++e) {
    top[e] = -INFINITY;
    for (int s = lane; on[e] && s < P.nsplit; s += 32) top[e] = fmax_nan(top[e], P.part_lse[at[e] + (long long)s * per]);
    sum[e] = o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < R; ++e)
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top[e] = fmax_nan(top[e], __shfl_xor_sync(~0u, top[e], x));
#pragma unroll 4
  for (int s = first; s < P.nsplit; s += W) {
#pragma unroll
    for (int e = 0; e < R; ++e) {
      const long long x = at[e] + (long long)s * per;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on[e] && f < P.D) v = *reinterpret_cast<const float4*>(P.part_o + x * P.D + f);
      const float w = top[e] != -INFINITY ? expf(P.part_lse[x] - top[e]) : 0.f;  // NaN is passed on
      const bool some = w > 0.f;  // a split that saw nothing left no part
      sum[e] += w;
      o[e][0] += some ? w * v.x : 0.f;
      o[e][1] += some ? w * v.y : 0.f;
      o[e][2] += some ? w * v.z : 0.f;
      o[e][3] += some ? w * v.w : 0.f;
    }
  }
  if (W > 1) {
    sums[first][lane] = make_float4(o[0][0], o[0][1], o[0][2], o[0][3]);
    if (lane == 0) sums[first][32].x = sum[0];
    __syncthreads();
    if (first) return;
#pragma unroll
    for (int x = 1; x < W; ++x) {
      const float4 v = sums[x][lane];
      sum[0] += sums[x][32].x;
      o[0][0] += v.x;
      o[0][1] += v.y;
      o[0][2] += v.z;
      o[0][3] += v.w;
    }
  }
#pragma unroll
  for (int e = 0; e < R; ++e) {
    if (!on[e]) continue;
    const bool any = top[e] != -INFINITY;
    const float inv = any ? 1.f / sum[e] : 0.f;
    if (f < P.D)
      *reinterpret_cast<uint2*>(P.out + to[e]) =
          make_uint2(pack_bf16x2(o[e][0] * inv, o[e][1] * inv), pack_bf16x2(o[e][2] * inv, o[e][3] * inv));
    if (lane == 0 && P.lse) P.lse[to_lse[e]] = any ? top[e] + logf(sum[e]) : -INFINITY;
  }
}

// The shape of a call: units, splits along the keys.  Returns the rows of a unit:
// one or two tiles, or kFewRows for the kernel of few rows.
int cross_shape(const CrossCall& c, CrossParams* P) {
  P->Tq = c.Tq;
  P->S = c.S;
  P->Hk = c.Hk;
  P->G = c.Hq / c.Hk;
  P->D = c.D;
  P->gmul = 65536 / P->G + 1;
  if ((long long)c.Tq * P->G <= kFewRows) {
    const int units = c.B * c.Hk;
    P->tokens = c.Tq;
    P->qtiles = P->groups = 1;
    P->nsplit = few_splits(c.B, c.Hk, c.S);
    P->full = P->nsplit > kFewCluster ? 0 : units;  // (a cluster leaves no parts)
    return kFewRows;
  }
  P->tokens = kRows / P->G;
  P->qtiles = (c.Tq + P->tokens - 1) / P->tokens;
  P->ntiles = (c.S + kRows - 1) / kRows;
  // Up to 16 key tiles two CTAs of one query tile each share an SM, their starts
  // and ends under each other's work; beyond, one CTA of two tiles halves the keys
  // and values that are loaded.  Fresh inputs (pair / single, us): 2640 queries, 20 heads
  // of 112, 128 keys 15.9 / 14.4, 300 23.7 / 21.2, 1024 44.3 / 43.4, 2048 65.2 / 64.9,
  // 2640 78.9 / 79.2, 7920 181 / 190 (heads of 64: 180 / 172); 1024 queries, 16 heads of
  // 128, 4096 keys 48.9 / 51.3.  The rule does not look at the queries: with one query
  // tile (17 to 128 rows) over more than 16 key tiles a pair's second half is idle,
  // 20 heads of 112 over 2640 keys 22.4 / 18.9, over 7920 31.9 / 30.8, 8 requests of
  // them 123 / 126.
  const int nq = P->ntiles <= kSingleTiles ? 1 : 2;
  P->groups = (P->qtiles + nq - 1) / nq;
  const long long units = (long long)c.B * c.Hk * P->groups;
  const long long slots = num_sms() * (3 - nq);  // CTAs that run at a time
  // Units of a last, partial wave are split along the keys while a CTA keeps at
  // least two tiles, so that the wave is full and shorter; with fewer units than
  // slots that is all of them.
  const long long rest = units % slots;
  long long n = rest ? std::max<long long>(1, std::min<long long>(slots / rest, P->ntiles / 2)) : 1;
  P->full = n > 1 ? (unsigned)(units - rest) : (unsigned)units;
  if (c.mask && P->ntiles > kMaskTiles) {  // what a CTA can list
    n = std::max<long long>(n, (P->ntiles + kMaskTiles - 1) / kMaskTiles);
    P->full = 0;
  }
  P->per_split = (int)std::max<long long>(1, (P->ntiles + n - 1) / n);
  P->nsplit = std::max(1, (P->ntiles + P->per_split - 1) / P->per_split);
  P->most = P->full ? P->ntiles : P->per_split;
  return nq * kRows;
}

// CTAs of the split units.
long long split_blocks(const CrossCall& c, const CrossParams& P) {
  return ((long long)c.B * c.Hk * P.groups - P.full) * P.nsplit;
}

template <int NB, int NQ>
cudaError_t launch_nb(unsigned grid, cudaStream_t stream, const CUtensorMap& mq, const CUtensorMap& mk,
                      const CUtensorMap& mv, const CrossParams& P) {
  // more than a third (half) of an SM's shared memory: two CTAs (one) per SM, as
  // many as tensor memory has columns for
  constexpr int least = NQ == 1 ? 80 * 1024 : 116 * 1024;
  using L = CrossLayout<NB, NQ>;
  const int bytes = std::max<int>(least, L::mask + (P.mask ? P.most * L::mask_tile : 0));
  constexpr int most = std::max<int>(least, L::mask + (NQ == 1 ? kSingleTiles : kMaskTiles) * L::mask_tile);
  const cudaError_t e = allow_smem(gdn_cross_kernel<NB, NQ>, most);
  if (e != cudaSuccess) return e;
  ProfileScope ps(stream, kKernCross);
  return launch_after(gdn_cross_kernel<NB, NQ>, grid, Roles<NQ>::threads, bytes, stream, mq, mk, mv, P);
}

cudaError_t launch_tiles(const CrossCall& c, CrossParams* P, int nq, unsigned grid) {
  P->qb = c.q.batch_stride != 0;
  P->kb = c.k.batch_stride != 0;
  P->vb = c.v.batch_stride != 0;
  CUtensorMap mq, mk, mv;
  if (!make_heads_map(&mq, c.q.data, P->qb ? c.B : 1, c.Tq, c.Hk, P->G, c.D, c.q.batch_stride, c.q.token_stride,
                      P->tokens))
    return cudaErrorInvalidValue;
  if (c.S == 0) {
    mk = mv = mq;  // no key tile is ever loaded
  } else if (!make_heads_map(&mk, c.k.data, P->kb ? c.B : 1, c.S, c.Hk, 1, c.D, c.k.batch_stride,
                             c.k.token_stride, kRows) ||
             !make_heads_map(&mv, c.v.data, P->vb ? c.B : 1, c.S, c.Hk, 1, c.D, c.v.batch_stride,
                             c.v.token_stride, kRows)) {
    return cudaErrorInvalidValue;
  }
  cudaError_t e;
  if (nq == 1)
    e = c.D > 64 ? launch_nb<2, 1>(grid, c.stream, mq, mk, mv, *P) : launch_nb<1, 1>(grid, c.stream, mq, mk, mv, *P);
  else
    e = c.D > 64 ? launch_nb<2, 2>(grid, c.stream, mq, mk, mv, *P) : launch_nb<1, 2>(grid, c.stream, mq, mk, mv, *P);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

size_t cross_workspace_bytes(const CrossCall& c) {
  CrossParams P = {};
  const int per = cross_shape(c, &P);
  return (size_t)split_blocks(c, P) * per * (c.D + 1) * sizeof(float);
}

cudaError_t launch_cross(const CrossCall& c, void* ws) {
  CrossParams P = {};
  const int per = cross_shape(c, &P);
  const long long parts = split_blocks(c, P);
  P.mask = c.mask;
  P.mask_bs = c.mask_bs;
  P.scale_log2 = c.scale * 1.4426950408889634f;
  P.out = static_cast<__nv_bfloat16*>(c.out);
  P.lse = c.lse;
  P.part_o = static_cast<float*>(ws);
  P.part_lse = P.part_o + (size_t)parts * per * c.D;
  P.limit = c.limit;
  P.err = c.err;
  cudaError_t e = per == kFewRows ? launch_cross_few(c, P) : launch_tiles(c, &P, per / kRows, (unsigned)(P.full + parts));
  if (e != cudaSuccess) return e;
  if (parts > 0) {
    ProfileScope ps(c.stream, kKernCrossJoin);
    const unsigned rows = (unsigned)(parts / P.nsplit * per);  // (their parts fit the device's memory)
    const bool many = P.nsplit > kJoinSplits;
    const unsigned each = many ? 1 : 2 * kJoinWarps;  // rows of a block
    e = launch_after(many ? gdn_cross_join_kernel<kJoinWarps> : gdn_cross_join_kernel<1>, (rows + each - 1) / each,
                     kJoinThreads, 0, c.stream, P, per, rows);
    if (e == cudaSuccess) count_launches(1);
  }
  return e;
}

}  // namespace gdn
