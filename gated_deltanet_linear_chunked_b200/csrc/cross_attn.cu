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
//   warp 8         TMA producer: the Q tiles, then K_0 V_0 K_1 V_1 ... through a
//                  ring of four slots (128-byte swizzle: a box row is 128 bytes).
//   warps 9, 10    MMA issue for g = 0, 1, one lane each: S_g = Q_g K_j^T (M 128,
//                  N 128, K D) and O_g += P_g V_j (M 128, N D, K 128), both in
//                  TMEM; P_g is read from TMEM (bf16, over the first 64 columns of
//                  S_g), which leaves shared memory's bandwidth to K and V: from
//                  shared memory P alone would take 4 KB per 16 keys against V's
//                  2 D bytes x 16, more than the tensor core's time allows.
//   warps 0-3, 4-7 softmax of g = 0, 1, a row per thread (its TMEM lane): maximum,
//                  p = 2^(s c - m), sum, P back to TMEM; O is rescaled in TMEM
//                  only when the maximum has grown by more than 2^8 (until then p
//                  may reach 2^8, which fp32 sums and bf16 P hold as well as 1).
// P_g,j is used up before S_g,j+1 is written over it because one thread issues
// both and tensor-core operations of one thread complete in order; while one
// tile's softmax runs the other's products do.
// Masked keys: a CTA first reads its batch row's mask into one bit per key and
// lists the key tiles that have any, so tiles without are never loaded; in tiles
// with some, scores of masked keys become -inf whatever they were, and the masked
// rows of V are cleared in shared memory, since 0 * NaN would reach the sum.
// Few query tiles and many keys: the key tiles are split over CTAs, each leaves
// its normalised fp32 part and its lse, and gdn_cross_join_kernel joins them.
// Every wait is bounded; one that gives up sets the error word and the CTA drains
// its copies and MMAs before it frees TMEM.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "gdn_internal.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kQTiles = 2;
constexpr int kRows = 128;             // rows of a query tile, keys of a key tile
constexpr int kSlots = 4;              // ring of K and V tiles
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kThreads = 32 * (kMmaWarp + kQTiles);
constexpr uint32_t kTileCols = 256;    // TMEM columns of a tile: S (and P) [0, 128) | O [128, 128 + D)
constexpr uint32_t kBlock = kRows * 128;  // one 64-feature block of a 128-row tile, bytes
constexpr int kMaskTiles = 128;        // key tiles of one CTA under a mask, at most
constexpr float kRescaleLog2 = 8.f;
constexpr long long kDrainPolls = 1LL << 40;  // drains are bounded by the 2 s timer

struct CrossParams {
  int Tq, S, Hk, G, D;
  int tokens;            // query tokens per tile: 128 / G
  int qtiles, groups;    // query tiles of a (b, key head); CTAs along them (nq tiles each)
  int nq;
  int ntiles, nsplit, per_split;  // key tiles, CTAs along them, tiles of each
  int qb, kb, vb;        // batch coordinate factors: 0 for a broadcast batch
  const uint8_t* mask;
  long long mask_bs;
  float scale_log2;      // scale * log2(e)
  float* lse;            // [B, Hq, Tq] or nullptr
  float* part_o;         // nsplit > 1: [nsplit][B, Tq, Hq][D] fp32
  float* part_lse;       // nsplit > 1: [nsplit][B, Tq, Hq]
  long long rows;        // B * Tq * Hq
  long long limit;
  unsigned* err;
};

struct CrossAux {
  uint64_t q_full;
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[kQTiles], p_full[kQTiles], o_full[kQTiles], drain[kQTiles];
  uint32_t tmem;
  int abort;
  int count;                       // key tiles to walk
  uint32_t bits[kMaskTiles * 4];   // seen keys of each of the CTA's tiles (under a mask)
  uint8_t list[kMaskTiles];        // tiles with any
};

// Shared memory: Q tiles (later the output's), the ring, the barriers and mask.
struct CrossLayout {
  uint32_t tile, q, ring, aux, total;
};
__host__ __device__ inline CrossLayout cross_layout(int D) {
  CrossLayout L;
  L.tile = ((D + 63) / 64) * kBlock;
  L.q = 0;
  L.ring = kQTiles * L.tile;
  L.aux = L.ring + kSlots * L.tile;
  L.total = L.aux + (uint32_t)sizeof(CrossAux);
  return L;
}

__global__ void __launch_bounds__(kThreads, 1)
gdn_cross_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_out,
                 const __grid_constant__ CrossParams P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int D = P.D, nb = (D + 63) / 64;
  const CrossLayout L = cross_layout(D);
  CrossAux& aux = *reinterpret_cast<CrossAux*>(smem + L.aux);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // unit: ((b * Hk + hk) * groups + group) * nsplit + split
  const int split = blockIdx.x % P.nsplit, u = blockIdx.x / P.nsplit;
  const int group = u % P.groups, bh = u / P.groups;
  const int b = bh / P.Hk, hk = bh - b * P.Hk;
  const int tile0 = group * P.nq, nq = min(P.nq, P.qtiles - tile0);
  const int k0 = split * P.per_split, kn = min(P.per_split, P.ntiles - k0);  // key tiles of the split
  volatile int* abort_flag = &aux.abort;

  if (tid == 0) {
    mbar_init(&aux.q_full, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&aux.full[s], 1);
      mbar_init(&aux.empty[s], nq);
    }
    for (int g = 0; g < kQTiles; ++g) {
      mbar_init(&aux.s_full[g], 1);
      mbar_init(&aux.p_full[g], kRows);
      mbar_init(&aux.o_full[g], 1);
      mbar_init(&aux.drain[g], 1);
    }
    aux.abort = 0;
    aux.count = kn;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&aux.tmem, kTileCols * kQTiles);
    tmem_relinquish();
  }
  if (P.mask) {
    const uint8_t* mrow = P.mask + b * P.mask_bs;
    for (int w = warp; w < kn * 4; w += kThreads / 32) {
      const long long key = (long long)(k0 * 4 + w) * 32 + lane;
      const uint32_t bits = __ballot_sync(~0u, key < P.S && mrow[key] != 0);
      if (lane == 0) aux.bits[w] = bits;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (P.mask) {
    if (warp == 0) {
      int n = 0;
      for (int t0 = 0; t0 < kn; t0 += 32) {
        const int t = t0 + lane;
        const bool any = t < kn && (aux.bits[4 * t] | aux.bits[4 * t + 1] | aux.bits[4 * t + 2] |
                                    aux.bits[4 * t + 3]) != 0;
        const uint32_t bal = __ballot_sync(~0u, any);
        if (any) aux.list[n + __popc(bal & ((1u << lane) - 1))] = (uint8_t)t;
        n += __popc(bal);
      }
      if (lane == 0) aux.count = n;
    }
    __syncthreads();
  }
  const uint32_t tm = aux.tmem;
  const int n = aux.count;
  const bool masked = P.mask != nullptr;
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(P.err, kErrTimeout);
  };
  // ring item i: K (even i) or V (odd i) of listed tile i / 2
  auto slot_ptr = [&](int i) { return smem + L.ring + (i % kSlots) * L.tile; };
  auto wait_full = [&](int i) { return mbar_wait(&aux.full[i % kSlots], (i / kSlots) & 1, P.limit); };

  if (warp == kProducerWarp) {
    if (lane == 0 && n > 0) {
      const uint32_t qbytes = (uint32_t)P.tokens * P.G * 128;  // of one 64-feature block
      mbar_arrive_expect_tx(&aux.q_full, nq * nb * qbytes);
      for (int g = 0; g < nq; ++g)
        for (int c = 0; c < nb; ++c)
          tma_load_5d(smem + L.q + g * L.tile + c * kBlock, &tm_q, &aux.q_full, c * 64, 0,
                      (tile0 + g) * P.tokens, hk, b * P.qb);
      int issued = 0;
      for (int i = 0; i < 2 * n; ++i) {
        if (*abort_flag) break;
        if (i >= kSlots && !mbar_wait(&aux.empty[i % kSlots], (i / kSlots - 1) & 1, P.limit)) {
          fail();
          break;
        }
        const int tile = k0 + (masked ? aux.list[i / 2] : i / 2);
        uint64_t* bar = &aux.full[i % kSlots];
        mbar_arrive_expect_tx(bar, L.tile);
        for (int c = 0; c < nb; ++c)
          tma_load_5d(slot_ptr(i) + c * kBlock, i & 1 ? &tm_v : &tm_k, bar, c * 64, 0, tile * kRows, hk,
                      b * (i & 1 ? P.vb : P.kb));
        ++issued;
      }
      // every load has landed before shared memory goes
      mbar_wait(&aux.q_full, 0, kDrainPolls);
      for (int i = max(0, issued - kSlots); i < issued; ++i)
        mbar_wait(&aux.full[i % kSlots], (i / kSlots) & 1, kDrainPolls);
    }
  } else if (warp >= kMmaWarp) {
    const int g = warp - kMmaWarp;
    if (lane == 0 && g < nq && n > 0) {
      const uint32_t idS = idesc_bf16(kRows, kRows, 0, 0), idO = idesc_bf16(kRows, D, 0, 1);
      const uint32_t tS = tm + g * kTileCols, tO = tS + kRows;
      const uint64_t dq = sdesc_sw128(smem_u32(smem + L.q + g * L.tile), 16);
      bool ok = mbar_wait(&aux.q_full, 0, P.limit);
      if (!ok) fail();
      for (int j = 0; ok && j <= n; ++j) {
        if (*abort_flag) break;
        if (j > 0) {
          const int i = 2 * (j - 1) + 1;
          if (!wait_full(i) || !mbar_wait(&aux.p_full[g], (j - 1) & 1, P.limit)) {
            fail();
            break;
          }
          tc_fence_after_sync();
          // O_g += P_g V: P in TMEM (8 columns per 16 keys), V MN-major
          const uint64_t dv = sdesc_sw128(smem_u32(slot_ptr(i)), kBlock);
#pragma unroll
          for (int ks = 0; ks < kRows / 16; ++ks)
            mma_bf16_ts(tO, tS + ks * 8, dv + ks * (2048 >> 4), idO, j > 1 || ks > 0);
          mma_commit(&aux.empty[i % kSlots]);
        }
        if (j < n) {
          const int i = 2 * j;
          if (!wait_full(i)) {
            fail();
            break;
          }
          tc_fence_after_sync();
          // S_g = Q_g K^T: both K-major
          const uint64_t dk = sdesc_sw128(smem_u32(slot_ptr(i)), 16);
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t at = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
            mma_bf16(tS, dq + at, dk + at, idS, ks > 0);
          }
          mma_commit(&aux.s_full[g]);
          mma_commit(&aux.empty[i % kSlots]);
        } else {
          mma_commit(&aux.o_full[g]);
        }
      }
      mma_commit(&aux.drain[g]);
      mbar_wait(&aux.drain[g], 0, kDrainPolls);
    }
  } else if ((warp >> 2) < nq) {
    const int g = warp >> 2;
    const int r = tid & (kRows - 1);
    const uint32_t tS = tm + g * kTileCols + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = tS + kRows;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (__any_sync(~0u, *abort_flag != 0)) {
        ok = false;
        break;
      }
      if (!__all_sync(~0u, mbar_wait(&aux.s_full[g], j & 1, P.limit))) {
        if (lane == 0) fail();
        ok = false;
        break;
      }
      tc_fence_after_sync();
      float s[kRows];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<float(*)[32]>(s + 32 * c));
      tmem_wait_ld();
      // the seen keys of the tile
      uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
      const int tile = masked ? aux.list[j] : j;
      if (masked) {
#pragma unroll
        for (int c = 0; c < 4; ++c) bits[c] = aux.bits[4 * tile + c];
      } else {
        const int left = P.S - (k0 + tile) * kRows;  // > 0
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (left < 32 * (c + 1)) bits[c] = left <= 32 * c ? 0u : (1u << (left - 32 * c)) - 1;
      }
      const bool part = (bits[0] & bits[1] & bits[2] & bits[3]) != ~0u;  // uniform over the CTA
      if (part) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (!(bits[i / 32] >> (i % 32) & 1)) s[i] = -INFINITY;
        if (masked) {  // clear the masked rows of V
          const int i = 2 * j + 1;
          if (!__all_sync(~0u, wait_full(i))) {
            if (lane == 0) fail();
            ok = false;
            break;
          }
          if (!(bits[r / 32] >> (r % 32) & 1)) {
            for (int c = 0; c < nb * 8; ++c)
              *reinterpret_cast<uint4*>(slot_ptr(i) + (c >> 3) * kBlock + r * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
      }
      float acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmax3(s[e], s[e + 8], s[e + 16]);
#pragma unroll
      for (int i = 24; i + 16 <= 120; i += 16)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmax3(acc[e], s[i + e], s[i + 8 + e]);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaxf(acc[e], s[120 + e]);
      float mx = fmax3(fmax3(acc[0], acc[1], acc[2]), fmax3(acc[3], acc[4], acc[5]), fmaxf(acc[6], acc[7]));
      mx *= P.scale_log2;
      float m_new = m_run, alpha = 1.f;
      bool resc = false;
      if (mx > m_run + kRescaleLog2) {
        m_new = mx;
        alpha = ex2_approx(m_run - m_new);  // 0 on the first tile
        resc = j > 0;
      }
      if (__any_sync(~0u, resc)) {  // P V of the tile before is done: S of this one came after it
        const float a = resc ? alpha : 1.f;
        for (int c0 = 0; c0 < D; c0 += 16) {
          float o[16];
          tmem_ld16(tO + c0, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= a;
          tmem_st16(tO + c0, o);
        }
      }
      // p = 2^(s c - m), two at a time: one pair in four on the FMA pipe, the
      // rest on the special-function unit; P packed to bf16 into TMEM as it goes
      const uint64_t c2 = f2_pack(P.scale_log2, P.scale_log2), nm2 = f2_pack(-m_new, -m_new);
      uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint64_t x = f2_fma(f2_pack(s[32 * c + i], s[32 * c + i + 1]), c2, nm2);
          uint64_t p2;
          float a, e;
          if ((i & 7) == 6) {
            p2 = exp2_poly2(x);
            f2_unpack(p2, a, e);
          } else {
            f2_unpack(x, a, e);
            a = ex2_approx(a);
            e = ex2_approx(e);
            p2 = f2_pack(a, e);
          }
          sum2[(i >> 1) & 3] = f2_add(sum2[(i >> 1) & 3], p2);
          pk[i >> 1] = pack_bf16x2(a, e);
        }
        tmem_st16u(tS + 16 * c, pk);
      }
      const uint64_t sa = f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3]));
      float rs0, rs1;
      f2_unpack(sa, rs0, rs1);
      l_run = l_run * alpha + (rs0 + rs1);
      m_run = m_new;
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&aux.p_full[g]);
    }
    if (ok && n > 0 && !__all_sync(~0u, mbar_wait(&aux.o_full[g], 0, P.limit))) {
      if (lane == 0) fail();
      ok = false;
    }
    ok = named_barrier_and(1 + g, kRows, ok);  // all rows of the tile agree before it is stored
    if (ok) {
      tc_fence_after_sync();
      const int Hq = P.Hk * P.G;
      const int t = (tile0 + g) * P.tokens + r / P.G, head = hk * P.G + r % P.G;
      const bool row = r < P.tokens * P.G && t < P.Tq;
      const float lse = n > 0 ? (m_run + log2f(l_run)) * 0.6931471805599453f : -INFINITY;
      const float inv = n > 0 ? 1.f / l_run : 0.f;
      if (P.nsplit > 1) {
        const long long at = (long long)split * P.rows + ((long long)b * P.Tq + t) * Hq + head;
        if (row) P.part_lse[at] = lse;
        if (n > 0) {
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            tmem_ld16(tO + c0, o);
            tmem_wait_ld();
            if (row) {
              float4* to = reinterpret_cast<float4*>(P.part_o + at * D + c0);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                to[e] = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
            }
          }
        }
      } else {
        if (row && P.lse) P.lse[((long long)b * Hq + head) * P.Tq + t] = lse;
        // every S MMA has completed (or none was issued and Q never loaded):
        // the tile's Q buffer takes its output
        uint8_t* so = smem + L.q + g * L.tile + r * 128;
        for (int c0 = 0; c0 < D; c0 += 16) {
          float o[16];
          if (n > 0) {
            tmem_ld16(tO + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= inv;
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0.f;
          }
          uint8_t* blk = so + (c0 >> 6) * kBlock;
          const int c = (c0 & 63) >> 3;
          *reinterpret_cast<uint4*>(blk + ((c ^ (r & 7)) << 4)) = pack8_bf16(o);
          *reinterpret_cast<uint4*>(blk + (((c + 1) ^ (r & 7)) << 4)) = pack8_bf16(o + 8);
        }
        fence_proxy_async_smem();
        named_barrier(1 + g, kRows);
        if (r == 0) {
          for (int c = 0; c < nb; ++c)
            tma_store_5d(&tm_out, smem + L.q + g * L.tile + c * kBlock, c * 64, 0, (tile0 + g) * P.tokens, hk, b);
          bulk_commit();
          bulk_wait_all();
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tm, kTileCols * kQTiles);
  }
}

// Joins the splits: out = sum_i w_i o_i with w_i = e^(lse_i - lse).  A warp per
// row, four features a lane.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
gdn_cross_join_kernel(const __grid_constant__ CrossParams P, __nv_bfloat16* out) {
  const long long row = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= P.rows) return;
  float top = -INFINITY;
  for (int i = 0; i < P.nsplit; ++i) top = fmaxf(top, P.part_lse[i * P.rows + row]);
  const bool any = top > -INFINITY;
  float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int f = lane * 4;
  for (int i = 0; any && i < P.nsplit; ++i) {
    const float w = expf(P.part_lse[i * P.rows + row] - top);
    sum += w;
    if (w > 0.f && f < P.D) {  // a split that saw nothing left no part
      const float4 x = *reinterpret_cast<const float4*>(P.part_o + (i * P.rows + row) * P.D + f);
      o[0] += w * x.x;
      o[1] += w * x.y;
      o[2] += w * x.z;
      o[3] += w * x.w;
    }
  }
  const float inv = any ? 1.f / sum : 0.f;
  if (f < P.D) {
    uint2 u = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    *reinterpret_cast<uint2*>(out + row * P.D + f) = u;
  }
  if (lane == 0 && P.lse) {
    const int Hq = P.Hk * P.G;
    const long long bt = row / Hq, b = bt / P.Tq;
    P.lse[(b * Hq + (row - bt * Hq)) * P.Tq + (bt - b * P.Tq)] = any ? top + logf(sum) : -INFINITY;
  }
}

// The shape of a call: tiles, CTAs along queries and splits along keys.
void cross_shape(const CrossCall& c, CrossParams* P) {
  P->Tq = c.Tq;
  P->S = c.S;
  P->Hk = c.Hk;
  P->G = c.Hq / c.Hk;
  P->D = c.D;
  P->tokens = kRows / P->G;
  P->qtiles = (c.Tq + P->tokens - 1) / P->tokens;
  P->nq = std::min(kQTiles, P->qtiles);
  P->groups = (P->qtiles + P->nq - 1) / P->nq;
  P->ntiles = (c.S + kRows - 1) / kRows;
  P->rows = (long long)c.B * c.Tq * c.Hq;
  // split the keys while a CTA keeps at least two tiles and the GPU has room
  const long long units = (long long)c.B * c.Hk * P->groups;
  long long n = std::max<long long>(1, std::min<long long>(num_sms() / units, P->ntiles / 2));
  if (c.mask) n = std::max<long long>(n, (P->ntiles + kMaskTiles - 1) / kMaskTiles);
  P->per_split = (int)std::max<long long>(1, (P->ntiles + n - 1) / n);
  P->nsplit = std::max(1, (P->ntiles + P->per_split - 1) / P->per_split);
}

}  // namespace

size_t cross_workspace_bytes(const CrossCall& c) {
  CrossParams P = {};
  cross_shape(c, &P);
  return P.nsplit > 1 ? (size_t)P.nsplit * P.rows * (c.D + 1) * sizeof(float) : 0;
}

cudaError_t launch_cross(const CrossCall& c, void* ws) {
  CrossParams P = {};
  cross_shape(c, &P);
  P.mask = c.mask;
  P.mask_bs = c.mask_bs;
  P.scale_log2 = c.scale * 1.4426950408889634f;
  P.lse = c.lse;
  P.part_o = static_cast<float*>(ws);
  P.part_lse = P.part_o + (size_t)P.nsplit * P.rows * c.D;
  P.limit = c.limit;
  P.err = c.err;
  P.qb = c.q.batch_stride != 0;
  P.kb = c.k.batch_stride != 0;
  P.vb = c.v.batch_stride != 0;
  CUtensorMap mq, mk, mv, mo;
  const long long ots = (long long)c.Hq * c.D;
  if (!make_heads_map(&mq, c.q.data, P.qb ? c.B : 1, c.Tq, c.Hk, P.G, c.D, c.q.batch_stride,
                      c.q.token_stride, P.tokens) ||
      !make_heads_map(&mo, c.out, c.B, c.Tq, c.Hk, P.G, c.D, c.Tq * ots, ots, P.tokens))
    return cudaErrorInvalidValue;
  if (c.S == 0) {
    mk = mv = mq;  // no key tile is ever loaded
  } else if (!make_heads_map(&mk, c.k.data, P.kb ? c.B : 1, c.S, c.Hk, 1, c.D, c.k.batch_stride,
                             c.k.token_stride, kRows) ||
             !make_heads_map(&mv, c.v.data, P.vb ? c.B : 1, c.S, c.Hk, 1, c.D, c.v.batch_stride,
                             c.v.token_stride, kRows)) {
    return cudaErrorInvalidValue;
  }
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static bool done[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(gdn_cross_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)cross_layout(128).total);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  // more than half an SM's shared memory: one CTA (all of TMEM) per SM
  const uint32_t smem = std::max(cross_layout(c.D).total, 116u * 1024);
  const unsigned grid = (unsigned)((long long)c.B * c.Hk * P.groups * P.nsplit);
  {
    ProfileScope ps(c.stream, kKernCross);
    gdn_cross_kernel<<<grid, kThreads, smem, c.stream>>>(mq, mk, mv, mo, P);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (P.nsplit > 1) {
    ProfileScope ps(c.stream, kKernCrossJoin);
    const unsigned blocks = (unsigned)((P.rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
    gdn_cross_join_kernel<<<blocks, kJoinThreads, 0, c.stream>>>(P, static_cast<__nv_bfloat16*>(c.out));
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
  }
  return e;
}

}  // namespace gdn
