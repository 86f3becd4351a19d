// cross_attn_bwd.cu -- gradients of the attention to the encoder's states.
//
//   P = e^(s - lse) (0 at masked keys),  delta = sum_f dO O,  dP = dO V^T,
//   dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
// the last two summed over the query heads of a key head as well: they are rows
// of the same products, packed as in the forward (row = token * G + head).
//
// Two passes instead of one over the same tiles.  One pass that makes all three
// gradients needs five products per tile but has to add dQ (or dK and dV) up
// across CTAs, by atomics, whose order changes the result, or through partial
// sums of full size; two passes take seven products and every sum stays in a
// CTA's TMEM, in a fixed order.
//   gdn_cross_stat_kernel  -lse log2 e and -delta of every packed row; -inf and 0
//                  for the rows that are none (past the tokens, or with no key),
//                  for which 2^(s - inf) = 0.
//   gdn_cross_bwd_kernel   dQ: a CTA per query tile (and share of the key tiles, where
//                  there are few query tiles) walks the key tiles.
//                  dK, dV: a CTA per key tile and share of the query tiles; the
//                  products are transposed, S^T = K Q^T and dP^T = V dO^T, so that
//                  a TMEM lane is a key, P^T and dS^T are left operands out of
//                  TMEM, and dK and dV add up there.
//   gdn_cross_grad_join_kernel  adds the shares up where there are several.
// P and dS enter the products as bf16, and where there is one key tile as the sum of
// two bf16: their rounding is as large as the result's own, and with few keys the
// rounding of out in delta comes to it (22 keys: error of dq 1.5 times that of one
// rounding, of dv 1.4; 1.1 and 1.0 with two terms; the products they cost are not what
// bounds calls that small: 333 queries of 77 keys 19.1 -> 21 us).
// No maximum is searched and no row's threads meet: lse is known.  16 warps take
// a 128 x 128 tile, 32 columns a thread; one warp copies, one issues products.
// 2 x 4095 queries of 16 heads over 2641 keys of 4, 128 wide, a fifth masked: 442 us on
// fresh inputs, 1140 TFLOP/s of the seven products, tensor core 64% busy; TMEM is full, so
// a tile's exponentials and its products take turns in part.  2640 queries over 225 of
// 300 keys, 20 heads of 112: 48 us, of which the row statistics and the join of the shares
// 13: short tiles, one CTA an SM, their starts and ends bare.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "gdn_internal.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kRows = 128;
constexpr int kCols = 32;               // columns of a softmax thread
constexpr int kSoftmaxWarps = 16;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kProducerWarp = kSoftmaxWarps;
constexpr int kMmaWarp = kProducerWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr uint32_t kBlock = kRows * 128;
constexpr int kStatThreads = 256;
constexpr long long kDrainPolls = 1LL << 40;

struct BwdParams {
  int Tq, S, Hk, G, D;
  int tokens, qtiles, ntiles;   // tokens and tiles of queries, tiles of keys
  int gmul;                     // r / G = r * gmul >> 16 for rows r < 128
  int nsplit, per_split;        // dkv: shares of the query tiles, tiles of each
  int qsplit, per_qsplit;       // dq: shares of the (listed) key tiles, tiles of each
  unsigned dkv_blocks;          // ntiles * nsplit of every (b, key head)
  int qb, kb, vb;
  const uint32_t* bits;         // under a mask: seen keys, [B][ntiles][4], one bit each
  const int* list;              // ... and [B][ntiles + 1]: the tiles with any, their number last
  float scale, scale_log2;
  __nv_bfloat16 *dq, *dk, *dv;
  const float* stat;            // [B * Hk][qtiles][2][128]: -lse log2 e, -delta
  float* part;                  // nsplit > 1: [nsplit][2 (dk, dv)][B * Hk][ntiles][128][D]
  long long part_rows;          // B * Hk * ntiles * 128
  float* qpart;                 // qsplit > 1: [qsplit][B * Hk][qtiles][128][D]
  long long qpart_rows;         // B * Hk * qtiles * 128
  long long limit;
  unsigned* err;
};

// The mask of batch row b as bits and as a list of the tiles with any seen key.
// One block per batch row; the list is made by its first warp.
__device__ void mask_lists(const uint8_t* mrow, int S, int ntiles, uint32_t* bits, int* list) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w = warp; w < ntiles * 4; w += kStatThreads / 32) {
    const long long key = (long long)w * 32 + lane;
    const uint32_t x = __ballot_sync(~0u, key < S && mrow[key] != 0);
    if (lane == 0) bits[w] = x;
  }
  __syncthreads();
  if (warp) return;
  int n = 0;
  for (int t0 = 0; t0 < ntiles; t0 += 32) {
    const int t = t0 + lane;
    const bool any = t < ntiles && (bits[4 * t] | bits[4 * t + 1] | bits[4 * t + 2] | bits[4 * t + 3]) != 0;
    const uint32_t bal = __ballot_sync(~0u, any);
    if (any) list[n + __popc(bal & ((1u << lane) - 1))] = t;
    n += __popc(bal);
  }
  if (lane == 0) list[ntiles] = n;
}

// The seen keys of tile t of batch row b, as four words.
__device__ __forceinline__ uint4 seen_keys(const BwdParams& P, int b, int t) {
  if (P.bits) return *reinterpret_cast<const uint4*>(P.bits + ((long long)b * P.ntiles + t) * 4);
  const int left = P.S - t * kRows;
  uint32_t w[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) w[c] = left >= 32 * (c + 1) ? ~0u : left <= 32 * c ? 0u : (1u << (left - 32 * c)) - 1;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t word_of(const uint4& w, int c) {
  return c == 0 ? w.x : c == 1 ? w.y : c == 2 ? w.z : w.w;
}

// ---------------------------------------------------------------- row stats
// Sixteen lanes per packed row, 8 features a lane; four rows of a group are loaded
// before any is summed.  Under a mask, the last B blocks turn the rows of the mask
// into bits and lists instead.
// With at most kFewKeys keys (template argument) delta is formed from them instead,
// sum_j P_j dO.v_j: dO.out holds the rounding of out, which weighs the more the fewer
// keys there are (2 keys: error of dq 2.1 times that of one rounding, against 1.1).
struct FewKeys {
  const __nv_bfloat16 *q, *k, *v;
  long long q_bs, q_ts, k_bs, k_ts, v_bs, v_ts;
};
constexpr int kFewKeys = 8;
constexpr int kStatRows = 4;
constexpr int kStatBlockRows = kStatThreads / 16 * kStatRows;
template <bool kFew>
__global__ void __launch_bounds__(kStatThreads)
gdn_cross_stat_kernel(const __nv_bfloat16* out, const __nv_bfloat16* d_out, const float* lse, float* stat,
                      long long rows, unsigned row_blocks, const uint8_t* mask, long long mask_bs,
                      const __grid_constant__ BwdParams P, const __grid_constant__ FewKeys F) {
  pdl_wait();  // inputs may come from the kernel in front
  pdl_trigger();
  if (blockIdx.x >= row_blocks) {
    const int b = blockIdx.x - row_blocks;
    mask_lists(mask + b * mask_bs, P.S, P.ntiles, const_cast<uint32_t*>(P.bits) + (long long)b * P.ntiles * 4,
               const_cast<int*>(P.list) + (long long)b * (P.ntiles + 1));
    return;
  }
  const int l = threadIdx.x & 15, Hq = P.Hk * P.G;
  const long long first = (long long)blockIdx.x * kStatBlockRows + threadIdx.x / 16;
  uint4 x[kStatRows], y[kStatRows];  // out (kFew: the query) and dO
  float lg[kStatRows];
  int at_b[kStatRows], at_hk[kStatRows];
#pragma unroll
  for (int i = 0; i < kStatRows; ++i) {
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
    lg[i] = -INFINITY;
    at_b[i] = at_hk[i] = -1;
    const long long row = first + i * (kStatThreads / 16);
    const int r = (int)(row % kRows), dt = r * P.gmul >> 16;
    const unsigned tile = (unsigned)(row / kRows), bh = tile / P.qtiles, qt = tile - bh * P.qtiles;
    const unsigned b = bh / P.Hk, hk = bh - b * P.Hk;
    const int t = qt * P.tokens + dt, head = hk * P.G + r - dt * P.G;
    if (row >= rows || r >= P.tokens * P.G || t >= P.Tq) continue;
    const long long at = (((long long)b * P.Tq + t) * Hq + head) * P.D + l * 8;
    at_b[i] = b;
    at_hk[i] = hk;
    if (l * 8 < P.D) {
      x[i] = *reinterpret_cast<const uint4*>(kFew ? F.q + b * F.q_bs + t * F.q_ts + head * P.D + l * 8 : out + at);
      y[i] = *reinterpret_cast<const uint4*>(d_out + at);
    }
    lg[i] = lse[((long long)b * Hq + head) * P.Tq + t];
  }
#pragma unroll
  for (int i = 0; i < kStatRows; ++i) {
    float u[8], v[8], d = 0.f;
    unpack8_bf16(x[i], u);
    unpack8_bf16(y[i], v);
    if (kFew) {
      for (int s = 0; s < P.S; ++s) {
        const bool on = at_b[i] >= 0 && (!mask || mask[at_b[i] * mask_bs + s] != 0);
        uint4 ku = make_uint4(0, 0, 0, 0), vu = ku;
        if (on && l * 8 < P.D) {
          ku = *reinterpret_cast<const uint4*>(F.k + at_b[i] * F.k_bs + s * F.k_ts + at_hk[i] * P.D + l * 8);
          vu = *reinterpret_cast<const uint4*>(F.v + at_b[i] * F.v_bs + s * F.v_ts + at_hk[i] * P.D + l * 8);
        }
        float kf[8], vf[8], qk = 0.f, dp = 0.f;
        unpack8_bf16(ku, kf);
        unpack8_bf16(vu, vf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          qk = fmaf(u[e], kf[e], qk);
          dp = fmaf(v[e], vf[e], dp);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          qk += __shfl_xor_sync(~0u, qk, o);
          dp += __shfl_xor_sync(~0u, dp, o);
        }
        if (on) d = fmaf(exp2f(fmaf(qk, P.scale_log2, lg[i] * -1.4426950408889634f)), dp, d);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(u[e], v[e], d);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
    }
    const long long row = first + i * (kStatThreads / 16);
    const bool on = lg[i] != -INFINITY;  // (a NaN row's gradients are NaN)
    if (l == 0 && row < rows) {
      float* to = stat + row / kRows * (2 * kRows) + row % kRows;
      to[0] = on ? lg[i] * -1.4426950408889634f : -INFINITY;
      to[kRows] = on ? -d : 0.f;
    }
  }
}

// 2^x of pair i of a thread's 16, x <= 0 up to rounding: one in four on the FMA pipe (to
// 7.5e-5, far under the rounding of P and dS to bf16; 2^-125 for -inf, of rows
// whose Q, dO or result are nothing), the others on the special-function unit, which
// alone would take 1024 cycles for a tile, half of its products' time.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x, int i) {
  if ((i & 3) == 3) return exp2_poly2<true>(x);
  float a, e;
  f2_unpack(x, a, e);
  return f2_pack(ex2_approx(a), ex2_approx(e));
}

// What rounding a and b to the packed pair left, as a packed pair.
__device__ __forceinline__ uint32_t rest_of(float a, float b, uint32_t pair) {
  return pack_bf16x2(a - __uint_as_float(pair << 16), b - __uint_as_float(pair & 0xFFFF0000u));
}

// Columns [c0, c0 + n) (n 16 or 32) of a warp's 32 rows out of TMEM, times `mul`
// (zeros if there is nothing), as bf16 to dst(row) or as fp32 to part(row).
template <typename Dst, typename Part>
__device__ __forceinline__ void put_columns(uint32_t src, int n, bool any, float mul, uint8_t* stage, int lane,
                                            bool whole, Dst dst, Part part) {
  float o[kCols];
  if (any) {
    if (n == kCols)
      tmem_ld32(src, o);
    else
      tmem_ld16(src, *reinterpret_cast<float(*)[16]>(o));
    tmem_wait_ld();
  }
#pragma unroll
  for (int e = 0; e < kCols; ++e) o[e] = any ? o[e] * mul : 0.f;
  if (whole) {
    const uint4 v[4] = {pack8_bf16(o), pack8_bf16(o + 8), pack8_bf16(o + 16), pack8_bf16(o + 24)};
    store_rows<4>(stage, lane, v, n / 8, dst);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* f = o + 16 * h + 4 * e;
      v[e] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    if (16 * h < n) store_rows<4>(stage, lane, v, 4, [&](int r) -> void* { return part(r) + 16 * h; });
  }
}

// ----------------------------------------------------------------------- dQ
// TMEM: S of even and odd key tiles [0, 128), [128, 256) (dS over them), dP
// [256, 384), dQ [384, 384 + D).  With two S the product for the next tile runs
// under this one's exponentials.
// K tiles have three places, V tiles two: K is needed until its dQ, V only until dP.
constexpr int kKs = 3, kVs = 2;
struct DqAux {
  uint64_t q_full, k_full[kKs], k_empty[kKs], v_full[kVs], v_empty[kVs];
  uint64_t s_full[2], dp_full, dp_free, ds_full[2], dq_full, drain;
  uint32_t tmem;
  int abort;
};
template <int NB>
struct DqLayout {
  static constexpr uint32_t tile = NB * kBlock;
  static constexpr uint32_t q = 0, g = tile, k = 2 * tile, v = k + kKs * tile;
  static constexpr uint32_t aux = v + kVs * tile;
  static constexpr uint32_t total = aux + (uint32_t)sizeof(DqAux);
};

// How a call's key tiles are taken: all by a CTA of dQ, or shared out, or there is one
// and dS has two terms.
enum Mode { kWhole, kShared, kOne };
template <int NB, Mode kMode>
__device__ __forceinline__ void dq_tile(uint8_t* smem, unsigned block, const CUtensorMap& tm_q,
                                        const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                                        const CUtensorMap& tm_v, const BwdParams& P) {
  using L = DqLayout<NB>;
  constexpr bool kShares = kMode == kShared;
  DqAux& aux = *reinterpret_cast<DqAux*>(smem + L::aux);
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  // unit: ((b * Hk + hk) * qtiles + tile) * qsplit + split
  const int split = kShares ? block % P.qsplit : 0, u = kShares ? block / P.qsplit : block;
  const int qt = u % P.qtiles, bh = u / P.qtiles;
  const int b = bh / P.Hk, hk = bh - b * P.Hk;
  const int D = P.D;
  volatile int* abort_flag = &aux.abort;
  if (tid == 0) {
    mbar_init(&aux.q_full, 1);
    for (int s = 0; s < kKs; ++s) {
      mbar_init(&aux.k_full[s], 1);
      mbar_init(&aux.k_empty[s], 1);
    }
    for (int s = 0; s < kVs; ++s) {
      mbar_init(&aux.v_full[s], 1);
      mbar_init(&aux.v_empty[s], 1);
    }
    mbar_init(&aux.s_full[0], 1);
    mbar_init(&aux.s_full[1], 1);
    mbar_init(&aux.dp_full, 1);
    mbar_init(&aux.dp_free, kSoftmaxWarps);
    mbar_init(&aux.ds_full[0], kSoftmaxWarps);
    mbar_init(&aux.ds_full[1], kSoftmaxWarps);
    mbar_init(&aux.dq_full, 1);
    mbar_init(&aux.drain, 1);
    aux.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&aux.tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();  // the row statistics and mask lists
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_trigger();  // with tensor memory in hand: the next kernel's blocks may want it too
  constexpr uint32_t tm = 0;  // all 512 columns: the allocation starts at the first
  constexpr uint32_t tDP = tm + 256, tDQ = tm + 384;
  const int* list = P.bits ? P.list + (long long)b * (P.ntiles + 1) : nullptr;
  const int j0 = split * P.per_qsplit, all_tiles = list ? list[P.ntiles] : P.ntiles;
  // (a reduction's result is uniform: the issuing warp's loop stays in uniform registers)
  const int n = __reduce_max_sync(~0u, kShares ? max(0, min(all_tiles - j0, P.per_qsplit)) : all_tiles);
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(P.err, kErrTimeout);
  };

  if (warp == kProducerWarp) {
    if (lane == 0 && n > 0) {
      const uint32_t bytes = (uint32_t)P.tokens * P.G * 128 * NB;
      mbar_arrive_expect_tx(&aux.q_full, 2 * bytes);
      for (int c = 0; c < NB; ++c) {
        tma_load_5d(smem + L::q + c * kBlock, &tm_q, &aux.q_full, c * 64, 0, qt * P.tokens, hk, b * P.qb);
        tma_load_5d(smem + L::g + c * kBlock, &tm_do, &aux.q_full, c * 64, 0, qt * P.tokens, hk, b);
      }
      int j = 0;
      for (; j < n; ++j) {
        if (*abort_flag) break;
        const int ks = j % kKs, vs = j % kVs, t = list ? list[j0 + j] : j0 + j;
        if ((j >= kKs && !mbar_wait(&aux.k_empty[ks], (j / kKs - 1) & 1, P.limit)) ||
            (j >= kVs && !mbar_wait(&aux.v_empty[vs], (j / kVs - 1) & 1, P.limit))) {
          fail();
          break;
        }
        mbar_arrive_expect_tx(&aux.k_full[ks], L::tile);
        for (int c = 0; c < NB; ++c)
          tma_load_5d(smem + L::k + ks * L::tile + c * kBlock, &tm_k, &aux.k_full[ks], c * 64, 0, t * kRows, hk,
                      b * P.kb);
        mbar_arrive_expect_tx(&aux.v_full[vs], L::tile);
        for (int c = 0; c < NB; ++c)
          tma_load_5d(smem + L::v + vs * L::tile + c * kBlock, &tm_v, &aux.v_full[vs], c * 64, 0, t * kRows, hk,
                      b * P.vb);
      }
      // every load has landed before shared memory goes
      mbar_wait(&aux.q_full, 0, kDrainPolls);
      for (int i = max(0, j - kKs); i < j; ++i) mbar_wait(&aux.k_full[i % kKs], (i / kKs) & 1, kDrainPolls);
      for (int i = max(0, j - kVs); i < j; ++i) mbar_wait(&aux.v_full[i % kVs], (i / kVs) & 1, kDrainPolls);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t idS = idesc_bf16(kRows, kRows, 0, 0), idQ = idesc_bf16(kRows, D, 0, 1);
    const uint64_t dq = sdesc_sw128(smem_u32(smem + L::q), 16), dg = sdesc_sw128(smem_u32(smem + L::g), 16);
    const uint64_t dk = sdesc_sw128(smem_u32(smem + L::k), 16), dv = sdesc_sw128(smem_u32(smem + L::v), 16);
    const uint64_t dkn = sdesc_sw128(smem_u32(smem + L::k), kBlock);
    auto all = [&](uint64_t* bar, uint32_t ph) { return __all_sync(~0u, mbar_wait(bar, ph, P.limit)); };
    // rows of A times rows of B over the features, both K-major
    auto product = [&](uint32_t d, uint64_t a, uint64_t bb) {
#pragma unroll
      for (int ks = 0; ks < 4 * NB; ++ks) {
        const uint32_t at = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
        if (ks < D / 16) mma_bf16_elect(d, a + at, bb + at, idS, ks > 0);
      }
    };
    auto issue_s = [&](int j) {
      const int s = j % kKs;
      if (!all(&aux.k_full[s], (j / kKs) & 1)) return false;
      tc_fence_after_sync();
      product(tm + (j & 1) * 128, dq, dk + (s * L::tile >> 4));
      mma_commit_elect(&aux.s_full[j & 1]);
      return true;
    };
    auto issue_dp = [&](int j) {
      const int s = j % kVs;
      if (!all(&aux.v_full[s], (j / kVs) & 1)) return false;
      if (j > 0 && !all(&aux.dp_free, (j - 1) & 1)) return false;
      tc_fence_after_sync();
      product(tDP, dg, dv + (s * L::tile >> 4));
      mma_commit_elect(&aux.dp_full);
      mma_commit_elect(&aux.v_empty[s]);
      return true;
    };
    bool ok = true;
    if (n > 0) ok = all(&aux.q_full, 0) && issue_s(0) && issue_dp(0);
    for (int j = 0; ok && j < n; ++j) {
      if (j + 1 < n) ok = issue_s(j + 1) && issue_dp(j + 1);
      ok = ok && all(&aux.ds_full[j & 1], (j >> 1) & 1);
      if (!ok) break;
      tc_fence_after_sync();
      // dQ += dS K: dS in TMEM (8 columns per 16 keys, 32 keys over their own
      // scores' columns), K MN-major
      const int s = j % kKs;
#pragma unroll
      for (int ks = 0; ks < kRows / 16; ++ks)
        mma_bf16_ts_elect(tDQ, tm + (j & 1) * 128 + (ks >> 1) * 32 + (ks & 1) * 8,
                          dkn + ((s * L::tile + ks * 2048) >> 4), idQ, j > 0 || ks > 0);
      if (kMode == kOne) {
#pragma unroll
        for (int ks = 0; ks < kRows / 16; ++ks)
          mma_bf16_ts_elect(tDQ, tm + (j & 1) * 128 + (ks >> 1) * 32 + (ks & 1) * 8 + kCols / 2,
                            dkn + ((s * L::tile + ks * 2048) >> 4), idQ, true);
      }
      mma_commit_elect(&aux.k_empty[s]);
    }
    if (!ok && lane == 0) fail();
    mma_commit_elect(&aux.dq_full);
    mma_commit_elect(&aux.drain);
    mbar_wait(&aux.drain, 0, kDrainPolls);
    __syncwarp();
  } else {
    const int r = (warp & 3) * 32 + lane, cg = warp >> 2;  // row; columns [32 cg, 32 cg + 32)
    const uint32_t trow = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const float* st = P.stat + ((long long)bh * P.qtiles + qt) * (2 * kRows) + r;
    const uint64_t c2 = f2_pack(P.scale_log2, P.scale_log2);
    const uint64_t nl = f2_pack(st[0], st[0]), nd = f2_pack(st[kRows], st[kRows]);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint4 keys = seen_keys(P, b, list ? list[j0 + j] : j0 + j);
      if (!__all_sync(~0u, *abort_flag == 0 && mbar_wait(&aux.s_full[j & 1], (j >> 1) & 1, P.limit))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t ts = trow + (j & 1) * 128 + kCols * cg;
      const uint32_t seen = word_of(keys, cg);
      float x[kCols];
      uint64_t p[kCols / 2];
      tmem_ld32(ts, x);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) p[i] = exp2_pair(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), c2, nl), i);
      if (!__all_sync(~0u, mbar_wait(&aux.dp_full, j & 1, P.limit))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      tmem_ld32(trow + tDP + kCols * cg, x);
      tmem_wait_ld();
      tc_fence_before_sync();
      mbar_arrive_warp(&aux.dp_free, lane);
      uint32_t pk[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) {
        float a, e;
        f2_unpack(f2_mul(p[i], f2_add(f2_pack(x[2 * i], x[2 * i + 1]), nd)), a, e);
        pk[i] = pack_bf16x2(a, e);
      }
      if (seen != ~0u) {  // dS of masked keys is 0 whatever their scores and values are
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i)
          pk[i] &= (seen >> (2 * i) & 1 ? 0xFFFFu : 0u) | (seen >> (2 * i + 1) & 1 ? 0xFFFF0000u : 0u);
      }
      tmem_st16u(ts, pk);
      if (kMode == kOne) {  // what the rounding left, beside it
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          float a, e;
          f2_unpack(f2_mul(p[i], f2_add(f2_pack(x[2 * i], x[2 * i + 1]), nd)), a, e);
          pk[i] = rest_of(a, e, pk[i]);
          pk[i] &= (seen >> (2 * i) & 1 ? 0xFFFFu : 0u) | (seen >> (2 * i + 1) & 1 ? 0xFFFF0000u : 0u);
        }
        tmem_st16u(ts + kCols / 2, pk);
      }
      if (P.bits && (keys.x & keys.y & keys.z & keys.w) != ~0u) {
        // clear the masked rows of K (its product with Q is done): 0 * NaN would reach dQ
        const int key = tid >> 2, part = tid & 3;  // four threads a row
        if (!(word_of(keys, key >> 5) >> (key & 31) & 1)) {
          uint8_t* row = smem + L::k + (j % kKs) * L::tile + key * 128 + part * 32;
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            *reinterpret_cast<uint4*>(row + c * kBlock) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(row + c * kBlock + 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive_warp(&aux.ds_full[j & 1], lane);
    }
    if (ok && !__all_sync(~0u, mbar_wait(&aux.dq_full, 0, P.limit))) ok = false;
    if (!ok && lane == 0) fail();
    ok = named_barrier_and(1, kSoftmaxThreads, ok && *abort_flag == 0);
    if (ok) {
      tc_fence_after_sync();
      // every product has completed: Q's (and dO's) buffer takes the rows, 2 KB a warp
      const int Hq = P.Hk * P.G, tok0 = qt * P.tokens, c0 = kCols * cg, r0 = (warp & 3) * 32;
      __nv_bfloat16* to = P.dq + (((long long)b * P.Tq + tok0) * Hq + hk * P.G) * D + c0;
      float* part = kShares ? P.qpart + (split * P.qpart_rows + ((long long)bh * P.qtiles + qt) * kRows) * D + c0 : nullptr;
      if (c0 < D)
        put_columns(
            trow + tDQ + c0, min(kCols, D - c0), n > 0, P.scale, smem + L::q + warp * 2048, lane,
            !kShares,
            [&](int i) -> void* {
              const int q = r0 + i, dt = q * P.gmul >> 16, dh = q - dt * P.G;  // row = token * G + head
              return dt < P.tokens && tok0 + dt < P.Tq ? to + ((long long)dt * Hq + dh) * D : nullptr;
            },
            [&](int i) { return part + (long long)(r0 + i) * D; });
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(aux.tmem, 512);
  }
}

// -------------------------------------------------------------------- dK, dV
// TMEM: S^T [0, 128) (P^T over it), dP^T [128, 256) (dS^T over it), dV
// [256, 256 + D), dK [384, 384 + D).  P^T is handed on before dP^T is looked at:
// dV += P^T dO and the next S^T run under the second half of the softmax, and
// dK += dS^T Q and the next dP^T under the first half of the next.
// Q and dO tiles take turns through a ring of five places, Q_i the item 2 i and dO_i
// the item 2 i + 1: Q_i+2 is on its way one step early.
constexpr int kRing = 5;
struct DkvAux {
  uint64_t kv_full, full[kRing], empty[kRing];
  uint64_t s_full, p_full, dp_full, ds_full, out_full, drain;
  uint32_t tmem;
  int abort;
  __align__(16) float nl[2][kRows], nd[2][kRows];  // -lse log2 e and -delta of two query tiles
};
template <int NB>
struct DkvLayout {
  static constexpr uint32_t tile = NB * kBlock;
  static constexpr uint32_t k = 0, v = tile, ring = 2 * tile;
  static constexpr uint32_t aux = ring + kRing * tile;
  static constexpr uint32_t total = aux + (uint32_t)sizeof(DkvAux);
};

template <int NB, Mode kMode>
__device__ __forceinline__ void dkv_tile(uint8_t* smem, unsigned block, const CUtensorMap& tm_q,
                                         const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                                         const CUtensorMap& tm_v, const BwdParams& P) {
  using L = DkvLayout<NB>;
  DkvAux& aux = *reinterpret_cast<DkvAux*>(smem + L::aux);
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  // unit: ((b * Hk + hk) * ntiles + tile) * nsplit + split
  const int split = block % P.nsplit, u = block / P.nsplit;
  const int kt = u % P.ntiles, bh = u / P.ntiles;
  const int b = bh / P.Hk, hk = bh - b * P.Hk;
  const int i0 = split * P.per_split, i1 = min(P.qtiles, i0 + P.per_split);
  const int D = P.D;
  volatile int* abort_flag = &aux.abort;
  if (tid == 0) {
    mbar_init(&aux.kv_full, 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&aux.full[s], 1);
      mbar_init(&aux.empty[s], 1);
    }
    mbar_init(&aux.s_full, 1);
    mbar_init(&aux.p_full, kSoftmaxWarps);
    mbar_init(&aux.dp_full, 1);
    mbar_init(&aux.ds_full, kSoftmaxWarps);
    mbar_init(&aux.out_full, 1);
    mbar_init(&aux.drain, 1);
    aux.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&aux.tmem, 512);
    tmem_relinquish();
  }
  // rows of Q and dO past the packed ones are never loaded, and a product runs
  // over them: they have to be numbers
  for (int i = P.tokens * P.G * 8 + tid; i < kRows * 8; i += kThreads)
    for (int c = 0; c < kRing * NB; ++c)
      *reinterpret_cast<uint4*>(smem + L::ring + c * kBlock + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  pdl_wait();  // the row statistics and mask bits
  const uint4 keys = seen_keys(P, b, kt);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_trigger();  // as in dq_tile
  constexpr uint32_t tm = 0;
  constexpr uint32_t tDP = tm + 128, tDV = tm + 256, tDK = tm + 384;
  const bool any = (keys.x | keys.y | keys.z | keys.w) != 0;
  const int n = __reduce_max_sync(~0u, any ? i1 - i0 : 0);  // uniform, as for dQ
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(P.err, kErrTimeout);
  };

  if (warp == kProducerWarp) {
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(&aux.kv_full, 2 * L::tile);
      for (int c = 0; c < NB; ++c) {
        tma_load_5d(smem + L::k + c * kBlock, &tm_k, &aux.kv_full, c * 64, 0, kt * kRows, hk, b * P.kb);
        tma_load_5d(smem + L::v + c * kBlock, &tm_v, &aux.kv_full, c * 64, 0, kt * kRows, hk, b * P.vb);
      }
      const uint32_t bytes = (uint32_t)P.tokens * P.G * 128 * NB;
      int x = 0;
      for (; x < 2 * n; ++x) {
        if (*abort_flag) break;
        const int s = x % kRing, qt = i0 + x / 2;
        if (x >= kRing && !mbar_wait(&aux.empty[s], (x / kRing - 1) & 1, P.limit)) {
          fail();
          break;
        }
        mbar_arrive_expect_tx(&aux.full[s], bytes);
        for (int c = 0; c < NB; ++c)
          tma_load_5d(smem + L::ring + s * L::tile + c * kBlock, x & 1 ? &tm_do : &tm_q, &aux.full[s], c * 64, 0,
                      qt * P.tokens, hk, x & 1 ? b : b * P.qb);
      }
      mbar_wait(&aux.kv_full, 0, kDrainPolls);
      for (int y = max(0, x - kRing); y < x; ++y) mbar_wait(&aux.full[y % kRing], (y / kRing) & 1, kDrainPolls);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (n > 0) {
      const uint32_t idS = idesc_bf16(kRows, kRows, 0, 0), idO = idesc_bf16(kRows, D, 0, 1);
      const uint64_t dk = sdesc_sw128(smem_u32(smem + L::k), 16), dv = sdesc_sw128(smem_u32(smem + L::v), 16);
      // ring item x as a right operand: K-major, and MN-major
      auto rowwise = [&](int x) { return sdesc_sw128(smem_u32(smem + L::ring + x % kRing * L::tile), 16); };
      auto colwise = [&](int x) { return sdesc_sw128(smem_u32(smem + L::ring + x % kRing * L::tile), kBlock); };
      auto all = [&](uint64_t* bar, uint32_t ph) { return __all_sync(~0u, mbar_wait(bar, ph, P.limit)); };
      auto product = [&](uint32_t d, uint64_t a, uint64_t bb) {  // over the features, both K-major
#pragma unroll
        for (int ks = 0; ks < 4 * NB; ++ks) {
          const uint32_t at = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
          if (ks < D / 16) mma_bf16_elect(d, a + at, bb + at, idS, ks > 0);
        }
      };
      auto add = [&](uint32_t d, uint32_t a, uint64_t bb, bool more) {  // over the queries, A in TMEM
#pragma unroll
        for (int ks = 0; ks < kRows / 16; ++ks)
          mma_bf16_ts_elect(d, a + (ks >> 1) * 32 + (ks & 1) * 8, bb + ks * (2048 >> 4), idO, more || ks > 0);
      };
      auto landed = [&](int x) { return all(&aux.full[x % kRing], (x / kRing) & 1); };
      bool ok = all(&aux.kv_full, 0) && landed(0);
      if (ok) {
        tc_fence_after_sync();
        product(tm, dk, rowwise(0));
        mma_commit_elect(&aux.s_full);
        ok = landed(1);
      }
      if (ok) {
        tc_fence_after_sync();
        product(tDP, dv, rowwise(1));
        mma_commit_elect(&aux.dp_full);
      }
      for (int i = 0; ok && i < n; ++i) {
        const int q = 2 * i, g = 2 * i + 1;
        ok = all(&aux.p_full, i & 1);
        if (!ok) break;
        tc_fence_after_sync();
        add(tDV, tm, colwise(g), i > 0);
        if (kMode == kOne) add(tDV, tm + kCols / 2, colwise(g), true);
        mma_commit_elect(&aux.empty[g % kRing]);
        if (i + 1 < n) {
          ok = landed(q + 2);
          if (!ok) break;
          tc_fence_after_sync();
          product(tm, dk, rowwise(q + 2));
          mma_commit_elect(&aux.s_full);
        }
        ok = all(&aux.ds_full, i & 1);
        if (!ok) break;
        tc_fence_after_sync();
        add(tDK, tDP, colwise(q), i > 0);
        if (kMode == kOne) add(tDK, tDP + kCols / 2, colwise(q), true);
        mma_commit_elect(&aux.empty[q % kRing]);
        if (i + 1 < n) {
          ok = landed(g + 2);
          if (!ok) break;
          tc_fence_after_sync();
          product(tDP, dv, rowwise(g + 2));
          mma_commit_elect(&aux.dp_full);
        }
      }
      if (!ok && lane == 0) fail();
      mma_commit_elect(&aux.out_full);
      mma_commit_elect(&aux.drain);
      mbar_wait(&aux.drain, 0, kDrainPolls);
    }
    __syncwarp();
  } else {
    const int cg = warp >> 2;  // a key per lane; queries [32 cg, 32 cg + 32)
    const uint32_t trow = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t seen = word_of(keys, warp & 3);
    const uint32_t keep = seen >> lane & 1 ? ~0u : 0u;  // both halves of a packed pair
    const uint64_t c2 = f2_pack(P.scale_log2, P.scale_log2);
    // Warp 0 brings the next tile's -lse log2 e, warp 1 its -delta, each written while
    // no one reads that place: nl under this tile's first half (every thread is past
    // the last tile's), nd under its second.
    const float* stat = P.stat + ((long long)bh * P.qtiles + i0) * (2 * kRows) + lane * 4;
    if (n > 0) {
      if (warp < 2)
        *reinterpret_cast<float4*>((warp ? aux.nd : aux.nl)[0] + lane * 4) =
            *reinterpret_cast<const float4*>(stat + warp * kRows);
      named_barrier(1, kSoftmaxThreads);
    }
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      float4 coming = make_float4(0.f, 0.f, 0.f, 0.f);
      if (warp < 2 && i + 1 < n)
        coming = *reinterpret_cast<const float4*>(stat + (long long)(i + 1) * (2 * kRows) + warp * kRows);
      if (!__all_sync(~0u, *abort_flag == 0 && mbar_wait(&aux.s_full, i & 1, P.limit))) {
        ok = false;
        break;
      }
      if (i > 0) mbar_wait(&aux.p_full, (i - 1) & 1, 2);  // complete: acquires what warp 0 wrote
      tc_fence_after_sync();
      float x[kCols];
      uint64_t p[kCols / 2];
      uint32_t pk[kCols / 2];
      tmem_ld32(trow + kCols * cg, x);
      tmem_wait_ld();
      const uint4* nl = reinterpret_cast<const uint4*>(aux.nl[i & 1] + kCols * cg);
#pragma unroll
      for (int c = 0; c < kCols / 4; ++c) {
        const uint4 y = nl[c];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t neg = f2_pack(__uint_as_float(h ? y.z : y.x), __uint_as_float(h ? y.w : y.y));
          float a, e;
          p[2 * c + h] = exp2_pair(f2_fma(f2_pack(x[4 * c + 2 * h], x[4 * c + 2 * h + 1]), c2, neg), 2 * c + h);
          f2_unpack(p[2 * c + h], a, e);
          pk[2 * c + h] = pack_bf16x2(a, e);
        }
      }
      if (seen != ~0u) {  // a masked key's lane: 0 whatever its scores are
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) pk[c] &= keep;
      }
      tmem_st16u(trow + kCols * cg, pk);
      if (kMode == kOne) {
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
          float a, e;
          f2_unpack(p[c], a, e);
          pk[c] = rest_of(a, e, pk[c]) & keep;
        }
        tmem_st16u(trow + kCols * cg + kCols / 2, pk);
      }
      if (warp == 0) *reinterpret_cast<float4*>(aux.nl[(i + 1) & 1] + lane * 4) = coming;
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive_warp(&aux.p_full, lane);
      if (!__all_sync(~0u, mbar_wait(&aux.dp_full, i & 1, P.limit))) {
        ok = false;
        break;
      }
      if (i > 0) mbar_wait(&aux.ds_full, (i - 1) & 1, 2);  // ... and warp 1
      tc_fence_after_sync();
      tmem_ld32(trow + tDP + kCols * cg, x);
      tmem_wait_ld();
      const uint4* nd = reinterpret_cast<const uint4*>(aux.nd[i & 1] + kCols * cg);
#pragma unroll
      for (int c = 0; c < kCols / 4; ++c) {
        const uint4 y = nd[c];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t neg = f2_pack(__uint_as_float(h ? y.z : y.x), __uint_as_float(h ? y.w : y.y));
          float a, e;
          f2_unpack(f2_mul(p[2 * c + h], f2_add(f2_pack(x[4 * c + 2 * h], x[4 * c + 2 * h + 1]), neg)), a, e);
          pk[2 * c + h] = pack_bf16x2(a, e);
        }
      }
      if (seen != ~0u) {
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) pk[c] &= keep;
      }
      tmem_st16u(trow + tDP + kCols * cg, pk);
      if (kMode == kOne) {
#pragma unroll
        for (int c = 0; c < kCols / 4; ++c) {
          const uint4 y = nd[c];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t neg = f2_pack(__uint_as_float(h ? y.z : y.x), __uint_as_float(h ? y.w : y.y));
            float a, e;
            f2_unpack(f2_mul(p[2 * c + h], f2_add(f2_pack(x[4 * c + 2 * h], x[4 * c + 2 * h + 1]), neg)), a, e);
            pk[2 * c + h] = rest_of(a, e, pk[2 * c + h]) & keep;
          }
        }
        tmem_st16u(trow + tDP + kCols * cg + kCols / 2, pk);
      }
      if (warp == 1) *reinterpret_cast<float4*>(aux.nd[(i + 1) & 1] + lane * 4) = coming;
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive_warp(&aux.ds_full, lane);
    }
    if (ok && n > 0 && !__all_sync(~0u, mbar_wait(&aux.out_full, 0, P.limit))) ok = false;
    if (!ok && lane == 0) fail();
    ok = named_barrier_and(1, kSoftmaxThreads, ok && *abort_flag == 0);
    if (ok) {
      tc_fence_after_sync();
      // dK, then dV: to the share's part, or as bf16 where they belong; every product
      // has completed, so K's (and V's) buffer takes the rows, 2 KB a warp
      const int c0 = kCols * cg, r0 = (warp & 3) * 32;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (c0 >= D) break;
        __nv_bfloat16* to = (which ? P.dv : P.dk) + (((long long)b * P.S + kt * kRows) * P.Hk + hk) * D + c0;
        float* part = P.part + ((2 * split + which) * P.part_rows + ((long long)bh * P.ntiles + kt) * kRows) * D + c0;
        put_columns(
            trow + (which ? tDV : tDK) + c0, min(kCols, D - c0), n > 0, which ? 1.f : P.scale,
            smem + L::k + warp * 2048, lane, P.nsplit == 1,
            [&](int i) -> void* { return kt * kRows + r0 + i < P.S ? to + (long long)(r0 + i) * P.Hk * D : nullptr; },
            [&](int i) { return part + (long long)(r0 + i) * D; });
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(aux.tmem, 512);
  }
}

// One grid for both: the dK, dV tiles first, which are longer, then the dQ tiles,
// so that neither's last wave leaves SMs idle.
template <int NB, Mode kMode>
__global__ void __launch_bounds__(kThreads, 1)
gdn_cross_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ BwdParams P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (threadIdx.x == 0) {
    prefetch_map(&tm_q);
    prefetch_map(&tm_do);
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
  }
  if (blockIdx.x < P.dkv_blocks)
    dkv_tile<NB, kMode>(smem, blockIdx.x, tm_q, tm_do, tm_k, tm_v, P);
  else
    dq_tile<NB, kMode>(smem, blockIdx.x - P.dkv_blocks, tm_q, tm_do, tm_k, tm_v, P);
}

// dK, dV and dQ = the sums of their shares, in their order.  A thread per four
// features: kv of dK in the first kv_blocks, as many of dV, then q of dQ.  Every
// number of rows or features is below 2^32, as their fp32 shares fit the memory.
__global__ void __launch_bounds__(256)
gdn_cross_grad_join_kernel(const __grid_constant__ BwdParams P, unsigned kv, unsigned kv_blocks, unsigned q) {
  pdl_wait();
  const int which = blockIdx.x >= 2 * kv_blocks ? 2 : blockIdx.x >= kv_blocks;
  const unsigned i = (blockIdx.x - which * kv_blocks) * 256 + threadIdx.x;
  if (i >= (which < 2 ? kv : q)) return;
  const unsigned d4 = P.D / 4, row = i / d4;
  const int f = (int)(i - row * d4) * 4;
  const float* from;
  long long step;
  int n;
  if (which < 2) {  // row ((b * S) + s) * Hk + hk
    const unsigned bs = row / P.Hk, hk = row - bs * P.Hk, b = bs / P.S, t = bs - b * P.S;
    from = P.part + (which * P.part_rows + (long long)(b * P.Hk + hk) * P.ntiles * kRows + t) * P.D + f;
    step = 2 * P.part_rows * P.D;
    n = P.nsplit;
  } else {  // row ((b * Tq) + t) * Hq + head
    const unsigned Hq = P.Hk * P.G, bt = row / Hq, head = row - bt * Hq, b = bt / P.Tq, t = bt - b * P.Tq;
    const unsigned hk = head / P.G, qt = t / P.tokens, r = (t - qt * P.tokens) * P.G + head - hk * P.G;
    from = P.qpart + (((long long)(b * P.Hk + hk) * P.qtiles + qt) * kRows + r) * P.D + f;
    step = P.qpart_rows * P.D;
    n = P.qsplit;
  }
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int x = 0; x < n; ++x) {
    const float4 v = *reinterpret_cast<const float4*>(from + x * step);
    o[0] += v.x;
    o[1] += v.y;
    o[2] += v.z;
    o[3] += v.w;
  }
  __nv_bfloat16* to = which == 2 ? P.dq : which ? P.dv : P.dk;
  *reinterpret_cast<uint2*>(to + (long long)row * P.D + f) =
      make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
}

void bwd_shape(const CrossCall& c, BwdParams* P) {
  P->Tq = c.Tq;
  P->S = c.S;
  P->Hk = c.Hk;
  P->G = c.Hq / c.Hk;
  P->D = c.D;
  P->tokens = kRows / P->G;
  P->gmul = 65536 / P->G + 1;
  P->qtiles = (c.Tq + P->tokens - 1) / P->tokens;
  P->ntiles = (c.S + kRows - 1) / kRows;
  P->part_rows = (long long)c.B * c.Hk * P->ntiles * kRows;
  // Shares of the query tiles: the fewest tile steps over all waves of CTAs,
  // a CTA's start and end counting as three steps and a share's fp32 part as two.
  const long long units = (long long)c.B * c.Hk * P->ntiles;
  const int sms = num_sms();
  double best = 1e300;
  P->nsplit = 1;
  for (int s = 1; s <= 16 && s <= P->qtiles; ++s) {
    const long long waves = (units * s + sms - 1) / sms;
    const double cost = (double)waves * ((P->qtiles + s - 1) / s + 3 + (s > 1 ? 2 : 0));
    if (cost < best) {
      best = cost;
      P->nsplit = s;
    }
  }
  P->per_split = (P->qtiles + P->nsplit - 1) / P->nsplit;
  P->nsplit = (P->qtiles + P->per_split - 1) / P->per_split;
  P->dkv_blocks = (unsigned)(units * P->nsplit);
  // Shares of the key tiles: few query tiles over many keys would leave the other SMs
  // idle at the end (a token of 16 heads over 8192 keys 69.4 us whole, 14.2 shared out,
  // 2 x 64 queries of 8 heads 120 and 94).  A dK, dV step takes 1.4 times a dQ step;
  // the grid takes its work over all SMs or its longest CTA, whichever is longer.
  const long long qunits = (long long)c.B * c.Hk * P->qtiles;
  P->qpart_rows = qunits * kRows;
  const double dkv = 1.4 * (P->per_split + 3);
  best = 1e300;
  P->qsplit = 1;
  for (int s = 1; s <= 16 && (s == 1 || s <= P->ntiles / 4); ++s) {
    const double dq = (P->ntiles + s - 1) / s + 3 + (s > 1 ? 2 : 0);
    const double cost = std::max({(P->dkv_blocks * dkv + qunits * s * dq) / sms, dq, dkv}) +
                        (s > 1 && P->nsplit == 1 ? 3 : 0);  // a join's launch
    if (cost < best) {
      best = cost;
      P->qsplit = s;
    }
  }
  P->per_qsplit = (P->ntiles + P->qsplit - 1) / P->qsplit;
  P->qsplit = (P->ntiles + P->per_qsplit - 1) / P->per_qsplit;
}

// Scratch: the row stats, under a mask its bits and lists, then the shares' parts.
struct BwdScratch {
  size_t bits, list, part, qpart, total;
};
BwdScratch bwd_scratch(const CrossCall& c, const BwdParams& P) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  BwdScratch s;
  s.bits = up((size_t)c.B * c.Hk * P.qtiles * 2 * kRows * sizeof(float));
  s.list = s.bits + (c.mask ? up((size_t)c.B * P.ntiles * 4 * sizeof(uint32_t)) : 0);
  s.part = s.list + (c.mask ? up((size_t)c.B * (P.ntiles + 1) * sizeof(int)) : 0);
  s.qpart = s.part + (P.nsplit > 1 ? (size_t)2 * P.nsplit * P.part_rows * c.D * sizeof(float) : 0);
  s.total = s.qpart + (P.qsplit > 1 ? (size_t)P.qsplit * P.qpart_rows * c.D * sizeof(float) : 0);
  return s;
}

template <int NB>
cudaError_t launch_nb(const CrossCall& c, const BwdParams& P, const CUtensorMap& mq, const CUtensorMap& mg,
                      const CUtensorMap& mk, const CUtensorMap& mv) {
  // more than half an SM's shared memory: one CTA (all of TMEM) per SM
  constexpr int bytes = std::max({(int)DqLayout<NB>::total, (int)DkvLayout<NB>::total, 116 * 1024});
  const auto kernel = P.qsplit > 1    ? gdn_cross_bwd_kernel<NB, kShared>
                      : P.ntiles == 1 ? gdn_cross_bwd_kernel<NB, kOne>
                                      : gdn_cross_bwd_kernel<NB, kWhole>;
  cudaError_t e = allow_smem(kernel, bytes);
  if (e != cudaSuccess) return e;
  ProfileScope ps(c.stream, kKernCrossBwd);
  e = launch_after(kernel, P.dkv_blocks + (unsigned)(c.B * c.Hk * P.qtiles * P.qsplit), kThreads, bytes, c.stream,
                   mq, mg, mk, mv, P);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

size_t cross_backward_workspace_bytes(const CrossCall& c) {
  BwdParams P = {};
  bwd_shape(c, &P);
  return bwd_scratch(c, P).total;
}

cudaError_t launch_cross_backward(const CrossCall& c, void* ws) {
  BwdParams P = {};
  bwd_shape(c, &P);
  const BwdScratch at = bwd_scratch(c, P);
  uint8_t* base = static_cast<uint8_t*>(ws);
  P.bits = c.mask ? reinterpret_cast<const uint32_t*>(base + at.bits) : nullptr;
  P.list = c.mask ? reinterpret_cast<const int*>(base + at.list) : nullptr;
  P.dq = static_cast<__nv_bfloat16*>(c.dq);
  P.dk = static_cast<__nv_bfloat16*>(c.dk);
  P.dv = static_cast<__nv_bfloat16*>(c.dv);
  P.scale = c.scale;
  P.scale_log2 = c.scale * 1.4426950408889634f;
  P.stat = static_cast<const float*>(ws);
  P.part = reinterpret_cast<float*>(base + at.part);
  P.qpart = reinterpret_cast<float*>(base + at.qpart);
  P.limit = c.limit;
  P.err = c.err;
  P.qb = c.q.batch_stride != 0;
  P.kb = c.k.batch_stride != 0;
  P.vb = c.v.batch_stride != 0;
  CUtensorMap mq, mg, mk, mv;
  const long long ots = (long long)c.Hq * c.D;
  if (!make_heads_map(&mq, c.q.data, P.qb ? c.B : 1, c.Tq, c.Hk, P.G, c.D, c.q.batch_stride, c.q.token_stride,
                      P.tokens) ||
      !make_heads_map(&mg, c.d_out, c.B, c.Tq, c.Hk, P.G, c.D, c.Tq * ots, ots, P.tokens) ||
      !make_heads_map(&mk, c.k.data, P.kb ? c.B : 1, c.S, c.Hk, 1, c.D, c.k.batch_stride, c.k.token_stride,
                      kRows) ||
      !make_heads_map(&mv, c.v.data, P.vb ? c.B : 1, c.S, c.Hk, 1, c.D, c.v.batch_stride, c.v.token_stride,
                      kRows))
    return cudaErrorInvalidValue;
  const long long rows = (long long)c.B * c.Hk * P.qtiles * kRows;
  cudaError_t e;
  {
    ProfileScope ps(c.stream, kKernCrossStat);
    const unsigned blocks = (unsigned)((rows + kStatBlockRows - 1) / kStatBlockRows);
    const FewKeys few = {static_cast<const __nv_bfloat16*>(c.q.data), static_cast<const __nv_bfloat16*>(c.k.data),
                         static_cast<const __nv_bfloat16*>(c.v.data), c.q.batch_stride, c.q.token_stride,
                         c.k.batch_stride, c.k.token_stride, c.v.batch_stride, c.v.token_stride};
    e = launch_after(c.S <= kFewKeys ? gdn_cross_stat_kernel<true> : gdn_cross_stat_kernel<false>,
                     blocks + (c.mask ? c.B : 0), kStatThreads, 0, c.stream,
                     static_cast<const __nv_bfloat16*>(c.out), static_cast<const __nv_bfloat16*>(c.d_out),
                     (const float*)c.lse, static_cast<float*>(ws), rows, blocks, c.mask, c.mask_bs, P, few);
  }
  if (e != cudaSuccess) return e;
  count_launches(1);
  e = c.D > 64 ? launch_nb<2>(c, P, mq, mg, mk, mv)
               : launch_nb<1>(c, P, mq, mg, mk, mv);
  if (e != cudaSuccess || (P.nsplit == 1 && P.qsplit == 1)) return e;
  ProfileScope ps(c.stream, kKernCrossGradJoin);
  const unsigned kv = P.nsplit > 1 ? (unsigned)((long long)c.B * c.S * c.Hk * (c.D / 4)) : 0;
  const unsigned q = P.qsplit > 1 ? (unsigned)((long long)c.B * c.Tq * c.Hq * (c.D / 4)) : 0;
  const unsigned kv_blocks = (unsigned)(((long long)kv + 255) / 256);
  e = launch_after(gdn_cross_grad_join_kernel, 2 * kv_blocks + (unsigned)(((long long)q + 255) / 256), 256, 0,
                   c.stream, P, kv, kv_blocks, q);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace gdn
