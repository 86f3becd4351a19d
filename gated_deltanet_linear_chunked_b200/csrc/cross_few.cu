// cross_few.cu -- the attention to the encoder's states for a few query rows: at
// most 16 of them, tokens times the query heads of a key head, as when one token is
// generated at a time.
//
// Nothing but the keys and values is large, so the kernel is a stream over them: a
// warp takes every W-th group of 16 keys of its (b, key head), W being all warps on
// it, and keeps three groups of K and V on their way into its own piece of shared
// memory (16-byte asynchronous copies, no barrier between warps).  The 16 rows are
// one mma.sync tile (m16n8k16: S = Q K^T over the features, then O += P V), with
// the running maximum and sum of each row in registers; a 128-row tcgen05 tile would
// spend its time on 112 rows that are none.  Masked keys are not copied: their rows
// arrive as zeros (so that 0 * NaN never arises), their scores become -inf, and
// groups without any seen key are skipped.  The warps of a CTA join in shared
// memory, up to eight CTAs of one (b, key head) in each other's as a cluster, more
// through gdn_cross_join_kernel.  Bound by its start (the mask's bytes, then the first
// keys) and end: 8 requests of one token, 16 query heads on 4 key heads of 128, over 4096
// keys, a seventh of them masked, 18.5 us from memory (3.1 TB/s), DRAM at 33% while it
// runs; repeated on the same tensors, out of L2, 14.0 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cross_attn.cuh"
#include "gdn_internal.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kKeys = 16;     // keys of a group
constexpr int kDepth = 3;     // groups on their way per warp

struct FewParams {
  CrossParams c;
  const __nv_bfloat16 *q, *k, *v;
  long long q_bs, q_ts, k_bs, k_ts, v_bs, v_ts;
  int cluster;  // the CTAs of a (b, key head) are one cluster
};

// Shared memory of a warp: kDepth x (K, V) groups of 16 rows of D features, 16-byte
// piece c of row r at piece c ^ (r & 7) (rows of D / 8 pieces; D = 16 has two).
template <int NK>
struct FewLayout {
  static constexpr int pieces = 2 * NK;                    // of a row
  static constexpr uint32_t group = kKeys * pieces * 16;   // K or V of a group, bytes
  static constexpr uint32_t warp = kDepth * 2 * group;
  // the joined rows: [kWarps][16][D] fp32 and the rows' maxima and sums
  static constexpr uint32_t join = kWarps * 16 * (16 * NK) * 4;
  static constexpr uint32_t total = (kWarps * warp > join ? kWarps * warp : join) + kWarps * 16 * 8;
};

template <int NK>  // D / 16
__global__ void __launch_bounds__(32 * kWarps, 2)
gdn_cross_few_kernel(const __grid_constant__ FewParams F) {
  extern __shared__ __align__(128) uint8_t smem[];
  using L = FewLayout<NK>;
  constexpr int D = 16 * NK, kPieces = L::pieces;
  const CrossParams& P = F.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % P.nsplit, bh = blockIdx.x / P.nsplit;
  const int b = bh / P.Hk, hk = bh - b * P.Hk;
  const int rows = P.tokens * P.G;  // of the 16
  const int Hq = P.Hk * P.G;
  pdl_wait();  // inputs may come from the kernel in front
  pdl_trigger();

  // piece c of row r of a group: swizzled within aligned runs of eight pieces, or of
  // the whole row where it has fewer; rows of 6, 10, 12, 14 pieces keep their tail
  auto piece = [&](int r, int c) -> uint32_t {
    constexpr int run = kPieces >= 8 ? 8 : kPieces >= 4 ? 4 : 2;
    const int base = c & ~(run - 1);
    const int cc = base + run <= kPieces ? base + ((c ^ r) & (run - 1)) : c;
    return (uint32_t)(r * kPieces + cc) * 16;
  };

  const int workers = P.nsplit * kWarps, me = split * kWarps + warp;
  const int groups = (P.S + kKeys - 1) / kKeys;
  const uint8_t* mrow = P.mask ? P.mask + b * P.mask_bs : nullptr;
  const __nv_bfloat16* kbase = F.k + b * F.k_bs + hk * D;
  const __nv_bfloat16* vbase = F.v + b * F.v_bs + hk * D;
  const uint32_t base = smem_u32(smem) + warp * L::warp;

  // which of the 16 keys of group i are seen: the lane's mask byte, and the vote
  auto look = [&](int i) -> bool {
    const long long key = (long long)i * kKeys + (lane & 15);
    return i < groups && key < P.S && (!mrow || mrow[key] != 0);
  };
  auto vote = [&](bool on) -> uint32_t { return __ballot_sync(~0u, on) & 0xFFFFu; };
  auto fetch = [&](int i, uint32_t seen, int slot) {
    if (seen) {
      const uint32_t dk = base + slot * 2 * L::group, dv = dk + L::group;
#pragma unroll
      for (int x = 0; x < kKeys * kPieces; x += 32) {
        const int y = x + lane, r = y / kPieces, c = y - r * kPieces;
        if (kKeys * kPieces % 32 == 0 || y < kKeys * kPieces) {
          const bool on = seen >> r & 1;
          const long long key = on ? (long long)i * kKeys + r : 0;
          copy16(dk + piece(r, c), kbase + key * F.k_ts + c * 8, on);
          copy16(dv + piece(r, c), vbase + key * F.v_ts + c * 8, on);
        }
      }
    }
    copy_commit();
  };

  // seen bits of the groups in flight, and of the one to be fetched next: all their
  // bytes are asked for before the first is waited for
  uint32_t seen[kDepth], coming;
  {
    bool on[kDepth];
#pragma unroll
    for (int s = 0; s < kDepth; ++s) on[s] = look(me + s * workers);
#pragma unroll
    for (int s = 0; s < kDepth; ++s) seen[s] = vote(on[s]);
    coming = seen[kDepth - 1];
  }
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) fetch(me + s * workers, seen[s], s);

  // Q as left operands, row r = token * G + head, straight from memory
  uint32_t qa[NK][4];
  {
    const int g = lane >> 2, t2 = (lane & 3) * 2;
    const __nv_bfloat16* row[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i, dt = r * P.gmul >> 16, dh = r - dt * P.G;
      row[i] = r < rows ? F.q + b * F.q_bs + dt * F.q_ts + (hk * P.G + dh) * D : nullptr;
    }
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat16* p = row[i & 1];
        qa[ks][i] = p ? *reinterpret_cast<const uint32_t*>(p + 16 * ks + t2 + 8 * (i >> 1)) : 0u;
      }
  }

  float m[2] = {kLowest, kLowest}, l[2] = {0.f, 0.f};
  float o[2 * NK][4];
#pragma unroll
  for (int i = 0; i < 2 * NK; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  int slot = 0;
  for (int i = me; i < groups; i += workers) {
    // the slot used two groups ago takes the group two ahead
    const int into = slot >= 1 ? slot - 1 : kDepth - 1;
    const uint32_t next = coming;
    __syncwarp();  // every lane is done with that slot
    fetch(i + (kDepth - 1) * workers, next, into);
    const bool later = look(i + kDepth * workers);
    copy_wait<kDepth - 1>();
    __syncwarp();
    coming = vote(later);
    const uint32_t now = seen[0];
#pragma unroll
    for (int s = 0; s + 1 < kDepth; ++s) seen[s] = seen[s + 1];
    seen[kDepth - 2] = next;
    if (now) {
      const uint32_t tk = base + slot * 2 * L::group, tv = tk + L::group;
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      const int mat = lane >> 3, mr = lane & 7;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        uint32_t kb[4];  // keys 0-7: features 0-7, 8-15; keys 8-15: the same
        ldmatrix_x4(tk + piece(mr + 8 * (mat >> 1), 2 * ks + (mat & 1)), kb);
        mma_16816(s0, qa[ks], kb[0], kb[1]);
        mma_16816(s1, qa[ks], kb[2], kb[3]);
      }
      // lane: rows lane / 4 and that + 8, keys 2 (lane % 4) + {0, 1} and those + 8
      const int t2 = (lane & 3) * 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool a = now >> (t2 + e) & 1, c = now >> (t2 + 8 + e) & 1;
        s0[e] = a ? s0[e] * P.scale_log2 : -INFINITY;
        s0[2 + e] = a ? s0[2 + e] * P.scale_log2 : -INFINITY;
        s1[e] = c ? s1[e] * P.scale_log2 : -INFINITY;
        s1[2 + e] = c ? s1[2 + e] * P.scale_log2 : -INFINITY;
      }
      uint32_t pa[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(fmaxf(s0[2 * h], s0[2 * h + 1]), fmaxf(s1[2 * h], s1[2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
        const float mn = fmaxf(m[h], mx);  // finite: p of a score of -inf is 0; NaN is ignored here, but not
                                           // in p and the row's sum
        const float alpha = exp2f(m[h] - mn);
        m[h] = mn;
        const float p0 = exp2f(s0[2 * h] - mn), p1 = exp2f(s0[2 * h + 1] - mn);
        const float p2 = exp2f(s1[2 * h] - mn), p3 = exp2f(s1[2 * h + 1] - mn);
        l[h] = l[h] * alpha + ((p0 + p1) + (p2 + p3));  // this lane's four keys
        pa[h] = pack_bf16x2(p0, p1);
        pa[2 + h] = pack_bf16x2(p2, p3);
#pragma unroll
        for (int f = 0; f < 2 * NK; ++f) {
          o[f][2 * h] *= alpha;
          o[f][2 * h + 1] *= alpha;
        }
      }
#pragma unroll
      for (int f = 0; f < NK; ++f) {
        uint32_t vb[4];  // features 0-7: keys 0-7, 8-15; features 8-15: the same
        ldmatrix_x4_trans(tv + piece(mr + 8 * (mat & 1), 2 * f + (mat >> 1)), vb);
        mma_16816(o[2 * f], pa, vb[0], vb[1]);
        mma_16816(o[2 * f + 1], pa, vb[2], vb[3]);
      }
    }
    slot = slot + 1 == kDepth ? 0 : slot + 1;
  }
  copy_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(~0u, l[h], 1);
    l[h] += __shfl_xor_sync(~0u, l[h], 2);
  }

  // join the CTA's warps: rows and their (m, l) over the groups' memory
  __syncthreads();
  float* ow = reinterpret_cast<float*>(smem) + warp * 16 * D;
  float2* ml = reinterpret_cast<float2*>(smem + L::total - kWarps * 16 * 8);
  {
    const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
    for (int f = 0; f < 2 * NK; ++f) {
      *reinterpret_cast<float2*>(ow + g * D + 8 * f + t2) = make_float2(o[f][0], o[f][1]);
      *reinterpret_cast<float2*>(ow + (g + 8) * D + 8 * f + t2) = make_float2(o[f][2], o[f][3]);
    }
    if ((lane & 3) == 0) {
      ml[warp * 16 + g] = make_float2(m[0], l[0]);
      ml[warp * 16 + g + 8] = make_float2(m[1], l[1]);
    }
  }
  __syncthreads();
  // this CTA's rows: normalised, and their lse
  constexpr int kMine = (16 * D / 4 + 32 * kWarps - 1) / (32 * kWarps);  // pieces of a thread
  float4 mine[kMine];
  float mine_lse[kMine];
#pragma unroll
  for (int p = 0; p < kMine; ++p) {
    const int x = threadIdx.x + p * 32 * kWarps, r = x / (D / 4), f = (x - r * (D / 4)) * 4;
    mine[p] = make_float4(0.f, 0.f, 0.f, 0.f);
    mine_lse[p] = -INFINITY;
    if (r >= rows) continue;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * 16 + r].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = ml[w * 16 + r];
      const float a = v.y != 0.f ? exp2f(v.x - top) : 0.f;  // (a NaN sum counts)
      const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * 16 + r) * D + f);
      sum += a * v.y;
      mine[p].x += a * y.x;
      mine[p].y += a * y.y;
      mine[p].z += a * y.z;
      mine[p].w += a * y.w;
    }
    const bool any = sum != 0.f;  // else no key is seen, or every score is -inf
    const float inv = any ? 1.f / sum : 0.f;
    mine[p] = make_float4(mine[p].x * inv, mine[p].y * inv, mine[p].z * inv, mine[p].w * inv);
    mine_lse[p] = any ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
  auto put = [&](int r, int f, const float4& v, float lse) {
    const int dt = r * P.gmul >> 16, head = hk * P.G + r - dt * P.G;
    if (f == 0 && P.lse) P.lse[((long long)b * Hq + head) * P.Tq + dt] = lse;
    *reinterpret_cast<uint2*>(P.out + (((long long)b * P.Tq + dt) * Hq + head) * D + f) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  };
  if (!F.cluster) {
#pragma unroll
    for (int p = 0; p < kMine; ++p) {
      const int x = threadIdx.x + p * 32 * kWarps, r = x / (D / 4), f = (x - r * (D / 4)) * 4;
      if (r >= rows) continue;
      if (P.nsplit == 1) {
        put(r, f, mine[p], mine_lse[p]);
      } else {
        const long long at = (long long)blockIdx.x * kFewRows + r;
        if (f == 0) P.part_lse[at] = mine_lse[p];
        *reinterpret_cast<float4*>(P.part_o + at * D + f) = mine[p];
      }
    }
    return;
  }
  // The CTAs of a cluster share the (b, key head): each leaves its rows in its own
  // shared memory, then takes every nsplit-th row and joins it from all of them.
  float* left = reinterpret_cast<float*>(smem);  // [16][D] | lse [16]
  __syncthreads();
#pragma unroll
  for (int p = 0; p < kMine; ++p) {
    const int x = threadIdx.x + p * 32 * kWarps, r = x / (D / 4), f = (x - r * (D / 4)) * 4;
    if (r >= rows) continue;
    *reinterpret_cast<float4*>(left + r * D + f) = mine[p];
    if (f == 0) left[16 * D + r] = mine_lse[p];
  }
  cluster_sync();
  const uint32_t at = smem_u32(left);
  for (int x = threadIdx.x; x < (rows - split + P.nsplit - 1) / P.nsplit * (D / 4); x += 32 * kWarps) {
    const int r = split + x / (D / 4) * P.nsplit, f = x % (D / 4) * 4;
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < P.nsplit; ++s) top = fmax_nan(top, cluster_load(cluster_addr(at + (16 * D + r) * 4, s)));
    const bool any = top != -INFINITY;  // NaN is passed on
    for (int s = 0; any && s < P.nsplit; ++s) {
      const float w = expf(cluster_load(cluster_addr(at + (16 * D + r) * 4, s)) - top);
      const float4 v = cluster_load4(cluster_addr(at + (r * D + f) * 4, s));
      sum += w;
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    }
    const float inv = any ? 1.f / sum : 0.f;
    put(r, f, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), any ? top + logf(sum) : -INFINITY);
  }
  cluster_sync();  // no CTA's shared memory goes while another reads it
}

template <int NK>
cudaError_t launch_nk(const FewParams& F, unsigned grid, cudaStream_t stream) {
  constexpr int bytes = FewLayout<NK>::total;
  const cudaError_t e = allow_smem(gdn_cross_few_kernel<NK>, bytes);
  if (e != cudaSuccess) return e;
  ProfileScope ps(stream, kKernCrossFew);
  return launch_after_in_clusters(gdn_cross_few_kernel<NK>, grid, 32 * kWarps, bytes, stream,
                                  F.cluster ? (unsigned)F.c.nsplit : 1u, F);
}

}  // namespace

// Two CTAs an SM, each warp at least two groups of keys; where that is nine or ten
// CTAs, eight, which are a cluster and join without a second kernel (one token over
// 4096 keys, heads of 112 and 128, eight / all, us: ten CTAs, 28 key heads, 15.5-16.8 /
// 15.6-15.9; nine, 30 and 32 key heads, 16.1 / 17.1 and 15.4-16.6 / 16.5-17.7).
int few_splits(int B, int Hk, int S) {
  const long long units = (long long)B * Hk;
  const long long most = ((S + kKeys - 1) / kKeys) / (2 * kWarps);
  const int n = (int)std::max<long long>(1, std::min<long long>(2 * num_sms() / units, most));
  return n > kFewCluster && n <= kFewCluster + 2 ? kFewCluster : n;
}

cudaError_t launch_cross_few(const CrossCall& c, const CrossParams& P) {
  FewParams F;
  F.c = P;
  F.cluster = P.nsplit > 1 && P.nsplit <= kFewCluster;
  F.q = static_cast<const __nv_bfloat16*>(c.q.data);
  F.k = static_cast<const __nv_bfloat16*>(c.k.data);
  F.v = static_cast<const __nv_bfloat16*>(c.v.data);
  F.q_bs = c.B > 1 ? c.q.batch_stride : 0;
  F.q_ts = c.q.token_stride;
  F.k_bs = c.B > 1 ? c.k.batch_stride : 0;
  F.k_ts = c.k.token_stride;
  F.v_bs = c.B > 1 ? c.v.batch_stride : 0;
  F.v_ts = c.v.token_stride;
  const unsigned grid = (unsigned)(c.B * c.Hk * P.nsplit);
  cudaError_t e;
  switch (c.D / 16) {
    case 1: e = launch_nk<1>(F, grid, c.stream); break;
    case 2: e = launch_nk<2>(F, grid, c.stream); break;
    case 3: e = launch_nk<3>(F, grid, c.stream); break;
    case 4: e = launch_nk<4>(F, grid, c.stream); break;
    case 5: e = launch_nk<5>(F, grid, c.stream); break;
    case 6: e = launch_nk<6>(F, grid, c.stream); break;
    case 7: e = launch_nk<7>(F, grid, c.stream); break;
    default: e = launch_nk<8>(F, grid, c.stream); break;
  }
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace gdn
