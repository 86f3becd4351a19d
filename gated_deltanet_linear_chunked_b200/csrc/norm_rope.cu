// norm_rope.cu -- what a softmax block does to its queries and keys before the
// attention: an RMS norm of every head and the rotary positions, in one pass,
// and the gradients of both.
//
// For one head row x of D features, weight w and the rotation's first R:
//   r = (mean(x^2) + eps)^(-1/2),  x^ = r x,  y = w x^     (or y = x: no norm)
//   (y_a, y_b) -> A (y_a cos t - y_b sin t,  y_a sin t + y_b cos t)
// for each of the R/2 pairs, t = position * frequency.  The gradient turns
// d_out back (t -> -t), g = A R(-t) d_out, and then
//   dw = sum over rows of g x^,   dx = r (g w - x^ mean(g w x^)).
//
// Both are streams over memory: every row is read once and written once, and
// nothing but the angles and the weights' gradient crosses rows.  A row belongs
// to a group of G lanes (a power of two, all in one warp), each of which holds
// two 16-byte pieces of it.  In the half layout the two pieces are the two sides
// of the same pairs (features i and i + R/2), in the interleaved one they are
// neighbours: either way a lane turns its pairs alone, and only the sum of
// squares crosses lanes.  A block takes TB tokens of the queries or of the keys;
// it forms the cosines and sines of its tokens once, in shared memory, each
// group takes its token's into registers and keeps them for all of its heads.
// Angles are formed in 64 bits and reduced to a fraction of a turn there: a
// position of 10^6 has an angle whose 32-bit rounding is already 0.06.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_internal.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kBwdBlocks = 3 * 148;          // per side: persistent blocks of the backward, at most
constexpr long long kMaxStride = 1ll << 40;  // elements

// One side (queries or keys) of a call.
struct Side {
  const void* x;      // forward: input; backward: the forward's input
  const void* dy;     // backward: gradient of the output
  void* out;          // forward: output; backward: gradient of the input
  const float* w;     // [D], or nullptr: ones
  long long x_bs, x_ts, dy_bs, dy_ts, o_bs, o_ts;  // elements
  int H;
  int log_tb;         // tokens per block = 1 << log_tb
  unsigned blocks;    // blocks of this side
};

struct NormRopeParams {
  Side side[2];
  const void* pos;
  const double* freq;
  long long pos_bs;
  int pos_wide;        // positions are int64, else int32
  int axes, sec1, sec2;  // pairs below sec1: axis 0, below sec2: axis 1, else axis 2
  int T, D, R;
  long long tokens;    // B * T
  float amplitude, eps;
  int interleaved;
  int norm;
  int inverse;         // turn by -t
  float* partial;      // backward: [blocks][D] sums of g x^, queries' blocks first
};

template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ uint4 raw(const void* p) { return *static_cast<const uint4*>(p); }
  static __device__ __forceinline__ void open(uint4 u, float (&f)[8]) { unpack8_bf16(u, f); }
  static __device__ __forceinline__ uint4 close(const float (&f)[8]) { return pack8_bf16(f); }
};
template <> struct Vec<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ uint4 raw(const void* p) { return *static_cast<const uint4*>(p); }
  static __device__ __forceinline__ void open(uint4 u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 close(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

// The two pieces of lane l (of G) of a row, as indices of V-feature pieces,
// and whether they hold pairs that turn.  D and R are multiples of 16, so a
// pair never crosses a piece.
struct Pieces {
  int a, b;
  bool present, turns_a, turns_b;
};
template <int V>
__device__ __forceinline__ Pieces pieces_of(int l, int D, int R, bool interleaved) {
  Pieces p;
  const int h = R / (2 * V);
  p.present = l < D / (2 * V);
  if (interleaved) {
    p.a = 2 * l;
    p.b = 2 * l + 1;
    p.turns_a = p.a * V < R;
    p.turns_b = p.b * V < R;
  } else {
    p.turns_a = p.turns_b = l < h;
    p.a = l < h ? l : 2 * h + 2 * (l - h);
    p.b = l < h ? l + h : p.a + 1;
  }
  return p;
}

// cos and sin (times the amplitude) of the pair `i` of token n, t = turns.
__device__ __forceinline__ float2 angle(const NormRopeParams& P, long long n, int i) {
  const long long b = n / P.T, t = n - b * P.T;
  const int axis = i < P.sec1 ? 0 : i < P.sec2 ? 1 : 2;
  const long long at = b * P.pos_bs + t * P.axes + axis;
  const double pos = P.pos_wide ? (double)static_cast<const long long*>(P.pos)[at]
                                : (double)static_cast<const int*>(P.pos)[at];
  // turns = position * frequency / 2 pi; only its fraction matters
  const double turns = pos * P.freq[i] * 0.15915494309189533577;
  const float frac = (float)(turns - rint(turns));
  float s, c;
  sincospif(2.f * frac, &s, &c);
  return make_float2(c * P.amplitude, (P.inverse ? -s : s) * P.amplitude);
}

// Turns a lane's pairs in place: `c`, `s` hold its V pairs' cosines and sines,
// in the half layout pair j is (a[j], b[j]), in the interleaved one pairs
// 0 .. V/2-1 are (a[2j], a[2j+1]) and V/2 .. V-1 are b's.  Features that do not
// turn are left alone (not multiplied by 1 and 0: their neighbour may be infinite).
template <int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float (&c)[V],
                                     const float (&s)[V], const Pieces& pc, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
      if (pc.turns_a) {
        a[2 * j] = a0 * c[j] - a1 * s[j];
        a[2 * j + 1] = a0 * s[j] + a1 * c[j];
      }
      if (pc.turns_b) {
        b[2 * j] = b0 * c[V / 2 + j] - b1 * s[V / 2 + j];
        b[2 * j + 1] = b0 * s[V / 2 + j] + b1 * c[V / 2 + j];
      }
    }
  } else if (pc.turns_a) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float a0 = a[j], b0 = b[j];
      a[j] = a0 * c[j] - b0 * s[j];
      b[j] = a0 * s[j] + b0 * c[j];
    }
  }
}

// The block's side, its first token and its index within the side.
__device__ __forceinline__ int my_side(const NormRopeParams& P, unsigned* block) {
  *block = blockIdx.x;
  if (blockIdx.x < P.side[0].blocks) return 0;
  *block -= P.side[0].blocks;
  return 1;
}

// Fills tab[token][pair] for the tokens n0 .. n0 + tb - 1.
__device__ __forceinline__ void fill_angles(const NormRopeParams& P, float2* tab, long long n0, int tb) {
  const int pairs = P.R / 2;
  for (int i = threadIdx.x; i < tb * pairs; i += kThreads) {
    const int tk = i / pairs;
    if (n0 + tk < P.tokens) tab[i] = angle(P, n0 + tk, i - tk * pairs);
  }
}

// A lane's V pairs from its token's row of the table; pairs that do not turn
// get cos 1, sin 0.
template <int V>
__device__ __forceinline__ void take_angles(const NormRopeParams& P, const float2* row, const Pieces& pc,
                                            int l, float (&c)[V], float (&s)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool on = pc.present && (P.interleaved && j >= V / 2 ? pc.turns_b : pc.turns_a);
    const float2 v = on ? row[l * V + j] : make_float2(1.f, 0.f);
    c[j] = v.x;
    s[j] = v.y;
  }
}

template <int V>
__device__ __forceinline__ void take_weights(const float* w, const Pieces& pc, float (&wa)[V], float (&wb)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) wa[j] = wb[j] = 1.f;
  if (w && pc.present) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      wa[j] = w[pc.a * V + j];
      wb[j] = w[pc.b * V + j];
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads)
gdn_norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
  using VT = Vec<T>;
  constexpr int V = VT::V, kGroups = kThreads / G;
  extern __shared__ float2 tab[];
  unsigned block;
  const Side& S = P.side[my_side(P, &block)];
  const int tb = 1 << S.log_tb, per = kGroups >> S.log_tb;  // tokens; groups per token
  const long long n0 = (long long)block << S.log_tb;
  const int l = threadIdx.x % G, grp = threadIdx.x / G;
  const int tk = grp / per, h0 = grp - tk * per;
  const bool interleaved = P.interleaved;
  const Pieces pc = pieces_of<V>(l, P.D, P.R, interleaved);
  if (P.R > 0) fill_angles(P, tab, n0, tb);
  float wa[V], wb[V], c[V], s[V];
  take_weights<V>(S.w, pc, wa, wb);
  __syncthreads();
  take_angles<V>(P, tab + tk * (P.R / 2), pc, l, c, s);
  const long long n = n0 + tk;
  const bool on = n < P.tokens;
  const long long b = n / P.T, t = n - b * P.T;
  const T* x = static_cast<const T*>(S.x) + (on ? b * S.x_bs + t * S.x_ts : 0);
  T* out = static_cast<T*>(S.out) + (on ? b * S.o_bs + t * S.o_ts : 0);
  const float inv_d = 1.f / P.D;
  // the trip count is the block's, so that the group sums see whole warps
  for (int h1 = 0; h1 < S.H; h1 += per) {
    const int h = h1 + h0;
    const bool act = on && pc.present && h < S.H;
    float a[V], e[V];
    uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
    if (act) {
      ra = VT::raw(x + (long long)h * P.D + pc.a * V);
      rb = VT::raw(x + (long long)h * P.D + pc.b * V);
    }
    VT::open(ra, a);
    VT::open(rb, e);
    if (P.norm) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) ss += a[j] * a[j] + e[j] * e[j];
      const float r = rsqrtf(group_sum<G>(ss) * inv_d + P.eps);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        a[j] *= r * wa[j];
        e[j] *= r * wb[j];
      }
    }
    turn<V>(a, e, c, s, pc, interleaved);
    if (act) {
      *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.a * V) = VT::close(a);
      *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.b * V) = VT::close(e);
    }
  }
}

// The gradients.  Blocks are persistent: each walks its side's token tiles with
// a stride of the side's blocks, so that the weight's gradient leaves as one
// partial row per block, which gdn_norm_rope_reduce_kernel adds up in a fixed
// order (no atomics: the same call gives the same bits).
template <typename T, int G>
__global__ void __launch_bounds__(kThreads)
gdn_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams P) {
  using VT = Vec<T>;
  constexpr int V = VT::V, kGroups = kThreads / G;
  extern __shared__ float2 tab[];
  unsigned block;
  const Side& S = P.side[my_side(P, &block)];
  const int tb = 1 << S.log_tb, per = kGroups >> S.log_tb;
  const long long tiles = (P.tokens + tb - 1) >> S.log_tb;
  const int l = threadIdx.x % G, grp = threadIdx.x / G;
  const int tk = grp / per, h0 = grp - tk * per;
  const bool interleaved = P.interleaved;
  const Pieces pc = pieces_of<V>(l, P.D, P.R, interleaved);
  float wa[V], wb[V], da[V], db[V];
  take_weights<V>(S.w, pc, wa, wb);
#pragma unroll
  for (int j = 0; j < V; ++j) da[j] = db[j] = 0.f;
  const float inv_d = 1.f / P.D;
  for (long long tile = block; tile < tiles; tile += S.blocks) {
    const long long n0 = tile << S.log_tb;
    float c[V], s[V];
    if (P.R > 0) {
      __syncthreads();  // the table's readers of the tile before
      fill_angles(P, tab, n0, tb);
      __syncthreads();
    }
    take_angles<V>(P, tab + tk * (P.R / 2), pc, l, c, s);
    const long long n = n0 + tk;
    const bool on = n < P.tokens;
    const long long b = n / P.T, t = n - b * P.T;
    const T* x = static_cast<const T*>(S.x) + (on ? b * S.x_bs + t * S.x_ts : 0);
    const T* dy = static_cast<const T*>(S.dy) + (on ? b * S.dy_bs + t * S.dy_ts : 0);
    T* out = static_cast<T*>(S.out) + (on ? b * S.o_bs + t * S.o_ts : 0);
    for (int h1 = 0; h1 < S.H; h1 += per) {
      const int h = h1 + h0;
      const bool act = on && pc.present && h < S.H;
      float a[V], e[V], ga[V], ge[V];
      uint4 ra = make_uint4(0, 0, 0, 0), rb = ra, rc = ra, rd = ra;
      if (act) {
        ra = VT::raw(x + (long long)h * P.D + pc.a * V);
        rb = VT::raw(x + (long long)h * P.D + pc.b * V);
        rc = VT::raw(dy + (long long)h * P.D + pc.a * V);
        rd = VT::raw(dy + (long long)h * P.D + pc.b * V);
      }
      VT::open(ra, a);
      VT::open(rb, e);
      VT::open(rc, ga);
      VT::open(rd, ge);
      turn<V>(ga, ge, c, s, pc, interleaved);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ss += a[j] * a[j] + e[j] * e[j];
        dot += ga[j] * wa[j] * a[j] + ge[j] * wb[j] * e[j];
      }
      ss = group_sum<G>(ss);
      dot = group_sum<G>(dot);
      const float r = rsqrtf(ss * inv_d + P.eps);
      const float m = dot * r * inv_d;  // mean(g w x^)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xa = a[j] * r, xe = e[j] * r;
        da[j] += ga[j] * xa;
        db[j] += ge[j] * xe;
        ga[j] = r * (ga[j] * wa[j] - xa * m);
        ge[j] = r * (ge[j] * wb[j] - xe * m);
      }
      if (act) {
        *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.a * V) = VT::close(ga);
        *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.b * V) = VT::close(ge);
      }
    }
  }
  // the block's sums: first over the groups of a warp, then over its warps
  __shared__ float red[kThreads / 32][128];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int o = 16; o >= G; o >>= 1) {
      da[j] += __shfl_xor_sync(~0u, da[j], o);
      db[j] += __shfl_xor_sync(~0u, db[j], o);
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane < G && pc.present) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      red[warp][pc.a * V + j] = da[j];
      red[warp][pc.b * V + j] = db[j];
    }
  }
  __syncthreads();
  if (threadIdx.x < P.D) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) sum += red[w][threadIdx.x];
    P.partial[(size_t)blockIdx.x * P.D + threadIdx.x] = sum;
  }
  pdl_trigger();
}

// dw[side][f] = sum over the side's blocks of partial[block][f]: one block per
// (side, 16 features), 16 lanes across features and 32 rows at a time.
constexpr int kRedCols = 16, kRedRows = 32;
__global__ void __launch_bounds__(kRedCols * kRedRows)
gdn_norm_rope_reduce_kernel(const float* partial, unsigned n0, unsigned n1, int D, float* dw0, float* dw1) {
  pdl_wait();
  __shared__ float red[kRedRows][kRedCols + 1];
  const int col = threadIdx.x % kRedCols, row = threadIdx.x / kRedCols;
  const int f = blockIdx.x * kRedCols + col;
  const unsigned lo = blockIdx.y ? n0 : 0, hi = blockIdx.y ? n0 + n1 : n0;
  float* dw = blockIdx.y ? dw1 : dw0;
  float sum = 0.f;
  for (unsigned i = lo + row; i < hi; i += kRedRows) sum += partial[(size_t)i * D + f];
  red[row][col] = sum;
  __syncthreads();
  if (row == 0 && dw) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kRedRows; ++i) s += red[i][col];
    dw[f] = s;
  }
}

// ------------------------------------------------------------------- host
int lanes_per_row(int D, int V) {
  int g = 1;
  while (g < D / (2 * V)) g *= 2;
  return g;
}

// Tokens per block: enough groups on each token that a group takes about four
// of its heads (the angles, once in registers, serve them all), fewer tokens
// while the grid does not fill the GPU.
int log_tokens_per_block(int groups, int H, long long tokens, int sms) {
  int per = 1;
  while (per < groups && per * 4 < H) per *= 2;
  int lt = 0;
  while ((per << (lt + 1)) <= groups) ++lt;
  while (lt > 0 && (tokens >> lt) < 2 * sms) --lt;
  return lt;
}

template <typename T, int G>
cudaError_t launch_g(NormRopeParams& P, bool backward, cudaStream_t stream) {
  constexpr int groups = kThreads / G;
  const int sms = num_sms();
  size_t smem = 0;
  for (Side& S : P.side) {
    S.blocks = 0;
    S.log_tb = 0;
    if (!S.H) continue;
    S.log_tb = log_tokens_per_block(groups, S.H, P.tokens, sms);
    const long long tiles = (P.tokens + (1 << S.log_tb) - 1) >> S.log_tb;
    S.blocks = (unsigned)tiles;
    if (backward) S.blocks = (unsigned)std::min<long long>(tiles, kBwdBlocks);
    smem = std::max(smem, (size_t)(1 << S.log_tb) * (P.R / 2) * sizeof(float2));
  }
  const unsigned grid = P.side[0].blocks + P.side[1].blocks;
  if (backward) {
    ProfileScope ps(stream, kKernNormRopeBwd);
    gdn_norm_rope_bwd_kernel<T, G><<<grid, kThreads, smem, stream>>>(P);
  } else {
    ProfileScope ps(stream, kKernNormRope);
    gdn_norm_rope_kernel<T, G><<<grid, kThreads, smem, stream>>>(P);
  }
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(NormRopeParams& P, bool backward, cudaStream_t stream) {
  // D / 16 pieces of two for bf16 (1 to 8), D / 8 for fp32 (2 to 16)
  constexpr int kLeast = Vec<T>::V == 8 ? 1 : 2;
  switch (lanes_per_row(P.D, Vec<T>::V) / kLeast) {
    case 1: return launch_g<T, kLeast>(P, backward, stream);
    case 2: return launch_g<T, 2 * kLeast>(P, backward, stream);
    case 4: return launch_g<T, 4 * kLeast>(P, backward, stream);
    default: return launch_g<T, 8 * kLeast>(P, backward, stream);
  }
}

// A [B, T, H, D] view with its strides in bytes, for the overlap checks.
struct View {
  const uint8_t* p;
  long long bs, ts, row;  // bytes; row = H * D elements
  int B, T;
  Range range() const {
    return {(uintptr_t)p, (uintptr_t)p + (B - 1) * bs + (T - 1) * ts + row};
  }
};

// Whether no two rows of the view share memory: tokens inside batch rows, or
// batch rows inside tokens (a sequence-first buffer).
bool rows_apart(const View& v) {
  const bool in_b = (v.T == 1 || v.ts >= v.row) && (v.B == 1 || v.bs >= (v.T - 1) * v.ts + v.row);
  const bool in_t = (v.B == 1 || v.bs >= v.row) && (v.T == 1 || v.ts >= (v.B - 1) * v.bs + v.row);
  return in_b || in_t;
}

// Whether two views share memory.  Views of one packed buffer interleave: with
// equal strides and no row of either reaching into the other's, they do not.
bool views_clash(const View& a, const View& b) {
  if (!overlaps(a.range(), b.range())) return false;
  if (a.bs == b.bs && a.ts == b.ts) {
    const View& lo = a.p <= b.p ? a : b;
    const View& hi = a.p <= b.p ? b : a;
    View both = lo;
    both.row = (hi.p - lo.p) + hi.row;
    if (hi.p - lo.p >= lo.row && rows_apart(both)) return false;
  }
  return true;
}

bool same_view(const View& a, const View& b) {
  return a.p == b.p && (a.bs == b.bs || a.B == 1) && (a.ts == b.ts || a.T == 1);
}

struct Call {
  const gdn_rows* in[2];    // the forward's inputs (the rope's: unused in its backward)
  const gdn_rows* dy[2];    // backward: gradients of the outputs
  const gdn_rows* out[2];   // outputs, or gradients of the inputs
  const float* w[2];
  float* dw[2];
  const gdn_rotation* rot;
  int B, T, H[2], D;
  float eps;
  gdn_dtype dtype;
  void* stream;
  bool norm, backward, inverse;
};

gdn_status run(const Call& c) {
  // ---- pure host checks
  if (c.dtype != GDN_F32 && c.dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (c.B < 0 || c.T < 0 || c.H[0] < 0 || c.H[1] < 0 || c.D < 0) return GDN_ERR_INVALID_ARG;
  if (!(c.eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (!supported_dim(c.D)) return GDN_ERR_UNSUPPORTED;
  if ((long long)c.B * c.T > 0x3FFFFFFFll || (long long)c.H[0] + c.H[1] > (1 << 20))
    return GDN_ERR_UNSUPPORTED;
  const gdn_rotation* r = c.rot;
  if (r) {
    if (r->rot_dim < 0 || r->rot_dim > c.D || r->axes < 1 || r->axes > 3) return GDN_ERR_INVALID_ARG;
    if (r->layout != GDN_ROPE_HALF && r->layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
    if (r->rot_dim % 16) return GDN_ERR_UNSUPPORTED;
    int pairs = 0;
    for (int i = 0; i < r->axes; ++i) {
      if (r->section[i] < 0 || r->section[i] > r->rot_dim / 2) return GDN_ERR_INVALID_ARG;
      pairs += r->section[i];
    }
    if (pairs != r->rot_dim / 2) return GDN_ERR_INVALID_ARG;
    if (r->position_bytes != 4 && r->position_bytes != 8) return GDN_ERR_INVALID_ARG;
    if (r->position_batch_stride < 0 || r->position_batch_stride > kMaxStride) return GDN_ERR_INVALID_ARG;
  }
  const int R = r ? r->rot_dim : 0;
  const bool empty = c.B == 0 || c.T == 0 || c.H[0] + c.H[1] == 0;
  if (empty && !(c.backward && (c.dw[0] || c.dw[1]))) return GDN_OK;
  const int es = c.dtype == GDN_BF16 ? 2 : 4;

  View in[2], dy[2], out[2];
  Range fixed[8];  // contiguous buffers that are read
  int nfixed = 0;
  const void* ptrs[16];
  int nptr = 0;
  auto view = [&](const gdn_rows* v, int s, View* to) {
    if (!v || !v->data || !aligned16(v->data)) return false;
    if (v->batch_stride < 0 || v->batch_stride > kMaxStride || v->token_stride < 0 ||
        v->token_stride > kMaxStride)
      return false;
    if ((v->batch_stride * es) % 16 || (v->token_stride * es) % 16) return false;
    *to = {static_cast<const uint8_t*>(v->data), v->batch_stride * es, v->token_stride * es,
           (long long)c.H[s] * c.D * es, c.B, c.T};
    ptrs[nptr++] = v->data;
    return true;
  };
  auto read = [&](const void* p, size_t bytes) {
    if (!p) return;
    fixed[nfixed++] = range_of(p, bytes);
    ptrs[nptr++] = p;
  };
  for (int s = 0; s < 2; ++s) {
    if (c.dw[s] && !aligned16(c.dw[s])) return GDN_ERR_INVALID_ARG;
    if (c.w[s] && !aligned16(c.w[s])) return GDN_ERR_INVALID_ARG;
    if (c.w[s] && c.H[s]) read(c.w[s], (size_t)c.D * 4);
    if (empty || !c.H[s]) continue;
    if (!view(c.in[s], s, &in[s]) || !view(c.out[s], s, &out[s])) return GDN_ERR_INVALID_ARG;
    if (c.backward && !view(c.dy[s], s, &dy[s])) return GDN_ERR_INVALID_ARG;
    if (!rows_apart(out[s])) return GDN_ERR_ALIAS;
  }
  if (R > 0 && !empty) {
    if (!r->positions || !r->inv_freq || (uintptr_t)r->positions % r->position_bytes ||
        (uintptr_t)r->inv_freq % 8)
      return GDN_ERR_INVALID_ARG;
    read(r->positions, (size_t)((c.B - 1) * r->position_batch_stride + (long long)c.T * r->axes) *
                           r->position_bytes);
    read(r->inv_freq, (size_t)R / 2 * 8);
  }
  // what is written overlaps nothing else, except that an output may be
  // exactly the rows it is computed from
  for (int s = 0; s < 2 && !empty; ++s) {
    if (!c.H[s]) continue;
    for (int i = 0; i < 2; ++i) {
      if (!c.H[i]) continue;
      if (views_clash(out[s], in[i]) && !(s == i && same_view(out[s], in[i]))) return GDN_ERR_ALIAS;
      if (c.backward && views_clash(out[s], dy[i]) && !(s == i && same_view(out[s], dy[i])))
        return GDN_ERR_ALIAS;
      if (i > s && views_clash(out[s], out[i])) return GDN_ERR_ALIAS;
    }
    for (int i = 0; i < nfixed; ++i)
      if (overlaps(out[s].range(), fixed[i])) return GDN_ERR_ALIAS;
  }
  for (int s = 0; s < 2; ++s) {
    if (!c.dw[s]) continue;
    const Range w = range_of(c.dw[s], (size_t)c.D * 4);
    for (int i = 0; i < nfixed; ++i)
      if (overlaps(w, fixed[i])) return GDN_ERR_ALIAS;
    for (int i = 0; i < 2 && !empty; ++i)
      if (c.H[i] && (overlaps(w, in[i].range()) || overlaps(w, dy[i].range()) || overlaps(w, out[i].range())))
        return GDN_ERR_ALIAS;
    ptrs[nptr++] = c.dw[s];
  }
  if (c.dw[0] && c.dw[1] &&
      overlaps(range_of(c.dw[0], (size_t)c.D * 4), range_of(c.dw[1], (size_t)c.D * 4)))
    return GDN_ERR_ALIAS;

  // ---- device checks
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  for (int i = 0; i < nptr; ++i) {
    const gdn_status st = check_device_pointer(ptrs[i], dev);
    if (st != GDN_OK) return st;
  }
  cudaGetLastError();
  cudaStream_t stream = static_cast<cudaStream_t>(c.stream);
  if (empty) {  // no rows: the weights' gradients are zero
    cudaError_t e = cudaSuccess;
    for (int s = 0; s < 2; ++s)
      if (c.dw[s] && e == cudaSuccess) e = cudaMemsetAsync(c.dw[s], 0, (size_t)c.D * 4, stream);
    return finish(stream, e, nullptr);
  }

  NormRopeParams P = {};
  for (int s = 0; s < 2; ++s) {
    Side& S = P.side[s];
    S.H = c.H[s];
    S.w = c.w[s];
    if (!S.H) continue;
    S.x = c.in[s]->data;
    S.x_bs = c.in[s]->batch_stride;
    S.x_ts = c.in[s]->token_stride;
    S.out = c.out[s]->data;
    S.o_bs = c.out[s]->batch_stride;
    S.o_ts = c.out[s]->token_stride;
    if (c.backward) {
      S.dy = c.dy[s]->data;
      S.dy_bs = c.dy[s]->batch_stride;
      S.dy_ts = c.dy[s]->token_stride;
    }
  }
  P.T = c.T;
  P.D = c.D;
  P.R = R;
  P.tokens = (long long)c.B * c.T;
  P.eps = c.eps;
  P.norm = c.norm;
  P.inverse = c.inverse;
  if (r) {
    P.pos = r->positions;
    P.freq = r->inv_freq;
    P.pos_bs = r->position_batch_stride;
    P.pos_wide = r->position_bytes == 8;
    P.axes = r->axes;
    P.sec1 = r->section[0];
    P.sec2 = P.sec1 + (r->axes > 1 ? r->section[1] : R);
    P.amplitude = r->amplitude;
    P.interleaved = r->layout == GDN_ROPE_INTERLEAVED;
  }
  if (!c.backward) {
    const cudaError_t e = c.dtype == GDN_BF16 ? launch_t<__nv_bfloat16>(P, false, stream)
                                              : launch_t<float>(P, false, stream);
    return finish(stream, e, nullptr);
  }
  OpScratch sc;
  unsigned int* err = nullptr;
  const gdn_status st =
      op_scratch(dev, stream, (size_t)2 * kBwdBlocks * c.D * sizeof(float), &err, &sc);
  if (st != GDN_OK) return st;
  P.partial = static_cast<float*>(sc.p);
  cudaError_t e = c.dtype == GDN_BF16 ? launch_t<__nv_bfloat16>(P, true, stream)
                                      : launch_t<float>(P, true, stream);
  if (e == cudaSuccess && (c.dw[0] || c.dw[1])) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c.D / kRedCols, 2);
    cfg.blockDim = dim3(kRedCols * kRedRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    ProfileScope ps(stream, kKernNormRopeReduce);
    e = cudaLaunchKernelEx(&cfg, gdn_norm_rope_reduce_kernel, (const float*)P.partial,
                           P.side[0].blocks, P.side[1].blocks, c.D, c.dw[0], c.dw[1]);
    if (e == cudaSuccess) count_launches(1);
  }
  const cudaError_t f = op_scratch_done(sc);
  return finish(stream, e == cudaSuccess ? f : e, nullptr);
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_rope(const gdn_rows* q, const gdn_rows* k, const gdn_rotation* rotation, int inverse,
                    const gdn_rows* q_out, const gdn_rows* k_out, int B, int T, int Hq, int Hk, int D,
                    gdn_dtype dtype, void* stream) {
  gdn::Call c = {{q, k}, {nullptr, nullptr}, {q_out, k_out}, {nullptr, nullptr}, {nullptr, nullptr},
                 rotation, B, T, {Hq, Hk}, D, 0.f, dtype, stream, false, false, inverse != 0};
  if (!rotation) return GDN_ERR_INVALID_ARG;
  return gdn::run(c);
}

gdn_status gdn_qk_norm_rope(const gdn_rows* q, const gdn_rows* k, const float* q_weight,
                            const float* k_weight, const gdn_rotation* rotation, const gdn_rows* q_out,
                            const gdn_rows* k_out, int B, int T, int Hq, int Hk, int D, float eps,
                            gdn_dtype dtype, void* stream) {
  gdn::Call c = {{q, k}, {nullptr, nullptr}, {q_out, k_out}, {q_weight, k_weight}, {nullptr, nullptr},
                 rotation, B, T, {Hq, Hk}, D, eps, dtype, stream, true, false, false};
  return gdn::run(c);
}

gdn_status gdn_qk_norm_rope_backward(const gdn_rows* q, const gdn_rows* k, const float* q_weight,
                                     const float* k_weight, const gdn_rotation* rotation,
                                     const gdn_rows* dq_out, const gdn_rows* dk_out, const gdn_rows* dq,
                                     const gdn_rows* dk, float* dq_weight, float* dk_weight, int B, int T,
                                     int Hq, int Hk, int D, float eps, gdn_dtype dtype, void* stream) {
  gdn::Call c = {{q, k}, {dq_out, dk_out}, {dq, dk}, {q_weight, k_weight}, {dq_weight, dk_weight},
                 rotation, B, T, {Hq, Hk}, D, eps, dtype, stream, true, true, true};
  return gdn::run(c);
}

}  // extern "C"
