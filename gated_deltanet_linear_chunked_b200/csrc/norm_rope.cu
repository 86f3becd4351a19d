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
// squares crosses lanes.  A block takes a tile of tokens, all heads of queries and
// keys; it forms the cosines and sines of its tokens once, in shared memory, each
// group takes its token's into registers, with the weights of its side folded in,
// and keeps them for its heads, two of which are always on their way from memory.
// Angles are formed in 64 bits and reduced to a fraction of a turn there: a
// position of 10^6 has an angle whose 32-bit rounding is already 0.06.
// Inputs from memory: 65536 tokens, 16 + 4 heads of 128 in fp32 220 us (6.1 TB/s, bound
// by memory), 2640 tokens, 20 + 20 heads of 112 in bf16 12.2 us (3.9 TB/s: 880 blocks for
// 444 places, each forming its angles before it stores).  The gradients, which read
// twice as much and hold the weights' sums in registers, are bound by latency at 16
// warps an SM: the same 22.9 us (3.1 TB/s), 4 x 4096 tokens, 16 + 4 heads of 128 in bf16
// 60 us (4.2 TB/s).  Repeated on the same tensors, so largely out of L2: 10.1, 18.8
// and 60 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_internal.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr long long kMaxStride = 1ll << 40;  // elements

// One side (queries or keys) of a call.
struct Side {
  const void* x;      // forward: input; backward: the forward's input
  const void* dy;     // backward: gradient of the output
  void* out;          // forward: output; backward: gradient of the input
  const float* w;     // [D], or nullptr: ones
  long long x_bs, x_ts, dy_bs, dy_ts, o_bs, o_ts;  // elements
  int H;
  int per;            // groups of lanes per token
};

struct NormRopeParams {
  Side side[2];
  const void* pos;
  const double* freq;
  long long pos_bs;
  int pos_wide;        // positions are int64, else int32
  int axes, sec1, sec2;  // pairs below sec1: axis 0, below sec2: axis 1, else axis 2
  int T, D, R;
  unsigned tokens;     // B * T
  int heads;           // heads of a group, at most
  int tb;              // tokens of a tile: what a block's groups take at a time
  unsigned tiles;
  float amplitude, eps;
  int interleaved;
  int norm;
  int inverse;         // turn by -t
  float* partial;      // backward: [side][block][D] sums of g x^
};

// 16 bytes of a row as packed fp32 pairs: V features, V / 2 pairs.
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void open(uint4 u, uint64_t* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint4 close(const uint64_t* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2_unpack(f[i], a, b);
      w[i] = pack_bf16x2(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void open(uint4 u, uint64_t* f) {
    f[0] = f2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
    f[1] = f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 close(const uint64_t* f) {
    float a, b, c, d;
    f2_unpack(f[0], a, b);
    f2_unpack(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
};
__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }
__device__ __forceinline__ uint64_t f2_swap(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return f2_pack(b, a);
}

// The two pieces of lane l (of G) of a row, as indices of V-feature pieces,
// and whether they hold pairs that turn.  D and R are multiples of 16, so a
// pair never crosses a piece.
struct Pieces {
  int a, b;
  bool present, turns_a, turns_b;
};
template <int V, bool interleaved>
__device__ __forceinline__ Pieces pieces_of(int l, int D, int R) {
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
__device__ __forceinline__ float2 angle(const NormRopeParams& P, unsigned n, int i) {
  const unsigned b = n / (unsigned)P.T, t = n - b * P.T;
  const int axis = i < P.sec1 ? 0 : i < P.sec2 ? 1 : 2;
  const long long at = b * P.pos_bs + (long long)t * P.axes + axis;
  const double pos = P.pos_wide ? (double)static_cast<const long long*>(P.pos)[at]
                                : (double)static_cast<const int*>(P.pos)[at];
  // turns = position * frequency / 2 pi; only its fraction matters
  const double turns = pos * P.freq[i] * 0.15915494309189533577;
  const float frac = (float)(turns - rint(turns));
  float s, c;
  sincospif(2.f * frac, &s, &c);
  return make_float2(c * P.amplitude, (P.inverse ? -s : s) * P.amplitude);
}

// A lane holds 2V features as V packed pairs, piece a's V / 2 first.  Turning is
//   out = x * c1 + partner * c2,
// the partner of piece a's features being piece b's in the half layout (c2 = -s,
// and +s the other way), and each packed pair's own other half in the interleaved
// one (c2 = (-s, s)).  Features that do not turn are only scaled by c1 (a product
// with 0 would let an infinite neighbour in).
template <int V, bool interleaved>
__device__ __forceinline__ void turn(uint64_t (&x)[V], const uint64_t (&c1)[V], const uint64_t (&c2)[V],
                                     const Pieces& pc) {
  constexpr int N = V / 2;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (interleaved) {
      const uint64_t a = f2_mul(x[j], c1[j]), b = f2_mul(x[N + j], c1[N + j]);
      x[j] = pc.turns_a ? f2_fma(f2_swap(x[j]), c2[j], a) : a;
      x[N + j] = pc.turns_b ? f2_fma(f2_swap(x[N + j]), c2[N + j], b) : b;
    } else {
      const uint64_t a = f2_mul(x[j], c1[j]), b = f2_mul(x[N + j], c1[N + j]);
      const uint64_t a2 = f2_fma(x[N + j], c2[j], a), b2 = f2_fma(x[j], c2[N + j], b);
      x[j] = pc.turns_a ? a2 : a;
      x[N + j] = pc.turns_a ? b2 : b;
    }
  }
}

// A group's place in a block: its token of the tile (or none), its side, and the
// heads h0, h0 + per, ... of that side it takes.
struct Place {
  int token, side, h0;
};
__device__ __forceinline__ Place place_of(const NormRopeParams& P, int grp) {
  const int per = P.side[0].per + P.side[1].per;
  Place p;
  p.token = grp / per;
  const int i = grp - p.token * per;
  p.side = i >= P.side[0].per;
  p.h0 = p.side ? i - P.side[0].per : i;
  return p;
}

// The angles' table: for every token of a tile, lane l of a group and j < V / 2, the
// cosines and sines of the lane's pairs V l + 2 j and V l + 2 j + 1 as
// (cos, cos, sin, sin), at [token][j][l] so that a group's lanes read side by side.
template <int V, int G>
__device__ __forceinline__ void fill_angles(const NormRopeParams& P, float* tab, unsigned n0) {
  const int pairs = P.R / 2;
  for (int i = threadIdx.x; i < P.tb * pairs; i += kThreads) {
    const int tk = i / pairs, p = i - tk * pairs;
    if (n0 + tk >= P.tokens) continue;
    const float2 a = angle(P, n0 + tk, p);
    float* to = tab + (((tk * (V / 2) + p % V / 2) * G + p / V) * 4 + p % 2);
    to[0] = a.x;
    to[2] = a.y;
  }
}
// Entry j of a lane: cosines and sines of two pairs (1 and 0 where nothing turns).
__device__ __forceinline__ float4 angles_at(const float4* row, bool on, int j, int G) {
  return on ? row[j * G] : make_float4(1.f, 1.f, 0.f, 0.f);
}

// A lane's factors c1, c2 (see turn) from its token's row of the table and the
// weights of its features, wx of the feature itself and wp of its partner:
// turned = wx x c1 + wp partner c2 with the weights folded in (pass ones to leave
// them out).
template <int V, int G, bool interleaved>
__device__ __forceinline__ void take_angles(const float4* row, const Pieces& pc, const uint64_t (&w)[V],
                                            uint64_t (&c1)[V], uint64_t (&c2)[V]) {
  constexpr int N = V / 2;
  float wf[2 * V];
#pragma unroll
  for (int j = 0; j < V; ++j) f2_unpack(w[j], wf[2 * j], wf[2 * j + 1]);
  const bool on_a = pc.turns_a && pc.present, on_b = pc.turns_b && pc.present;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (interleaved) {  // pairs V l + j (piece a) and V l + N + j (piece b)
      const float4 fa = angles_at(row, on_a, j / 2, G), fb = angles_at(row, on_b, (N + j) / 2, G);
      const float ca = j % 2 ? fa.y : fa.x, sa = j % 2 ? fa.w : fa.z;
      const float cb = j % 2 ? fb.y : fb.x, sb = j % 2 ? fb.w : fb.z;
      c1[j] = f2_pack(wf[2 * j] * ca, wf[2 * j + 1] * ca);
      c2[j] = f2_pack(-wf[2 * j + 1] * sa, wf[2 * j] * sa);
      c1[N + j] = f2_pack(wf[V + 2 * j] * cb, wf[V + 2 * j + 1] * cb);
      c2[N + j] = f2_pack(-wf[V + 2 * j + 1] * sb, wf[V + 2 * j] * sb);
    } else {  // pairs V l + 2 j and V l + 2 j + 1
      const float4 f = angles_at(row, on_a, j, G);
      c1[j] = f2_pack(wf[2 * j] * f.x, wf[2 * j + 1] * f.y);
      c2[j] = f2_pack(-wf[V + 2 * j] * f.z, -wf[V + 2 * j + 1] * f.w);
      c1[N + j] = f2_pack(wf[V + 2 * j] * f.x, wf[V + 2 * j + 1] * f.y);
      c2[N + j] = f2_pack(wf[2 * j] * f.z, wf[2 * j + 1] * f.w);
    }
  }
}

// 16 bytes of shared memory that the compiler is not to keep in registers.
__device__ __forceinline__ float4 reread(uint32_t addr) {
  uint32_t r[4];
  ld_shared_v4(addr, r);
  return make_float4(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]), __uint_as_float(r[3]));
}

// The turn of a gradient, its factors straight from the table, read anew for every
// head: kept in registers they make the gradient kernel spill (the chunk's gradients
// 23.8 us against 21.0; a third block per SM at 80 registers spills as well, 28.5).
template <int V, int G, bool interleaved>
__device__ __forceinline__ void turn_from(uint32_t row, uint64_t (&x)[V], const Pieces& pc) {
  constexpr int N = V / 2;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (interleaved) {
      if (j % 2) continue;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        if (!(side ? pc.turns_b : pc.turns_a)) continue;
        const float4 f = reread(row + ((side * N + j) / 2) * G * 16);
        uint64_t* y = x + side * N + j;
        y[0] = f2_fma(f2_swap(y[0]), f2_pack(-f.z, f.z), f2_mul(y[0], f2_pack(f.x, f.x)));
        y[1] = f2_fma(f2_swap(y[1]), f2_pack(-f.w, f.w), f2_mul(y[1], f2_pack(f.y, f.y)));
      }
    } else if (pc.turns_a) {
      const float4 f = reread(row + j * G * 16);
      const uint64_t c = f2_pack(f.x, f.y), s = f2_pack(f.z, f.w), ns = f2_pack(-f.z, -f.w);
      const uint64_t a = f2_fma(x[N + j], ns, f2_mul(x[j], c));
      x[N + j] = f2_fma(x[j], s, f2_mul(x[N + j], c));
      x[j] = a;
    }
  }
}

// The weights of a lane's features (ones without).
template <int V>
__device__ __forceinline__ void take_weights(const float* w, const Pieces& pc, uint64_t (&to)[V]) {
  constexpr int N = V / 2;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int f = j < N ? pc.a * V + 2 * j : pc.b * V + 2 * (j - N);
    to[j] = w && pc.present ? *reinterpret_cast<const uint64_t*>(w + f) : f2_pack(1.f, 1.f);
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <typename T, int G, bool interleaved>
__global__ void __launch_bounds__(kThreads, 3)
gdn_norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
  using VT = Vec<T>;
  constexpr int V = VT::V, N = V / 2;
  extern __shared__ __align__(16) float tab[];
  const int l = threadIdx.x % G;
  const Place pl = place_of(P, threadIdx.x / G);
  const Side& S = P.side[pl.side];
  const int tk = pl.token, h0 = pl.h0;
  const unsigned n0 = blockIdx.x * P.tb, n = n0 + tk;
  const Pieces pc = pieces_of<V, interleaved>(l, P.D, P.R);
  const bool on = pc.present && tk < P.tb && n < P.tokens;
  const unsigned bu = on ? n / (unsigned)P.T : 0, tu = on ? n - bu * P.T : 0;
  const long long b = bu, t = tu;
  const T* x = static_cast<const T*>(S.x) + b * S.x_bs + t * S.x_ts;
  T* out = static_cast<T*>(S.out) + b * S.o_bs + t * S.o_ts;
  pdl_wait();  // inputs may come from the kernel in front
  pdl_trigger();
  // two heads' loads are always under way, the first before the angles
  uint4 ring[2][2];
  auto fetch = [&](uint4 (&to)[2], int h) {
    to[0] = to[1] = make_uint4(0, 0, 0, 0);
    if (on && h < S.H) {
      to[0] = load16(x + (long long)h * P.D + pc.a * V);
      to[1] = load16(x + (long long)h * P.D + pc.b * V);
    }
  };
  fetch(ring[0], h0);
  fetch(ring[1], h0 + S.per);
  uint64_t c1[V], c2[V];
  {
    uint64_t w[V];
    take_weights<V>(S.w, pc, w);
    if (P.R > 0) {
      fill_angles<V, G>(P, tab, n0);
      __syncthreads();
    }
    take_angles<V, G, interleaved>(reinterpret_cast<const float4*>(tab) + min(tk, P.tb - 1) * (N * G) + l, pc, w, c1, c2);
  }
  const float inv_d = 1.f / P.D;
  auto work = [&](const uint4 (&from)[2], int h) {
    uint64_t v[V];
    VT::open(from[0], v);
    VT::open(from[1], v + N);
    if (P.norm) {
      uint64_t s2[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < V; ++j) s2[j & 1] = f2_fma(v[j], v[j], s2[j & 1]);
      float sa, sb;
      f2_unpack(f2_add(s2[0], s2[1]), sa, sb);
      const float r = rsqrtf(group_sum<G>(sa + sb) * inv_d + P.eps);
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = f2_mul(v[j], r2);
    }
    turn<V, interleaved>(v, c1, c2, pc);
    if (on && h < S.H) {
      *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.a * V) = VT::close(v);
      *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.b * V) = VT::close(v + N);
    }
  };
  // the trip count is the block's, so that the group sums see whole warps
  for (int i = 0, h = h0; i < P.heads; i += 2, h += 2 * S.per) {
    work(ring[0], h);
    if (i + 1 >= P.heads) break;
    fetch(ring[0], h + 2 * S.per);
    work(ring[1], h + S.per);
    fetch(ring[1], h + 3 * S.per);
  }
}

// The gradients.  Blocks are persistent: each walks its side's token tiles with
// a stride of the side's blocks, so that the weight's gradient leaves as one
// partial row per block, which gdn_norm_rope_reduce_kernel adds up in a fixed
// order (no atomics: the same call gives the same bits).  Two heads on their way
// instead of one took longer (the chunk's gradients 23.1 us for 21.1 in rotation).
template <typename T, int G, bool interleaved>
__global__ void __launch_bounds__(kThreads, 2)
gdn_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams P) {
  using VT = Vec<T>;
  constexpr int V = VT::V, N = V / 2;
  extern __shared__ __align__(16) float tab[];
  const int l = threadIdx.x % G, grp = threadIdx.x / G;
  const Place pl = place_of(P, grp);
  const Side& S = P.side[pl.side];
  const int tk = pl.token, h0 = pl.h0;
  const Pieces pc = pieces_of<V, interleaved>(l, P.D, P.R);
  pdl_wait();  // inputs may come from the kernel in front
  pdl_trigger();
  const uint32_t row = smem_u32(tab) + (min(tk, P.tb - 1) * (N * G) + l) * 16;
  uint64_t w[V], dw[V];
  take_weights<V>(S.w, pc, w);
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = 0;
  const float inv_d = 1.f / P.D;
  for (unsigned tile = blockIdx.x; tile < P.tiles; tile += gridDim.x) {
    const unsigned n0 = tile * P.tb, n = n0 + tk;
    const bool on = pc.present && tk < P.tb && n < P.tokens;
    const unsigned bu = on ? n / (unsigned)P.T : 0, tu = on ? n - bu * P.T : 0;
    const long long b = bu, t = tu;
    const T* x = static_cast<const T*>(S.x) + b * S.x_bs + t * S.x_ts;
    const T* dy = static_cast<const T*>(S.dy) + b * S.dy_bs + t * S.dy_ts;
    T* out = static_cast<T*>(S.out) + b * S.o_bs + t * S.o_ts;
    // the next head's loads are always under way, the first before the angles
    uint4 ring[4];
    auto fetch = [&](int h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ring[i] = make_uint4(0, 0, 0, 0);
      if (on && h < S.H) {
        ring[0] = load16(x + (long long)h * P.D + pc.a * V);
        ring[1] = load16(x + (long long)h * P.D + pc.b * V);
        ring[2] = load16(dy + (long long)h * P.D + pc.a * V);
        ring[3] = load16(dy + (long long)h * P.D + pc.b * V);
      }
    };
    fetch(h0);
    if (P.R > 0) {
      __syncthreads();  // the table's readers of the tile before
      fill_angles<V, G>(P, tab, n0);
      __syncthreads();
    }
    for (int i = 0, h = h0; i < P.heads; ++i, h += S.per) {
      uint64_t v[V], g[V];
      VT::open(ring[0], v);
      VT::open(ring[1], v + N);
      VT::open(ring[2], g);
      VT::open(ring[3], g + N);
      fetch(h + S.per);
      // A place without a row (a token or head past the end) holds zeros, and adds zeros
      // to dw: its part of the table was never written, and r of its sum of squares may
      // be infinite.
      const bool mine = on && h < S.H;
      if (mine) turn_from<V, G, interleaved>(row, g, pc);
      uint64_t s2[2] = {0, 0}, d2[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        s2[0] = f2_fma(v[j], v[j], s2[0]);
        s2[1] = f2_fma(v[j + 1], v[j + 1], s2[1]);
        d2[0] = f2_fma(f2_mul(g[j], w[j]), v[j], d2[0]);
        d2[1] = f2_fma(f2_mul(g[j + 1], w[j + 1]), v[j + 1], d2[1]);
      }
      float sa, sb, da, db;
      f2_unpack(f2_add(s2[0], s2[1]), sa, sb);
      f2_unpack(f2_add(d2[0], d2[1]), da, db);
      const float ss = group_sum<G>(sa + sb), dot = group_sum<G>(da + db);
      const float r = mine ? rsqrtf(ss * inv_d + P.eps) : 0.f;
      const float m = -dot * r * inv_d;  // -mean(g w x^)
      const uint64_t r2 = f2_pack(r, r), m2 = f2_pack(m, m);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
#pragma unroll
        for (int e = j; e < j + 2; ++e) {
          const uint64_t hat = f2_mul(v[e], r2);
          dw[e] = f2_fma(g[e], hat, dw[e]);
          g[e] = f2_mul(r2, f2_fma(hat, m2, f2_mul(g[e], w[e])));
        }
      }
      if (mine) {
        *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.a * V) = VT::close(g);
        *reinterpret_cast<uint4*>(out + (long long)h * P.D + pc.b * V) = VT::close(g + N);
      }
    }
  }
  // the block's sums: every group's row to shared memory (over the angles), then a
  // thread per side and feature adds the side's up in their order
  float* red = reinterpret_cast<float*>(tab);
  __syncthreads();
  if (pc.present) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int f = j < N ? pc.a * V + 2 * j : pc.b * V + 2 * (j - N);
      *reinterpret_cast<uint64_t*>(red + grp * P.D + f) = dw[j];
    }
  }
  __syncthreads();
  const int per = P.side[0].per + P.side[1].per;
  for (int i = threadIdx.x; i < 2 * P.D; i += kThreads) {
    const int side = i >= P.D, f = i - side * P.D;
    const int lo = side ? P.side[0].per : 0, hi = side ? per : P.side[0].per;
    float sum = 0.f;
    for (int k = 0; k < P.tb; ++k)
      for (int x = lo; x < hi; ++x) sum += red[(k * per + x) * P.D + f];
    P.partial[((size_t)side * gridDim.x + blockIdx.x) * P.D + f] = sum;
  }
}

// dw[side][f] = sum over the side's blocks of partial[block][f]: one block per
// (side, 16 features), 16 lanes across features and 32 rows at a time.  About 2 us,
// most of them its launch.
constexpr int kRedCols = 16, kRedRows = 32;
__global__ void __launch_bounds__(kRedCols * kRedRows)
gdn_norm_rope_reduce_kernel(const float* partial, unsigned blocks, int D, float* dw0, float* dw1) {
  pdl_wait();
  __shared__ float red[kRedRows][kRedCols + 1];
  const int col = threadIdx.x % kRedCols, row = threadIdx.x / kRedCols;
  const int per = D / kRedCols, side = blockIdx.x / per, f = (blockIdx.x - side * per) * kRedCols + col;
  float* dw = side ? dw1 : dw0;
  const float* from = partial + (size_t)side * blocks * D + f;
  float sum = 0.f;
  for (unsigned i = row; i < blocks; i += kRedRows) sum += from[(size_t)i * D];
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

// How a block's groups are shared out: for m heads a group, ceil(H / m) groups of
// each side to a token.  The angles, once in registers, serve m heads, and a tile
// starts once for them, which counts as 1.5 heads; m is the one that takes the
// least time over all waves of tiles (`slots` blocks run at a time).  The chunk of
// 2640 tokens, 20 + 20 heads of 112 in bf16: m = 4, three tokens to a tile, 880
// tiles for 444 slots; m = 5 would leave a second wave half empty.
bool share_groups(int groups, int slots, NormRopeParams* P) {
  double best = 0;
  const int most = std::max(P->side[0].H, P->side[1].H);
  for (int m = 1; m <= most; ++m) {
    const int per0 = (P->side[0].H + m - 1) / m, per1 = (P->side[1].H + m - 1) / m;
    if (per0 + per1 > groups) continue;
    const unsigned tb = std::min<unsigned>(groups / (per0 + per1), P->tokens);
    const unsigned tiles = (P->tokens + tb - 1) / tb;
    const double time = (double)((tiles + slots - 1) / slots) * (m + 1.5);
    if (best == 0 || time < best) {
      best = time;
      P->side[0].per = per0;
      P->side[1].per = per1;
      P->heads = m;
      P->tb = tb;
      P->tiles = tiles;
    }
    if (m > 64 && best > 0) break;
  }
  return best > 0;
}

template <typename T, int G>
cudaError_t launch_g(NormRopeParams& P, bool backward, cudaStream_t stream, unsigned* blocks) {
  constexpr int groups = kThreads / G;
  const int slots = (backward ? 2 : 3) * num_sms();  // blocks that run at a time
  if (!share_groups(groups, slots, &P)) return cudaErrorInvalidValue;
  const unsigned grid = backward ? std::min<unsigned>(P.tiles, slots) : P.tiles;
  size_t smem = (size_t)P.tb * (Vec<T>::V / 2) * G * 16;
  if (backward) smem = std::max(smem, (size_t)groups * P.D * sizeof(float));
  *blocks = grid;
  ProfileScope ps(stream, backward ? kKernNormRopeBwd : kKernNormRope);
  void (*kernel)(const NormRopeParams) =
      backward ? (P.interleaved ? gdn_norm_rope_bwd_kernel<T, G, true> : gdn_norm_rope_bwd_kernel<T, G, false>)
               : (P.interleaved ? gdn_norm_rope_kernel<T, G, true> : gdn_norm_rope_kernel<T, G, false>);
  const cudaError_t e = launch_after(kernel, grid, kThreads, smem, stream, P);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename T>
cudaError_t launch_t(NormRopeParams& P, bool backward, cudaStream_t stream, unsigned* blocks) {
  // D / 16 pieces of two for bf16 (1 to 8), D / 8 for fp32 (2 to 16)
  constexpr int kLeast = Vec<T>::V == 8 ? 1 : 2;
  switch (lanes_per_row(P.D, Vec<T>::V) / kLeast) {
    case 1: return launch_g<T, kLeast>(P, backward, stream, blocks);
    case 2: return launch_g<T, 2 * kLeast>(P, backward, stream, blocks);
    case 4: return launch_g<T, 4 * kLeast>(P, backward, stream, blocks);
    default: return launch_g<T, 8 * kLeast>(P, backward, stream, blocks);
  }
}

// A [B, T, H, D] view with its strides in bytes (0 where the extent is at most 1), for
// the overlap checks.
struct View {
  const uint8_t* p;
  long long bs, ts, row;  // bytes; row = H * D elements
  int B, T;
  Range range() const {
    return {(uintptr_t)p, (uintptr_t)p + (B - 1) * bs + (T - 1) * ts + row};
  }
};

// A stride that is never stepped by is not looked at.
long long used(long long stride, int extent) { return extent > 1 ? stride : 0; }

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
  return a.p == b.p && a.bs == b.bs && a.ts == b.ts;
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
  long long pos_bs = 0;
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
    pos_bs = used(r->position_batch_stride, c.B);
    if (pos_bs < 0 || pos_bs > kMaxStride) return GDN_ERR_INVALID_ARG;
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
    const long long bs = used(v->batch_stride, c.B), ts = used(v->token_stride, c.T);
    if (bs < 0 || bs > kMaxStride || ts < 0 || ts > kMaxStride) return false;
    if ((bs * es) % 16 || (ts * es) % 16) return false;
    *to = {static_cast<const uint8_t*>(v->data), bs * es, ts * es, (long long)c.H[s] * c.D * es, c.B, c.T};
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
    read(r->positions, (size_t)((c.B - 1) * pos_bs + (long long)c.T * r->axes) *
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
    S.x = in[s].p;
    S.x_bs = in[s].bs / es;
    S.x_ts = in[s].ts / es;
    S.out = const_cast<uint8_t*>(out[s].p);
    S.o_bs = out[s].bs / es;
    S.o_ts = out[s].ts / es;
    if (c.backward) {
      S.dy = dy[s].p;
      S.dy_bs = dy[s].bs / es;
      S.dy_ts = dy[s].ts / es;
    }
  }
  P.T = c.T;
  P.D = c.D;
  P.R = R;
  P.tokens = (unsigned)c.B * c.T;
  P.eps = c.eps;
  P.norm = c.norm;
  P.inverse = c.inverse;
  if (r) {
    P.pos = r->positions;
    P.freq = r->inv_freq;
    P.pos_bs = pos_bs;
    P.pos_wide = r->position_bytes == 8;
    P.axes = r->axes;
    P.sec1 = r->section[0];
    P.sec2 = P.sec1 + (r->axes > 1 ? r->section[1] : R);
    P.amplitude = r->amplitude;
    P.interleaved = r->layout == GDN_ROPE_INTERLEAVED;
  }
  unsigned blocks = 0;
  if (!c.backward) {
    const cudaError_t e = c.dtype == GDN_BF16 ? launch_t<__nv_bfloat16>(P, false, stream, &blocks)
                                              : launch_t<float>(P, false, stream, &blocks);
    return finish(stream, e, nullptr);
  }
  OpScratch sc;
  unsigned int* err = nullptr;
  // two rows of partial sums per block, at most two blocks an SM
  const gdn_status st = op_scratch(dev, stream, (size_t)4 * num_sms() * c.D * sizeof(float), &err, &sc);
  if (st != GDN_OK) return st;
  P.partial = static_cast<float*>(sc.p);
  cudaError_t e = c.dtype == GDN_BF16 ? launch_t<__nv_bfloat16>(P, true, stream, &blocks)
                                      : launch_t<float>(P, true, stream, &blocks);
  if (e == cudaSuccess && (c.dw[0] || c.dw[1])) {
    ProfileScope ps(stream, kKernNormRopeReduce);
    e = launch_after(gdn_norm_rope_reduce_kernel, 2 * (c.D / kRedCols), kRedCols * kRedRows, 0, stream,
                     (const float*)P.partial, blocks, c.D, c.dw[0], c.dw[1]);
    if (e == cudaSuccess) count_launches(1);
  }
  const cudaError_t f = op_scratch_done(&sc);
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
