// cross_api.cu -- the cross-attention entry points (include/gdn.h): host-side
// checks, tensor maps, scratch and launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr long long kMaxStride = 1ll << 36;  // elements: TMA strides stay below 2^40 bytes

// Whether a view is one that the TMA maps can take: data aligned to 16 bytes, strides
// in range and multiples of 16 bytes.  A stride that is never stepped by is not
// looked at, and comes back as 0.
bool good_view(const gdn_rows* v, int B, int T, gdn_rows* to) {
  if (!v || !v->data || !aligned16(v->data)) return false;
  *to = {v->data, B > 1 ? v->batch_stride : 0, T > 1 ? v->token_stride : 0};
  if (to->batch_stride < 0 || to->batch_stride > kMaxStride || to->token_stride < 0 || to->token_stride > kMaxStride)
    return false;
  return to->batch_stride % 8 == 0 && to->token_stride % 8 == 0 && (T <= 1 || to->token_stride != 0);
}

Range range_of_view(const gdn_rows& v, int B, int T, long long row) {
  if (B == 0 || T == 0) return {0, 0};
  const uintptr_t lo = (uintptr_t)v.data;
  return {lo, lo + (uintptr_t)(2 * ((B - 1) * v.batch_stride + (T - 1) * v.token_stride + row))};
}

struct Checked {
  CrossCall c;
  Range reads[8];  // at most q, k, v, mask, out, d_out, lse
  int nreads;
  const void* ptrs[16];
  int nptrs;
  bool nothing;  // nothing to compute
};

// The checks both directions share, none of which makes a CUDA call.
gdn_status check_inputs(const gdn_rows* q, const gdn_rows* k, const gdn_rows* v, const unsigned char* mask,
                        long long mask_bs, int B, int Tq, int S, int Hq, int Hk, int D, float scale,
                        gdn_dtype dtype, void* stream, Checked* o) {
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (B < 0 || Tq < 0 || S < 0 || Hq < 0 || Hk < 0 || D < 0) return GDN_ERR_INVALID_ARG;
  // 0 times the -infinity of a masked score is no number
  if (!(scale > 0.f) || !std::isnormal(scale) || !std::isnormal(scale * 1.5f)) return GDN_ERR_INVALID_ARG;
  if (B <= 1) mask_bs = 0;  // not stepped by
  if (mask_bs < 0 || mask_bs > kMaxStride) return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_BF16 || !supported_dim(D)) return GDN_ERR_UNSUPPORTED;
  if (Hq > 0 && (Hk == 0 || Hq % Hk)) return GDN_ERR_INVALID_ARG;
  if (Hq > 0 && Hq / Hk > 128) return GDN_ERR_UNSUPPORTED;
  // one-dimensional grids over (batch, head, tile): query and key tiles are at
  // least a token each
  if (S > (1 << 30) || Tq > (1 << 30) || (double)B * Hq * (Tq / 16.0 + S / 16.0 + 2.0) > 1.0e9)
    return GDN_ERR_UNSUPPORTED;
  CrossCall& c = o->c;
  c = CrossCall{};
  c.B = B; c.Tq = Tq; c.S = S; c.Hq = Hq; c.Hk = Hk; c.D = D;
  c.scale = scale;
  c.stream = static_cast<cudaStream_t>(stream);
  o->nreads = o->nptrs = 0;
  o->nothing = B == 0 || Hq == 0;
  if (o->nothing) return GDN_OK;
  if (Tq > 0) {
    if (!good_view(q, B, Tq, &c.q)) return GDN_ERR_INVALID_ARG;
    if (B == 1) c.q.batch_stride = 1;  // not used; nonzero, so that it is no broadcast
    o->reads[o->nreads++] = range_of_view(c.q, B, Tq, (long long)Hq * D);
    o->ptrs[o->nptrs++] = q->data;
  }
  if (S > 0) {
    if (!good_view(k, B, S, &c.k) || !good_view(v, B, S, &c.v)) return GDN_ERR_INVALID_ARG;
    if (B == 1) c.k.batch_stride = c.v.batch_stride = 1;
    o->reads[o->nreads++] = range_of_view(c.k, B, S, (long long)Hk * D);
    o->reads[o->nreads++] = range_of_view(c.v, B, S, (long long)Hk * D);
    o->ptrs[o->nptrs++] = k->data;
    o->ptrs[o->nptrs++] = v->data;
    if (mask) {
      c.mask = mask;
      c.mask_bs = mask_bs;
      o->reads[o->nreads++] = range_of(mask, (size_t)((B - 1) * mask_bs + S));
      o->ptrs[o->nptrs++] = mask;
    }
  }
  return GDN_OK;
}

gdn_status check_device(const Checked& o, int* dev) {
  if (cudaGetDevice(dev) != cudaSuccess) {
    cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  for (int i = 0; i < o.nptrs; ++i) {
    const gdn_status st = check_device_pointer(o.ptrs[i], *dev);
    if (st != GDN_OK) return st;
  }
  cudaGetLastError();
  return GDN_OK;
}

using EncodeTiledFn = decltype(&cuTensorMapEncodeTiled);

// The driver's tensor-map encoder, looked up once.
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

}  // namespace

bool make_heads_map(CUtensorMap* m, const void* base, int nb, int T, int Hk, int G, int D,
                    long long batch_stride, long long token_stride, int box_tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  // a stride that is never stepped by still has to be a valid one
  const cuuint64_t ts = T > 1 ? (cuuint64_t)token_stride * 2 : (cuuint64_t)Hk * G * D * 2;
  const cuuint64_t bs = nb > 1 ? (cuuint64_t)batch_stride * 2 : ts * (cuuint64_t)T;
  const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)T, (cuuint64_t)Hk, (cuuint64_t)nb};
  const cuuint64_t strides[4] = {(cuuint64_t)D * 2, ts, (cuuint64_t)G * D * 2, bs};
  const cuuint32_t box[5] = {64, (cuuint32_t)G, (cuuint32_t)box_tokens, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdn

extern "C" {

gdn_status gdn_cross_attention(const gdn_rows* q, const gdn_rows* k, const gdn_rows* v,
                               const unsigned char* key_mask, long long mask_batch_stride, void* out,
                               float* lse, int B, int Tq, int S, int Hq, int Hk, int D, float scale,
                               gdn_dtype dtype, void* stream) {
  using namespace gdn;
  Checked o;
  gdn_status st = check_inputs(q, k, v, key_mask, mask_batch_stride, B, Tq, S, Hq, Hk, D, scale, dtype,
                               stream, &o);
  if (st != GDN_OK || o.nothing || Tq == 0) return st;
  if (!out || !aligned16(out) || (lse && !aligned16(lse))) return GDN_ERR_INVALID_ARG;
  const Range ro = range_of(out, (size_t)B * Tq * Hq * D * 2);
  const Range rl = range_of(lse, lse ? (size_t)B * Tq * Hq * 4 : 0);
  if (overlaps(ro, rl)) return GDN_ERR_ALIAS;
  for (int i = 0; i < o.nreads; ++i)
    if (overlaps(ro, o.reads[i]) || overlaps(rl, o.reads[i])) return GDN_ERR_ALIAS;
  o.ptrs[o.nptrs++] = out;
  if (lse) o.ptrs[o.nptrs++] = lse;
  int dev = 0;
  st = check_device(o, &dev);
  if (st != GDN_OK) return st;
  CrossCall& c = o.c;
  c.out = out;
  c.lse = lse;
  OpScratch sc;
  st = op_scratch(dev, c.stream, cross_workspace_bytes(c), &c.err, &sc);
  if (st != GDN_OK) return st;
  c.limit = current_wait_limit();
  const cudaError_t e = launch_cross(c, sc.p);
  const cudaError_t f = op_scratch_done(&sc);
  return finish(c.stream, e == cudaSuccess ? f : e, c.err);
}

gdn_status gdn_cross_attention_backward(const gdn_rows* q, const gdn_rows* k, const gdn_rows* v,
                                        const unsigned char* key_mask, long long mask_batch_stride,
                                        const void* out, const float* lse, const void* d_out, void* dq,
                                        void* dk, void* dv, int B, int Tq, int S, int Hq, int Hk, int D,
                                        float scale, gdn_dtype dtype, void* stream) {
  using namespace gdn;
  Checked o;
  gdn_status st = check_inputs(q, k, v, key_mask, mask_batch_stride, B, Tq, S, Hq, Hk, D, scale, dtype,
                               stream, &o);
  if (st != GDN_OK) return st;
  const size_t qbytes = (size_t)B * Tq * Hq * D * 2, kbytes = (size_t)B * S * Hk * D * 2;
  if (qbytes == 0 && kbytes == 0) return GDN_OK;
  const size_t lbytes = (size_t)B * Tq * Hq * 4;
  const struct {
    const void* p;
    size_t bytes;
    bool written;
  } bufs[] = {{out, qbytes, false}, {d_out, qbytes, false}, {lse, lbytes, false},
              {dq, qbytes, true},   {dk, kbytes, true},     {dv, kbytes, true}};
  for (const auto& x : bufs) {
    if (x.bytes == 0) continue;
    if (!x.p || !aligned16(x.p)) return GDN_ERR_INVALID_ARG;
    if (!x.written) o.reads[o.nreads++] = range_of(x.p, x.bytes);
    o.ptrs[o.nptrs++] = x.p;
  }
  for (int i = 3; i < 6; ++i) {
    const Range w = range_of(bufs[i].p, bufs[i].bytes);
    for (int r = 0; r < o.nreads; ++r)
      if (overlaps(w, o.reads[r])) return GDN_ERR_ALIAS;
    for (int x = i + 1; x < 6; ++x)
      if (overlaps(w, range_of(bufs[x].p, bufs[x].bytes))) return GDN_ERR_ALIAS;
  }
  int dev = 0;
  st = check_device(o, &dev);
  if (st != GDN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (qbytes == 0 || kbytes == 0) {  // nothing attends: what there is of gradients is zero
    cudaError_t e = cudaSuccess;
    if (qbytes) e = cudaMemsetAsync(dq, 0, qbytes, s);
    if (kbytes) e = cudaMemsetAsync(dk, 0, kbytes, s);
    if (kbytes && e == cudaSuccess) e = cudaMemsetAsync(dv, 0, kbytes, s);
    return finish(s, e, nullptr);
  }
  CrossCall& c = o.c;
  c.out = const_cast<void*>(out);
  c.lse = const_cast<float*>(lse);
  c.d_out = d_out;
  c.dq = dq;
  c.dk = dk;
  c.dv = dv;
  OpScratch sc;
  st = op_scratch(dev, c.stream, cross_backward_workspace_bytes(c), &c.err, &sc);
  if (st != GDN_OK) return st;
  c.limit = current_wait_limit();
  const cudaError_t e = launch_cross_backward(c, sc.p);
  const cudaError_t f = op_scratch_done(&sc);
  return finish(c.stream, e == cudaSuccess ? f : e, c.err);
}

}  // extern "C"
