// torch_bind.cpp -- the torch side of the softmax blocks' operators, compiled.
//
// Argument marshalling only, as in api.py: checks that it was handed CUDA tensors
// of the expected shapes, types and strides, allocates outputs the caller did not
// supply, and passes pointers, sizes and the current CUDA stream to libgdn.so's C
// entry points, whose addresses api.py hands over once.  It is compiled because
// these operators' small calls take a few microseconds of GPU time: the same
// marshalling in Python took 9 of a call's 18.5 us (queries and keys of one token,
// normalised and rotated); now the call takes 6.6 us, 2.1 of them for its two new
// tensors and 2 for the launch.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <array>
#include <string>
#include <tuple>
#include <vector>

#include "gdn.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;
namespace py = pybind11;

decltype(&gdn_rope) f_rope = nullptr;
decltype(&gdn_qk_norm_rope) f_norm_rope = nullptr;
decltype(&gdn_qk_norm_rope_backward) f_norm_rope_bwd = nullptr;
decltype(&gdn_cross_attention) f_cross = nullptr;
decltype(&gdn_cross_attention_backward) f_cross_bwd = nullptr;

void connect(const py::dict& at) {
  auto get = [&](const char* name, auto& f) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(at[name].cast<uintptr_t>());
  };
  get("gdn_rope", f_rope);
  get("gdn_qk_norm_rope", f_norm_rope);
  get("gdn_qk_norm_rope_backward", f_norm_rope_bwd);
  get("gdn_cross_attention", f_cross);
  get("gdn_cross_attention_backward", f_cross_bwd);
}

// Calls an entry point without the interpreter's lock: it may wait, for another thread's
// launches on the stream or for room in its queue, and what it waits for may need Python.
template <typename... P, typename... A>
int enqueue(gdn_status (*entry)(P...), A... args) {
  py::gil_scoped_release release;
  return entry(args...);
}

using Shape = std::array<int64_t, 4>;

// Refusals, as Python's ValueError and TypeError.  Messages are put together as
// strings, without streams.
template <typename... A>
std::string join(const A&... parts) {
  std::string s;
  (s.append(parts), ...);
  return s;
}
#define REFUSE_VALUE(ok, ...)                              \
  do {                                                     \
    if (!(ok)) throw py::value_error(join(__VA_ARGS__));   \
  } while (0)
#define REFUSE_TYPE(ok, ...)                               \
  do {                                                     \
    if (!(ok)) throw py::type_error(join(__VA_ARGS__));    \
  } while (0)

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

void check(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
  REFUSE_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
  REFUSE_TYPE(t.scalar_type() == dtype, name, " must be ", c10::toString(dtype), ", got ",
              c10::toString(t.scalar_type()));
  REFUSE_VALUE(t.sizes() == shape, name, " must have shape ", text(shape), ", got ", text(t.sizes()));
}

void check_contiguous(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
  check(t, name, dtype, shape);
  REFUSE_VALUE(t.is_contiguous(), name, " must be contiguous");
}

// A [B, T, H, D] tensor whose heads and features are contiguous.
gdn_rows rows(const Tensor& t, const char* name, at::ScalarType dtype, const Shape& s) {
  check(t, name, dtype, s);
  REFUSE_VALUE((t.stride(3) == 1 && (t.stride(2) == s[3] || s[2] <= 1)) || t.numel() == 0, name,
                    " must have contiguous heads and features");
  return {t.data_ptr(), s[0] > 1 ? t.stride(0) : 0, s[1] > 1 ? t.stride(1) : 0};
}

// A new contiguous tensor on the device of `like`, straight from the allocator: the
// dispatcher's way to it takes half a microsecond more.
Tensor fresh(const Tensor& like, at::ScalarType type, at::IntArrayRef shape) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// The caller's tensor, or a new one of the type of `like`.
Tensor or_new(const OptTensor& t, const Tensor& like, at::IntArrayRef shape) {
  return t ? *t : fresh(like, like.scalar_type(), shape);
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

const float* weight(const OptTensor& w, const char* name, int64_t D) {
  if (!w) return nullptr;
  check_contiguous(*w, name, at::kFloat, {D});
  return w->data_ptr<float>();
}

struct Rotation {
  gdn_rotation r;
  bool on;
  const gdn_rotation* get() const { return on ? &r : nullptr; }
};

Rotation rotation(const OptTensor& positions, const OptTensor& inv_freq,
                  const std::optional<std::vector<int>>& sections, const std::string& layout, double amplitude,
                  int64_t B, int64_t T) {
  Rotation out = {};
  if (!positions && !inv_freq) return out;
  REFUSE_VALUE(positions && inv_freq, "positions and inv_freq go together");
  REFUSE_VALUE(layout == "half" || layout == "interleaved", "layout must be 'half' or 'interleaved'");
  const Tensor &p = *positions, &f = *inv_freq;
  const int64_t pairs = f.numel();
  const int64_t axes = sections ? (int64_t)sections->size() : 1;
  REFUSE_VALUE(axes >= 1 && axes <= 3, "sections must name 1 to 3 position axes");
  REFUSE_VALUE(p.is_cuda(), "positions must be a CUDA tensor");
  REFUSE_VALUE(f.is_cuda(), "inv_freq must be a CUDA tensor");
  REFUSE_TYPE(f.scalar_type() == at::kDouble && f.dim() == 1 && f.is_contiguous(),
                   "inv_freq must be a contiguous float64 vector");
  REFUSE_TYPE(p.scalar_type() == at::kInt || p.scalar_type() == at::kLong, "positions must be int32 or int64");
  // [T], [B, T] (one axis), [T, axes], [B, T, axes]
  const bool one = axes == 1 && ((p.dim() == 1 && p.size(0) == T) || (p.dim() == 2 && p.size(0) == B && p.size(1) == T));
  const int64_t d = p.dim() + (one ? 1 : 0);  // dimensions with the axes
  REFUSE_VALUE(one || (d == 2 && p.size(0) == T && p.size(1) == axes) ||
                        (d == 3 && p.size(0) == B && p.size(1) == T && p.size(2) == axes),
                    "positions must be [T], [B, T] (one axis), [T, ", std::to_string(axes), "] or [B, T, ",
               std::to_string(axes), "], got ", text(p.sizes()));
  const int64_t at_t = d == 3 ? 1 : 0;
  REFUSE_VALUE(B * T == 0 || ((axes == 1 || p.stride(at_t + 1) == 1) && (T == 1 || p.stride(at_t) == axes)),
                    "positions must be contiguous over tokens and axes");
  gdn_rotation& r = out.r;
  out.on = true;
  r.positions = p.data_ptr();
  r.inv_freq = f.data_ptr<double>();
  r.position_batch_stride = d == 3 && B > 1 ? p.stride(0) : 0;
  r.position_bytes = p.scalar_type() == at::kInt ? 4 : 8;
  r.axes = (int)axes;
  for (int64_t i = 0; i < axes; ++i) r.section[i] = sections ? (*sections)[i] : (int)pairs;
  r.rot_dim = (int)(2 * pairs);
  r.layout = layout == "half" ? GDN_ROPE_HALF : GDN_ROPE_INTERLEAVED;
  r.amplitude = (float)amplitude;
  return out;
}

// Sizes and types of q and k (k may be missing).
struct Heads {
  Shape q, k;
  int B, T, Hq, Hk, D;
  at::ScalarType type;
  gdn_dtype dtype;
};
Heads heads(const Tensor& q, const OptTensor& k) {
  REFUSE_VALUE(q.dim() == 4 && (!k || k->dim() == 4), "q, k must be [B,T,H,D]");
  Heads h;
  h.type = q.scalar_type();
  REFUSE_TYPE(h.type == at::kBFloat16 || h.type == at::kFloat, "q, k must be bfloat16 or float32, got ", c10::toString(h.type));
  h.dtype = h.type == at::kFloat ? GDN_F32 : GDN_BF16;
  h.q = {q.size(0), q.size(1), q.size(2), q.size(3)};
  h.k = {q.size(0), q.size(1), k ? k->size(2) : 0, q.size(3)};
  for (int64_t n : {h.q[0], h.q[1], h.q[2], h.q[3], h.k[2]})
    REFUSE_VALUE(n < (int64_t(1) << 31), "sizes must be below 2^31");
  h.B = (int)h.q[0];
  h.T = (int)h.q[1];
  h.Hq = (int)h.q[2];
  h.Hk = (int)h.k[2];
  h.D = (int)h.q[3];
  return h;
}

using Sections = std::optional<std::vector<int>>;

std::tuple<int, Tensor, OptTensor> rope(const Tensor& q, const OptTensor& k, const OptTensor& positions,
                                        const OptTensor& inv_freq, const Sections& sections,
                                        const std::string& layout, double amplitude, bool inverse,
                                        const OptTensor& q_out, const OptTensor& k_out) {
  const Heads h = heads(q, k);
  const gdn_rows vq = rows(q, "q", h.type, h.q);
  const gdn_rows vk = k ? rows(*k, "k", h.type, h.k) : gdn_rows{};
  const Rotation r = rotation(positions, inv_freq, sections, layout, amplitude, h.B, h.T);
  REFUSE_VALUE(r.on, "rope needs positions and inv_freq");
  const Tensor oq = or_new(q_out, q, h.q);
  const gdn_rows wq = rows(oq, "q_out", h.type, h.q);
  OptTensor ok;
  gdn_rows wk = {};
  if (k) {
    ok = or_new(k_out, q, h.k);
    wk = rows(*ok, "k_out", h.type, h.k);
  }
  const int st = enqueue(f_rope, &vq, k ? &vk : nullptr, r.get(), inverse, &wq, k ? &wk : nullptr, h.B, h.T, h.Hq, h.Hk, h.D,
                        h.dtype, stream_of(q));
  return {st, oq, ok};
}

std::tuple<int, Tensor, OptTensor> qk_norm_rope(const Tensor& q, const OptTensor& k, const OptTensor& q_weight,
                                                const OptTensor& k_weight, const OptTensor& positions,
                                                const OptTensor& inv_freq, double eps, const Sections& sections,
                                                const std::string& layout, double amplitude,
                                                const OptTensor& q_out, const OptTensor& k_out) {
  const Heads h = heads(q, k);
  const gdn_rows vq = rows(q, "q", h.type, h.q);
  const gdn_rows vk = k ? rows(*k, "k", h.type, h.k) : gdn_rows{};
  const float *gq = weight(q_weight, "q_weight", h.D), *gk = weight(k_weight, "k_weight", h.D);
  const Rotation r = rotation(positions, inv_freq, sections, layout, amplitude, h.B, h.T);
  const Tensor oq = or_new(q_out, q, h.q);
  const gdn_rows wq = rows(oq, "q_out", h.type, h.q);
  OptTensor ok;
  gdn_rows wk = {};
  if (k) {
    ok = or_new(k_out, q, h.k);
    wk = rows(*ok, "k_out", h.type, h.k);
  }
  const int st = enqueue(f_norm_rope, &vq, k ? &vk : nullptr, gq, gk, r.get(), &wq, k ? &wk : nullptr, h.B, h.T, h.Hq, h.Hk,
                             h.D, (float)eps, h.dtype, stream_of(q));
  return {st, oq, ok};
}

std::tuple<int, Tensor, OptTensor, Tensor, OptTensor> qk_norm_rope_backward(
    const Tensor& q, const OptTensor& k, const OptTensor& q_weight, const OptTensor& k_weight, const Tensor& dq_out,
    const OptTensor& dk_out, const OptTensor& positions, const OptTensor& inv_freq, double eps,
    const Sections& sections, const std::string& layout, double amplitude, const OptTensor& dq, const OptTensor& dk) {
  const Heads h = heads(q, k);
  const gdn_rows vq = rows(q, "q", h.type, h.q);
  const gdn_rows vk = k ? rows(*k, "k", h.type, h.k) : gdn_rows{};
  const float *gq = weight(q_weight, "q_weight", h.D), *gk = weight(k_weight, "k_weight", h.D);
  const Rotation r = rotation(positions, inv_freq, sections, layout, amplitude, h.B, h.T);
  REFUSE_VALUE(!k || dk_out, "dk_out must be given with k");
  const gdn_rows yq = rows(dq_out, "dq_out", h.type, h.q);
  const gdn_rows yk = k ? rows(*dk_out, "dk_out", h.type, h.k) : gdn_rows{};
  const Tensor oq = or_new(dq, q, h.q);
  const gdn_rows wq = rows(oq, "dq", h.type, h.q);
  const Tensor dwq = fresh(q, at::kFloat, {h.D});
  OptTensor ok, dwk;
  gdn_rows wk = {};
  if (k) {
    ok = or_new(dk, q, h.k);
    wk = rows(*ok, "dk", h.type, h.k);
    dwk = fresh(q, at::kFloat, {h.D});
  }
  const int st = enqueue(f_norm_rope_bwd, &vq, k ? &vk : nullptr, gq, gk, r.get(), &yq, k ? &yk : nullptr, &wq,
                                 k ? &wk : nullptr, dwq.data_ptr<float>(), k ? dwk->data_ptr<float>() : nullptr, h.B,
                                 h.T, h.Hq, h.Hk, h.D, (float)eps, h.dtype, stream_of(q));
  return {st, oq, ok, dwq, dwk};
}

// Sizes and views of a cross-attention call.
struct Cross {
  Shape q, k;
  gdn_rows vq, vk, vv;
  const unsigned char* mask;
  int64_t mask_bs;
  float scale;
};
Cross cross_args(const Tensor& q, const Tensor& k, const Tensor& v, const OptTensor& mask,
                 std::optional<double> scale) {
  REFUSE_VALUE(q.dim() == 4 && k.dim() == 4, "q must be [B,Tq,Hq,D] and k, v [B,S,Hk,D]");
  REFUSE_TYPE(q.scalar_type() == at::kBFloat16, "q, k, v must be bfloat16, got ", c10::toString(q.scalar_type()));
  Cross c = {};
  c.q = {q.size(0), q.size(1), q.size(2), q.size(3)};
  c.k = {q.size(0), k.size(1), k.size(2), q.size(3)};
  for (int64_t n : {c.q[0], c.q[1], c.q[2], c.q[3], c.k[1], c.k[2]})
    REFUSE_VALUE(n < (int64_t(1) << 31), "sizes must be below 2^31");
  c.vq = rows(q, "q", at::kBFloat16, c.q);
  c.vk = rows(k, "k", at::kBFloat16, c.k);
  c.vv = rows(v, "v", at::kBFloat16, c.k);
  if (mask) {
    REFUSE_VALUE(mask->is_cuda(), "key_mask must be a CUDA tensor");
    REFUSE_TYPE(mask->scalar_type() == at::kBool || mask->scalar_type() == at::kByte,
                     "key_mask must be bool or uint8, got ", c10::toString(mask->scalar_type()));
    REFUSE_VALUE(mask->dim() == 2 && mask->size(0) == c.q[0] && mask->size(1) == c.k[1],
                      "key_mask must have shape ", text({c.q[0], c.k[1]}), ", got ", text(mask->sizes()));
    REFUSE_VALUE(c.k[1] <= 1 || mask->stride(1) == 1, "key_mask must be contiguous over the keys");
    c.mask = static_cast<const unsigned char*>(mask->data_ptr());
    c.mask_bs = c.q[0] > 1 ? mask->stride(0) : 0;
  }
  c.scale = (float)(scale ? *scale : c.q[3] ? 1.0 / std::sqrt((double)c.q[3]) : 1.0);
  return c;
}

std::tuple<int, Tensor, OptTensor> cross_attention(const Tensor& q, const Tensor& k, const Tensor& v,
                                                   const OptTensor& mask, std::optional<double> scale,
                                                   const OptTensor& out, bool want_lse) {
  const Cross c = cross_args(q, k, v, mask, scale);
  const Tensor o = or_new(out, q, c.q);
  if (out) check_contiguous(o, "out", at::kBFloat16, c.q);
  OptTensor lse;
  if (want_lse) lse = fresh(q, at::kFloat, {c.q[0], c.q[2], c.q[1]});
  const int st = enqueue(f_cross, &c.vq, &c.vk, &c.vv, c.mask, c.mask_bs, o.data_ptr(), lse ? lse->data_ptr<float>() : nullptr,
                         (int)c.q[0], (int)c.q[1], (int)c.k[1], (int)c.q[2], (int)c.k[2], (int)c.q[3], c.scale,
                         GDN_BF16, stream_of(q));
  return {st, o, lse};
}

std::tuple<int, Tensor, Tensor, Tensor> cross_attention_backward(const Tensor& q, const Tensor& k, const Tensor& v,
                                                                 const Tensor& out, const Tensor& lse,
                                                                 const Tensor& d_out, const OptTensor& mask,
                                                                 std::optional<double> scale) {
  const Cross c = cross_args(q, k, v, mask, scale);
  check_contiguous(out, "out", at::kBFloat16, c.q);
  check_contiguous(lse, "lse", at::kFloat, {c.q[0], c.q[2], c.q[1]});
  check_contiguous(d_out, "d_out", at::kBFloat16, c.q);
  const Tensor dq = fresh(q, at::kBFloat16, c.q), dk = fresh(q, at::kBFloat16, c.k), dv = fresh(q, at::kBFloat16, c.k);
  const int st = enqueue(f_cross_bwd, &c.vq, &c.vk, &c.vv, c.mask, c.mask_bs, out.data_ptr(), lse.data_ptr<float>(),
                             d_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), (int)c.q[0], (int)c.q[1],
                             (int)c.k[1], (int)c.q[2], (int)c.k[2], (int)c.q[3], c.scale, GDN_BF16, stream_of(q));
  return {st, dq, dk, dv};
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("connect", &connect);
  m.def("rope", &rope);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_backward", &qk_norm_rope_backward);
  m.def("cross_attention", &cross_attention);
  m.def("cross_attention_backward", &cross_attention_backward);
}
