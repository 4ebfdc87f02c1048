// Python binding of the operators of a serving and a training step (argument checks,
// output tensors and the call of the C ABI in include/fa.h; no arithmetic).
//
// These calls run once a layer and a step, at sizes where the kernels take a few
// microseconds: in Python the same checks and allocations cost 11 to 20 us a call, here 2
// to 5.  The library is not linked: fa.py hands over the addresses of its entry points, so
// that whatever build it has loaded is the one that runs.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>

#include <cmath>
#include <cstdint>
#include <optional>
#include <sstream>
#include <string>
#include <tuple>

#include "fa.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

struct {
  decltype(&fa_qk_norm_rope) qk_norm_rope, qk_norm_rope_fp16;
  decltype(&fa_qk_norm_rope_bwd) qk_norm_rope_bwd, qk_norm_rope_bwd_fp16;
  decltype(&fa_append_paged) append_paged;
  decltype(&fa_extend_pages) extend_pages;
  decltype(&fa_decode_shared_prefix) decode_shared_prefix;
  decltype(&fa_last_error_string) last_error_string;
} api;
PyObject* error_class = nullptr;   // fa.FAError(code, where, message)

[[noreturn]] void refuse(int code, const char* where, const std::string& message) {
  py::object error = py::reinterpret_borrow<py::object>(error_class)(code, where, message);
  PyErr_SetObject(error_class, error.ptr());
  throw py::error_already_set();
}
void check(int code, const char* entry) {
  if (code != FA_OK) refuse(code, entry, api.last_error_string());
}
// A size as the C ABI takes it.
int size(const char* where, int64_t n) {
  if (n > INT32_MAX) refuse(FA_ERR_UNSUPPORTED, where, "a size does not fit 31 bits");
  return static_cast<int>(n);
}

std::string text(at::IntArrayRef sizes) {
  std::ostringstream s;
  s << sizes;
  return s.str();
}
// Shapes are compared with what the call's other tensors ask for; -1 is any size.
void shape(const char* where, const char* name, const Tensor& t,
           std::initializer_list<int64_t> want) {
  const at::IntArrayRef have = t.sizes(), need(want.begin(), want.size());
  bool same = have.size() == need.size();
  for (size_t i = 0; same && i < need.size(); ++i) same = need[i] == -1 || need[i] == have[i];
  if (!same)
    refuse(FA_ERR_INVALID_ARG, where,
           std::string(name) + " must have shape " + text(need) + ", not " + text(have));
}
void dtype(const char* where, const char* name, const Tensor& t, at::ScalarType want) {
  if (t.scalar_type() != want)
    refuse(FA_ERR_INVALID_ARG, where, std::string(name) + " must be " + at::toString(want) +
                                          ", not " + at::toString(t.scalar_type()));
}

// The kernels run on the current device: refuses tensors elsewhere.
struct Device {
  const char* where;
  int index;
  Device(const char* w, const Tensor& first) : where(w), index(-1) {
    if (first.is_cuda()) index = first.get_device();
    if (index < 0 || index != c10::cuda::current_device()) elsewhere();
  }
  void operator()(const Tensor& t) const {
    if (!t.is_cuda() || t.get_device() != index) elsewhere();
  }
  void operator()(const Maybe& t) const {
    if (t) (*this)(*t);
  }
  [[noreturn]] void elsewhere() const {
    refuse(FA_ERR_INVALID_ARG, where, "tensors must live on the current CUDA device");
  }
  fa_stream_t stream() const {
    return reinterpret_cast<fa_stream_t>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
  }
};

template <class T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <class T = void>
T* ptr(const Maybe& t) {
  return t ? ptr<T>(*t) : nullptr;
}
bool at16(const Tensor& t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0; }
// t contiguous and at a 16-byte boundary, copied where it is not.
Tensor aligned(const Tensor& t) {
  const Tensor c = t.contiguous();
  return at16(c) ? c : c.clone();
}
// (Past the dispatcher: 0.3 us less a tensor, 9.7 and 8.4 us for page extension's five.)
Tensor empty(const Tensor& like, at::ScalarType type, at::IntArrayRef sizes) {
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// t [..., H, D] as the library reads token-major rows: t itself where each token's heads
// are contiguous and one stride leads from token to token (a view of a QKV projection), a
// contiguous copy otherwise; and that stride in elements.
std::pair<Tensor, int64_t> head_rows(const Tensor& t) {
  const int64_t n = t.dim(), H = t.size(n - 2), D = t.size(n - 1);
  int64_t stride = H * D, span = 1;            // no step from token to token: any will do
  bool one = true;
  for (int64_t i = n - 3; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (span == 1)
      stride = t.stride(i);
    else if (t.stride(i) != stride * span)
      one = false;
    span *= t.size(i);
  }
  if (one && t.numel() > 0 && t.stride(n - 1) == 1 && (H == 1 || t.stride(n - 2) == D) &&
      stride >= H * D && stride % 8 == 0 && at16(t))
    return {t, stride};
  return {aligned(t), H * D};
}

// What the norm + rotation calls share.
struct NormRope {
  Tensor q, k, table, positions;
  Maybe q_weight, k_weight, pair_axis;
  int64_t q_stride, k_stride, tokens, Hq, Hkv, D, rot, max_pos, axes;
  bool bf16;
  NormRope(const char* where, const Device& device, const Tensor& q_in, const Tensor& k_in,
           const Maybe& qw, const Maybe& kw, const Tensor& tab, const Tensor& pos,
           const Maybe& axis, int lead) {
    device(k_in);
    device(qw);
    device(kw);
    device(tab);
    device(pos);
    const at::ScalarType type = q_in.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf)
      refuse(FA_ERR_INVALID_ARG, where, "q must be bf16 or fp16");
    bf16 = type == at::kBFloat16;
    dtype(where, "k", k_in, type);
    if (lead == 1) {
      shape(where, "q", q_in, {-1, -1, -1});
      shape(where, "k", k_in, {q_in.size(0), -1, q_in.size(2)});
    } else {
      shape(where, "q", q_in, {-1, -1, -1, -1});
      shape(where, "k", k_in, {q_in.size(0), q_in.size(1), -1, q_in.size(3)});
    }
    tokens = lead == 1 ? q_in.size(0) : q_in.size(0) * q_in.size(1);
    Hq = q_in.size(lead);
    Hkv = k_in.size(lead);
    D = q_in.size(lead + 1);
    for (const auto& [name, w] : {std::pair<const char*, const Maybe&>{"q_weight", qw},
                                  std::pair<const char*, const Maybe&>{"k_weight", kw}})
      if (w) {
        dtype(where, name, *w, type);
        shape(where, name, *w, {D});
      }
    dtype(where, "table", tab, at::kFloat);
    shape(where, "table", tab, {-1, -1});
    max_pos = tab.size(0);
    rot = tab.size(1);
    dtype(where, "positions", pos, at::kInt);
    if (pos.dim() == 1)
      shape(where, "positions", pos, {tokens});
    else
      shape(where, "positions", pos, {-1, tokens});
    axes = pos.dim() == 1 ? 1 : pos.size(0);
    if (axes != 1) {
      if (!axis)
        refuse(FA_ERR_INVALID_ARG, where, "pair_axis is needed with more than one axis");
      device(axis);
      dtype(where, "pair_axis", *axis, at::kByte);
      shape(where, "pair_axis", *axis, {rot / 2});
      pair_axis = axis->contiguous();
    }
    std::tie(q, q_stride) = head_rows(q_in);
    std::tie(k, k_stride) = head_rows(k_in);
    if (qw) q_weight = aligned(*qw);
    if (kw) k_weight = aligned(*kw);
    table = aligned(tab);
    positions = pos.contiguous();
  }
};

Tensor out_rows(const Tensor& q, int64_t B, int64_t N, int64_t H, int64_t D, bool heads_first) {
  return heads_first ? empty(q, q.scalar_type(), {B, H, N, D})
                     : empty(q, q.scalar_type(), {B, N, H, D});
}

std::tuple<Tensor, Tensor> qk_norm_rope(const Tensor& q, const Tensor& k, const Maybe& q_weight,
                                        const Maybe& k_weight, const Tensor& table,
                                        const Tensor& positions, const Maybe& pair_axis, double eps,
                                        bool interleaved, bool heads_first) {
  const char* where = "qk_norm_rope";
  const Device device(where, q);
  const NormRope a(where, device, q, k, q_weight, k_weight, table, positions, pair_axis, 2);
  const int64_t B = q.size(0), N = q.size(1);
  Tensor qo = out_rows(q, B, N, a.Hq, a.D, heads_first);
  Tensor ko = out_rows(q, B, N, a.Hkv, a.D, heads_first);
  auto fn = a.bf16 ? api.qk_norm_rope : api.qk_norm_rope_fp16;
  check(fn(ptr<void>(a.q), ptr<void>(a.k), ptr(a.q_weight), ptr(a.k_weight), ptr<float>(a.table),
           ptr<int32_t>(a.positions), ptr<uint8_t>(a.pair_axis), ptr<void>(qo), ptr<void>(ko),
           size(where, B), size(where, N), size(where, a.Hq),
           size(where, a.Hkv), size(where, a.D), a.q_stride, a.k_stride,
           size(where, a.rot), size(where, a.max_pos), size(where, a.axes),
           interleaved, heads_first, static_cast<float>(eps), device.stream()),
        "fa_qk_norm_rope");
  return {qo, ko};
}

std::tuple<Tensor, Tensor, Maybe, Maybe> qk_norm_rope_backward(
    const Tensor& q, const Tensor& k, const Tensor& dq_out, const Tensor& dk_out,
    const Maybe& q_weight, const Maybe& k_weight, const Tensor& table, const Tensor& positions,
    const Maybe& pair_axis, double eps, bool interleaved, bool heads_first) {
  const char* where = "qk_norm_rope_backward";
  const Device device(where, q);
  const NormRope a(where, device, q, k, q_weight, k_weight, table, positions, pair_axis, 2);
  const int64_t B = q.size(0), N = q.size(1);
  for (const auto& [name, g, H] :
       {std::tuple<const char*, const Tensor&, int64_t>{"dq_out", dq_out, a.Hq},
        std::tuple<const char*, const Tensor&, int64_t>{"dk_out", dk_out, a.Hkv}}) {
    device(g);
    dtype(where, name, g, q.scalar_type());
    if (heads_first)
      shape(where, name, g, {B, H, N, a.D});
    else
      shape(where, name, g, {B, N, H, a.D});
  }
  const Tensor dqo = aligned(dq_out), dko = aligned(dk_out);
  Tensor dq = out_rows(q, B, N, a.Hq, a.D, false), dk = out_rows(q, B, N, a.Hkv, a.D, false);
  Maybe dwq, dwk, scratch;
  if (q_weight) dwq = empty(q, at::kFloat, {a.D});
  if (k_weight) dwk = empty(q, at::kFloat, {a.D});
  if (q_weight || k_weight)
    scratch = empty(q, at::kFloat, {2 * FA_QK_NORM_ROPE_SCRATCH_ROWS * a.D});
  auto fn = a.bf16 ? api.qk_norm_rope_bwd : api.qk_norm_rope_bwd_fp16;
  check(fn(ptr<void>(a.q), ptr<void>(a.k), ptr<void>(dqo), ptr<void>(dko), ptr(a.q_weight),
           ptr(a.k_weight), ptr<float>(a.table), ptr<int32_t>(a.positions),
           ptr<uint8_t>(a.pair_axis), ptr<void>(dq), ptr<void>(dk), ptr<float>(dwq),
           ptr<float>(dwk), ptr<float>(scratch), size(where, B), size(where, N),
           size(where, a.Hq), size(where, a.Hkv), size(where, a.D), a.q_stride,
           a.k_stride, a.Hq * a.D, a.Hkv * a.D, size(where, a.rot),
           size(where, a.max_pos), size(where, a.axes), interleaved, heads_first,
           static_cast<float>(eps), device.stream()),
        "fa_qk_norm_rope_bwd");
  return {dq, dk, dwq, dwk};
}

void cache_shapes(const char* where, const Device& device, const Tensor& kcache,
                  const Tensor& vcache, int64_t Hkv, int64_t D) {
  device(kcache);
  device(vcache);
  dtype(where, "kcache", kcache, at::kBFloat16);
  dtype(where, "vcache", vcache, at::kBFloat16);
  shape(where, "kcache", kcache, {-1, -1, Hkv, D});
  shape(where, "vcache", vcache, {kcache.size(0), kcache.size(1), kcache.size(2), D});
}

Tensor append_paged(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& kcache,
                    const Tensor& vcache, const Tensor& slot_map, const Maybe& q_weight,
                    const Maybe& k_weight, const Tensor& table, const Tensor& positions,
                    const Maybe& pair_axis, double eps, bool interleaved) {
  const char* where = "append_paged";
  const Device device(where, q);
  dtype(where, "q", q, at::kBFloat16);
  const NormRope a(where, device, q, k, q_weight, k_weight, table, positions, pair_axis, 1);
  device(v);
  device(slot_map);
  dtype(where, "v", v, at::kBFloat16);
  dtype(where, "slot_map", slot_map, at::kLong);
  shape(where, "v", v, {a.tokens, a.Hkv, a.D});
  shape(where, "slot_map", slot_map, {a.tokens});
  cache_shapes(where, device, kcache, vcache, a.Hkv, a.D);
  if (!kcache.is_contiguous() || !vcache.is_contiguous())
    refuse(FA_ERR_INVALID_ARG, where,
           "the caches are written in place and must be contiguous");
  const auto [vr, v_stride] = head_rows(v);
  const Tensor slots = slot_map.contiguous();
  Tensor qo = empty(q, at::kBFloat16, {a.tokens, a.Hq, a.D});
  check(api.append_paged(ptr<void>(a.q), ptr<void>(a.k), ptr<void>(vr), ptr(a.q_weight),
                         ptr(a.k_weight), ptr<float>(a.table), ptr<int32_t>(a.positions),
                         ptr<uint8_t>(a.pair_axis), ptr<int64_t>(slots), ptr<void>(qo),
                         ptr<void>(kcache), ptr<void>(vcache), size(where, a.tokens),
                         size(where, a.Hq), size(where, a.Hkv), size(where, a.D),
                         size(where, kcache.size(1)), size(where, kcache.size(0)),
                         a.q_stride, a.k_stride, v_stride, size(where, a.rot),
                         size(where, a.max_pos), size(where, a.axes), interleaved,
                         static_cast<float>(eps), device.stream()),
        "fa_append_paged");
  return qo;
}

std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor> extend_pages(
    const Tensor& block_table, const Tensor& seq_lens, const Tensor& new_lens,
    const Tensor& free_pages, const Tensor& free_count, int64_t num_pages, int64_t max_tokens) {
  const char* where = "extend_pages";
  const Device device(where, block_table);
  shape(where, "block_table", block_table, {-1, -1});
  const int64_t B = block_table.size(0), max_pages = block_table.size(1);
  for (const auto& [name, t, n] :
       {std::tuple<const char*, const Tensor&, int64_t>{"seq_lens", seq_lens, B},
        std::tuple<const char*, const Tensor&, int64_t>{"new_lens", new_lens, B},
        std::tuple<const char*, const Tensor&, int64_t>{"free_pages", free_pages, num_pages},
        std::tuple<const char*, const Tensor&, int64_t>{"free_count", free_count, 1}}) {
    device(t);
    dtype(where, name, t, at::kInt);
    shape(where, name, t, {n});
  }
  dtype(where, "block_table", block_table, at::kInt);
  if (!block_table.is_contiguous())
    refuse(FA_ERR_INVALID_ARG, where, "block_table is written in place and must be contiguous");
  if (max_tokens < 0) refuse(FA_ERR_INVALID_ARG, where, "max_tokens must not be negative");
  const Tensor lens = seq_lens.contiguous(), add = new_lens.contiguous(),
               free = free_pages.contiguous();
  Tensor lens_out = empty(block_table, at::kInt, {B}), cu = empty(block_table, at::kInt, {B + 1}),
         left = empty(block_table, at::kInt, {1}),
         positions = empty(block_table, at::kInt, {max_tokens}),
         slots = empty(block_table, at::kLong, {max_tokens});
  check(api.extend_pages(ptr<int32_t>(block_table), ptr<int32_t>(lens), ptr<int32_t>(add),
                         ptr<int32_t>(free), ptr<int32_t>(free_count), ptr<int32_t>(lens_out),
                         ptr<int32_t>(left), ptr<int32_t>(cu), ptr<int32_t>(positions),
                         ptr<int64_t>(slots), size(where, B), size(where, max_pages),
                         size(where, num_pages), 16, size(where, max_tokens),
                         device.stream()),
        "fa_extend_pages");
  return {lens_out, cu, positions, slots, left};
}

std::tuple<Tensor, Maybe> decode_shared_prefix(const Tensor& q, const Tensor& kcache,
                                               const Tensor& vcache, const Tensor& block_table,
                                               const Tensor& seq_lens, const Tensor& prefix_table,
                                               const Tensor& prefix_pages,
                                               std::optional<double> scale, bool return_lse) {
  const char* where = "decode_shared_prefix";
  const Device device(where, q);
  dtype(where, "q", q, at::kBFloat16);
  shape(where, "q", q, {-1, -1, -1});
  const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
  cache_shapes(where, device, kcache, vcache, -1, D);
  for (const auto& [name, t] :
       {std::pair<const char*, const Tensor&>{"block_table", block_table},
        std::pair<const char*, const Tensor&>{"seq_lens", seq_lens},
        std::pair<const char*, const Tensor&>{"prefix_table", prefix_table},
        std::pair<const char*, const Tensor&>{"prefix_pages", prefix_pages}}) {
    device(t);
    dtype(where, name, t, at::kInt);
  }
  shape(where, "block_table", block_table, {B, -1});
  shape(where, "seq_lens", seq_lens, {B});
  shape(where, "prefix_table", prefix_table, {-1});
  shape(where, "prefix_pages", prefix_pages, {1});
  const Tensor qc = q.contiguous(), kc = kcache.contiguous(), vc = vcache.contiguous(),
               blocks = block_table.contiguous(), lens = seq_lens.contiguous(),
               prefix = prefix_table.contiguous();
  Tensor o = empty(q, at::kBFloat16, {B, Hq, D});
  Maybe lse;
  if (return_lse) lse = empty(q, at::kFloat, {B, Hq});
  const double s = scale ? *scale : 1.0 / std::sqrt(static_cast<double>(D));
  check(api.decode_shared_prefix(
            ptr<void>(qc), ptr<void>(kc), ptr<void>(vc), ptr<int32_t>(blocks), ptr<int32_t>(lens),
            ptr<int32_t>(prefix), ptr<int32_t>(prefix_pages), ptr<void>(o), size(where, B),
            size(where, Hq), size(where, kc.size(2)), size(where, D),
            size(where, kc.size(1)), static_cast<float>(s), device.stream(),
            size(where, blocks.size(1)), size(where, prefix.size(0)),
            size(where, kc.size(0)), ptr<float>(lse)),
        "fa_decode_shared_prefix");
  return {o, lse};
}

// Entry points by name (addresses in the library that fa.py has loaded), and FAError.
void bind(const py::dict& entry, const py::object& error) {
  auto set = [&](auto& slot, const char* name) {
    slot = reinterpret_cast<std::decay_t<decltype(slot)>>(entry[name].cast<uintptr_t>());
  };
  set(api.qk_norm_rope, "fa_qk_norm_rope");
  set(api.qk_norm_rope_fp16, "fa_qk_norm_rope_fp16");
  set(api.qk_norm_rope_bwd, "fa_qk_norm_rope_bwd");
  set(api.qk_norm_rope_bwd_fp16, "fa_qk_norm_rope_bwd_fp16");
  set(api.append_paged, "fa_append_paged");
  set(api.extend_pages, "fa_extend_pages");
  set(api.decode_shared_prefix, "fa_decode_shared_prefix");
  set(api.last_error_string, "fa_last_error_string");
  Py_XDECREF(error_class);
  error_class = error.inc_ref().ptr();
}

}  // namespace

PYBIND11_MODULE(_step, m) {
  m.attr("abi") = FA_BINDING_ABI;      // the torch and the Python that it was compiled for
  m.def("bind", &bind);
  m.def("head_rows", &head_rows);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_backward", &qk_norm_rope_backward);
  m.def("append_paged", &append_paged);
  m.def("extend_pages", &extend_pages);
  m.def("decode_shared_prefix", &decode_shared_prefix);
}
