// The Python side of a serving step's calls (add_rmsnorm_quant_act, paged_plan, rope_paged_append,
// attention_paged): argument checks, outputs and workspaces from torch's allocator, the current
// stream.  They are made once per layer and step, most often for a few tokens, where the GPU
// takes 3-10 us: in Python over ctypes a call took 11-14 us of host time, here 5-7, 2-3 of them the launch.
// The library itself stays the plain C one: its entry points are looked up in the handle that the
// package loaded.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/bitnet_b200.h"

namespace py = pybind11;

namespace {

struct {
  decltype(&bitnet_add_rmsnorm_quant_act) add_norm;
  decltype(&bitnet_paged_plan) plan;
  decltype(&bitnet_rope_paged_append) rope;
  decltype(&bitnet_attention_paged_workspace_bytes) attention_ws;
  decltype(&bitnet_attention_paged) attention;
} api;
PyObject* error_class = nullptr;  // BitnetError; kept for the process's life

template <typename F>
void look_up(F& f, void* handle, const char* name) {
  f = reinterpret_cast<F>(dlsym(handle, name));
  if (!f) throw py::import_error(std::string(name) + " is missing in the library");
}
void bind(uintptr_t handle, py::object error) {
  void* h = reinterpret_cast<void*>(handle);
  look_up(api.add_norm, h, "bitnet_add_rmsnorm_quant_act");
  look_up(api.plan, h, "bitnet_paged_plan");
  look_up(api.rope, h, "bitnet_rope_paged_append");
  look_up(api.attention_ws, h, "bitnet_attention_paged_workspace_bytes");
  look_up(api.attention, h, "bitnet_attention_paged");
  error_class = error.release().ptr();
}
void check(bitnet_status st, const char* where) {
  if (st == BITNET_OK) return;
  py::object e = py::reinterpret_borrow<py::object>(error_class)((int)st, where);
  PyErr_SetObject(error_class, e.ptr());
  throw py::error_already_set();
}

// The work of a call without the interpreter's lock: an allocation may wait for the device, and a launch for room in the
// stream's queue, which another Python thread or a host callback in that stream may have to make.  What `f` throws
// are C++ exceptions until the lock is held again.
template <typename F>
void unlocked(const char* where, F f) {
  bitnet_status st;
  {
    const py::gil_scoped_release release;
    st = f();
  }
  check(st, where);
}

// The call's device: that of its first tensor, which has to be the current one.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
    throw py::value_error(std::string(name) + " must be a CUDA tensor on the current device");
  return (int)t.get_device();
}
void* arg(int dev, const char* name, const at::Tensor& t, at::ScalarType type, int64_t numel) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    throw py::value_error(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor on cuda:" + std::to_string(dev));
  if (t.numel() != numel) throw py::value_error(std::string(name) + " must have " + std::to_string(numel) + " entries");
  return t.data_ptr();
}
int32_t* ints(int dev, const char* name, const at::Tensor& t, int64_t numel) {
  return reinterpret_cast<int32_t*>(arg(dev, name, t, at::kInt, numel));
}
bitnet_dtype float_code(const char* name, const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return BITNET_BF16;
  if (t.scalar_type() == at::kFloat) return BITNET_F32;
  throw py::value_error(std::string(name) + " must be of type bfloat16 or float32");
}
void dims(const char* name, const at::Tensor& t, int64_t n) {
  if (t.dim() != n) throw py::value_error(std::string(name) + " must have " + std::to_string(n) + " dimensions");
}
at::Tensor make(int dev, at::IntArrayRef size, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
}

// The bytes of contiguous tensors, and the refusal of overlaps that would let a kernel read what another part of it
// has already written.
struct Bytes {
  uintptr_t from, to;
  Bytes(const at::Tensor& t) : from(t.numel() ? reinterpret_cast<uintptr_t>(t.data_ptr()) : 0), to(t.numel() ? from + t.nbytes() : 0) {}
  bool meets(const Bytes& o) const { return from < o.to && o.from < to; }
  bool is(const Bytes& o) const { return from == o.from && to == o.to; }
};
// No output overlaps an input or another output.
void apart(std::initializer_list<Bytes> outs, std::initializer_list<Bytes> ins) {
  for (const Bytes* o = outs.begin(); o != outs.end(); ++o) {
    for (const Bytes& i : ins)
      if (o->meets(i)) throw py::value_error("an output must not overlap an input");
    for (const Bytes* p = outs.begin(); p != o; ++p)
      if (o->meets(*p)) throw py::value_error("outputs must not overlap one another");
  }
}

// `n` entries of 4 bytes of `buf` from entry `at` on, as a tensor of their own (an allocation takes 0.7 us, this 0.2).
at::Tensor part(const at::Tensor& buf, at::ScalarType type, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// The given stream made current for the call, so that what it allocates belongs to it.
struct OnStream {
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  explicit OnStream(const py::object& stream) {
    if (stream.is_none()) return;
    guard.emplace(c10::cuda::CUDAStream::unpack3(stream.attr("stream_id").cast<int64_t>(),
                                                 (c10::DeviceIndex)stream.attr("device_index").cast<int>(),
                                                 (c10::DeviceType)stream.attr("device_type").cast<int>()));
  }
  bitnet_stream get(int dev) const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

typedef std::optional<at::Tensor> Maybe;

py::tuple add_rmsnorm_quant_act(const at::Tensor& x, const at::Tensor& residual, const Maybe& gain, double eps, Maybe residual_out,
                                const std::optional<std::tuple<at::Tensor, at::Tensor, at::Tensor>>& out, const py::object& stream) {
  const OnStream on(stream);
  at::Tensor q, s, sq;
  unlocked("add_rmsnorm_quant_act", [&] {
    const int dev = device_of(x, "x");
    dims("x", x, 2);
    const int64_t T = x.size(0), K = x.size(1), n = T * K;
    const bitnet_dtype xt = float_code("x", x), rt = float_code("residual", residual);
    if (residual.sizes() != x.sizes()) throw py::value_error("residual must have the shape of x");
    const at::Tensor& g = gain ? *gain : residual;
    if (!residual_out) {
      residual_out = make(dev, {T, K}, residual.scalar_type());
    } else {
      if (residual_out->sizes() != x.sizes()) throw py::value_error("residual_out must have the shape of x");
      apart({*residual_out}, {x});
      if (!Bytes(*residual_out).is(residual)) apart({*residual_out}, {residual, g});  // in place, or elsewhere
    }
    if (out) {
      std::tie(q, s, sq) = *out;
      apart({q, s, sq, *residual_out}, {x});
      apart({q, s, sq}, {residual, g});
    } else {
      const int64_t second = (T + 3) / 4 * 4;  // 16-byte aligned
      const at::Tensor rows = make(dev, {second + T}, at::kInt);
      q = make(dev, {T, K}, at::kChar), s = part(rows, at::kFloat, 0, T), sq = part(rows, at::kInt, second, T);
    }
    return api.add_norm(arg(dev, "x", x, x.scalar_type(), n), xt, arg(dev, "residual", residual, residual.scalar_type(), n), rt,
                       gain ? reinterpret_cast<const float*>(arg(dev, "gain", *gain, at::kFloat, K)) : nullptr, (float)eps, T, K,
                       arg(dev, "residual_out", *residual_out, residual.scalar_type(), n),
                       reinterpret_cast<int8_t*>(arg(dev, "q", q, at::kChar, n)), reinterpret_cast<float*>(arg(dev, "s_x", s, at::kFloat, T)),
                       ints(dev, "sum_q", sq, T), on.get(dev));
  });
  return py::make_tuple(*residual_out, q, s, sq);
}

py::tuple paged_plan(const at::Tensor& new_lens, const at::Tensor& ctx_lens, const at::Tensor& block_table, const at::Tensor& free_pages,
                     const at::Tensor& n_free, int64_t page_size, int64_t T,
                     const std::optional<std::tuple<at::Tensor, at::Tensor, at::Tensor, at::Tensor, at::Tensor>>& out,
                     const py::object& stream) {
  const OnStream on(stream);
  at::Tensor cu, kv, pos, slots, left;
  unlocked("paged_plan", [&] {
    const int dev = device_of(new_lens, "new_lens");
    dims("block_table", block_table, 2);
    const int64_t B = block_table.size(0), width = block_table.size(1), n_list = free_pages.numel();
    if (T < 0) return BITNET_ERR_SHAPE;
    if (out) {
      std::tie(cu, kv, pos, slots, left) = *out;
      apart({cu, kv, pos, slots, left, block_table}, {new_lens, ctx_lens, free_pages, n_free});
    } else {
      apart({block_table}, {new_lens, ctx_lens, free_pages, n_free});
      const at::Tensor buf = make(dev, {2 * B + 2 + 2 * T}, at::kInt);  // 4-byte alignment is all that the step's calls need
      cu = part(buf, at::kInt, 0, B + 1), kv = part(buf, at::kInt, B + 1, B), pos = part(buf, at::kInt, 2 * B + 1, T);
      slots = part(buf, at::kInt, 2 * B + 1 + T, T), left = part(buf, at::kInt, 2 * B + 1 + 2 * T, 1);
    }
    return api.plan(ints(dev, "new_lens", new_lens, B), ints(dev, "ctx_lens", ctx_lens, B), B, page_size,
                   ints(dev, "block_table", block_table, B * width), width, ints(dev, "free_pages", free_pages, n_list), n_list,
                   ints(dev, "n_free", n_free, 1), T, ints(dev, "cu_new", cu, B + 1), ints(dev, "kv_lens", kv, B),
                   ints(dev, "positions", pos, T), ints(dev, "slots", slots, T), ints(dev, "n_free_out", left, 1), on.get(dev));
  });
  return py::make_tuple(cu, kv, pos, slots, left);
}

struct Pages {
  int64_t n, size;
  void *k, *v;
  Pages(int dev, const at::Tensor& kp, const at::Tensor& vp, int64_t Hkv, int64_t d) {
    if (kp.dim() != 4 || kp.sizes() != vp.sizes() || kp.size(1) != Hkv || kp.size(3) != d)
      throw py::value_error("k_pages and v_pages must be [n_pages, Hkv, page_size, d]");
    n = kp.size(0), size = kp.size(2);
    k = arg(dev, "k_pages", kp, at::kBFloat16, kp.numel()), v = arg(dev, "v_pages", vp, at::kBFloat16, vp.numel());
  }
};

at::Tensor rope_paged_append(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& positions,
                             const at::Tensor& slots, double theta, const at::Tensor& k_pages, const at::Tensor& v_pages, Maybe q_rot,
                             const py::object& stream) {
  const OnStream on(stream);
  unlocked("rope_paged_append", [&] {
    const int dev = device_of(q, "q");
    dims("q", q, 3);
    dims("k", k, 3);
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = k.size(1), n = T * Hq * d, nk = T * Hkv * d;
    const at::ScalarType type = q.scalar_type();
    const bitnet_dtype xt = float_code("q", q);
    if (k.size(0) != T || k.size(2) != d || v.sizes() != k.sizes()) throw py::value_error("k and v must be [T, Hkv, d]");
    const Pages pages(dev, k_pages, v_pages, Hkv, d);
    if (!q_rot) {
      q_rot = make(dev, {T, Hq, d}, at::kBFloat16);
      apart({k_pages, v_pages}, {q, k, v, positions, slots});
    } else {
      if (q_rot->sizes() != q.sizes()) throw py::value_error("q_rot must have the shape of q");
      apart({*q_rot, k_pages, v_pages}, {q, k, v, positions, slots});
    }
    return api.rope(arg(dev, "q", q, type, n), arg(dev, "k", k, type, nk), arg(dev, "v", v, type, nk), xt, T, Hq, Hkv, d,
                   ints(dev, "positions", positions, T), ints(dev, "slots", slots, T), theta, arg(dev, "q_rot", *q_rot, at::kBFloat16, n),
                   pages.k, pages.v, pages.n, pages.size, on.get(dev));
  });
  return *q_rot;
}

at::Tensor attention_paged(const at::Tensor& q_rot, const at::Tensor& k_pages, const at::Tensor& v_pages, const at::Tensor& block_table,
                           const at::Tensor& cu_new, const at::Tensor& kv_lens, int64_t max_new, at::ScalarType out_dtype, Maybe out,
                           Maybe ws, const py::object& stream) {
  const OnStream on(stream);
  unlocked("attention_paged", [&] {
    const int dev = device_of(q_rot, "q_rot");
    dims("q_rot", q_rot, 3);
    dims("block_table", block_table, 2);
    dims("k_pages", k_pages, 4);
    const int64_t T = q_rot.size(0), Hq = q_rot.size(1), d = q_rot.size(2), Hkv = k_pages.size(1), n = T * Hq * d;
    const int64_t B = block_table.size(0), width = block_table.size(1);
    const Pages pages(dev, k_pages, v_pages, Hkv, d);
    if (!out) {
      out = make(dev, {T, Hq, d}, out_dtype);
    } else {
      if (out->sizes() != q_rot.sizes()) throw py::value_error("out must have the shape of q_rot");
      apart({*out}, {k_pages, v_pages, block_table, cu_new, kv_lens});
      if (!Bytes(*out).is(q_rot)) apart({*out}, {q_rot});  // in place, or elsewhere
    }
    const bitnet_dtype ot = float_code("out", *out);
    if (!ws) {
      ws = make(dev, {std::max<int64_t>((int64_t)api.attention_ws(Hq, Hkv, max_new), 16)}, at::kByte);
    } else {
      apart({*ws, *out}, {k_pages, v_pages, block_table, cu_new, kv_lens});
      apart({*ws}, {q_rot});
    }
    const int64_t nws = ws->numel();
    return api.attention(arg(dev, "q_rot", q_rot, at::kBFloat16, n), pages.k, pages.v, ints(dev, "block_table", block_table, B * width),
                        ints(dev, "cu_new", cu_new, B + 1), ints(dev, "kv_lens", kv_lens, B), T, B, Hq, Hkv, d, pages.n, pages.size, width,
                        max_new, arg(dev, "out", *out, out->scalar_type(), n), ot, arg(dev, "ws", *ws, at::kByte, nws), (size_t)nws,
                        on.get(dev));
  });
  return *out;
}

}  // namespace

PYBIND11_MODULE(_serving, m) {
  m.attr("built_for") = SERVING_BUILT_FOR;  // looked for in the file before it is loaded
  m.def("bind", &bind);
  m.def("add_rmsnorm_quant_act", &add_rmsnorm_quant_act);
  m.def("paged_plan", &paged_plan);
  m.def("rope_paged_append", &rope_paged_append);
  m.def("attention_paged", &attention_paged);
}
