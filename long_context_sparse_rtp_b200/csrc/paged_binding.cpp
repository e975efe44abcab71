// paged_binding.cpp -- the Python binding of the paged-cache calls, as a CPython
// extension module: argument checks, allocation and marshalling only.
//
// A decode step makes up to four of these calls with 8 to 20 arguments each, and
// without a CUDA graph their cost on the host is what a small step costs.  Through
// ctypes an attention call took 31 us before its launches (a plan 32, a write 17);
// here the tensors are read in C++.  Positional arguments only: paged.py has the
// signatures users see.
//
// Outputs and workspaces come from torch's allocator on the call's stream, so that
// calls in flight at once, and captured graphs, each have their own.
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "rtp.h"

namespace {

constexpr int64_t kD = 128;
constexpr int64_t kAny = -1;  // any size
PyObject* g_error = nullptr;  // RtpError
PyObject* g_plan_names[6];    // the plan's outputs

struct Bad {  // becomes a ValueError
  std::string what;
};
struct Set {};  // a Python exception is set already

void need(bool ok, const char* what) {
  if (!ok) throw Bad{what};
}

bool none(PyObject* o) { return o == Py_None; }

int32_t to_int(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Set{};
  if (x < INT32_MIN || x > INT32_MAX) throw Bad{std::string(name) + ": out of range"};
  return (int32_t)x;
}

double to_double(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Set{};
  return x;
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    throw Bad{std::string(name) + ": expected a CUDA tensor"};
  return THPVariable_Unpack(o);
}

// A tensor of this type and shape on `dev`.
const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type,
                         std::initializer_list<int64_t> shape, c10::Device dev,
                         bool contiguous = true) {
  bool ok = THPVariable_Check(o);
  if (ok) {
    const at::Tensor& t = THPVariable_Unpack(o);
    ok = t.scalar_type() == type && t.device() == dev && t.dim() == (int64_t)shape.size();
    int64_t i = 0;
    for (int64_t n : shape) {
      ok = ok && (n == kAny || t.size(i) == n);
      ++i;
    }
    if (ok && contiguous && !t.is_contiguous())
      throw Bad{std::string(name) + ": expected a contiguous tensor"};
  }
  if (!ok) {
    std::string s;
    for (int64_t n : shape) s += (s.empty() ? "" : ", ") + (n == kAny ? "any" : std::to_string(n));
    throw Bad{std::string(name) + ": expected " + c10::toString(type) + " [" + s + "] on " + dev.str()};
  }
  return THPVariable_Unpack(o);
}

void* ptr(const at::Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }

struct Roles {
  uint8_t role[256];
  int32_t Hkv = 0, n_rkv = 0;
  explicit Roles(PyObject* o) {
    PyObject* seq = PySequence_Fast(o, "kv_role: expected a sequence");
    if (seq == nullptr) throw Set{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    bool ok = n > 0 && n <= 256;
    for (Py_ssize_t i = 0; ok && i < n; ++i) {
      const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
      if (x == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw Set{};
      }
      ok = x == 0 || x == 1;
      role[i] = (uint8_t)x;
      n_rkv += (int32_t)x;
    }
    Py_DECREF(seq);
    need(ok, "kv_role: expected one 0 or 1 per kv head");
    Hkv = (int32_t)n;
  }
};

// Makes the call's device and stream current for as long as it lives.  On a stream
// other than the caller's current one it tells the allocator who uses what: the
// caller's tensors are in use on the call's stream, what the call allocates there is
// used on the caller's stream too.  Inside a capture as well: a graph's pool hands what
// was dropped out again to the stream that it was allocated on, within the capture.
struct On {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  c10::cuda::CUDAStream theirs, ours;
  cudaStream_t stream;
  bool crossed = false;
  On(c10::Device dev, PyObject* s)
      : theirs(c10::cuda::getCurrentCUDAStream(dev.index())), ours(theirs) {
    if (none(s)) {
      device.set_device(dev);
      stream = ours.stream();
      return;
    }
    int64_t v[3];
    const char* names[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
      PyObject* x = PyObject_GetAttrString(s, names[i]);
      if (x == nullptr) throw Set{};
      v[i] = PyLong_AsLongLong(x);
      Py_DECREF(x);
      if (v[i] == -1 && PyErr_Occurred()) throw Set{};
    }
    need(v[1] == dev.index() && v[2] == (int64_t)c10::DeviceType::CUDA,
         "stream: expected a stream of the tensors' device");
    ours = c10::cuda::CUDAStream::unpack3(v[0], (c10::DeviceIndex)v[1], (c10::DeviceType)v[2]);
    guard.reset_stream(ours);
    stream = ours.stream();
    crossed = ours != theirs;
  }
  void record(const at::Tensor& t, c10::cuda::CUDAStream s) const {
    if (t.defined() && t.numel())
      c10::cuda::CUDACachingAllocator::get()->recordStream(t.storage().data_ptr(), s);
  }
  // The call's arguments: tensors among them are in use on its stream.
  void uses(PyObject* const* a, int n) const {
    for (int i = 0; crossed && i < n; ++i)
      if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).is_cuda())
        record(THPVariable_Unpack(a[i]), ours);
  }
  // What the call allocated for the caller.
  void gives(const at::Tensor& t) const {
    if (crossed) record(t, theirs);
  }
};

rtp_stream_t raw(cudaStream_t s) { return reinterpret_cast<rtp_stream_t>(s); }

at::Tensor empty(c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// A contiguous tensor on buf's storage (32-bit elements) from its element `offset`.
at::Tensor part(const at::Tensor& buf, int64_t offset, c10::IntArrayRef shape,
                at::ScalarType type = at::kInt) {
  const auto meta = c10::scalarTypeToTypeMeta(type);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()),
                                                          buf.key_set(), meta);
  t.unsafeGetTensorImpl()->set_storage_offset(offset * 4 / (int64_t)meta.itemsize());
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// A workspace that goes back to the allocator, in stream order, when it ends.
struct Workspace {
  size_t bytes;
  c10::DataPtr data;
  Workspace(rtp_paged_op op, int32_t B, int32_t H, const Roles* r, int32_t width)
      : bytes(rtp_paged_workspace_size(op, B, H, r ? r->Hkv : 0, r ? r->role : nullptr, width)),
        data(c10::cuda::CUDACachingAllocator::get()->allocate(bytes)) {}
};

void check(const char* fn, rtp_status st) {
  if (st == RTP_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", fn, (int)st);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Set{};
}

// [n_pages, page_size, Hkv, 128], in any order of strides; a size of 1 has none.
rtp_pages pages(const at::Tensor& t) {
  auto st = [&](int i) { return t.size(i) > 1 ? t.stride(i) : kD; };
  need(t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX, "pages: too many");
  return {ptr(t), st(0), st(1), st(2), (int32_t)t.size(0), (int32_t)t.size(1),
          t.scalar_type() == at::kBFloat16 ? RTP_KV_BF16 : RTP_KV_E4M3};
}

struct Cache {
  rtp_pages k, v;
  const float* k_scale = nullptr;
  const float* v_scale = nullptr;
  Cache(PyObject* kp, PyObject* vp, PyObject* ks, PyObject* vs, int64_t Hkv, c10::Device dev) {
    for (PyObject* o : {kp, vp}) {
      bool ok = THPVariable_Check(o);
      if (ok) {
        const at::Tensor& t = THPVariable_Unpack(o);
        ok = (t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat8_e4m3fn) &&
             t.device() == dev && t.dim() == 4 && t.size(3) == kD && t.stride(3) == 1;
      }
      need(ok, "k_pages, v_pages: expected bfloat16 or float8_e4m3fn [n_pages, page_size, Hkv, 128] "
               "on the other tensors' device, rows of 128 contiguous");
    }
    const at::Tensor &tk = THPVariable_Unpack(kp), &tv = THPVariable_Unpack(vp);
    need(tk.sizes() == tv.sizes() && tk.scalar_type() == tv.scalar_type(),
         "k_pages and v_pages differ in shape or type");
    need(tk.size(2) == Hkv, "k_pages, v_pages: another number of kv heads");
    k = pages(tk);
    v = pages(tv);
    k_scale = scale(ks, "k_scale", Hkv, dev);
    v_scale = scale(vs, "v_scale", Hkv, dev);
  }
  const float* scale(PyObject* o, const char* name, int64_t Hkv, c10::Device dev) {
    if (none(o)) return nullptr;
    need(k.type == RTP_KV_E4M3, "k_scale, v_scale: bfloat16 pages have none");
    return static_cast<const float*>(ptr(tensor(o, name, at::kFloat, {Hkv}, dev)));
  }
};

struct Rows {  // [n, heads, 128] (or [n, 1, heads, 128]) bf16: pointer and elements between rows
  void* p;
  int64_t stride;
};
Rows rows(PyObject* o, const char* name, int64_t n, int64_t heads, c10::Device dev, bool q) {
  const at::Tensor& t = q ? tensor(o, name, at::kBFloat16, {n, 1, heads, kD}, dev, false)
                          : tensor(o, name, at::kBFloat16, {n, heads, kD}, dev, false);
  const int64_t last = t.dim() - 1;
  if (t.stride(last) != 1 || (heads > 1 && t.stride(last - 1) != kD))
    throw Bad{std::string(name) + ": expected contiguous heads x 128 per row"};
  return {ptr(t), n > 1 ? t.stride(0) : heads * kD};
}

struct Table {
  const int32_t* p;
  int64_t stride;
  int32_t width;
  Table(PyObject* o, int64_t B, c10::Device dev) {
    const at::Tensor& t = tensor(o, "block_table", at::kInt, {B, kAny}, dev, false);
    need(t.size(1) <= 1 || t.stride(1) == 1, "block_table: expected contiguous rows");
    need(t.size(1) <= INT32_MAX, "block_table: too wide");
    width = (int32_t)t.size(1);
    stride = B > 1 ? t.stride(0) : width;
    p = static_cast<const int32_t*>(ptr(t));
  }
};

int32_t count(int64_t n, const char* what) {
  need(n <= INT32_MAX, what);
  return (int32_t)n;
}

const int32_t* i32(const at::Tensor& t) { return static_cast<const int32_t*>(ptr(t)); }
int32_t* i32_out(const at::Tensor& t) { return static_cast<int32_t*>(ptr(t)); }

// (seq_lens, n_new, block_table, free_pages, free_count, page_size, max_tokens,
//  row_tokens, release, six buffers or None, stream) -> dict of the six outputs
PyObject* plan(PyObject* const* a) {
  const at::Tensor& lens = cuda_tensor(a[0], "seq_lens");
  const c10::Device dev = lens.device();
  tensor(a[0], "seq_lens", at::kInt, {kAny}, dev);
  const int32_t B = count(lens.size(0), "seq_lens: too many requests");
  const at::Tensor& n_new = tensor(a[1], "n_new", at::kInt, {B}, dev);
  const Table tab(a[2], B, dev);
  const at::Tensor& pool = tensor(a[3], "free_pages", at::kInt, {kAny}, dev);
  const at::Tensor& free_count = tensor(a[4], "free_count", at::kInt, {1}, dev);
  const int32_t ps = to_int(a[5], "page_size"), T = to_int(a[6], "max_tokens"),
                row = to_int(a[7], "row_tokens");
  need(ps > 0 && T >= 0 && row >= 0, "page_size, max_tokens, row_tokens: expected no negative numbers");
  const uint8_t* release = nullptr;
  if (!none(a[8])) {
    const bool is_bool = THPVariable_Check(a[8]) && THPVariable_Unpack(a[8]).scalar_type() == at::kBool;
    release = static_cast<const uint8_t*>(
        ptr(tensor(a[8], "release", is_bool ? at::kBool : at::kByte, {B}, dev)));
  }
  const int64_t n_spans = std::min<int64_t>(T, T / ps + 2 * (int64_t)B);
  On on(dev, a[15]);
  on.uses(a, 15);
  // one allocation for what the caller gave no buffer for, and the workspace
  const size_t ws_bytes = rtp_paged_workspace_size(RTP_PAGED_PLAN, B, 0, 0, nullptr, 0);
  auto padded = [](int64_t ints) { return (ints + 63) / 64 * 64; };  // 256-byte places
  const at::Tensor buf =
      empty({padded(ws_bytes / 4) + 2 * padded(B) + padded(B + 1) + padded(T) +
             padded(4 * n_spans) + padded(1)}, at::kInt, dev);
  on.gives(buf);
  int64_t at = padded(ws_bytes / 4);
  at::Tensor out[6];
  auto take = [&](int i, const char* name, std::initializer_list<int64_t> shape,
                  std::initializer_list<int64_t> given) {
    if (!none(a[9 + i])) {
      out[i] = tensor(a[9 + i], name, at::kInt, given, dev);
      return;
    }
    out[i] = part(buf, at, c10::IntArrayRef(shape.begin(), shape.size()));
    at += padded(out[i].numel());
  };
  take(0, "seq_lens", {B}, {B});
  take(1, "cu_new", {B + 1}, {B + 1});
  take(2, "slot_map", {T}, {T});
  take(3, "spans", {n_spans, 4}, {kAny, 4});
  take(4, "free_count", {1}, {1});
  take(5, "admitted", {B}, {B});
  if (B == 0) {  // the library enqueues nothing: an empty batch
    out[1].zero_();
    out[2].fill_(-1);
    out[3].zero_().select(1, 0).fill_(-1);
    if (!out[4].is_same(free_count)) out[4].copy_(free_count);
  }
  check("rtp_paged_plan",
        rtp_paged_plan(B, ps, row, i32(lens), i32(n_new), release, const_cast<int32_t*>(tab.p),
                       tab.stride, tab.width, i32_out(pool),
                       count(pool.size(0), "free_pages: too many"), i32(free_count), T,
                       count(out[3].size(0), "spans: too many"), i32_out(out[0]), i32_out(out[1]),
                       i32_out(out[2]), i32_out(out[3]), i32_out(out[4]), i32_out(out[5]),
                       ptr(buf), ws_bytes, raw(on.stream)));
  PyObject* r = PyDict_New();
  if (r == nullptr) throw Set{};
  for (int i = 0; i < 6; ++i) {
    PyObject* t = THPVariable_Wrap(out[i]);
    const bool ok = t != nullptr && PyDict_SetItem(r, g_plan_names[i], t) == 0;
    Py_XDECREF(t);
    if (!ok) {
      Py_DECREF(r);
      throw Set{};
    }
  }
  return r;
}

int64_t batch(PyObject* o, const char* name, int64_t dims, const char* what) {
  const at::Tensor& t = cuda_tensor(o, name);
  need(t.dim() == dims, what);
  return t.size(0);
}

// (k, v, slot_map, k_pages, v_pages, k_scale, v_scale, stream)
PyObject* kv_write(PyObject* const* a) {
  const int32_t T = count(batch(a[0], "k", 3, "k: expected [T, Hkv, 128]"), "k: too many rows");
  const at::Tensor& k = THPVariable_Unpack(a[0]);
  const c10::Device dev = k.device();
  const int32_t Hkv = count(k.size(1), "k: too many heads");
  const Rows kr = rows(a[0], "k", T, Hkv, dev, false), vr = rows(a[1], "v", T, Hkv, dev, false);
  const at::Tensor& slot = tensor(a[2], "slot_map", at::kInt, {T}, dev);
  const Cache c(a[3], a[4], a[5], a[6], Hkv, dev);
  On on(dev, a[7]);
  on.uses(a, 7);
  check("rtp_paged_kv_write", rtp_paged_kv_write(T, Hkv, kr.p, kr.stride, vr.p, vr.stride, i32(slot),
                                                 c.k, c.v, c.k_scale, c.v_scale, raw(on.stream)));
  Py_RETURN_NONE;
}

// (k, v, spans, k_pages, v_pages, kv_role, bounds, bound_scale, k_scale, v_scale, stream)
PyObject* kv_append(PyObject* const* a) {
  const int32_t T = count(batch(a[0], "k", 3, "k: expected [T, Hkv, 128]"), "k: too many rows");
  const at::Tensor& k = THPVariable_Unpack(a[0]);
  const c10::Device dev = k.device();
  const Roles role(a[5]);
  need(k.size(1) == role.Hkv, "kv_role: another number of kv heads than k");
  const Rows kr = rows(a[0], "k", T, role.Hkv, dev, false), vr = rows(a[1], "v", T, role.Hkv, dev, false);
  const at::Tensor& spans = tensor(a[2], "spans", at::kInt, {kAny, 4}, dev);
  const Cache c(a[3], a[4], a[8], a[9], role.Hkv, dev);
  const at::Tensor& bounds =
      tensor(a[6], "bounds", at::kChar, {c.k.n_pages, role.n_rkv, 2, kD}, dev);
  const at::Tensor& scale = tensor(a[7], "bound_scale", at::kFloat, {c.k.n_pages, role.n_rkv}, dev);
  On on(dev, a[10]);
  on.uses(a, 10);
  check("rtp_paged_kv_append",
        rtp_paged_kv_append(T, role.Hkv, role.role, kr.p, kr.stride, vr.p, vr.stride, i32(spans),
                            count(spans.size(0), "spans: too many"), c.k, c.v, c.k_scale, c.v_scale,
                            static_cast<int8_t*>(ptr(bounds)), static_cast<float*>(ptr(scale)),
                            raw(on.stream)));
  Py_RETURN_NONE;
}

// (k, v, k_pages, v_pages, kv_role, k_scale, v_scale): raises what writing these rows
// to these pages would raise, by whichever call, and does nothing.
PyObject* check_rows(PyObject* const* a) {
  const int32_t T = count(batch(a[0], "k", 3, "k: expected [T, Hkv, 128]"), "k: too many rows");
  const c10::Device dev = THPVariable_Unpack(a[0]).device();
  const Roles role(a[4]);
  const Rows kr = rows(a[0], "k", T, role.Hkv, dev, false), vr = rows(a[1], "v", T, role.Hkv, dev, false);
  const Cache c(a[2], a[3], a[5], a[6], role.Hkv, dev);
  check("rtp_paged_kv_append",
        rtp_paged_kv_append(T, role.Hkv, role.role, kr.p, kr.stride, vr.p, vr.stride, nullptr, 0, c.k,
                            c.v, c.k_scale, c.v_scale, nullptr, nullptr, nullptr));
  Py_RETURN_NONE;
}

// What an entry point's CHECK form hands the library: no workspace, which is the last
// thing that a call with work to do is refused for, before anything is enqueued.
void check_only(const char* fn, rtp_status st) {
  check(fn, st == RTP_ERR_WORKSPACE_TOO_SMALL ? RTP_OK : st);
}

// (q, bounds, bound_scale, block_table, seq_lens, kv_role, page_size, n_sel, n_first,
//  n_recent, sel, sel_count, stream) -> (sel, sel_count)
// CHECK: raises what the call would raise, and does nothing.
template <bool CHECK>
PyObject* block_select(PyObject* const* a) {
  const int32_t B = count(batch(a[0], "q", 4, "q: expected [B, 1, H, 128]"), "q: too many requests");
  const at::Tensor& q = THPVariable_Unpack(a[0]);
  const c10::Device dev = q.device();
  const int32_t H = count(q.size(2), "q: too many heads");
  const Rows qr = rows(a[0], "q", B, H, dev, true);
  const Roles role(a[5]);
  const at::Tensor& bounds = tensor(a[1], "bounds", at::kChar, {kAny, role.n_rkv, 2, kD}, dev);
  const at::Tensor& scale =
      tensor(a[2], "bound_scale", at::kFloat, {bounds.size(0), role.n_rkv}, dev);
  const Table tab(a[3], B, dev);
  const at::Tensor& lens = tensor(a[4], "seq_lens", at::kInt, {B}, dev);
  const int32_t n_sel = to_int(a[7], "n_sel");
  need(n_sel >= 1, "n_sel: expected at least 1");
  auto call = [&](int32_t* sel, int32_t* n, void* ws, size_t ws_bytes, rtp_stream_t stream) {
    return rtp_paged_block_select(
        B, H, role.Hkv, role.role, qr.p, qr.stride, static_cast<const int8_t*>(ptr(bounds)),
        static_cast<const float*>(ptr(scale)), count(bounds.size(0), "bounds: too many pages"),
        to_int(a[6], "page_size"), tab.p, tab.stride, tab.width, i32(lens), n_sel,
        to_int(a[8], "n_first"), to_int(a[9], "n_recent"), sel, n, ws, ws_bytes, stream);
  };
  if (CHECK) {
    int32_t none_[2];
    check_only("rtp_paged_block_select", call(none_, none_, nullptr, 0, nullptr));
    Py_RETURN_NONE;
  }
  On on(dev, a[12]);
  on.uses(a, 12);
  const int64_t n_rows = (int64_t)B * role.n_rkv;
  at::Tensor buf;  // the outputs' one allocation
  if (none(a[10]) || none(a[11])) buf = empty({n_rows * (n_sel + (int64_t)1)}, at::kInt, dev);
  on.gives(buf);
  const at::Tensor sel = none(a[10]) ? part(buf, 0, {B, role.n_rkv, n_sel})
                                     : tensor(a[10], "sel", at::kInt, {B, role.n_rkv, n_sel}, dev);
  const at::Tensor n = none(a[11]) ? part(buf, n_rows * n_sel, {B, role.n_rkv})
                                   : tensor(a[11], "sel_count", at::kInt, {B, role.n_rkv}, dev);
  Workspace ws(RTP_PAGED_SELECT, B, H, &role, tab.width);
  check("rtp_paged_block_select",
        call(i32_out(sel), i32_out(n), ws.data.get(), ws.bytes, raw(on.stream)));
  return Py_BuildValue("NN", THPVariable_Wrap(sel), THPVariable_Wrap(n));
}

// (q, k_pages, v_pages, block_table, seq_lens, kv_role, window, n_sink, sel,
//  sel_count, k_scale, v_scale, scale, o, lse, stream) -> (o, lse)
// CHECK: raises what the call would raise, and does nothing; for sel the length of its
// lists, or None, and None for sel_count.
template <bool CHECK>
PyObject* attn_decode(PyObject* const* a) {
  const int32_t B = count(batch(a[0], "q", 4, "q: expected [B, 1, H, 128]"), "q: too many requests");
  const at::Tensor& q = THPVariable_Unpack(a[0]);
  const c10::Device dev = q.device();
  const int32_t H = count(q.size(2), "q: too many heads");
  const Rows qr = rows(a[0], "q", B, H, dev, true);
  const Roles role(a[5]);
  need(role.n_rkv == role.Hkv || !none(a[6]), "window: expected with local heads");
  const int32_t window = none(a[6]) ? 0 : to_int(a[6], "window");
  const Cache c(a[1], a[2], a[10], a[11], role.Hkv, dev);
  const Table tab(a[3], B, dev);
  const at::Tensor& lens = tensor(a[4], "seq_lens", at::kInt, {B}, dev);
  const int32_t *sel = nullptr, *n = nullptr;
  int32_t n_sel = 0;
  if (CHECK && !none(a[8])) {
    sel = n = i32(lens);
    n_sel = to_int(a[8], "n_sel");
  } else if (!CHECK) {
    need(none(a[8]) == none(a[9]), "sel and sel_count come together");
    if (!none(a[8])) {
      const at::Tensor& s = tensor(a[8], "sel", at::kInt, {B, role.n_rkv, kAny}, dev);
      sel = i32(s);
      n = i32(tensor(a[9], "sel_count", at::kInt, {B, role.n_rkv}, dev));
      n_sel = count(s.size(2), "sel: too many pages");
      need(role.n_rkv == 0 || n_sel >= 1, "sel: expected room for a page at least");
    }
  }
  const float scale = (float)to_double(a[12]);
  const Rows orow = none(a[13]) ? Rows{nullptr, H * kD} : rows(a[13], "o", B, H, dev, true);
  if (!none(a[14])) tensor(a[14], "lse", at::kFloat, {B, H, 1}, dev);
  auto call = [&](void* o, float* lse, void* ws, size_t ws_bytes, rtp_stream_t stream) {
    return rtp_paged_attn_decode(B, H, role.Hkv, role.role, window, to_int(a[7], "n_sink"), qr.p,
                                 qr.stride, c.k, c.v, c.k_scale, c.v_scale, tab.p, tab.stride,
                                 tab.width, i32(lens), sel, n, n_sel, scale, o, orow.stride, lse, ws,
                                 ws_bytes, stream);
  };
  if (CHECK) {
    check_only("rtp_paged_attn_decode",
               call(orow.p ? orow.p : qr.p, nullptr, nullptr, 0, nullptr));
    Py_RETURN_NONE;
  }
  On on(dev, a[15]);
  on.uses(a, 15);
  const int64_t o_ints = (int64_t)B * H * (kD / 2);
  at::Tensor buf;  // the outputs' one allocation
  if (none(a[13]) || none(a[14])) buf = empty({o_ints + (int64_t)B * H}, at::kInt, dev);
  on.gives(buf);
  const at::Tensor o = none(a[13]) ? part(buf, 0, {B, 1, H, kD}, at::kBFloat16)
                                   : THPVariable_Unpack(a[13]);
  const at::Tensor lse = none(a[14]) ? part(buf, o_ints, {B, H, 1}, at::kFloat)
                                     : THPVariable_Unpack(a[14]);
  Workspace ws(RTP_PAGED_ATTN, B, H, &role, tab.width);
  check("rtp_paged_attn_decode", call(ptr(o), static_cast<float*>(ptr(lse)), ws.data.get(),
                                      ws.bytes, raw(on.stream)));
  return Py_BuildValue("NN", THPVariable_Wrap(o), THPVariable_Wrap(lse));
}

// No C++ exception leaves an entry point.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Set&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<plan, 16>("plan"),
    method<kv_write, 8>("kv_write"),
    method<kv_append, 11>("kv_append"),
    method<block_select<false>, 13>("block_select"),
    method<attn_decode<false>, 16>("attn_decode"),
    method<check_rows, 7>("check_rows"),
    method<block_select<true>, 13>("check_block_select"),
    method<attn_decode<true>, 16>("check_attn_decode"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) {
  const char* names[6] = {"seq_lens", "cu_new", "slot_map", "spans", "free_count", "admitted"};
  for (int i = 0; i < 6; ++i)
    if ((g_plan_names[i] = PyUnicode_InternFromString(names[i])) == nullptr) return nullptr;
  return PyModule_Create(&g_module);
}
