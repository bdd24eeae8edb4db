// Python module _fmcache: the paged cache's calls (fm.h, "paged K/V cache")
// on torch tensors.  The serving calls take a few microseconds on the GPU;
// through ctypes their argument checks and conversions took 15 to 45
// microseconds of host time (GB300's Grace CPU), several times the kernels'.
// Checks, allocation of what the caller leaves out, and the call: no
// arithmetic happens here.  Work goes to the current stream of the tensors'
// device.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fm.h"

namespace {

// A Python exception has been set.
struct Raised {};

[[noreturn]] void refuse(const char* where, const std::string& what) {
  PyErr_SetString(PyExc_ValueError, (std::string(where) + ": " + what).c_str());
  throw Raised();
}

void check(fm_status st, const char* where) {
  if (st == FM_OK) return;
  // FMError, as the rest of the binding raises it
  PyObject* m = PyImport_ImportModule("masked_attention_bound_gb300._abi");
  if (m) {
    PyObject* r = PyObject_CallMethod(m, "check", "is", static_cast<int>(st), where);
    Py_XDECREF(r);
    Py_DECREF(m);
  }
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  throw Raised();
}

using Shape = std::initializer_list<int64_t>;

std::string text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

const at::Tensor& tensor(const char* where, const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(where, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

bool none(PyObject* o) { return o == Py_None; }

// One call: its name and the device that its tensors must be on.
struct Call {
  const char* where;
  c10::Device device;
  c10::cuda::OptionalCUDAGuard guard;

  Call(const char* w, const at::Tensor& first) : where(w), device(first.device()) {
    if (!device.is_cuda()) refuse(where, "the cache's tensors must be on a CUDA device");
    guard.set_device(device);
  }

  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

  void bf16(const char* name, const at::Tensor& t) const {
    if (t.scalar_type() != at::kBFloat16 || t.device() != device)
      refuse(where, std::string(name) + " must be a bf16 tensor on " + device.str());
    if (t.dim() < 1 || (t.stride(-1) != 1 && t.size(-1) != 1))
      refuse(where, std::string(name) + "'s head_dim must be the contiguous dimension");
  }

  void codes(const char* name, const at::Tensor& t) const {
    if (t.scalar_type() != at::kFloat8_e4m3fn || t.device() != device)
      refuse(where, std::string(name) + " must be a float8_e4m3fn tensor on " + device.str() + " where scales are given");
    if (t.dim() < 1 || (t.stride(-1) != 1 && t.size(-1) != 1))
      refuse(where, std::string(name) + "'s head_dim must be the contiguous dimension");
  }

  int32_t* ints(const char* name, const at::Tensor& t, Shape shape) const {
    if (t.scalar_type() != at::kInt || t.device() != device || t.sizes() != at::IntArrayRef(shape) ||
        !t.is_contiguous())
      refuse(where, std::string(name) + " must be a contiguous int32 tensor of shape " + text(shape) +
                        " on " + device.str());
    return static_cast<int32_t*>(t.data_ptr());
  }
  int32_t* ints(const char* name, PyObject* o, Shape shape) const {
    return ints(name, tensor(where, name, o), shape);
  }
  int32_t* ints_or_null(const char* name, PyObject* o, Shape shape) const {
    return none(o) ? nullptr : ints(name, o, shape);
  }

  int32_t* status(PyObject* o) const {
    if (none(o)) return nullptr;
    const at::Tensor& t = tensor(where, "status", o);
    if (t.scalar_type() != at::kInt || t.device() != device || t.numel() < 1)
      refuse(where, "status must be an int32 tensor on " + device.str());
    return static_cast<int32_t*>(t.data_ptr());
  }

  // straight from the allocator: by way of the dispatcher a call that makes
  // three took 8.8 us of host time, and takes 7.0 so
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
  }
  // `o`, or a new int32 tensor
  at::Tensor out(const char* name, PyObject* o, Shape shape) const {
    return none(o) ? empty(shape, at::kInt) : tensor(where, name, o);
  }

  at::Tensor workspace(PyObject* o, size_t bytes) const {
    if (bytes == 0) refuse(where, "sizes that the library does not take");
    if (none(o)) return empty({static_cast<int64_t>(bytes)}, at::kByte);
    const at::Tensor& t = tensor(where, "ws", o);
    if (t.device() != device || !t.is_contiguous())
      refuse(where, "ws must be a contiguous tensor on " + device.str());
    return t;
  }
};

// Strides of the dimensions [first, first + n) of t; a dimension of one
// element is never stepped along, whatever its stride.
void strides(int64_t* to, const at::Tensor& t, int first, int n, int64_t unstepped = 8) {
  for (int i = 0; i < n; ++i) to[i] = t.size(first + i) == 1 ? unstepped : t.stride(first + i);
}

// The description of pools and a page table; ks, vs: the scales of pools of
// e4m3 codes, None of bf16.
struct Cache {
  fm_cache c{};
  void *k, *v;
  float *k_scale = nullptr, *v_scale = nullptr;
  int32_t* table;

  bool coded() const { return k_scale != nullptr; }

  Cache(const Call& call, PyObject* ko, PyObject* vo, PyObject* to, bool one_layer, PyObject* ks, PyObject* vs) {
    const at::Tensor& kp = tensor(call.where, "k_pool", ko);
    const at::Tensor& vp = tensor(call.where, "v_pool", vo);
    const at::Tensor& tb = tensor(call.where, "table", to);
    if (none(ks) != none(vs)) refuse(call.where, "k_scale and v_scale must be given together");
    const bool scaled = !none(ks);
    if (scaled) {
      call.codes("k_pool", kp);
      call.codes("v_pool", vp);
    } else {
      call.bf16("k_pool", kp);
      call.bf16("v_pool", vp);
    }
    const int64_t dim = kp.dim();
    if ((dim != 4 && (dim != 5 || one_layer)) || vp.sizes() != kp.sizes() || tb.dim() != 2)
      refuse(call.where, one_layer ? "the pools must be one layer's, [pages][page_size][Hkv][d], and the "
                                     "page table [B][max_pages]"
                                   : "the pools must have one shape, [layers][pages][page_size][Hkv][d] or "
                                     "without layers, and the page table [B][max_pages]");
    for (int64_t i = 0; i < dim; ++i)
      if (kp.size(i) > INT32_MAX) refuse(call.where, "pools of more than 2^31 pages");
    if (tb.size(0) > INT32_MAX || tb.size(1) > INT32_MAX)
      refuse(call.where, "a page table of more than 2^31 rows or entries of a row");
    const int f = dim == 5;
    c.layers = f ? static_cast<int>(kp.size(0)) : 1;
    c.n_pages = static_cast<int>(kp.size(f));
    c.page_size = static_cast<int>(kp.size(f + 1));
    c.Hkv = static_cast<int>(kp.size(f + 2));
    c.d = static_cast<int>(kp.size(f + 3));
    c.B = static_cast<int>(tb.size(0));
    c.max_pages = static_cast<int>(tb.size(1));
    c.k_stride[0] = c.v_stride[0] = 16;
    strides(c.k_stride + !f, kp, 0, 3 + f, 16);
    strides(c.v_stride + !f, vp, 0, 3 + f, 16);
    if (scaled) {
      k_scale = scales(call, "k_scale", ks, f);
      v_scale = scales(call, "v_scale", vs, f);
    }
    table = call.ints("table", tb, {tb.size(0), tb.size(1)});
    k = kp.data_ptr();
    v = vp.data_ptr();
  }

 private:
  float* scales(const Call& call, const char* name, PyObject* o, bool layered) const {
    const at::Tensor& t = tensor(call.where, name, o);
    const int64_t want[4] = {c.layers, c.n_pages, c.Hkv, c.page_size / FM_SCALE_BLOCK};
    const at::IntArrayRef shape(want + !layered, 3 + layered);
    if (t.scalar_type() != at::kFloat || t.device() != call.device || t.sizes() != shape || !t.is_contiguous())
      refuse(call.where, std::string(name) + " must be a contiguous fp32 tensor of shape " + text(shape) + " on " +
                             call.device.str());
    return static_cast<float*>(t.data_ptr());
  }
};

PyObject* need(Py_ssize_t got, Py_ssize_t want) {
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return nullptr;
}

#define FM_BEGIN(count)                      \
  if (n != (count)) return need(n, (count)); \
  HANDLE_TH_ERRORS                           \
  try {
#define FM_END                  \
  }                             \
  catch (const Raised&) {       \
    return nullptr;             \
  }                             \
  END_HANDLE_TH_ERRORS

// New tokens' K and V, [total][Hkv][d], to one layer's pools; q, freqs,
// positions and q_out may be None.  Returns q's rotation, or None without q.
PyObject* append_any(const char* where, PyObject* qo, PyObject* ko, PyObject* vo, PyObject* cuo, PyObject* fo,
                     PyObject* kpo, PyObject* vpo, PyObject* to, PyObject* lo, PyObject* po, bool interleaved,
                     PyObject* oo, PyObject* ks, PyObject* vs, PyObject* st) {
  Call call(where, tensor(where, "k_pool", kpo));
  const Cache C(call, kpo, vpo, to, true, ks, vs);
  const at::Tensor& k = tensor(call.where, "k", ko);
  const at::Tensor& v = tensor(call.where, "v", vo);
  call.bf16("k", k);
  call.bf16("v", v);
  if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(1) != C.c.Hkv || k.size(2) != C.c.d)
    refuse(call.where, "k and v must be [total][Hkv][d]");
  const int64_t total = k.size(0);
  if (total > INT32_MAX) refuse(call.where, "more than 2^31 tokens");
  const int32_t* cu = call.ints("cu", cuo, {C.c.B + 1});
  const int32_t* lens = call.ints("lens", lo, {C.c.B});
  int32_t* status = call.status(st);
  fm_rotary r{};
  r.interleaved = interleaved;
  if (!none(fo)) {
    const at::Tensor& f = tensor(call.where, "freqs", fo);
    if (f.scalar_type() != at::kFloat || f.device() != call.device || f.dim() != 1 || !f.is_contiguous() ||
        f.size(0) > C.c.d / 2 || f.size(0) % 8 != 0)
      refuse(call.where, "freqs must be a contiguous fp32 tensor on " + call.device.str() +
                             " with half as many elements as a head has rotated ones, a multiple of 8");
    r.rot = static_cast<int>(2 * f.size(0));
    r.freqs = static_cast<const float*>(f.data_ptr());
    r.positions = call.ints_or_null("positions", po, {total});
  }
  at::Tensor out;
  if (!none(qo)) {
    const at::Tensor& q = tensor(call.where, "q", qo);
    call.bf16("q", q);
    if (q.dim() != 3 || q.size(0) != total || q.size(2) != C.c.d || q.size(1) > INT32_MAX)
      refuse(call.where, "q must be [total][H][d]");
    out = none(oo) ? call.empty(q.sizes(), at::kBFloat16) : tensor(call.where, "q_out", oo);
    call.bf16("q_out", out);
    if (out.sizes() != q.sizes()) refuse(call.where, "q_out must have q's shape");
    r.H = static_cast<int>(q.size(1));
    r.q = q.data_ptr();
    r.q_out = out.data_ptr();
    strides(r.q_stride, q, 0, 2);
    strides(r.o_stride, out, 0, 2);
  }
  if (total > 0) {
    int64_t k_stride[2], v_stride[2];
    strides(k_stride, k, 0, 2);
    strides(v_stride, v, 0, 2);
    const int n = static_cast<int>(total);
    if (none(qo) && none(fo) && !C.coded())
      check(fm_cache_append(&C.c, k.data_ptr(), v.data_ptr(), k_stride, v_stride, cu, n, C.k, C.v, C.table, lens,
                            status, call.stream()),
            "fm_cache_append");
    else
      check(fm_cache_append_rotary(&C.c, &r, k.data_ptr(), v.data_ptr(), k_stride, v_stride, cu, n, C.k, C.v,
                                   C.k_scale, C.v_scale, C.table, lens, status, call.stream()),
            "fm_cache_append_rotary");
  }
  if (none(qo)) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
}

// k, v, cu, k_pool, v_pool, table, lens, k_scale, v_scale, status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FM_BEGIN(10)
  return append_any("cache_append", Py_None, a[0], a[1], a[2], Py_None, a[3], a[4], a[5], a[6], Py_None, false,
                    Py_None, a[7], a[8], a[9]);
  FM_END
}

// q, k, v, cu, freqs, k_pool, v_pool, table, lens, positions, interleaved, q_out, k_scale, v_scale, status
PyObject* append_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FM_BEGIN(15)
  if (none(a[4])) refuse("cache_append_rotary", "freqs must be a tensor");
  const int inter = PyObject_IsTrue(a[10]);
  if (inter < 0) throw Raised();
  return append_any("cache_append_rotary", a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], inter != 0,
                    a[11], a[12], a[13], a[14]);
  FM_END
}

// q, k_pool, v_pool, table, lens, cu, scale, parents, max_nodes, o, lse, ws, k_scale, v_scale, status
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FM_BEGIN(15)
  const at::Tensor& q = tensor("tree_forward", "q", a[0]);
  Call call("tree_forward", q);
  const Cache C(call, a[1], a[2], a[3], true, a[12], a[13]);
  call.bf16("q", q);
  if (q.dim() != 3 || q.size(2) != C.c.d) refuse(call.where, "q must be [total][H][d]");
  const int64_t total = q.size(0), H = q.size(1);
  if (total > INT32_MAX || H > INT32_MAX) refuse(call.where, "more than 2^31 tokens or heads");
  const double scale = PyFloat_AsDouble(a[6]);
  if (scale == -1.0 && PyErr_Occurred()) throw Raised();
  const int32_t* lens = call.ints("lens", a[4], {C.c.B});
  const int32_t* cu = call.ints("cu", a[5], {C.c.B + 1});
  const int32_t* parents = call.ints_or_null("parents", a[7], {total});
  int64_t max_nodes = parents ? std::min<int64_t>(total, FM_TREE_MAX_NODES) : total;
  if (!none(a[8])) {
    max_nodes = PyLong_AsLongLong(a[8]);
    if (max_nodes == -1 && PyErr_Occurred()) throw Raised();
    if (max_nodes < 1 || max_nodes > INT32_MAX) refuse(call.where, "max_nodes must be positive");
  }
  const at::Tensor o = none(a[9]) ? call.empty(q.sizes(), at::kBFloat16) : tensor(call.where, "o", a[9]);
  const at::Tensor lse = none(a[10]) ? call.empty({H, total}, at::kFloat) : tensor(call.where, "lse", a[10]);
  call.bf16("o", o);
  if (o.sizes() != q.sizes() || lse.scalar_type() != at::kFloat || lse.device() != call.device ||
      !lse.is_contiguous() || lse.dim() != 2 || lse.size(0) != H || lse.size(1) != total)
    refuse(call.where, "o must have q's shape and lse be a contiguous fp32 [H][total]");
  if (total > 0) {
    fm_tree_desc d{};
    d.H = static_cast<int>(H);
    d.total = static_cast<int>(total);
    d.max_nodes = static_cast<int>(max_nodes);
    strides(d.q_stride, q, 0, 2);
    strides(d.o_stride, o, 0, 2);
    const at::Tensor ws = call.workspace(a[11], fm_tree_workspace_size(&C.c, &d));
    const float sc = static_cast<float>(scale);
    float* l = static_cast<float*>(lse.data_ptr());
    if (C.coded())
      check(fm_tree_fwd_fp8(&C.c, &d, q.data_ptr(), C.k, C.v, C.k_scale, C.v_scale, C.table, lens, cu, parents, sc,
                            o.data_ptr(), l, ws.data_ptr(), ws.nbytes(), call.status(a[14]), call.stream()),
            "fm_tree_fwd_fp8");
    else
      check(fm_tree_fwd(&C.c, &d, q.data_ptr(), C.k, C.v, C.table, lens, cu, parents, sc, o.data_ptr(), l,
                        ws.data_ptr(), ws.nbytes(), call.status(a[14]), call.stream()),
            "fm_tree_fwd");
  }
  PyObject* po = THPVariable_Wrap(o);
  PyObject* pl = THPVariable_Wrap(lse);
  PyObject* r = po && pl ? PyTuple_Pack(2, po, pl) : nullptr;
  Py_XDECREF(po);
  Py_XDECREF(pl);
  return r;
  FM_END
}

// accept, n_accept, cu, k_pool, v_pool, table, lens, lens_out, ref, k_scale, v_scale, status
PyObject* accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FM_BEGIN(12)
  Call call("cache_accept", tensor("cache_accept", "k_pool", a[3]));
  const Cache C(call, a[3], a[4], a[5], false, a[9], a[10]);
  const at::Tensor& acc = tensor(call.where, "accept", a[0]);
  const int64_t B = C.c.B;
  if (acc.dim() != 2 || acc.size(1) > INT32_MAX) refuse(call.where, "accept must be [B][max_accept]");
  const at::Tensor out = call.out("lens_out", a[7], {B});
  const int32_t* nodes = call.ints("accept", acc, {B, acc.size(1)});
  const int most = static_cast<int>(acc.size(1));
  const int32_t *take = call.ints("n_accept", a[1], {B}), *cu = call.ints("cu", a[2], {B + 1}),
                *lens = call.ints("lens", a[6], {B});
  int32_t *lens_out = call.ints("lens_out", out, {B}), *ref = call.ints_or_null("ref", a[8], {C.c.n_pages});
  if (C.coded())
    check(fm_cache_accept_fp8(&C.c, nodes, most, take, cu, C.k, C.v, C.k_scale, C.v_scale, C.table, lens, lens_out,
                              ref, call.status(a[11]), call.stream()),
          "fm_cache_accept_fp8");
  else
    check(fm_cache_accept(&C.c, nodes, most, take, cu, C.k, C.v, C.table, lens, lens_out, ref, call.status(a[11]),
                          call.stream()),
          "fm_cache_accept");
  return THPVariable_Wrap(out);
  FM_END
}

// parent, page_size, table, lens, ref, table_out, lens_out, ref_out, status
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FM_BEGIN(9)
  const at::Tensor& table = tensor("pages_fork", "table", a[2]);
  Call call("pages_fork", table);
  const at::Tensor& ref = tensor(call.where, "ref", a[4]);
  const long long page = PyLong_AsLongLong(a[1]);
  if (page == -1 && PyErr_Occurred()) throw Raised();
  if (table.dim() != 2 || ref.dim() != 1 || page < 1 || page > INT32_MAX)
    refuse(call.where, "table must be [B][max_pages], ref [pages] and page_size positive");
  if (table.size(0) > INT32_MAX || table.size(1) > INT32_MAX || ref.size(0) > INT32_MAX)
    refuse(call.where, "more than 2^31 rows, entries of a row or pages");
  const int64_t B = table.size(0), m = table.size(1), P = ref.size(0);
  fm_cache c{};
  c.B = static_cast<int>(B);
  c.max_pages = static_cast<int>(m);
  c.page_size = static_cast<int>(page);
  c.n_pages = static_cast<int>(P);
  const at::Tensor to = call.out("table_out", a[5], {B, m}), lo = call.out("lens_out", a[6], {B});
  const at::Tensor ro = none(a[7]) ? ref : tensor(call.where, "ref_out", a[7]);
  check(fm_pages_fork(&c, call.ints("parent", a[0], {B}), call.ints("table", table, {B, m}),
                      call.ints("lens", a[3], {B}), call.ints("ref", ref, {P}),
                      call.ints("table_out", to, {B, m}), call.ints("lens_out", lo, {B}),
                      call.ints("ref_out", ro, {P}), call.status(a[8]), call.stream()),
        "fm_pages_fork");
  PyObject* p[3] = {THPVariable_Wrap(to), THPVariable_Wrap(lo), THPVariable_Wrap(ro)};
  PyObject* r = p[0] && p[1] && p[2] ? PyTuple_Pack(3, p[0], p[1], p[2]) : nullptr;
  for (PyObject* x : p) Py_XDECREF(x);
  return r;
  FM_END
}

// grow, k_pool, v_pool, table, lens, ref, table_out, lens_out, ref_out, info, ws, k_scale, v_scale, status
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FM_BEGIN(14)
  Call call("pages_reserve", tensor("pages_reserve", "k_pool", a[1]));
  const Cache C(call, a[1], a[2], a[3], false, a[11], a[12]);
  const int64_t B = C.c.B, m = C.c.max_pages, P = C.c.n_pages;
  const at::Tensor info = call.out("info", a[9], {2});
  const at::Tensor ws = call.workspace(a[10], fm_pages_workspace_size(&C.c));
  int32_t *lens = call.ints("lens", a[4], {B}), *ref = call.ints("ref", a[5], {P});
  const int32_t* grow = call.ints("grow", a[0], {B});
  int32_t *to = none(a[6]) ? C.table : call.ints("table_out", a[6], {B, m}),
          *lo = none(a[7]) ? lens : call.ints("lens_out", a[7], {B}),
          *ro = none(a[8]) ? ref : call.ints("ref_out", a[8], {P}), *io = call.ints("info", info, {2});
  if (C.coded())
    check(fm_pages_reserve_fp8(&C.c, grow, C.k, C.v, C.k_scale, C.v_scale, C.table, lens, ref, to, lo, ro, io,
                               ws.data_ptr(), ws.nbytes(), call.status(a[13]), call.stream()),
          "fm_pages_reserve_fp8");
  else
    check(fm_pages_reserve(&C.c, grow, C.k, C.v, C.table, lens, ref, to, lo, ro, io, ws.data_ptr(), ws.nbytes(),
                           call.status(a[13]), call.stream()),
          "fm_pages_reserve");
  return THPVariable_Wrap(info);
  FM_END
}

// k_pool, v_pool, table, lens, ref, table_out, ref_out, n_live, ws, k_scale, v_scale, status
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FM_BEGIN(12)
  Call call("pages_compact", tensor("pages_compact", "k_pool", a[0]));
  const Cache C(call, a[0], a[1], a[2], false, a[9], a[10]);
  const int64_t B = C.c.B, m = C.c.max_pages, P = C.c.n_pages;
  const at::Tensor live = call.out("n_live", a[7], {1});
  const at::Tensor ws = call.workspace(a[8], fm_pages_workspace_size(&C.c));
  int32_t *ref = call.ints("ref", a[4], {P}), *lens = call.ints("lens", a[3], {B});
  int32_t *to = none(a[5]) ? C.table : call.ints("table_out", a[5], {B, m}),
          *ro = none(a[6]) ? ref : call.ints("ref_out", a[6], {P}), *out = call.ints("n_live", live, {1});
  if (C.coded())
    check(fm_pages_compact_fp8(&C.c, C.k, C.v, C.k_scale, C.v_scale, C.table, lens, ref, to, ro, out, ws.data_ptr(),
                               ws.nbytes(), call.status(a[11]), call.stream()),
          "fm_pages_compact_fp8");
  else
    check(fm_pages_compact(&C.c, C.k, C.v, C.table, lens, ref, to, ro, out, ws.data_ptr(), ws.nbytes(),
                           call.status(a[11]), call.stream()),
          "fm_pages_compact");
  return THPVariable_Wrap(live);
  FM_END
}

#define FM_FN(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"append", FM_FN(append)},   {"append_rotary", FM_FN(append_rotary)},
                         {"tree", FM_FN(tree)},
                         {"accept", FM_FN(accept)},   {"fork", FM_FN(fork)},
                         {"reserve", FM_FN(reserve)}, {"compact", FM_FN(compact)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fmcache", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fmcache() { return PyModule_Create(&module); }
