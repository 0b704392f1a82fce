// The Python face of the paged cache's calls (cache.py): checks and marshals
// torch tensors and calls the C entry points of littlebit.h.  A serving step
// makes several of these calls a layer, each a few microseconds on the GPU, so
// the marshalling is compiled: a call takes 3 (free) to 11 us (compact, three new
// tensors) on the host with its launches, 5 rotate, 4 write, 7 attend, against 20
// to 36 in Python.
//
// Every function takes what its wrapper in cache.py documents, runs on the
// current stream of the tensors' device (which is made current for the call),
// and makes its tensors there.  Arguments that do not fit raise ValueError;
// what the library refuses raises littlebit.LittleBitError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <memory>
#include <stdexcept>
#include <string>
#include <vector>

#include "littlebit.h"

namespace {

PyObject* g_fail = nullptr;   // littlebit._check(code, name): raises LittleBitError

struct PythonError {};        // a Python exception is set

using at::Tensor;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t v : t.sizes()) s += std::to_string(v) + ",";
  return s + ")";
}

void check(lb_status code, const char* name) {
  if (code == LB_OK) return;
  PyObject* r = PyObject_CallFunction(g_fail, "is", (int)code, name);
  Py_XDECREF(r);
  throw PythonError{};
}

// ------------------------------------------------------------------ arguments

struct Args {
  PyObject* const* v;
  Py_ssize_t n;

  Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t want) : v(args), n(count) {
    if (count != want) refuse("wrong number of arguments");
  }
  bool none(int i) const { return v[i] == Py_None; }
  int64_t integer(int i) const {
    const long long x = PyLong_AsLongLong(v[i]);
    if (x == -1 && PyErr_Occurred()) throw PythonError{};
    return x;
  }
  // A number that fits an int; one that does not is refused below as any other out of range.
  int small(int i) const {
    const int64_t x = integer(i);
    return x > INT32_MAX ? INT32_MAX : x < INT32_MIN ? INT32_MIN : (int)x;
  }
  double real(int i) const {
    const double x = PyFloat_AsDouble(v[i]);
    if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
    return x;
  }
  const Tensor& tensor(int i, const char* name) const { return as_tensor(v[i], name); }
  static const Tensor& as_tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    return t;
  }
  std::vector<PyObject*> list(int i, const char* name) const {
    if (!PyList_Check(v[i]) && !PyTuple_Check(v[i])) refuse(std::string(name) + " must be a list");
    PyObject** items = PySequence_Fast_ITEMS(v[i]);
    return std::vector<PyObject*>(items, items + PySequence_Fast_GET_SIZE(v[i]));
  }
};

void on(const Tensor& t, c10::Device device, const char* name) {
  if (t.device() != device) refuse(std::string(name) + " is on " + t.device().str() + ", not " + device.str());
}

lb_dtype dtype_of(const Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kHalf: return LB_F16;
    case at::kBFloat16: return LB_BF16;
    case at::kFloat: return LB_F32;
    case at::kChar: return LB_I8;
    default: refuse(std::string(name) + ": " + c10::toString(t.scalar_type()) + " is not supported");
  }
}

// A contiguous index tensor of n entries (-1: any); its address.
template <class T>
T* index_list(const Tensor& t, c10::Device device, const char* name, int64_t n) {
  on(t, device, name);
  const at::ScalarType want = sizeof(T) == 8 ? at::kLong : at::kInt;
  if (t.scalar_type() != want || t.dim() != 1 || !t.is_contiguous() || (n >= 0 && t.size(0) != n))
    refuse(std::string(name) + " must be a contiguous " + c10::toString(want) + " tensor of " +
           (n < 0 ? std::string("n") : std::to_string(n)) + " entries, got " + c10::toString(t.scalar_type()) + " " +
           shape_of(t));
  return static_cast<T*>(t.data_ptr());
}

// Rows (tokens, heads, width), or (tokens, width) for one head, unit stride within a row.
lb_rows rows_of(const Tensor& t, c10::Device device, const char* name, int64_t tokens, at::ScalarType dt) {
  on(t, device, name);
  const bool flat = t.dim() == 2;
  if ((t.dim() != 3 && !flat) || (t.size(-1) > 1 && t.stride(-1) != 1) || (tokens >= 0 && t.size(0) != tokens))
    refuse(std::string(name) + " must be (tokens, heads, width) or (tokens, width) with unit stride in its rows and " +
           (tokens < 0 ? std::string("any") : std::to_string(tokens)) + " tokens, got " + shape_of(t));
  if (t.scalar_type() != dt)
    refuse(std::string(name) + " must be " + c10::toString(dt) + ", got " + c10::toString(t.scalar_type()));
  const int64_t heads = flat ? 1 : t.size(1), width = t.size(-1);
  if (heads > INT32_MAX || width > INT32_MAX) refuse(std::string(name) + " is too large");
  return lb_rows{t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, heads > 1 ? t.stride(1) : 0, (int)heads, (int)width};
}

int count_of(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(std::string(name) + " has too many entries");
  return (int)n;
}

Tensor make(at::IntArrayRef shape, at::ScalarType dt, c10::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(dt).device(device));
}

void* stream_of(c10::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

PyObject* wrap(Tensor t) {
  PyObject* o = THPVariable_Wrap(std::move(t));
  if (!o) throw PythonError{};
  return o;
}

// ------------------------------------------------------------------ handles

// A cache: its tensors are kept alive by the Python object that holds the handle.
struct CacheHandle {
  std::vector<lb_plane> planes;
  std::vector<at::ScalarType> types;
  lb_cache c;
  c10::Device device{c10::kCUDA, 0};
};
constexpr const char* kCacheName = "littlebit.cache";

CacheHandle& cache_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, kCacheName);
  if (!p) throw PythonError{};
  return *static_cast<CacheHandle*>(p);
}

struct RopeHandle {
  lb_rotary r;
  c10::Device device{c10::kCUDA, 0};
};
constexpr const char* kRopeName = "littlebit.rotary";

RopeHandle& rope_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, kRopeName);
  if (!p) throw PythonError{};
  return *static_cast<RopeHandle*>(p);
}

template <class H>
void destroy(PyObject* o) {
  delete static_cast<H*>(PyCapsule_GetPointer(o, PyCapsule_GetName(o)));
}

// rotary(phases, rotary_dim, interleaved, scale)
PyObject* make_rotary(Args a) {
  const Tensor& phases = a.tensor(0, "phases");
  auto h = std::make_unique<RopeHandle>();
  h->device = phases.device();
  const int dim = a.small(1);
  h->r.phases = reinterpret_cast<const uint64_t*>(index_list<int64_t>(phases, h->device, "phases", dim / 2));
  h->r.rotary_dim = dim;
  h->r.interleaved = a.small(2) != 0;
  h->r.scale = (float)a.real(3);
  PyObject* o = PyCapsule_New(h.get(), kRopeName, destroy<RopeHandle>);
  if (!o) throw PythonError{};
  h.release();
  return o;
}

// cache(planes, table, length, refs)
PyObject* make_cache(Args a) {
  const auto planes = a.list(0, "planes");
  if (planes.empty()) refuse("a cache has at least one plane");
  auto h = std::make_unique<CacheHandle>();
  const Tensor& first = Args::as_tensor(planes[0], "planes[0]");
  h->device = first.device();
  if (first.dim() != 4) refuse("planes are (n_pages, heads, page_size, width)");
  const int64_t n_pages = first.size(0), page = first.size(2);
  for (size_t i = 0; i < planes.size(); ++i) {
    const std::string name = "planes[" + std::to_string(i) + "]";
    const Tensor& p = Args::as_tensor(planes[i], name.c_str());
    on(p, h->device, name.c_str());
    if (p.dim() != 4 || p.size(0) != n_pages || p.size(2) != page || (p.size(3) > 1 && p.stride(3) != 1))
      refuse(name + " must be (" + std::to_string(n_pages) + ", heads, " + std::to_string(page) +
             ", width) with unit stride in its rows, got " + shape_of(p));
    auto stride = [&](int d) { return p.size(d) > 1 ? p.stride(d) : 0; };
    h->planes.push_back(lb_plane{p.data_ptr(), stride(0), stride(1), stride(2), count_of(p.size(1), name.c_str()),
                                 count_of(p.size(3), name.c_str()), dtype_of(p, name.c_str())});
    h->types.push_back(p.scalar_type());
  }
  const Tensor& table = a.tensor(1, "table");
  on(table, h->device, "table");
  if (table.scalar_type() != at::kInt || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
    refuse("table must be an int32 tensor (n_slots, max_pages) with unit stride in its rows");
  lb_cache& c = h->c;
  c.planes = h->planes.data();
  c.n_planes = count_of((int64_t)h->planes.size(), "planes");
  c.n_pages = count_of(n_pages, "planes");
  c.page_size = count_of(page, "planes");
  c.n_slots = count_of(table.size(0), "table");
  c.max_pages = count_of(table.size(1), "table");
  c.table_stride = c.n_slots > 1 ? table.stride(0) : c.max_pages;
  c.table = static_cast<int32_t*>(table.data_ptr());
  c.length = index_list<int32_t>(a.tensor(2, "length"), h->device, "length", c.n_slots);
  c.refs = index_list<int32_t>(a.tensor(3, "refs"), h->device, "refs", c.n_pages);
  PyObject* o = PyCapsule_New(h.get(), kCacheName, destroy<CacheHandle>);
  if (!o) throw PythonError{};
  h.release();
  return o;
}

// ------------------------------------------------------------------ calls

// rotate(rope, xs, positions, outs or None, inverse) -> list
PyObject* rotate(Args a) {
  const RopeHandle& rope = rope_of(a.v[0]);
  const auto xs = a.list(1, "xs");
  const size_t n = xs.size();
  if (n == 0 || n > 8) refuse("xs must have one to eight tensors");
  const Tensor& positions = a.tensor(2, "positions");
  const int32_t* pos = index_list<int32_t>(positions, rope.device, "positions", -1);
  const int64_t tokens = positions.size(0);
  const Tensor& x0 = Args::as_tensor(xs[0], "xs[0]");
  const at::ScalarType dt = x0.scalar_type();
  const lb_dtype ldt = dtype_of(x0, "xs");
  std::vector<PyObject*> given;
  if (!a.none(3)) {
    given = a.list(3, "outs");
    if (given.size() != n) refuse("outs must have as many tensors as xs");
  }
  const c10::cuda::CUDAGuard guard(rope.device);
  lb_rows src[8], dst[8];
  std::vector<Tensor> outs(n);
  for (size_t i = 0; i < n; ++i) {
    const Tensor& x = Args::as_tensor(xs[i], "xs");
    src[i] = rows_of(x, rope.device, "xs", tokens, dt);
    outs[i] = given.empty() ? make(x.sizes(), dt, rope.device) : Args::as_tensor(given[i], "outs");
    dst[i] = rows_of(outs[i], rope.device, "outs", tokens, dt);
  }
  if (tokens)   // an empty tensor has no address
    check(littlebit_rotary(src, dst, (int)n, count_of(tokens, "positions"), ldt, pos, &rope.r, a.small(4) != 0,
                           stream_of(rope.device)),
          "littlebit_rotary");
  if (!given.empty()) {
    Py_INCREF(a.v[3]);
    return a.v[3];
  }
  PyObject* r = PyList_New((Py_ssize_t)n);
  for (size_t i = 0; i < n; ++i) PyList_SET_ITEM(r, (Py_ssize_t)i, wrap(std::move(outs[i])));
  return r;
}

// The (where, positions) tensors of `tokens` tokens, given or new, as a tuple.
struct Places {
  Tensor where, positions;
  int64_t* w;
  int32_t* p;
  int tokens;

  Places(const CacheHandle& h, const Args& a, int i_tokens, int i_out) {
    const int64_t n = a.integer(i_tokens);
    if (n < 0 || n > INT32_MAX) refuse("tokens must be a count");
    tokens = (int)n;
    if (a.none(i_out)) {
      where = make({n}, at::kLong, h.device);
      positions = make({n}, at::kInt, h.device);
    } else {
      const auto out = a.list(i_out, "out");
      if (out.size() != 2) refuse("out must be (where, positions)");
      where = Args::as_tensor(out[0], "where");
      positions = Args::as_tensor(out[1], "positions");
    }
    w = index_list<int64_t>(where, h.device, "where", n);
    p = index_list<int32_t>(positions, h.device, "positions", n);
  }
  PyObject* result() {
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, wrap(std::move(where)));
    PyTuple_SET_ITEM(r, 1, wrap(std::move(positions)));
    return r;
  }
};

// extend(cache, slots, starts, tokens, prefix, out or None) -> (where, positions)
PyObject* extend(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  const Tensor& slots = a.tensor(1, "slots");
  const int32_t* s = index_list<int32_t>(slots, h.device, "slots", -1);
  const int n = count_of(slots.size(0), "slots");
  const int32_t* starts = index_list<int32_t>(a.tensor(2, "starts"), h.device, "starts", n + 1ll);
  Places out(h, a, 3, 5);
  check(littlebit_cache_extend(&h.c, s, starts, n, out.tokens, a.small(4), out.w, out.p, stream_of(h.device)),
        "littlebit_cache_extend");
  return out.result();
}

// locate(cache, slots, starts, tokens, first or None, prefix, out or None) -> (where, positions)
PyObject* locate(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  const Tensor& slots = a.tensor(1, "slots");
  const int32_t* s = index_list<int32_t>(slots, h.device, "slots", -1);
  const int n = count_of(slots.size(0), "slots");
  const int32_t* starts = index_list<int32_t>(a.tensor(2, "starts"), h.device, "starts", n + 1ll);
  const int32_t* first = a.none(4) ? nullptr : index_list<int32_t>(a.tensor(4, "first"), h.device, "first", n);
  Places out(h, a, 3, 6);
  check(littlebit_cache_locate(&h.c, s, starts, first, n, out.tokens, a.small(5), out.w, out.p, stream_of(h.device)),
        "littlebit_cache_locate");
  return out.result();
}

// fork(cache, parents, children)
PyObject* fork_slots(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  const Tensor& parents = a.tensor(1, "parents");
  const int32_t* p = index_list<int32_t>(parents, h.device, "parents", -1);
  const int n = count_of(parents.size(0), "parents");
  const int32_t* c = index_list<int32_t>(a.tensor(2, "children"), h.device, "children", n);
  if (n == 0) Py_RETURN_NONE;
  const Tensor work = make({(int64_t)littlebit_cache_fork_work(n)}, at::kByte, h.device);
  check(littlebit_cache_fork(&h.c, p, c, n, work.data_ptr(), stream_of(h.device)), "littlebit_cache_fork");
  Py_RETURN_NONE;
}

// free(cache, slots)
PyObject* free_slots(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  const Tensor& slots = a.tensor(1, "slots");
  const int32_t* s = index_list<int32_t>(slots, h.device, "slots", -1);
  if (slots.size(0) == 0) Py_RETURN_NONE;
  check(littlebit_cache_free(&h.c, s, count_of(slots.size(0), "slots"), stream_of(h.device)), "littlebit_cache_free");
  Py_RETURN_NONE;
}

// compact(cache, table, refs, into) -> (table, refs, count): the cache's own tables, or with `into` new ones like them
PyObject* compact(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  Tensor table = a.tensor(1, "table"), refs = a.tensor(2, "refs");
  if (a.small(3)) {
    table = at::empty_strided(table.sizes(), table.strides(), table.options());
    refs = make({h.c.n_pages}, at::kInt, h.device);
  }
  const Tensor work = make({(int64_t)littlebit_cache_compact_work(h.c.n_pages)}, at::kByte, h.device);
  Tensor count = make({1}, at::kInt, h.device);
  check(littlebit_cache_compact(&h.c, static_cast<int32_t*>(table.data_ptr()), static_cast<int32_t*>(refs.data_ptr()),
                                static_cast<int32_t*>(count.data_ptr()), work.data_ptr(), stream_of(h.device)),
        "littlebit_cache_compact");
  PyObject* r = PyTuple_New(3);
  PyTuple_SET_ITEM(r, 0, wrap(std::move(table)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(refs)));
  PyTuple_SET_ITEM(r, 2, wrap(std::move(count)));
  return r;
}

// copy(cache, src, dst)
PyObject* copy_pages(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  const Tensor& src = a.tensor(1, "src");
  const int32_t* s = index_list<int32_t>(src, h.device, "src", -1);
  const int n = count_of(src.size(0), "src");
  const int32_t* d = index_list<int32_t>(a.tensor(2, "dst"), h.device, "dst", n);
  if (n == 0) Py_RETURN_NONE;
  check(littlebit_cache_copy(&h.c, s, d, n, stream_of(h.device)), "littlebit_cache_copy");
  Py_RETURN_NONE;
}

// The planes of a list of plane numbers, all of one type.
std::vector<int> planes_of(const CacheHandle& h, const Args& a, int i, at::ScalarType& dt) {
  std::vector<int> r;
  for (PyObject* o : a.list(i, "planes")) {
    const long long p = PyLong_AsLongLong(o);
    if (p == -1 && PyErr_Occurred()) throw PythonError{};
    if (p < 0 || p >= h.c.n_planes) refuse("there is no plane " + std::to_string(p));
    if (r.empty()) dt = h.types[p];
    else if (h.types[p] != dt) refuse("the planes of one call must have one dtype");
    r.push_back((int)p);
  }
  if (r.empty() || r.size() > 8) refuse("planes must have one to eight entries");
  return r;
}

// write(cache, planes, rows, where, rope or None, positions or None, rotated, q or None, q_out or None) -> q_out
PyObject* write_rows(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  at::ScalarType dt = at::kHalf;
  const std::vector<int> planes = planes_of(h, a, 1, dt);
  const auto rows = a.list(2, "rows");
  const size_t n = planes.size();
  if (rows.size() != n || n > 7) refuse("planes and rows must be lists of the same length, seven at most");
  const Tensor& where = a.tensor(3, "where");
  const int64_t* w = index_list<int64_t>(where, h.device, "where", -1);
  const int tokens = count_of(where.size(0), "where");
  lb_rows src[8];
  for (size_t i = 0; i < n; ++i) src[i] = rows_of(Args::as_tensor(rows[i], "rows"), h.device, "rows", tokens, dt);
  unsigned bits = 0;
  for (PyObject* o : a.list(6, "rotated")) {
    const long long i = PyLong_AsLongLong(o);
    if (i == -1 && PyErr_Occurred()) throw PythonError{};
    if (i < 0 || i >= (long long)n) refuse("rotated: " + std::to_string(i) + " is not a place in planes");
    bits |= 1u << i;
  }
  const lb_rotary* rope = nullptr;
  const int32_t* pos = nullptr;
  if (!a.none(4)) {
    const RopeHandle& r = rope_of(a.v[4]);
    if (r.device != h.device) refuse("rope is on " + r.device.str() + ", not " + h.device.str());
    rope = &r.r;
  }
  if (!a.none(5)) pos = index_list<int32_t>(a.tensor(5, "positions"), h.device, "positions", tokens);
  if ((bits || !a.none(7)) && (!rope || a.none(5))) refuse("rotating needs rope and positions");
  if (a.none(7) && !a.none(8)) refuse("q_out without q");
  lb_rows q, qo;
  Tensor out;
  if (!a.none(7)) {
    const Tensor& t = a.tensor(7, "q");
    q = rows_of(t, h.device, "q", tokens, dt);
    out = a.none(8) ? make(t.sizes(), dt, h.device) : a.tensor(8, "q_out");
    qo = rows_of(out, h.device, "q_out", tokens, dt);
  }
  if (tokens)
    check(littlebit_cache_write(&h.c, planes.data(), src, (int)n, tokens, w, rope, pos, bits, a.none(7) ? nullptr : &q,
                                a.none(7) ? nullptr : &qo, stream_of(h.device)),
          "littlebit_cache_write");
  if (a.none(7)) Py_RETURN_NONE;
  return wrap(std::move(out));
}

// read(cache, planes, where, outs or None) -> list
PyObject* read_rows(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  at::ScalarType dt = at::kHalf;
  const std::vector<int> planes = planes_of(h, a, 1, dt);
  const size_t n = planes.size();
  const Tensor& where = a.tensor(2, "where");
  const int64_t* w = index_list<int64_t>(where, h.device, "where", -1);
  const int tokens = count_of(where.size(0), "where");
  std::vector<PyObject*> given;
  if (!a.none(3)) {
    given = a.list(3, "outs");
    if (given.size() != n) refuse("outs must have as many tensors as planes");
  }
  std::vector<Tensor> outs(n);
  lb_rows dst[8];
  for (size_t i = 0; i < n; ++i) {
    const lb_plane& P = h.planes[planes[i]];
    outs[i] = given.empty() ? make({tokens, P.heads, P.width}, dt, h.device) : Args::as_tensor(given[i], "outs");
    dst[i] = rows_of(outs[i], h.device, "outs", tokens, dt);
  }
  if (tokens)
    check(littlebit_cache_read(&h.c, planes.data(), dst, (int)n, tokens, w, stream_of(h.device)),
          "littlebit_cache_read");
  if (!given.empty()) {
    Py_INCREF(a.v[3]);
    return a.v[3];
  }
  PyObject* r = PyList_New((Py_ssize_t)n);
  for (size_t i = 0; i < n; ++i) PyList_SET_ITEM(r, (Py_ssize_t)i, wrap(std::move(outs[i])));
  return r;
}

// attend(cache, q, slots, starts, k, v, prefix, most_q or None, scale or None, out or None) -> out
PyObject* attend(Args a) {
  const CacheHandle& h = cache_of(a.v[0]);
  const c10::cuda::CUDAGuard guard(h.device);
  const Tensor& q = a.tensor(1, "q");
  const int k = a.small(4), v = a.small(5), prefix = a.small(6);
  if (k < 0 || k >= h.c.n_planes || v < 0 || v >= h.c.n_planes) refuse("k and v must be planes of the cache");
  const lb_rows cq = rows_of(q, h.device, "q", -1, h.types[k]);
  const int tokens = count_of(q.size(0), "q");
  const Tensor& slots = a.tensor(2, "slots");
  const int32_t* s = index_list<int32_t>(slots, h.device, "slots", -1);
  const int n = count_of(slots.size(0), "slots");
  const int32_t* starts = index_list<int32_t>(a.tensor(3, "starts"), h.device, "starts", n + 1ll);
  const int most_q = !a.none(7) ? a.small(7) : n > 0 && tokens > 0 ? (tokens - 1) / n + 1 : 1;   // None: the mean
  const double scale = a.none(8) ? 1.0 / std::sqrt((double)cq.width) : a.real(8);
  Tensor out = a.none(9) ? make(q.sizes(), q.scalar_type(), h.device) : a.tensor(9, "out");
  const lb_rows co = rows_of(out, h.device, "out", tokens, h.types[k]);
  if (tokens == 0) return wrap(std::move(out));
  const size_t size = littlebit_cache_attend_work(&h.c, k, cq.heads, tokens, n, most_q, prefix >= 0);
  const Tensor work = make({(int64_t)size}, at::kByte, h.device);
  check(littlebit_cache_attend(&h.c, k, v, &cq, tokens, s, starts, n, prefix, most_q, (float)scale, &co,
                               work.data_ptr(), size, stream_of(h.device)),
        "littlebit_cache_attend");
  return wrap(std::move(out));
}

// on_fail(callable)
PyObject* on_fail(Args a) {
  Py_XDECREF(g_fail);
  Py_INCREF(a.v[0]);
  g_fail = a.v[0];
  Py_RETURN_NONE;
}

// No C++ exception passes into Python's C code.
template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(Args(args, n, N));
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyMethodDef g_methods[] = {
    {"on_fail", (PyCFunction)(void (*)())entry<on_fail, 1>, METH_FASTCALL, nullptr},
    {"rotary", (PyCFunction)(void (*)())entry<make_rotary, 4>, METH_FASTCALL, nullptr},
    {"cache", (PyCFunction)(void (*)())entry<make_cache, 4>, METH_FASTCALL, nullptr},
    {"rotate", (PyCFunction)(void (*)())entry<rotate, 5>, METH_FASTCALL, nullptr},
    {"extend", (PyCFunction)(void (*)())entry<extend, 6>, METH_FASTCALL, nullptr},
    {"locate", (PyCFunction)(void (*)())entry<locate, 7>, METH_FASTCALL, nullptr},
    {"fork", (PyCFunction)(void (*)())entry<fork_slots, 3>, METH_FASTCALL, nullptr},
    {"free", (PyCFunction)(void (*)())entry<free_slots, 2>, METH_FASTCALL, nullptr},
    {"compact", (PyCFunction)(void (*)())entry<compact, 4>, METH_FASTCALL, nullptr},
    {"copy", (PyCFunction)(void (*)())entry<copy_pages, 3>, METH_FASTCALL, nullptr},
    {"write", (PyCFunction)(void (*)())entry<write_rows, 9>, METH_FASTCALL, nullptr},
    {"read", (PyCFunction)(void (*)())entry<read_rows, 4>, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void (*)())entry<attend, 10>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cache", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache(void) { return PyModule_Create(&g_module); }
