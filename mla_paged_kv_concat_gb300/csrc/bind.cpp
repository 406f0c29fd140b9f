// Python binding of the calls around the decode (batch tables, gather, kv_b
// products, prompt attention): checks the tensors, allocates what was not
// given, takes the current stream and calls the C entry points of
// include/mla.h.  Nothing is computed here.
//
// Compiled, because these calls are short: through ctypes and Python checks
// one took 34 to 74 us of host time, more than most of the kernels; now 3.5 to
// 9.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/mla.h"

namespace {

using at::Tensor;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;
constexpr auto kI64 = at::kLong;
constexpr int64_t kNope = 128, kV = 128, kRope = 64;

struct BadValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PyError {};  // a Python exception is set

// The text is put together only when the check fails: for every check of a
// call it took longer than the rest of the call.
#define CHECK(ok, what)                \
  do {                                 \
    if (!(ok)) throw BadValue(what);   \
  } while (0)

// The arguments of one call in order, with the device and stream they run on.
struct Call {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  c10::DeviceIndex dev = -1;
  bool own_stream = false;  // a stream was given
  c10::optional<c10::cuda::CUDAStream> stream;

  PyObject* next() {
    if (i >= n) throw BadValue("too few arguments");
    return a[i++];
  }
  // A CUDA tensor, or an undefined one for None.
  Tensor tensor(const char* name, bool optional = false) {
    PyObject* o = next();
    if (o == Py_None && optional) return Tensor();
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
      throw PyError();
    }
    const Tensor& t = THPVariable_Unpack(o);
    CHECK(t.is_cuda(), std::string(name) + " must be a CUDA tensor");
    if (dev < 0) dev = c10::cuda::current_device();
    CHECK(t.device().index() == dev,
          std::string(name) + " is not on the current device cuda:" + std::to_string(dev));
    return t;
  }
  Tensor maybe(const char* name) { return tensor(name, true); }
  int64_t integer() {
    PyObject* o = next();
    PyObject* x = PyNumber_Index(o);
    if (!x) throw PyError();
    const long long v = PyLong_AsLongLong(x);
    Py_DECREF(x);
    if (v == -1 && PyErr_Occurred()) throw PyError();
    return v;
  }
  int small(const char* name) {
    const int64_t v = integer();
    CHECK(v >= INT32_MIN && v <= INT32_MAX, std::string(name) + " does not fit 32 bits");
    return static_cast<int>(v);
  }
  // A truth value: a bool, an integer or NumPy's bool, which is no integer.
  bool truth() {
    if (i < n && std::strncmp(Py_TYPE(a[i])->tp_name, "numpy.bool", 10) == 0) {
      const int v = PyObject_IsTrue(next());
      if (v < 0) throw PyError();
      return v != 0;
    }
    return integer() != 0;
  }
  double real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw PyError();
    return v;
  }
  // The stream argument (None: the current one); after the tensors.
  void take_stream() {
    PyObject* o = next();
    if (dev < 0) dev = c10::cuda::current_device();
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev);
      return;
    }
    int64_t v[3];
    const char* names[3] = {"stream_id", "device_index", "device_type"};
    for (int k = 0; k < 3; ++k) {
      PyObject* x = PyObject_GetAttrString(o, names[k]);
      if (!x) throw PyError();
      v[k] = PyLong_AsLongLong(x);
      Py_DECREF(x);
      if (v[k] == -1 && PyErr_Occurred()) throw PyError();
    }
    stream = c10::cuda::CUDAStream(c10::Stream::unpack3(
        v[0], static_cast<c10::DeviceIndex>(v[1]), static_cast<c10::DeviceType>(v[2])));
    CHECK(stream->device_index() == dev,
          "the stream is not on the current device cuda:" + std::to_string(dev));
    own_stream = true;
  }
  void* s() const { return stream->stream(); }
  // Memory of the stream that the kernels run on.  A block of the current
  // stream's pool may still be in use by work queued there, which a kernel on
  // another stream does not wait for.  The caller may use what is returned on
  // its own current stream too, so such a block is not given out again before
  // that.
  template <typename F>
  Tensor allocate(bool returned, F&& f) const {
    if (!own_stream) return f();
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(dev);
    const c10::cuda::CUDAStreamGuard guard(*stream);
    Tensor t = f();
    if (returned && current != *stream) t.record_stream(current);
    return t;
  }
  Tensor empty(at::IntArrayRef size, at::ScalarType dtype, bool returned = true) const {
    return allocate(returned, [&] {
      return at::empty(size, at::TensorOptions().dtype(dtype).device(at::kCUDA, dev));
    });
  }
  Tensor zeros(at::IntArrayRef size, at::ScalarType dtype) const {
    return allocate(true, [&] {
      return at::zeros(size, at::TensorOptions().dtype(dtype).device(at::kCUDA, dev));
    });
  }
};

std::string dims(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// dtype, shape (-1: any size) and unit last stride of a tensor that is given.
void typed(const Tensor& t, at::ScalarType dtype, std::initializer_list<int64_t> shape,
           const char* name) {
  if (!t.defined()) return;
  CHECK(t.scalar_type() == dtype, std::string(name) + " must be " + c10::toString(dtype) +
                                      ", not " + c10::toString(t.scalar_type()));
  const auto s = t.sizes();
  bool ok = s.size() == shape.size();
  if (ok) {
    size_t k = 0;
    for (int64_t x : shape) {
      ok = ok && (x < 0 || x == s[k]);
      ++k;
    }
  }
  CHECK(ok, std::string(name) + " has the wrong shape " + dims(s));
  CHECK(t.numel() == 0 || s.back() == 1 || t.stride(-1) == 1,
        std::string(name) + " must have unit last stride");
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(ptr(t));
}

// (row, head) strides of [tokens][heads][dims]; those of dimensions of size
// 1, which torch leaves arbitrary, as in a dense tensor.
struct Strides {
  int64_t row = 0, head = 0;
  Strides() = default;
  explicit Strides(const Tensor& t) {
    const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
    head = H > 1 ? t.stride(1) : D;
    row = T > 1 ? t.stride(0) : (H > 1 ? H * head : D);
  }
};
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }
int as_int(int64_t x, const char* name) {
  CHECK(x <= INT32_MAX, std::string(name) + " does not fit 32 bits");
  return static_cast<int>(x);
}

PyObject* wrap(const Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw PyError();
  return o;
}
PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw PyError();
  Py_ssize_t k = 0;
  for (const Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw PyError();
    }
    PyTuple_SET_ITEM(r, k++, o);
  }
  return r;
}

// Raises MlaError for a status other than MLA_OK.
void done(mla_status st, const char* where) {
  if (st == MLA_OK) return;
  PyObject* m = PyImport_ImportModule("mla_paged_kv_concat_gb300._lib");
  PyObject* r = m ? PyObject_CallMethod(m, "check", "is", static_cast<int>(st), where) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(m);
  throw PyError();
}

// Runs a call; C++ exceptions end here.
template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, F&& f) {
  try {
    Call c{a, n};
    return f(c);
  } catch (const PyError&) {
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "call failed");
  return nullptr;
}

// (query_lens, context_lens, req_block_table, free_blocks, free_count,
//  block_size, num_blocks, num_tokens (-1: from the token outputs), req_ids,
//  block_table, seq_lens, cu_q, cu_k, positions, slot_mapping,
//  free_count_out, err_count, stream)
PyObject* batch_build(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [](Call& c) {
    Tensor query = c.tensor("query_lens"), context = c.tensor("context_lens");
    Tensor table = c.tensor("req_block_table"), free_blocks = c.tensor("free_blocks");
    Tensor count = c.tensor("free_count");
    const int bs = c.small("block_size"), nb = c.small("num_blocks");
    int64_t tokens = c.integer();
    Tensor ids = c.maybe("req_ids"), bt = c.maybe("block_table"), seq = c.maybe("seq_lens");
    Tensor cu_q = c.maybe("cu_seqlens_q"), cu_k = c.maybe("cu_seqlens_k");
    Tensor pos = c.maybe("positions"), slot = c.maybe("slot_mapping");
    Tensor count_out = c.maybe("free_count_out"), err = c.maybe("err_count");
    c.take_stream();
    typed(query, kI32, {-1}, "query_lens");
    const int64_t B = query.size(0);
    typed(table, kI32, {-1, -1}, "req_block_table");
    const int64_t rows = table.size(0), maxb = table.size(1);
    if (tokens < 0) {
      const Tensor& given = pos.defined() ? pos : slot;
      CHECK(given.defined() && given.dim() == 1,
            "num_tokens is needed when no token output is given");
      tokens = given.size(0);
    }
    if (!bt.defined()) bt = c.zeros({B, maxb}, kI32);
    if (!seq.defined()) seq = c.empty({B}, kI32);
    if (!cu_q.defined()) cu_q = c.empty({B + 1}, kI32);
    if (!cu_k.defined()) cu_k = c.empty({B + 1}, kI32);
    if (!pos.defined()) pos = c.empty({tokens}, kI64);
    if (!slot.defined()) slot = c.empty({tokens}, kI64);
    if (!count_out.defined()) count_out = c.empty({1}, kI32);
    typed(context, kI32, {B}, "context_lens");
    typed(ids, kI32, {B}, "req_ids");
    typed(free_blocks, kI32, {-1}, "free_blocks");
    typed(count, kI32, {1}, "free_count");
    typed(count_out, kI32, {1}, "free_count_out");
    typed(bt, kI32, {B, maxb}, "block_table");
    typed(seq, kI32, {B}, "seq_lens");
    typed(cu_q, kI32, {B + 1}, "cu_seqlens_q");
    typed(cu_k, kI32, {B + 1}, "cu_seqlens_k");
    typed(pos, kI64, {tokens}, "positions");
    typed(slot, kI64, {tokens}, "slot_mapping");
    typed(err, kI32, {1}, "err_count");
    done(mla_batch_build(ptr<int32_t>(ids), ptr<int32_t>(query), ptr<int32_t>(context),
                         as_int(B, "the number of requests"), ptr<int32_t>(table),
                         rows > 1 ? table.stride(0) : maxb, as_int(rows, "the table's rows"),
                         as_int(maxb, "the table's columns"), bs, nb, ptr<int32_t>(free_blocks),
                         as_int(free_blocks.size(0), "the stack"), ptr<int32_t>(count),
                         ptr<int32_t>(count_out), as_int(tokens, "num_tokens"),
                         ptr<int32_t>(bt), B > 1 ? bt.stride(0) : maxb, ptr<int32_t>(seq),
                         ptr<int32_t>(cu_q), ptr<int32_t>(cu_k), ptr<int64_t>(pos),
                         ptr<int64_t>(slot), ptr<int>(err), c.s()),
         "mla_batch_build");
    return tuple({bt, seq, cu_q, cu_k, pos, slot, count_out});
  });
}

// (held_lens, req_block_table, free_blocks, free_count, block_size,
//  num_blocks, req_ids, free_count_out, err_count, stream)
PyObject* blocks_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [](Call& c) {
    Tensor held = c.tensor("held_lens"), table = c.tensor("req_block_table");
    Tensor free_blocks = c.tensor("free_blocks"), count = c.tensor("free_count");
    const int bs = c.small("block_size"), nb = c.small("num_blocks");
    Tensor ids = c.maybe("req_ids"), count_out = c.maybe("free_count_out");
    Tensor err = c.maybe("err_count");
    c.take_stream();
    if (!count_out.defined()) count_out = count;
    typed(held, kI32, {-1}, "held_lens");
    const int64_t B = held.size(0);
    typed(table, kI32, {-1, -1}, "req_block_table");
    typed(ids, kI32, {B}, "req_ids");
    typed(free_blocks, kI32, {-1}, "free_blocks");
    typed(count, kI32, {1}, "free_count");
    typed(count_out, kI32, {1}, "free_count_out");
    typed(err, kI32, {1}, "err_count");
    const int64_t rows = table.size(0), maxb = table.size(1);
    done(mla_blocks_release(ptr<int32_t>(ids), ptr<int32_t>(held),
                            as_int(B, "the number of requests"), ptr<int32_t>(table),
                            rows > 1 ? table.stride(0) : maxb, as_int(rows, "the table's rows"),
                            as_int(maxb, "the table's columns"), bs, nb,
                            ptr<int32_t>(free_blocks), as_int(free_blocks.size(0), "the stack"),
                            ptr<int32_t>(count), ptr<int32_t>(count_out), ptr<int>(err), c.s()),
         "mla_blocks_release");
    return wrap(count_out);
  });
}

// (kv_cache, kv_dtype (-1: from the tensor), block_table, cu_seqlens,
//  num_tokens (-1: from kv_c), kv_lora_rank (-1: the row less 64),
//  seq_starts, kv_scale, kv_c, k_pe, err_count, stream)
PyObject* gather_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [](Call& c) {
    Tensor cache = c.tensor("kv_cache");
    int fmt = c.small("kv_dtype");
    Tensor table = c.tensor("block_table"), cu = c.tensor("cu_seqlens");
    int64_t tokens = c.integer(), R = c.integer();
    Tensor starts = c.maybe("seq_starts"), scale = c.maybe("kv_scale");
    Tensor kv_c = c.maybe("kv_c"), k_pe = c.maybe("k_pe"), err = c.maybe("err_count");
    c.take_stream();
    if (fmt < 0) {
      switch (cache.scalar_type()) {
        case at::kBFloat16: fmt = MLA_KV_BF16; break;
        case at::kByte:
        case at::kFloat8_e4m3fn: fmt = MLA_KV_FP8_E4M3; break;
        case at::kFloat8_e5m2: fmt = MLA_KV_FP8_E5M2; break;
        default: throw BadValue("unsupported cache dtype");
      }
    }
    CHECK(cache.element_size() == (fmt == MLA_KV_BF16 ? 2u : 1u),
          "kv_cache_dtype does not fit the cache");
    CHECK(cache.dim() == 3 && cache.stride(2) == 1 && cache.stride(1) == cache.size(2),
          "cache rows must be dense");
    const int64_t nb = cache.size(0), bs = cache.size(1), d = cache.size(2);
    if (R < 0) R = d - kRope;
    const int64_t P = d - R;
    typed(table, kI32, {-1, -1}, "block_table");
    const int64_t B = table.size(0);
    if (tokens < 0) {
      CHECK(kv_c.defined() && kv_c.dim() == 2, "num_tokens is needed when kv_c is not given");
      tokens = kv_c.size(0);
    }
    CHECK(R > 0 && P > 0, "kv_lora_rank does not fit the cache");
    if (!kv_c.defined()) kv_c = c.empty({tokens, R}, kBf16);
    if (!k_pe.defined()) k_pe = c.empty({tokens, P}, kBf16);
    typed(cu, kI32, {B + 1}, "cu_seqlens");
    typed(starts, kI32, {B}, "seq_starts");
    typed(kv_c, kBf16, {tokens, R}, "kv_c");
    typed(k_pe, kBf16, {tokens, P}, "k_pe");
    typed(err, kI32, {1}, "err_count");
    CHECK(!scale.defined() || (scale.scalar_type() == at::kFloat && scale.numel() == 1),
          "kv_scale must be one float32");
    done(mla_gather_cache(ptr(cache), static_cast<mla_kv_dtype>(fmt), as_int(nb, "the cache"),
                          as_int(bs, "the block size"), nb > 1 ? cache.stride(0) : bs * d,
                          static_cast<int>(R), static_cast<int>(P), ptr<int32_t>(table),
                          B > 1 ? table.stride(0) : table.size(1),
                          as_int(table.size(1), "the block table"), ptr<int32_t>(cu),
                          ptr<int32_t>(starts), as_int(B, "the number of sequences"),
                          as_int(tokens, "num_tokens"), ptr<float>(scale), ptr(kv_c),
                          row_stride(kv_c), ptr(k_pe), row_stride(k_pe), ptr<int>(err), c.s()),
         "mla_gather_cache");
    return tuple({kv_c, k_pe});
  });
}

// The kv_b weight [heads * 256][R]; returns R.
int64_t kv_b(const Tensor& w, int64_t heads) {
  typed(w, kBf16, {heads * (kNope + kV), -1}, "w_kv_b");
  return w.size(1);
}

// (kv_c, w_kv_b, num_heads, k_nope, v, err_count, stream)
PyObject* expand_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [](Call& c) {
    Tensor x = c.tensor("kv_c"), w = c.tensor("w_kv_b");
    const int H = c.small("num_heads");
    Tensor k = c.maybe("k_nope"), v = c.maybe("v"), err = c.maybe("err_count");
    c.take_stream();
    CHECK(H > 0, "num_heads must be positive");
    const int64_t R = kv_b(w, H);
    typed(x, kBf16, {-1, R}, "kv_c");
    const int64_t T = x.size(0);
    CHECK(k.defined() == v.defined(), "give both k_nope and v, or neither");
    if (!k.defined()) {
      k = c.empty({T, H, kNope}, kBf16);
      v = c.empty({T, H, kV}, kBf16);
    }
    typed(k, kBf16, {T, H, kNope}, "k_nope");
    typed(v, kBf16, {T, H, kV}, "v");
    typed(err, kI32, {1}, "err_count");
    const Strides sk(k), sv(v);
    done(mla_expand_kv(ptr(x), row_stride(x), as_int(T, "the number of tokens"), ptr(w),
                       w.stride(0), H, as_int(R, "kv_lora_rank"), kNope, kV, ptr(k), sk.row,
                       sk.head, ptr(v), sv.row, sv.head, ptr<int>(err), c.s()),
         "mla_expand_kv");
    return tuple({k, v});
  });
}

// (x, w_kv_b, out, err_count, stream); absorb: [T][H][128] -> [T][H][R],
// project: [T][H][R] -> [T][H][128]
PyObject* head_product(PyObject* const* a, Py_ssize_t n, bool absorb) {
  return guarded(a, n, [absorb](Call& c) {
    Tensor x = c.tensor(absorb ? "q_nope" : "o"), w = c.tensor("w_kv_b");
    Tensor out = c.maybe("out"), err = c.maybe("err_count");
    c.take_stream();
    CHECK(x.dim() == 3, "the input must be [tokens, heads, dims]");
    const int64_t T = x.size(0), H = x.size(1);
    const int64_t R = kv_b(w, H);
    const int64_t in = absorb ? kNope : R, cols = absorb ? R : kV;
    typed(x, kBf16, {T, H, in}, absorb ? "q_nope" : "o");
    if (!out.defined()) out = c.empty({T, H, cols}, kBf16);
    typed(out, kBf16, {T, H, cols}, "out");
    typed(err, kI32, {1}, "err_count");
    const Strides si(x), so(out);
    const auto fn = absorb ? mla_absorb_q : mla_project_v;
    done(fn(ptr(x), si.row, si.head, as_int(T, "the number of tokens"), ptr(w), w.stride(0),
            as_int(H, "the number of heads"), as_int(R, "kv_lora_rank"), kNope, kV, ptr(out),
            so.row, so.head, ptr<int>(err), c.s()),
         absorb ? "mla_absorb_q" : "mla_project_v");
    return wrap(out);
  });
}
PyObject* absorb_q(PyObject*, PyObject* const* a, Py_ssize_t n) { return head_product(a, n, true); }
PyObject* project_v(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return head_product(a, n, false);
}

// (q, q_pe, k_nope, v, k_pe, cu_q, cu_k, sm_scale, causal, num_kv_splits,
//  workspace, out, lse, err_count, stream)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [](Call& c) {
    Tensor q = c.tensor("q"), q_pe = c.maybe("q_pe"), k = c.tensor("k_nope"), v = c.tensor("v");
    Tensor k_pe = c.tensor("k_pe"), cu_q = c.tensor("cu_seqlens_q"), cu_k = c.tensor("cu_seqlens_k");
    const float sm_scale = static_cast<float>(c.real());
    const int causal = c.truth();
    const int splits = c.small("num_kv_splits");
    Tensor ws = c.maybe("workspace"), out = c.maybe("out"), lse = c.maybe("lse");
    Tensor err = c.maybe("err_count");
    c.take_stream();
    CHECK(q.dim() == 3 && k_pe.dim() == 2, "q must be [tokens, heads, dims], k_pe [keys, 64]");
    const int64_t T = q.size(0), H = q.size(1), Tk = k_pe.size(0), P = k_pe.size(1);
    typed(cu_q, kI32, {-1}, "cu_seqlens_q");
    const int64_t B = cu_q.size(0) - 1;
    CHECK(B >= 0, "cu_seqlens_q must not be empty");
    if (!out.defined()) out = c.empty({T, H, kV}, kBf16);
    if (!lse.defined()) lse = c.empty({T, H}, at::kFloat);
    typed(q, kBf16, {T, H, kNope + (q_pe.defined() ? 0 : P)}, "q");
    typed(q_pe, kBf16, {T, H, P}, "q_pe");
    typed(k, kBf16, {Tk, H, kNope}, "k_nope");
    typed(v, kBf16, {Tk, H, kV}, "v");
    typed(k_pe, kBf16, {Tk, P}, "k_pe");
    typed(cu_k, kI32, {B + 1}, "cu_seqlens_k");
    typed(out, kBf16, {T, H, kV}, "out");
    typed(lse, at::kFloat, {T, H}, "lse");
    typed(err, kI32, {1}, "err_count");
    CHECK(lse.is_contiguous(), "lse must be contiguous");
    const int Ti = as_int(T, "the number of tokens"), Hi = as_int(H, "the number of heads");
    const size_t need = mla_prefill_workspace_bytes(Ti, Hi, splits, kV);
    if (need && !ws.defined()) {
      CHECK(need <= static_cast<size_t>(INT64_MAX), "the workspace does not fit");
      ws = c.empty({static_cast<int64_t>(need)}, at::kByte, false);
    }
    CHECK(!ws.defined() || ws.is_contiguous(), "workspace must be contiguous");
    const Strides sq(q), sk(k), sv(v), so(out), sp = q_pe.defined() ? Strides(q_pe) : Strides();
    done(mla_prefill(ptr(q), sq.row, sq.head, ptr(q_pe), sp.row, sp.head, Ti, Hi, ptr(k), sk.row,
                     sk.head, ptr(v), sv.row, sv.head, ptr(k_pe), row_stride(k_pe),
                     as_int(Tk, "the number of keys"), kNope, as_int(P, "rope_dim"), kV,
                     ptr<int32_t>(cu_q), ptr<int32_t>(cu_k), as_int(B, "the number of sequences"),
                     causal, sm_scale, splits, ptr(ws), ws.defined() ? ws.nbytes() : 0, ptr(out),
                     so.row, so.head, ptr<float>(lse), ptr<int>(err), c.s()),
         "mla_prefill");
    return tuple({out, lse});
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef kMethods[] = {
    method<batch_build>("batch_build"),   method<blocks_release>("blocks_release"),
    method<gather_cache>("gather_cache"), method<expand_kv>("expand_kv"),
    method<absorb_q>("absorb_q"),         method<project_v>("project_v"),
    method<prefill>("prefill"),           {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&kModule); }
