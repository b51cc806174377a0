// The step calls that take torch tensors, as a Python extension module: argument checks and
// marshalling for pa_rope_and_cache, pa_attention, pa_beam_topk and pa_beam_gather.
//
// These calls take a few microseconds on the GPU and come once per layer and step, so what the host
// does for them counts: reading the tensors' fields here costs about one microsecond a call, where
// the same checks in Python through ctypes took nine.  The library's functions are those of the
// library that the binding has loaded (bind), so another build of it can be named as before.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "pa.h"

namespace {

// What a call raises: ValueError for arguments, the binding's PAError for a status.
struct ArgError {
  std::string text;
};
struct PyFailure {};  // a Python error is set

void need(bool ok, const char* text) {
  if (!ok) throw ArgError{text};
}

PyObject* pa_error = nullptr;  // binding.PAError

decltype(&::pa_rope_and_cache) fn_rope = nullptr;
decltype(&::pa_attention) fn_attention = nullptr;
decltype(&::pa_beam_topk) fn_topk = nullptr;
decltype(&::pa_beam_gather) fn_gather = nullptr;

// ---- arguments --------------------------------------------------------------------------------

// Names of a function's arguments, the first `required` of which must be given.
struct Signature {
  const char* name;
  int required, count;
  const char* args[24];
  PyObject* keys[24];  // interned
};

void unpack(Signature& s, PyObject* const* args, Py_ssize_t n, PyObject* kwnames, PyObject** out) {
  if (!s.keys[0])
    for (int i = 0; i < s.count; ++i) s.keys[i] = PyUnicode_InternFromString(s.args[i]);
  for (int i = 0; i < s.count; ++i) out[i] = nullptr;
  if (n > s.count) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", s.name, s.count, n);
    throw PyFailure{};
  }
  for (Py_ssize_t i = 0; i < n; ++i) out[i] = args[i];
  const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < nk; ++k) {
    PyObject* key = PyTuple_GET_ITEM(kwnames, k);
    int at = -1;
    for (int i = 0; i < s.count && at < 0; ++i)
      if (key == s.keys[i]) at = i;
    for (int i = 0; i < s.count && at < 0; ++i)
      if (PyUnicode_Compare(key, s.keys[i]) == 0) at = i;
    if (at < 0 || out[at]) {
      PyErr_Format(PyExc_TypeError, "%s() got %s argument '%U'", s.name,
                   at < 0 ? "an unexpected keyword" : "multiple values for", key);
      throw PyFailure{};
    }
    out[at] = args[n + k];
  }
  for (int i = 0; i < s.required; ++i)
    if (!out[i]) {
      PyErr_Format(PyExc_TypeError, "%s() missing argument '%s'", s.name, s.args[i]);
      throw PyFailure{};
    }
}

bool given(PyObject* o) { return o && o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!o || !THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw PyFailure{};
  }
  return THPVariable_Unpack(o);
}

const at::Tensor* optional(PyObject* o, const char* name) { return given(o) ? &tensor(o, name) : nullptr; }

double number(PyObject* o, double otherwise) {
  if (!o) return otherwise;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFailure{};
  return v;
}

int integer(PyObject* o, int otherwise) {
  if (!o) return otherwise;
  PyObject* i = PyNumber_Index(o);
  if (!i) throw PyFailure{};
  const long v = PyLong_AsLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw PyFailure{};
  need(v >= INT32_MIN && v <= INT32_MAX, "an integer argument does not fit 32 bits");
  return static_cast<int>(v);
}

// Sizes go to the C ABI as 32-bit integers.
int size32(int64_t v) {
  need(v <= INT32_MAX, "a tensor's size does not fit 32 bits");
  return static_cast<int>(v);
}

// Every tensor must live on the current device: the library takes device pointers and launches
// there.
class Devices {
 public:
  void add(const at::Tensor& t) {
    need(t.is_cuda(), "tensors must be CUDA tensors (the library takes device pointers)");
    if (dev_ < 0) dev_ = c10::cuda::current_device();
    if (t.get_device() != dev_) throw ArgError{"tensors must be on the current device (cuda:" + std::to_string(dev_) + ")"};
  }
  void add(const at::Tensor* t) {
    if (t) add(*t);
  }
  int32_t* error_flag(PyObject* o) {
    const at::Tensor* t = optional(o, "err_flag");
    if (!t) return nullptr;
    add(*t);
    need(t->scalar_type() == at::kInt && t->numel() >= 1, "err_flag must be an int32 tensor of at least one element");
    return static_cast<int32_t*>(t->data_ptr());
  }
  pa_stream_t stream(PyObject* o) {
    if (!given(o)) return reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev_)).stream());
    PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
    if (!handle) {  // an integer handle
      PyErr_Clear();
      handle = o;
      Py_INCREF(handle);
    }
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred()) throw PyFailure{};
    return reinterpret_cast<pa_stream_t>(p);
  }

 private:
  int dev_ = -1;
};

pa_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return PA_BF16;
  need(t.scalar_type() == at::kFloat, "unsupported dtype (bfloat16 or float32)");
  return PA_F32;
}

void contiguous(const at::Tensor& t, const char* text) { need(t.is_contiguous(), text); }
void contiguous(const at::Tensor* t, const char* text) {
  if (t) contiguous(*t, text);
}

// Elements between the tokens of [T, H, D] rows whose heads lie side by side.
int64_t token_rows(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) throw ArgError{std::string(name) + " must be [T, heads, D]"};
  const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
  if (!((t.stride(2) == 1 || D == 1) && (t.stride(1) == D || H == 1)))
    throw ArgError{std::string(name) + ": the heads of a token must be contiguous"};
  if (T <= 1) return H * D;  // (the stride of a single token is arbitrary)
  if (t.stride(0) < H * D) throw ArgError{std::string(name) + ": tokens must not overlap"};
  return t.stride(0);
}

// Run `body` and turn what it throws into a Python error; a status that is not PA_OK into PAError.
template <typename Body>
PyObject* call(const char* name, const Body& body) {
  try {
    pa_status st = PA_OK;
    PyObject* result = body(st);
    if (st == PA_OK) {
      Py_INCREF(result);
      return result;
    }
    PyObject* e = PyObject_CallFunction(pa_error, "is", static_cast<int>(st), name);
    if (e) {
      PyErr_SetObject(pa_error, e);
      Py_DECREF(e);
    }
  } catch (const ArgError& e) {
    PyErr_SetString(PyExc_ValueError, e.text.c_str());
  } catch (const PyFailure&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The C call itself runs without the interpreter lock: a full launch queue blocks it.
template <typename F, typename... Args>
pa_status unlocked(F fn, Args... args) {
  PyThreadState* state = PyEval_SaveThread();
  const pa_status st = fn(args...);
  PyEval_RestoreThread(state);
  return st;
}

// ---- the calls --------------------------------------------------------------------------------

Signature rope_sig{"pa_rope_and_cache", 9, 13,
                   {"q_out", "q", "k", "v", "k_pool", "v_pool", "positions", "slot_mapping", "inv_freq", "layout",
                    "attn_factor", "err_flag", "stream"}, {}};

PyObject* rope(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return call("pa_rope_and_cache", [&](pa_status& st) -> PyObject* {
    PyObject* a[24];
    unpack(rope_sig, args, n, kw, a);
    const at::Tensor &q_out = tensor(a[0], "q_out"), &q = tensor(a[1], "q"), &k = tensor(a[2], "k"),
                     &v = tensor(a[3], "v"), &kp = tensor(a[4], "k_pool"), &vp = tensor(a[5], "v_pool"),
                     &pos = tensor(a[6], "positions"), &slots = tensor(a[7], "slot_mapping"),
                     &inv = tensor(a[8], "inv_freq");
    need(kp.dim() == 4 && vp.sizes() == kp.sizes(), "pools must be [NB, bs, Hkv, D]");
    const int64_t NB = kp.size(0), bs = kp.size(1), Hkv = kp.size(2), D = kp.size(3);
    const int64_t qs = token_rows(q, "q"), ks = token_rows(k, "k"), vs = token_rows(v, "v");
    const int64_t T = q.size(0), Hq = q.size(1);
    need(q.size(2) == D && k.size(0) == T && k.size(1) == Hkv && k.size(2) == D && v.sizes() == k.sizes(),
         "q/k/v shape mismatch");
    need(q_out.sizes() == q.sizes(), "q_out must have q's shape");
    need(pos.scalar_type() == at::kInt && pos.numel() == T, "positions int32 [T]");
    need(slots.scalar_type() == at::kLong && slots.numel() == T, "slot_mapping int64 [T]");
    need(inv.scalar_type() == at::kDouble && inv.dim() == 1, "inv_freq float64 [rotary_dim / 2]");
    const auto dt = q.scalar_type();
    need(k.scalar_type() == dt && v.scalar_type() == dt && q_out.scalar_type() == dt && kp.scalar_type() == dt &&
             vp.scalar_type() == dt,
         "q, k, v, q_out and pools share a dtype");
    for (const at::Tensor* t : {&q_out, &kp, &vp, &pos, &slots, &inv})
      contiguous(*t, "q_out, pools and index tensors must be contiguous");
    Devices on;
    for (const at::Tensor* t : {&q_out, &q, &k, &v, &kp, &vp, &pos, &slots, &inv}) on.add(*t);
    int32_t* err = on.error_flag(a[11]);
    st = unlocked(fn_rope, q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), kp.data_ptr(), vp.data_ptr(),
                  static_cast<const int32_t*>(pos.data_ptr()), static_cast<const int64_t*>(slots.data_ptr()),
                  static_cast<const double*>(inv.data_ptr()), size32(T), size32(Hq), size32(Hkv), size32(D), size32(bs),
                  size32(NB), qs, ks, vs, size32(2 * inv.numel()), static_cast<pa_rope_layout>(integer(a[9], PA_ROPE_HALF)),
                  static_cast<float>(number(a[10], 1.0)), dtype_of(q), err, on.stream(a[12]));
    return Py_None;
  });
}

Signature attention_sig{"pa_attention", 9, 17,
                        {"out", "q", "k_pool", "v_pool", "block_tables", "seq_lens", "query_starts", "max_query_len",
                         "scale", "softcap", "alibi_slopes", "window", "prefix_lens", "first_keys", "workspace",
                         "err_flag", "stream"}, {}};

PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return call("pa_attention", [&](pa_status& st) -> PyObject* {
    PyObject* a[24];
    unpack(attention_sig, args, n, kw, a);
    const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "q"), &kp = tensor(a[2], "k_pool"),
                     &vp = tensor(a[3], "v_pool"), &tables = tensor(a[4], "block_tables"),
                     &lens = tensor(a[5], "seq_lens"), &starts = tensor(a[6], "query_starts");
    const at::Tensor *slopes = optional(a[10], "alibi_slopes"), *prefix = optional(a[12], "prefix_lens"),
                     *first = optional(a[13], "first_keys"), *ws = optional(a[14], "workspace");
    const int64_t stride = token_rows(q, "q");
    need(out.sizes() == q.sizes(), "out must have q's shape");
    need(kp.dim() == 4 && vp.sizes() == kp.sizes(), "pools must be [NB, bs, Hkv, D]");
    need(tables.dim() == 2 && tables.scalar_type() == at::kInt, "block_tables int32 [B, MB]");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), B = tables.size(0);
    need(kp.size(3) == D, "head dim mismatch");
    need(lens.scalar_type() == at::kInt && lens.numel() == B, "seq_lens int32 [B]");
    need(starts.scalar_type() == at::kInt && starts.numel() == B + 1, "query_starts int32 [B + 1]");
    need(!slopes || (slopes->scalar_type() == at::kFloat && slopes->numel() == Hq), "alibi_slopes float32 [Hq]");
    need(!prefix || (prefix->scalar_type() == at::kInt && prefix->numel() == B), "prefix_lens int32 [B]");
    need(!first || (first->scalar_type() == at::kInt && first->numel() == T), "first_keys int32 [T]");
    const auto dt = q.scalar_type();
    need(out.scalar_type() == dt && kp.scalar_type() == dt && vp.scalar_type() == dt, "q, out and pools share a dtype");
    for (const at::Tensor* t : {&out, &kp, &vp, &tables, &lens, &starts, slopes, prefix, first, ws})
      contiguous(t, "out, pools, index tensors and workspace must be contiguous");
    Devices on;
    for (const at::Tensor* t : {&out, &q, &kp, &vp, &tables, &lens, &starts, slopes, prefix, first, ws}) on.add(t);
    int32_t* err = on.error_flag(a[15]);
    pa_attention_mods mods{};
    mods.softcap = static_cast<float>(number(a[9], 0.0));
    mods.window = integer(a[11], 0);
    if (slopes) mods.alibi_slopes = static_cast<const float*>(slopes->data_ptr());
    if (prefix) mods.prefix_lens = static_cast<const int32_t*>(prefix->data_ptr());
    if (first) mods.first_keys = static_cast<const int32_t*>(first->data_ptr());
    st = unlocked(fn_attention, out.data_ptr(), q.data_ptr(), kp.data_ptr(), vp.data_ptr(),
                  static_cast<const int32_t*>(tables.data_ptr()), static_cast<const int32_t*>(lens.data_ptr()),
                  static_cast<const int32_t*>(starts.data_ptr()), size32(T), size32(B), integer(a[7], 0), size32(Hq),
                  size32(kp.size(2)), size32(D), size32(kp.size(1)), size32(tables.size(1)), size32(kp.size(0)), stride,
                  static_cast<float>(number(a[8], 1.0)), &mods, dtype_of(q), ws ? ws->data_ptr() : nullptr,
                  ws ? ws->nbytes() : 0, err, on.stream(a[16]));
    return a[0];
  });
}

Signature topk_sig{"pa_beam_topk", 5, 9,
                   {"scores", "parents", "tokens", "logits", "cum_scores", "finished", "eos_token", "workspace",
                    "stream"}, {}};

PyObject* beam_topk(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return call("pa_beam_topk", [&](pa_status& st) -> PyObject* {
    PyObject* a[24];
    unpack(topk_sig, args, n, kw, a);
    const at::Tensor &scores = tensor(a[0], "scores"), &parents = tensor(a[1], "parents"),
                     &tokens = tensor(a[2], "tokens"), &logits = tensor(a[3], "logits"),
                     &cum = tensor(a[4], "cum_scores");
    const at::Tensor *finished = optional(a[5], "finished"), *ws = optional(a[7], "workspace");
    need(logits.dim() == 3, "logits must be [N, W, V]");
    const int64_t N = logits.size(0), W = logits.size(1), V = logits.size(2);
    need((logits.stride(2) == 1 || V == 1) && (N <= 1 || W <= 1 || logits.stride(0) == W * logits.stride(1)),
         "logits: rows contiguous, at one stride");
    const int64_t row = W > 1 ? logits.stride(1) : N > 1 ? logits.stride(0) : V;
    need(scores.dim() == 2 && scores.size(0) == N && scores.scalar_type() == at::kFloat, "scores float32 [N, k]");
    need(parents.sizes() == scores.sizes() && parents.scalar_type() == at::kInt, "parents int32 [N, k]");
    need(tokens.sizes() == scores.sizes() && tokens.scalar_type() == at::kInt, "tokens int32 [N, k]");
    need(cum.scalar_type() == at::kFloat && cum.dim() == 2 && cum.size(0) == N && cum.size(1) == W,
         "cum_scores float32 [N, W]");
    need(!finished || ((finished->scalar_type() == at::kBool || finished->scalar_type() == at::kByte) &&
                       finished->sizes() == cum.sizes()),
         "finished bool or uint8 [N, W]");
    for (const at::Tensor* t : {&scores, &parents, &tokens, &cum, finished, ws})
      contiguous(t, "tensors must be contiguous");
    Devices on;
    for (const at::Tensor* t : {&scores, &parents, &tokens, &logits, &cum, finished, ws}) on.add(t);
    st = unlocked(fn_topk, static_cast<float*>(scores.data_ptr()), static_cast<int32_t*>(parents.data_ptr()),
                  static_cast<int32_t*>(tokens.data_ptr()), logits.data_ptr(),
                  static_cast<const float*>(cum.data_ptr()),
                  finished ? static_cast<const uint8_t*>(finished->data_ptr()) : nullptr, integer(a[6], 0), size32(N),
                  size32(W), size32(V), size32(scores.size(1)), row, dtype_of(logits), ws ? ws->data_ptr() : nullptr,
                  ws ? ws->nbytes() : 0, on.stream(a[8]));
    return Py_None;
  });
}

Signature gather_sig{"pa_beam_gather", 3, 5, {"dst", "src", "parents", "err_flag", "stream"}, {}};

PyObject* beam_gather(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return call("pa_beam_gather", [&](pa_status& st) -> PyObject* {
    PyObject* a[24];
    unpack(gather_sig, args, n, kw, a);
    const at::Tensor &dst = tensor(a[0], "dst"), &src = tensor(a[1], "src"), &parents = tensor(a[2], "parents");
    need(parents.dim() == 2 && parents.scalar_type() == at::kInt, "parents int32 [N, k]");
    const int64_t N = parents.size(0), k = parents.size(1);
    need(src.dim() >= 2 && src.size(0) == N, "src must be [N, W, ...]");
    need(dst.scalar_type() == src.scalar_type() && dst.dim() == src.dim() && dst.size(0) == N && dst.size(1) == k &&
             dst.sizes().slice(2) == src.sizes().slice(2),
         "dst must be [N, k, ...]");
    for (const at::Tensor* t : {&dst, &src, &parents}) contiguous(*t, "tensors must be contiguous");
    Devices on;
    for (const at::Tensor* t : {&dst, &src, &parents}) on.add(*t);
    int32_t* err = on.error_flag(a[3]);
    const int64_t W = src.size(1), count = src.numel();
    if (count > 0 && k > 0)
      st = unlocked(fn_gather, dst.data_ptr(), src.data_ptr(), static_cast<const int32_t*>(parents.data_ptr()),
                    size32(N), size32(W), size32(k), static_cast<int64_t>(src.nbytes()) / (N * W), err, on.stream(a[4]));
    return a[0];
  });
}

// bind(PAError, addresses of the four functions): before any call.
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* error = nullptr;
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "OKKKK", &error, &f[0], &f[1], &f[2], &f[3])) return nullptr;
  Py_INCREF(error);
  Py_XDECREF(pa_error);
  pa_error = error;
  fn_rope = reinterpret_cast<decltype(fn_rope)>(f[0]);
  fn_attention = reinterpret_cast<decltype(fn_attention)>(f[1]);
  fn_topk = reinterpret_cast<decltype(fn_topk)>(f[2]);
  fn_gather = reinterpret_cast<decltype(fn_gather)>(f[3]);
  Py_RETURN_NONE;
}

#define PA_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(PAError, addresses): the library's functions"},
    {"pa_rope_and_cache", PA_FAST(rope),
     "pa_rope_and_cache(q_out, q, k, v, k_pool, v_pool, positions, slot_mapping, inv_freq, layout=PA_ROPE_HALF,\n"
     "                  attn_factor=1.0, err_flag=None, stream=None)\n\n"
     "Rotate q [T,Hq,D] into q_out and k [T,Hkv,D] into its slots, v unchanged into its own (see\n"
     "include/pa.h); the rotated part of a head is 2 * inv_freq.numel() elements."},
    {"pa_attention", PA_FAST(attention),
     "pa_attention(out, q, k_pool, v_pool, block_tables, seq_lens, query_starts, max_query_len, scale,\n"
     "             softcap=0.0, alibi_slopes=None, window=0, prefix_lens=None, first_keys=None,\n"
     "             workspace=None, err_flag=None, stream=None)\n\n"
     "out[T,Hq,D] = attention of q's ragged query tokens over the paged cache (see include/pa.h):\n"
     "sequence b's tokens are rows query_starts[b] .. query_starts[b + 1] - 1.  Returns out."},
    {"pa_beam_topk", PA_FAST(beam_topk),
     "pa_beam_topk(scores, parents, tokens, logits, cum_scores, finished=None, eos_token=0, workspace=None,\n"
     "             stream=None)\n\n"
     "The k best candidates of every request (scores, parents, tokens: [N, k]) from logits [N, W, V]\n"
     "and the beams' scores so far [N, W] (see include/pa.h)."},
    {"pa_beam_gather", PA_FAST(beam_gather),
     "pa_beam_gather(dst, src, parents, err_flag=None, stream=None)\n\n"
     "dst[n][i] = src[n][parents[n][i]]: per-beam states [N, W, ...] in the order of parents [N, k].\n"
     "Returns dst."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module{PyModuleDef_HEAD_INIT, "_calls", "Checked calls of libpagedattn on torch tensors.", -1, methods,
                   nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
