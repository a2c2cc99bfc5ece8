// attention_binding.cpp -- Python binding of include/nvfp4_attention.h: argument checks,
// result tensors and marshalling in C++ (a call on one token takes the GPU a few
// microseconds; the same work in Python would take several times that).
#include "binding.h"
#include "nvfp4_attention.h"

namespace {

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}

// A tokens x heads x values tensor on `dev` with contiguous values.  Axes of one entry are
// not stepped over: their stride does not count.
nvfp4_tokens tokens(const at::Tensor& t, const char* name, c10::Device dev) {
  if (t.dim() != 3) type_error(std::string(name) + " must be a 3-D tensor (tokens, heads, values)");
  on_device(t, name, dev);
  if (t.size(2) > 1 && t.stride(2) != 1) value_error(std::string(name) + " must have unit stride along a head's values");
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}
nvfp4_tokens tokens(const at::Tensor& t, const char* name, c10::Device dev, int64_t T, int64_t H, int64_t D,
                    at::ScalarType type) {
  const nvfp4_tokens v = tokens(t, name, dev);
  if (t.size(0) != T || t.size(1) != H || t.size(2) != D)
    value_error(std::string(name) + " must have shape (" + std::to_string(T) + ", " + std::to_string(H) + ", " +
                std::to_string(D) + ") (got " + shape_of(t) + ")");
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + c10::toString(type) + " (got " + c10::toString(t.scalar_type()) + ")");
  return v;
}
// The same for a result: given or made, and no two of its values in one place.
nvfp4_tokens result(const at::Tensor* given, at::Tensor& made, const char* name, c10::Device dev, int64_t T, int64_t H,
                    int64_t D, at::ScalarType type) {
  if (!given) {
    made = fresh({T, H, D}, type, dev);
    return tokens(made, name, dev);
  }
  const nvfp4_tokens v = tokens(*given, name, dev, T, H, D, type);
  const int64_t ts = v.token_stride, hs = v.head_stride;
  const bool apart = T <= 1 || H <= 1 ? (T <= 1 || ts >= D) && (H <= 1 || hs >= D)
                                      : (hs >= D && ts >= (H - 1) * hs + D) || (ts >= D && hs >= (T - 1) * ts + D);
  if (!apart) value_error(std::string(name) + " must not overlap itself");
  return v;
}
PyObject* returned(PyObject* o, const at::Tensor* given_, at::Tensor& made) {
  return given_ ? given(o) : THPVariable_Wrap(std::move(made));
}

struct Heads {
  int64_t T, Hq, Hk, D;
};
Heads heads_of(const at::Tensor& q, const at::Tensor& k) {
  if (q.dim() != 3) type_error("q must be a 3-D tensor (tokens, heads, values)");
  if (k.dim() != 3) type_error("k must be a 3-D tensor (tokens, heads, values)");
  return {q.size(0), q.size(1), k.size(1), q.size(2)};
}
int int_size(int64_t n, const char* where) {
  if (n > INT_MAX) throw Status{NVFP4_ERR_SHAPE, where};
  return (int)n;
}

struct Rotation {
  const int32_t* positions;
  const float* inv_freq;
  int rotated;
};
Rotation rotation(PyObject* pos, PyObject* freq, int64_t T, c10::Device dev, const char* where) {
  const at::Tensor &p = needed(pos, "positions"), &f = needed(freq, "inv_freq");
  if (f.dim() != 1) type_error("inv_freq must be a 1-D tensor");
  void* pp = vector(&p, "positions", T, dev, at::kInt);
  void* fp = vector(&f, "inv_freq", f.size(0), dev, at::kFloat);
  return {static_cast<int32_t*>(pp), static_cast<float*>(fp), int_size(f.size(0), where)};
}
struct Gammas {
  void *q, *k;
  int bf16;
};
Gammas gammas(const at::Tensor* gq, const at::Tensor* gk, int64_t D, c10::Device dev) {
  int b = 0;
  if (gq) b = is_bf16(gq->scalar_type(), "gamma_q");
  if (gk) b = is_bf16(gk->scalar_type(), "gamma_k");
  if (gq && gk && gq->scalar_type() != gk->scalar_type()) type_error("gamma_q and gamma_k must have the same type");
  return {vector(gq, "gamma_q", D, dev), vector(gk, "gamma_k", D, dev), b};
}

// (q, k, positions, inv_freq, gamma_q, gamma_k, eps, norm, interleaved, out_q, out_k, out_dtype) -> (q, k)
PyObject* qk_rope(PyObject* const* a) {
  const at::Tensor &q = needed(a[0], "q"), &k = needed(a[1], "k");
  const at::Tensor *gq = tensor(a[4], "gamma_q"), *gk = tensor(a[5], "gamma_k"), *oq = tensor(a[9], "out_q"),
                   *ok = tensor(a[10], "out_k");
  const double eps = number(a[6]);
  const bool norm = truth(a[7]), inter = truth(a[8]);
  const c10::Device dev = q.device();
  const Heads n = heads_of(q, k);
  const at::ScalarType xt = q.scalar_type();
  const int xb = is_bf16(xt, "q");
  const nvfp4_tokens qv = tokens(q, "q", dev), kv = tokens(k, "k", dev, n.T, n.Hk, n.D, xt);
  const Rotation r = rotation(a[2], a[3], n.T, dev, "nvfp4_qk_rope");
  const Gammas g = gammas(gq, gk, n.D, dev);
  const at::ScalarType yt = dtype_of(a[11], oq ? oq->scalar_type() : ok ? ok->scalar_type() : xt);
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor mq, mk;
  const nvfp4_tokens oqv = result(oq, mq, "out_q", dev, n.T, n.Hq, n.D, yt),
                     okv = result(ok, mk, "out_k", dev, n.T, n.Hk, n.D, yt);
  check(nvfp4_qk_rope(&qv, &kv, xb, n.T, int_size(n.Hq, "nvfp4_qk_rope"), int_size(n.Hk, "nvfp4_qk_rope"),
                      int_size(n.D, "nvfp4_qk_rope"), r.rotated, inter, r.positions, r.inv_freq, norm, (float)eps, g.q,
                      g.k, g.bf16, &oqv, &okv, is_bf16(yt, "out_dtype"), stream_of(dev)),
        "nvfp4_qk_rope");
  return tuple(returned(a[9], oq, mq), returned(a[10], ok, mk));
}

// (dq, dk, q, k, positions, inv_freq, gamma_q, gamma_k, eps, norm, interleaved, out_q, out_k, want_dgamma)
//   -> (dq, dk, dgamma_q, dgamma_k)
PyObject* qk_rope_backward(PyObject* const* a) {
  const char* where = "nvfp4_qk_rope_backward";
  const at::Tensor &dq = needed(a[0], "dq"), &dk = needed(a[1], "dk");
  const at::Tensor *q = tensor(a[2], "q"), *k = tensor(a[3], "k"), *gq = tensor(a[6], "gamma_q"),
                   *gk = tensor(a[7], "gamma_k"), *oq = tensor(a[11], "out_q"), *ok = tensor(a[12], "out_k");
  const double eps = number(a[8]);
  const bool norm = truth(a[9]), inter = truth(a[10]), want = truth(a[13]) && norm;
  if (norm && (!q || !k)) type_error("q and k must be tensors (the gradient of the norm needs them)");
  if (!q != !k) type_error("q and k must be given together");
  const c10::Device dev = dq.device();
  const Heads n = heads_of(dq, dk);
  const at::ScalarType yt = dq.scalar_type(), xt = q ? q->scalar_type() : yt;
  const int yb = is_bf16(yt, "dq"), xb = is_bf16(xt, "q");
  const nvfp4_tokens dqv = tokens(dq, "dq", dev), dkv = tokens(dk, "dk", dev, n.T, n.Hk, n.D, yt);
  nvfp4_tokens qv = {}, kv = {};
  if (q) {
    qv = tokens(*q, "q", dev, n.T, n.Hq, n.D, xt);
    kv = tokens(*k, "k", dev, n.T, n.Hk, n.D, xt);
  }
  const Rotation r = rotation(a[4], a[5], n.T, dev, where);
  const Gammas g = gammas(gq, gk, n.D, dev);
  const int Hq = int_size(n.Hq, where), Hk = int_size(n.Hk, where), D = int_size(n.D, where);
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor mq, mk;
  const nvfp4_tokens oqv = result(oq, mq, "out_q", dev, n.T, n.Hq, n.D, xt),
                     okv = result(ok, mk, "out_k", dev, n.T, n.Hk, n.D, xt);
  Floats f(dev);
  const int64_t aq = want ? f.add(n.D) : 0, ak = want ? f.add(n.D) : 0;
  f.make();
  Workspace ws;
  if (want) ws = Workspace(nvfp4_qk_rope_backward_workspace(n.T, Hq, Hk, D), "nvfp4_qk_rope_backward_workspace", dev);
  check(nvfp4_qk_rope_backward(&dqv, &dkv, yb, &qv, &kv, xb, n.T, Hq, Hk, D, r.rotated, inter, r.positions, r.inv_freq,
                               norm, (float)eps, g.q, g.k, g.bf16, &oqv, &okv, want ? f.ptr(aq) : nullptr,
                               want ? f.ptr(ak) : nullptr, ws.p, ws.n, stream_of(dev)),
        where);
  return tuple(returned(a[11], oq, mq), returned(a[12], ok, mk), want ? THPVariable_Wrap(f.view(aq, n.D)) : none(),
               want ? THPVariable_Wrap(f.view(ak, n.D)) : none());
}

// The cache's five tensors (k_codes, k_scales, v_codes, v_scales, alpha).
nvfp4_kv_cache cache_of(PyObject* const* a, c10::Device dev, const char* where) {
  static const char* names[4] = {"k_codes", "k_scales", "v_codes", "v_scales"};
  const at::Tensor* t[4];
  for (int i = 0; i < 4; ++i) {
    t[i] = &needed(a[i], names[i]);
    if (t[i]->dim() != 4) type_error(std::string(names[i]) + " must be a 4-D tensor (pages, heads, rows, bytes)");
    if (t[i]->scalar_type() != at::kByte) type_error(std::string(names[i]) + " must be torch.uint8");
    on_device(*t[i], names[i], dev);
    if (t[i]->size(3) > 1 && t[i]->stride(3) != 1) value_error(std::string(names[i]) + " must have contiguous rows");
  }
  const at::Tensor& kc = *t[0];
  const int64_t P = kc.size(0), H = kc.size(1), S = kc.size(2), D = 2 * kc.size(3);
  if (D % 32 != 0) throw Status{NVFP4_ERR_SHAPE, where};
  for (int i = 1; i < 4; ++i) {
    const int64_t bytes = i == 2 ? D / 2 : D / 16;
    if (t[i]->size(0) != P || t[i]->size(1) != H || t[i]->size(2) != S || t[i]->size(3) != bytes)
      value_error(std::string(names[i]) + " must have shape (" + std::to_string(P) + ", " + std::to_string(H) + ", " +
                  std::to_string(S) + ", " + std::to_string(bytes) + ") (got " + shape_of(*t[i]) + ")");
  }
  int64_t st[4][3];  // axes of one entry are not stepped over
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 3; ++j) st[i][j] = t[i]->size(j) > 1 ? t[i]->stride(j) : 0;
  for (int j = 0; j < 3; ++j)
    if (st[0][j] != st[2][j] || st[1][j] != st[3][j]) value_error("keys and values must have the same strides");
  const at::Tensor& alpha = needed(a[4], "alpha");
  nvfp4_kv_cache c = {};
  c.alpha_dev = static_cast<float*>(vector(&alpha, "alpha", 2, dev, at::kFloat));
  c.k_codes = static_cast<uint8_t*>(t[0]->data_ptr());
  c.k_scales = static_cast<uint8_t*>(t[1]->data_ptr());
  c.v_codes = static_cast<uint8_t*>(t[2]->data_ptr());
  c.v_scales = static_cast<uint8_t*>(t[3]->data_ptr());
  c.pages = P;
  c.heads = int_size(H, where);
  c.page_size = int_size(S, where);
  c.dim = int_size(D, where);
  c.code_page = st[0][0];
  c.code_head = st[0][1];
  c.code_row = st[0][2];
  c.scale_page = st[1][0];
  c.scale_head = st[1][1];
  c.scale_row = st[1][2];
  return c;
}

// (starts, lengths, table)
nvfp4_batch batch_of(PyObject* const* a, c10::Device dev) {
  const at::Tensor &s = needed(a[0], "starts"), &l = needed(a[1], "lengths"), &t = needed(a[2], "pages");
  if (l.dim() != 1) type_error("lengths must be a 1-D tensor");
  if (t.dim() != 2) type_error("pages must be a 2-D tensor (sequences, pages of each)");
  const int64_t B = l.size(0);
  nvfp4_batch b = {};
  b.starts = static_cast<int32_t*>(vector(&s, "starts", B + 1, dev, at::kInt));
  b.lengths = static_cast<int32_t*>(vector(&l, "lengths", B, dev, at::kInt));
  on_device(t, "pages", dev);
  if (t.scalar_type() != at::kInt) type_error("pages must be torch.int32");
  if (t.size(0) != B) value_error("pages must have a row for each of the " + std::to_string(B) + " lengths");
  if (t.size(1) > 1 && t.stride(1) != 1) value_error("pages must have unit stride along columns");
  b.table = static_cast<int32_t*>(t.data_ptr());
  b.sequences = B;
  b.table_width = t.size(1);
  b.table_stride = B > 1 ? t.stride(0) : 0;
  return b;
}
int* status_of(PyObject* o, c10::Device dev) {
  return static_cast<int*>(vector(tensor(o, "status"), "status", 1, dev, at::kInt));
}

// (k, v, k_codes, k_scales, v_codes, v_scales, alpha, starts, lengths, pages, status) -> None
PyObject* cache_write(PyObject* const* a) {
  const char* where = "nvfp4_cache_write";
  const at::Tensor &k = needed(a[0], "k"), &v = needed(a[1], "v");
  const c10::Device dev = k.device();
  const nvfp4_tokens kv = tokens(k, "k", dev);
  const at::ScalarType t = k.scalar_type();
  const int b = is_bf16(t, "k");
  const nvfp4_kv_cache c = cache_of(a + 2, dev, where);
  const int64_t T = k.size(0);
  tokens(k, "k", dev, T, c.heads, c.dim, t);
  const nvfp4_tokens vv = tokens(v, "v", dev, T, c.heads, c.dim, t);
  const nvfp4_batch batch = batch_of(a + 7, dev);
  int* status = status_of(a[10], dev);
  c10::cuda::CUDAGuard guard(dev);
  check(nvfp4_cache_write(&kv, &vv, b, T, &c, &batch, status, stream_of(dev)), where);
  return none();
}

// (k_codes, k_scales, v_codes, v_scales, alpha, starts, lengths, pages, tokens, out_k, out_v, out_dtype, want_k,
//  want_v, status) -> (k, v)
PyObject* cache_read(PyObject* const* a) {
  const char* where = "nvfp4_cache_read";
  const c10::Device dev = needed(a[0], "k_codes").device();
  const nvfp4_kv_cache c = cache_of(a, dev, where);
  const nvfp4_batch batch = batch_of(a + 5, dev);
  const at::Tensor *ok = tensor(a[9], "out_k"), *ov = tensor(a[10], "out_v");
  const bool want[2] = {truth(a[12]), truth(a[13])};
  const at::ScalarType t = dtype_of(a[11], ok ? ok->scalar_type() : ov ? ov->scalar_type() : at::kBFloat16);
  int64_t T = 0;
  if (a[8] != Py_None)
    T = integer(a[8]);
  else if (ok || ov)
    T = (ok ? ok : ov)->dim() > 0 ? (ok ? ok : ov)->size(0) : 0;
  else
    type_error("tokens must be an integer where no result tensor is given");
  if (T < 0 || T > INT_MAX) throw Status{NVFP4_ERR_SHAPE, where};
  int* status = status_of(a[14], dev);
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor mk, mv;
  nvfp4_tokens k = {}, v = {};
  if (want[0]) k = result(ok, mk, "out_k", dev, T, c.heads, c.dim, t);
  if (want[1]) v = result(ov, mv, "out_v", dev, T, c.heads, c.dim, t);
  check(nvfp4_cache_read(&k, &v, is_bf16(t, "out_dtype"), T, &c, &batch, status, stream_of(dev)), where);
  return tuple(want[0] ? returned(a[9], ok, mk) : none(), want[1] ? returned(a[10], ov, mv) : none());
}

// (q, k_codes, k_scales, v_codes, v_scales, alpha, starts, lengths, pages, scale, causal, window, sinks, out, want_lse,
//  status) -> (o, lse)
PyObject* cache_attention(PyObject* const* a) {
  const char* where = "nvfp4_cache_attention";
  const at::Tensor& q = needed(a[0], "q");
  const c10::Device dev = q.device();
  const nvfp4_tokens qv = tokens(q, "q", dev);
  if (q.scalar_type() != at::kBFloat16)
    type_error(std::string("q must be torch.bfloat16 (got ") + c10::toString(q.scalar_type()) + ")");
  const nvfp4_kv_cache c = cache_of(a + 1, dev, where);
  const int64_t T = q.size(0), H = q.size(1);
  tokens(q, "q", dev, T, H, c.dim, at::kBFloat16);
  const nvfp4_batch batch = batch_of(a + 6, dev);
  const double scale = a[9] == Py_None ? 1.0 / std::sqrt((double)c.dim) : number(a[9]);
  const bool causal = truth(a[10]), lse = truth(a[14]);
  const int64_t window = integer(a[11]), sinks = integer(a[12]);
  const at::Tensor* out = tensor(a[13], "out");
  int* status = status_of(a[15], dev);
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor made, ml;
  const nvfp4_tokens ov = result(out, made, "out", dev, T, H, c.dim, at::kBFloat16);
  if (lse) ml = fresh({T, H}, at::kFloat, dev);
  const int hq = int_size(H, where);
  const Workspace ws(nvfp4_cache_attention_workspace(T, hq, c.heads, c.dim, batch.sequences),
                     "nvfp4_cache_attention_workspace", dev);
  check(nvfp4_cache_attention(&qv, T, hq, &c, &batch, (float)scale, causal, window, sinks, &ov,
                              lse ? ml.data_ptr<float>() : nullptr, ws.p, ws.n, status, stream_of(dev)),
        where);
  return tuple(returned(a[13], out, made), lse ? THPVariable_Wrap(std::move(ml)) : none());
}

PyMethodDef methods[] = {method<qk_rope, 12>("qk_rope"),
                         method<qk_rope_backward, 14>("qk_rope_backward"),
                         method<cache_write, 11>("cache_write"),
                         method<cache_read, 15>("cache_read"),
                         method<cache_attention, 16>("cache_attention"),
                         {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nvfp4_attention", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nvfp4_attention() { return PyModule_Create(&module); }
