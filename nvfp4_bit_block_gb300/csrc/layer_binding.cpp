// layer_binding.cpp -- Python binding of include/nvfp4_layer.h: argument checks,
// result tensors and marshalling in C++.
//
// A call on one token takes the GPU about 4 us; the same checks and allocations
// in Python took 18 us more (one call of the layer norm with its statistics and
// amax: 22 us).  The small fp32 results of a call share one allocation.
#include "binding.h"
#include "nvfp4_layer.h"

namespace {

// An activation's code; a number that an int does not hold is none, and refused as the library would.
int activation(PyObject* o, const char* where) {
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  if (over != 0 || v < INT_MIN || v > INT_MAX) throw Status{NVFP4_ERR_FLAGS, where};
  return (int)v;
}

// (x, gamma, beta, eps, out, out_dtype, want_stats, want_amax) -> (y, mean, rstd, amax)
PyObject* layernorm(PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x");
  const at::Tensor *gamma = tensor(a[1], "gamma"), *beta = tensor(a[2], "beta");
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  const bool stats = truth(a[6]), amax = truth(a[7]);
  const c10::Device dev = x.device();
  const Matrix xm = matrix(x, "x", dev);
  const int xb = is_bf16(x.scalar_type(), "x");
  const int64_t M = x.size(0), N = x.size(1);
  int wb = 0;
  if (gamma) wb = is_bf16(gamma->scalar_type(), "gamma");
  if (beta) wb = is_bf16(beta->scalar_type(), "beta");
  if (gamma && beta && gamma->scalar_type() != beta->scalar_type()) type_error("gamma and beta must have the same type");
  void *gp = vector(gamma, "gamma", N, dev), *bp = vector(beta, "beta", N, dev);
  const at::Tensor* out = tensor(a[4], "out");
  const at::ScalarType yt = dtype_of(a[5], out ? out->scalar_type() : x.scalar_type());
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor made;
  if (!out) made = new_matrix(M, N, yt, dev);
  const Matrix ym = matrix(out ? *out : made, "out", dev, M, N, yt);
  Floats f(dev);
  const int64_t am = stats ? f.add(M) : 0, ar = stats ? f.add(M) : 0, aa = amax ? f.add(2) : 0;
  f.make();
  check(nvfp4_layernorm(xm.p, M, N, xm.ld, xb, gp, bp, wb, (float)eps, ym.p, ym.ld, is_bf16(yt, "out"),
                        stats ? f.ptr(am) : nullptr, stats ? f.ptr(ar) : nullptr, amax ? f.ptr(aa) : nullptr,
                        stream_of(dev)),
        "nvfp4_layernorm");
  if (stats && N == 0) {  // the library writes none; the mean of no values is 0 / 0
    f.view(am, M).fill_(NAN);
    f.view(ar, M).fill_(NAN);
  }
  return tuple(out ? given(a[4]) : THPVariable_Wrap(std::move(made)), stats ? THPVariable_Wrap(f.view(am, M)) : none(),
               stats ? THPVariable_Wrap(f.view(ar, M)) : none(), amax ? THPVariable_Wrap(f.view(aa, 2)) : none());
}

// (dy, x, mean, rstd, gamma, dres, out, want_dgamma, want_dbeta) -> (dx, dgamma, dbeta)
PyObject* layernorm_backward(PyObject* const* a) {
  const at::Tensor &dy = needed(a[0], "dy"), &x = needed(a[1], "x"), &mean = needed(a[2], "mean"),
                   &rstd = needed(a[3], "rstd");
  const at::Tensor *gamma = tensor(a[4], "gamma"), *dres = tensor(a[5], "dres"), *out = tensor(a[6], "out");
  const bool dgamma = truth(a[7]), dbeta = truth(a[8]);
  const c10::Device dev = x.device();
  const Matrix xm = matrix(x, "x", dev);
  const at::ScalarType xt = x.scalar_type();
  const int xb = is_bf16(xt, "x");
  const int64_t M = x.size(0), N = x.size(1);
  const int dyb = is_bf16(dy.scalar_type(), "dy");
  const Matrix dm = matrix(dy, "dy", dev, M, N, dy.scalar_type());
  const Matrix rm = dres ? matrix(*dres, "dres", dev, M, N, xt) : Matrix();
  void *mp = vector(&mean, "mean", M, dev, at::kFloat), *sp = vector(&rstd, "rstd", M, dev, at::kFloat);
  const int wb = gamma ? is_bf16(gamma->scalar_type(), "gamma") : 0;
  void* gp = vector(gamma, "gamma", N, dev);
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor made;
  if (!out) made = new_matrix(M, N, xt, dev);
  const Matrix om = matrix(out ? *out : made, "out", dev, M, N, xt);
  Floats f(dev);
  const int64_t ag = dgamma ? f.add(N) : 0, ab = dbeta ? f.add(N) : 0;
  f.make();
  const Workspace ws(nvfp4_layernorm_backward_workspace(M, N), "nvfp4_layernorm_backward_workspace", dev);
  check(nvfp4_layernorm_backward(dm.p, dm.ld, dyb, xm.p, xm.ld, xb, M, N, static_cast<float*>(mp),
                                 static_cast<float*>(sp), gp, wb, rm.p, rm.ld, om.p, om.ld,
                                 dgamma ? f.ptr(ag) : nullptr, dbeta ? f.ptr(ab) : nullptr, ws.p, ws.n, stream_of(dev)),
        "nvfp4_layernorm_backward");
  return tuple(out ? given(a[6]) : THPVariable_Wrap(std::move(made)), dgamma ? THPVariable_Wrap(f.view(ag, N)) : none(),
               dbeta ? THPVariable_Wrap(f.view(ab, N)) : none());
}

// (qa, sfa, alpha_a, qb, sfb, alpha_b, bias, act, residual, out, out_dtype, want_z, want_amax, status) -> (d, z, amax)
PyObject* linear(PyObject* const* a) {
  const at::Tensor &qa = needed(a[0], "qa"), &sfa = needed(a[1], "sfa"), &aa = needed(a[2], "alpha_a"),
                   &qb = needed(a[3], "qb"), &sfb = needed(a[4], "sfb"), &ab = needed(a[5], "alpha_b");
  const at::Tensor *bias = tensor(a[6], "bias"), *res = tensor(a[8], "residual"), *out = tensor(a[9], "out"),
                   *status = tensor(a[13], "status");
  const int act = activation(a[7], "nvfp4_linear");
  const bool want_z = truth(a[11]), want_amax = truth(a[12]);
  if (qa.dim() != 2 || qb.dim() != 2) type_error("qa and qb must be 2-D tensors");
  const c10::Device dev = qa.device();
  const int64_t M = qa.size(0), N = qb.size(0), half = qa.size(1), K = 2 * half;
  if (qb.size(1) != half) value_error("A and B must have the same K");
  const int64_t cols = (K / 16 + 3) / 4 * 4;  // scale columns of the tiled layout
  const auto u8 = at::kByte;
  void *ap = vector(&qa, "qa", M * half, dev, u8), *bp = vector(&qb, "qb", N * half, dev, u8);
  void *sap = vector(&sfa, "sfa", (M + 127) / 128 * 128 * cols, dev, u8);
  void *sbp = vector(&sfb, "sfb", (N + 127) / 128 * 128 * cols, dev, u8);
  void *aap = vector(&aa, "alpha_a", 1, dev, at::kFloat), *abp = vector(&ab, "alpha_b", 1, dev, at::kFloat);
  const int biasb = bias ? is_bf16(bias->scalar_type(), "bias") : 0;
  void* biasp = vector(bias, "bias", N, dev);
  void* stp = vector(status, "status", 1, dev, at::kInt);
  const at::ScalarType ot = dtype_of(a[10], out ? out->scalar_type() : at::kBFloat16);
  const int ob = is_bf16(ot, "out");
  if (want_amax && !ob) type_error("want_amax goes with a bfloat16 result (what nvfp4_quantize takes)");
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor made, z, amax;
  if (!out) made = new_matrix(M, N, ot, dev);
  const Matrix dm = matrix(out ? *out : made, "out", dev, M, N, ot);
  const Matrix rm = res ? matrix(*res, "residual", dev, M, N, ot) : Matrix();
  if (want_z) z = new_matrix(M, N, ot, dev);
  if (want_amax) amax = fresh({2}, at::kFloat, dev);
  const Workspace ws(nvfp4_linear_workspace(M, N, K), "nvfp4_linear_workspace", dev);
  auto bytes = [](void* p) { return static_cast<const uint8_t*>(p); };
  check(nvfp4_linear(bytes(ap), bytes(sap), static_cast<float*>(aap), bytes(bp), bytes(sbp), static_cast<float*>(abp), M,
                     N, K, biasp, biasb, act, rm.p, rm.ld, want_z ? z.data_ptr() : nullptr, N, dm.p, dm.ld, ob,
                     want_amax ? amax.data_ptr<float>() : nullptr, ws.p, ws.n, static_cast<int*>(stp), stream_of(dev)),
        "nvfp4_linear");
  return tuple(out ? given(a[9]) : THPVariable_Wrap(std::move(made)), want_z ? THPVariable_Wrap(std::move(z)) : none(),
               want_amax ? THPVariable_Wrap(std::move(amax)) : none());
}

// (dy, z, act, out, want_dz, want_dbias) -> (dz, dbias)
PyObject* act_backward(PyObject* const* a) {
  const at::Tensor& dy = needed(a[0], "dy");
  const at::Tensor *z = tensor(a[1], "z"), *out = tensor(a[3], "out");
  const int act = activation(a[2], "nvfp4_act_backward");
  const bool want_dz = truth(a[4]), want_dbias = truth(a[5]);
  const c10::Device dev = dy.device();
  const Matrix dm = matrix(dy, "dy", dev);
  const at::ScalarType t = dy.scalar_type();
  const int b = is_bf16(t, "dy");
  const int64_t M = dy.size(0), N = dy.size(1);
  const Matrix zm = z ? matrix(*z, "z", dev, M, N, t) : Matrix();
  c10::cuda::CUDAGuard guard(dev);
  at::Tensor made, dbias;
  Matrix om;
  if (want_dz) {
    if (!out) made = new_matrix(M, N, t, dev);
    om = matrix(out ? *out : made, "out", dev, M, N, t);
  }
  Workspace ws;
  if (want_dbias) {
    dbias = fresh({N}, at::kFloat, dev);
    ws = Workspace(nvfp4_act_backward_workspace(M, N), "nvfp4_act_backward_workspace", dev);
  }
  check(nvfp4_act_backward(dm.p, dm.ld, zm.p, zm.ld, M, N, b, act, om.p, om.ld,
                           want_dbias ? dbias.data_ptr<float>() : nullptr, ws.p, ws.n, stream_of(dev)),
        "nvfp4_act_backward");
  return tuple(!want_dz ? none() : (out ? given(a[3]) : THPVariable_Wrap(std::move(made))),
               want_dbias ? THPVariable_Wrap(std::move(dbias)) : none());
}

PyMethodDef methods[] = {method<layernorm, 8>("layernorm"), method<layernorm_backward, 9>("layernorm_backward"),
                         method<linear, 14>("linear"), method<act_backward, 6>("act_backward"), {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nvfp4_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nvfp4_layer() { return PyModule_Create(&module); }
