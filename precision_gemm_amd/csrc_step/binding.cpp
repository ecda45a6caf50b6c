// CPython binding of the norms and of the AdamW step on torch tensors: argument checks, output
// allocation and marshalling, nothing else.
//
// Arguments come by position from precision_gemm_amd/norm.py and optimizer.py, which document them and
// make the tensors' device current.  A call returns its outputs, or the library's status as an int
// where that is not LORA_OK.
#include "../csrc_attn/binding_util.hpp"

namespace {

int32_t width(const Tensor& t, const char* name) {
  if (t.dim() != 2 || t.size(1) > INT32_MAX) throw Refused(std::string(name) + " must be [tokens, channels]");
  return (int32_t)t.size(1);
}

// x, weight, bias, residual, eps, rms, out, sum_out, stream -> (y, h), h None where y has taken its place
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensor& x = req(a[0], "x");
    const int32_t T = tokens(x, "x"), K = width(x, "x");
    const at::Device dev = x.device();
    const Rows rx = rows(x, "x", K, T, dev);
    const float* w = static_cast<float*>(need_or_null(opt(a[1], "weight"), "weight", at::kFloat, {K}, dev));
    const float* b = static_cast<float*>(need_or_null(opt(a[2], "bias"), "bias", at::kFloat, {K}, dev));
    const Tensor *res = opt(a[3], "residual"), *out = opt(a[6], "out"), *so = opt(a[7], "sum_out");
    if (so && !res) throw Refused("sum_out is for a residual");
    const float eps = (float)number(a[4]);
    const bool rms = truth(a[5], "rms");
    Rows rr{nullptr, K}, rs{nullptr, K};
    if (res) rr = rows(*res, "residual", K, T, dev);
    const Tensor y = out ? *out : empty({T, K}, at::kBFloat16, dev);
    const Tensor h = !res ? x : so ? *so : empty({T, K}, at::kBFloat16, dev);
    const Rows ry = rows(y, "out", K, T, dev);
    if (res) rs = rows(h, "sum_out", K, T, dev);
    const lora_status s = lora_layer_norm(rx.p, rx.ld, rr.p, rr.ld, T, K, w, b, eps, rms, ry.p, ry.ld, rs.p, rs.ld, stream(a[8]));
    if (s != LORA_OK) return status(s);
    if (!res && T > 0 && ry.p == rx.p) return Py_BuildValue("(NO)", THPVariable_Wrap(y), Py_None);
    return Py_BuildValue("(NN)", THPVariable_Wrap(y), THPVariable_Wrap(h));
  });
}

// dy, h, weight, dsum, eps, rms, weight_grad, bias_grad, dx, dweight, dbias, workspace, stream -> (dx, dweight, dbias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const Tensor &dy = req(a[0], "dy"), &h = req(a[1], "h");
    const int32_t T = tokens(dy, "dy"), K = width(dy, "dy");
    const at::Device dev = dy.device();
    const Rows rg = rows(dy, "dy", K, T, dev), rh = rows(h, "h", K, T, dev);
    const float* w = static_cast<float*>(need_or_null(opt(a[2], "weight"), "weight", at::kFloat, {K}, dev));
    const Tensor *ds = opt(a[3], "dsum"), *out = opt(a[8], "dx"), *ow = opt(a[9], "dweight"), *ob = opt(a[10], "dbias"),
                 *ws = opt(a[11], "workspace");
    const float eps = (float)number(a[4]);
    const bool rms = truth(a[5], "rms"), want_w = truth(a[6], "weight_grad"), want_b = truth(a[7], "bias_grad");
    if ((ow && !want_w) || (ob && !want_b)) throw Refused("dweight and dbias are for gradients that are wanted");
    Rows rs{nullptr, K};
    if (ds) rs = rows(*ds, "dsum", K, T, dev);
    const Tensor dx = out ? *out : empty({T, K}, at::kBFloat16, dev);
    const Rows rx = rows(dx, "dx", K, T, dev);
    Tensor dw, db, work;
    void* pw = nullptr;
    if (want_w) dw = ow ? *ow : empty({K}, at::kFloat, dev);
    if (want_b) db = ob ? *ob : empty({K}, at::kFloat, dev);
    if (want_w || want_b) {
      work = ws ? *ws : empty({std::max<int64_t>(16, (int64_t)lora_layer_norm_backward_workspace_bytes(T, K))}, at::kByte, dev);
      pw = need(work, "workspace", at::kByte, {work.numel()}, dev);
    }
    const lora_status s = lora_layer_norm_backward(
        rg.p, rg.ld, rh.p, rh.ld, w, rs.p, rs.ld, T, K, eps, rms, rx.p, rx.ld,
        want_w ? static_cast<float*>(need(dw, "dweight", at::kFloat, {K}, dev)) : nullptr,
        want_b ? static_cast<float*>(need(db, "dbias", at::kFloat, {K}, dev)) : nullptr, pw, pw ? (size_t)work.numel() : 0,
        stream(a[12]));
    if (s != LORA_OK) return status(s);
    PyObject* none[2] = {want_w ? THPVariable_Wrap(dw) : Py_NewRef(Py_None), want_b ? THPVariable_Wrap(db) : Py_NewRef(Py_None)};
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dx), none[0], none[1]);
  });
}

// tiles, group_first, state_bits, hyper, active, steps, clip, grad_norm, status, workspace, stream -> grad_norm or None
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Tensor &tiles = req(a[0], "tiles"), &first = req(a[1], "group_first");
    const at::Device dev = tiles.device();
    const int64_t n_tiles = tiles.size(0);
    const int32_t G = tokens(first, "group_first") - 1;
    const void* pl = need(tiles, "tiles", at::kByte, {n_tiles, (int64_t)sizeof(lora_adamw_tile)}, dev);
    const void* pf = need(first, "group_first", at::kInt, {(int64_t)G + 1}, dev);
    const void* ph = need(req(a[3], "hyper"), "hyper", at::kDouble, {G, 6}, dev);
    const void* pa = need_or_null(opt(a[4], "active"), "active", at::kInt, {G}, dev);
    void* ps = need(req(a[5], "steps"), "steps", at::kInt, {G}, dev);
    const bool clip = truth(a[6], "clip");
    const Tensor *on = opt(a[7], "grad_norm"), &ws = req(a[9], "workspace");
    if (on && !clip) throw Refused("grad_norm is for a step that clips");
    Tensor norm;
    if (clip) norm = on ? *on : empty({G}, at::kFloat, dev);
    void* pw = need(ws, "workspace", at::kByte, {ws.numel()}, dev);
    const lora_status s = lora_adamw_step(
        static_cast<const lora_adamw_tile*>(pl), n_tiles, static_cast<const int32_t*>(pf), G, int32(a[2]),
        static_cast<const double*>(ph), static_cast<const int32_t*>(pa), static_cast<int32_t*>(ps),
        clip ? static_cast<float*>(need(norm, "grad_norm", at::kFloat, {G}, dev)) : nullptr, status_word(a[8], dev), pw,
        (size_t)ws.numel(), stream(a[10]));
    if (s != LORA_OK) return status(s);
    if (!clip) Py_RETURN_NONE;
    return THPVariable_Wrap(norm);
  });
}

PyMethodDef methods[] = {ENTRY(layer_norm), ENTRY(layer_norm_backward), ENTRY(adamw_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&module); }
