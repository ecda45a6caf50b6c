// CPython binding of the attention block's calls on torch tensors: argument checks, output
// allocation and marshalling, nothing else.  A decode step's append or head norm takes 3.2 us
// on the GPU; the same binding through ctypes took 14 to 15 us of host time a call, four
// times the work it launches, this one 5.5 to 6.1.
//
// Arguments come by position from precision_gemm_amd/attention.py, which documents them and makes
// the tensors' device current.  A call returns its outputs, or the library's status as an int
// where that is not LORA_OK.
#include "binding_util.hpp"

namespace {

// The rotation's arguments.
struct Rope {
  int32_t n_axes = 0;  // 0: one position a token
  const uint8_t* pair_axes = nullptr;
  const int32_t* pos = nullptr;
  const float* table = nullptr;
  int32_t max_pos = 0, rot = 0, interleaved = 0;
  const float *qw = nullptr, *kw = nullptr;
  float eps = 0.f;
};
Rope rope(PyObject* positions, PyObject* pair_axes, PyObject* cos_sin, PyObject* q_weight, PyObject* k_weight, PyObject* eps,
          PyObject* interleaved, int64_t T, int64_t D, const at::Device& dev) {
  Rope r;
  if (pair_axes != Py_None && cos_sin == Py_None) throw Refused("pair_axes is for a rotation: it needs cos_sin");
  if (const Tensor* t = opt(cos_sin, "cos_sin")) {
    if (t->dim() != 2 || t->size(0) > INT32_MAX || t->size(1) > INT32_MAX) throw Refused("cos_sin must be [positions, rot]");
    r.max_pos = (int32_t)t->size(0);
    r.rot = (int32_t)t->size(1);
    r.table = static_cast<float*>(need(*t, "cos_sin", at::kFloat, {r.max_pos, r.rot}, dev));
    const Tensor& pos = req(positions, "positions");
    if (pair_axes == Py_None) {
      r.pos = static_cast<int32_t*>(need(pos, "positions", at::kInt, {T}, dev));
    } else {
      if (!PyBytes_Check(pair_axes) || PyBytes_GET_SIZE(pair_axes) != r.rot / 2)
        throw Refused("pair_axes must be bytes, an axis for each of the " + std::to_string(r.rot / 2) + " pairs");
      if (pos.dim() != 2 || pos.size(0) < 1 || pos.size(0) > 4) throw Refused("with pair_axes, positions must be [1 to 4 axes, tokens]");
      r.n_axes = (int32_t)pos.size(0);
      r.pair_axes = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(pair_axes));
      for (int32_t i = 0; i < r.rot / 2; ++i)
        if (r.pair_axes[i] >= r.n_axes) throw Refused("pair_axes names axis " + std::to_string(r.pair_axes[i]) + " of " + std::to_string(r.n_axes));
      r.pos = static_cast<int32_t*>(need(pos, "positions", at::kInt, {r.n_axes, T}, dev));
    }
  }
  const Tensor *qw = opt(q_weight, "q_weight"), *kw = opt(k_weight, "k_weight");
  if (!qw != !kw) throw Refused("q_weight and k_weight go together");
  r.qw = static_cast<float*>(need_or_null(qw, "q_weight", at::kFloat, {D}, dev));
  r.kw = static_cast<float*>(need_or_null(kw, "k_weight", at::kFloat, {D}, dev));
  r.eps = (float)number(eps);
  r.interleaved = truth(interleaved, "interleaved");
  return r;
}

// A paged cache's arguments.
struct Cache { int32_t fmt; void *k, *v; const float *ks, *vs; int32_t n_pages, n_kv, page, D; };
Cache cache(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso, const at::Device& dev) {
  const Tensor &k = req(ko, "k_cache"), &v = req(vo, "v_cache");
  const at::ScalarType type = k.scalar_type();
  if ((type != at::kBFloat16 && type != at::kFloat8_e4m3fn) || k.dim() != 4)
    throw Refused("k_cache must be [pages, kv heads, page size, head_dim] in bfloat16 or float8_e4m3fn");
  for (int64_t n : k.sizes())
    if (n > INT32_MAX) throw Refused("k_cache is too large");
  Cache c{type == at::kBFloat16 ? LORA_KV_BF16 : LORA_KV_FP8_E4M3, nullptr, nullptr, nullptr, nullptr, (int32_t)k.size(0),
          (int32_t)k.size(1), (int32_t)k.size(2), (int32_t)k.size(3)};
  const Tensor *ks = opt(kso, "k_scale"), *vs = opt(vso, "v_scale");
  if (c.fmt == LORA_KV_BF16 && (ks || vs)) throw Refused("k_scale and v_scale are for an 8-bit cache");
  if (c.fmt != LORA_KV_BF16 && (!ks || !vs)) throw Refused("an 8-bit cache needs k_scale and v_scale");
  c.v = need(v, "v_cache", type, k.sizes(), dev);
  c.k = need(k, "k_cache", type, k.sizes(), dev);
  c.ks = static_cast<float*>(need_or_null(ks, "k_scale", at::kFloat, {c.n_kv}, dev));
  c.vs = static_cast<float*>(need_or_null(vs, "v_scale", at::kFloat, {c.n_kv}, dev));
  return c;
}

// qkv, positions, n_q, n_kv, D, cos_sin, q_weight, k_weight, eps, interleaved, q_out, k_out, status, pair_axes, stream
// -> (q, k)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const Tensor& qkv = req(a[0], "qkv");
    const int32_t T = tokens(qkv, "qkv"), n_q = int32(a[2]), n_kv = int32(a[3]), D = int32(a[4]);
    const at::Device dev = qkv.device();
    const Rows x = rows(qkv, "qkv", ((int64_t)n_q + 2ll * n_kv) * D, T, dev);
    const Rope r = rope(a[1], a[13], a[5], a[6], a[7], a[8], a[9], T, D, dev);
    const Tensor *qo = opt(a[10], "q_out"), *ko = opt(a[11], "k_out");
    if (n_q < 1 || n_kv < 1 || D < 1) return status(LORA_ERR_INVALID_ARG);
    const Tensor q = qo ? *qo : empty({T, n_q, D}, at::kBFloat16, dev), k = ko ? *ko : empty({T, n_kv, D}, at::kBFloat16, dev);
    const Rows ro = rows(q, "q_out", (int64_t)n_q * D, T, dev), rk = rows(k, "k_out", (int64_t)n_kv * D, T, dev);
    int32_t* word = status_word(a[12], dev);
    const lora_status s =
        r.n_axes ? lora_qk_norm_rope_axes(x.p, x.ld, r.pos, r.n_axes, r.pair_axes, T, n_q, n_kv, D, r.table, r.max_pos, r.rot,
                                          r.interleaved, r.qw, r.kw, r.eps, ro.p, ro.ld, rk.p, rk.ld, word, stream(a[14]))
                 : lora_qk_norm_rope(x.p, x.ld, r.pos, T, n_q, n_kv, D, r.table, r.max_pos, r.rot, r.interleaved, r.qw, r.kw,
                                     r.eps, ro.p, ro.ld, rk.p, rk.ld, word, stream(a[14]));
    if (s != LORA_OK) return status(s);
    return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(k));
  });
}

// qkv, positions, dq, dk, dv, cos_sin, q_weight, k_weight, eps, interleaved, dqkv, dq_weight, dk_weight, workspace, status,
// pair_axes, stream -> (dqkv, dq_weight, dk_weight)
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const Tensor &dq = req(a[2], "dq"), &dk = req(a[3], "dk");
    if (dq.dim() != 3 || dk.dim() != 3) throw Refused("dq and dk must be [tokens, heads, head_dim]");
    const int32_t T = tokens(dq, "dq"), n_q = (int32_t)dq.size(1), n_kv = (int32_t)dk.size(1), D = (int32_t)dq.size(2);
    const at::Device dev = dq.device();
    const int64_t width = ((int64_t)n_q + 2ll * n_kv) * D;
    void* pq = need(dq, "dq", at::kBFloat16, {T, n_q, D}, dev);
    void* pk = need(dk, "dk", at::kBFloat16, {T, n_kv, D}, dev);
    const Tensor* dv = opt(a[4], "dv");
    void* pv = need_or_null(dv, "dv", at::kBFloat16, {T, n_kv, D}, dev);
    const Rope r = rope(a[1], a[15], a[5], a[6], a[7], a[8], a[9], T, D, dev);
    const Rows x = r.qw ? rows(req(a[0], "qkv"), "qkv", width, T, dev) : Rows{nullptr, width};
    const Tensor* out = opt(a[10], "dqkv");
    if (!out && !dv) throw Refused("without dv, dqkv has to be given (its value columns are not written)");
    const Tensor dqkv = out ? *out : empty({T, width}, at::kBFloat16, dev);
    const Rows d = rows(dqkv, "dqkv", width, T, dev);
    Tensor dqw, dkw, ws;
    if (r.qw) {
      const Tensor *qw = opt(a[11], "dq_weight"), *kw = opt(a[12], "dk_weight"), *w = opt(a[13], "workspace");
      dqw = qw ? *qw : empty({D}, at::kFloat, dev);
      dkw = kw ? *kw : empty({D}, at::kFloat, dev);
      ws = w ? *w : empty({std::max<int64_t>(16, (int64_t)lora_qk_norm_rope_backward_workspace_bytes(T, D))}, at::kByte, dev);
    }
    float* gq = r.qw ? static_cast<float*>(need(dqw, "dq_weight", at::kFloat, {D}, dev)) : nullptr;
    float* gk = r.qw ? static_cast<float*>(need(dkw, "dk_weight", at::kFloat, {D}, dev)) : nullptr;
    int32_t* word = status_word(a[14], dev);
    void* pw = r.qw ? need(ws, "workspace", at::kByte, {ws.numel()}, dev) : nullptr;
    const size_t bytes = r.qw ? (size_t)ws.numel() : 0;
    const uint16_t *g0 = static_cast<uint16_t*>(pq), *g1 = static_cast<uint16_t*>(pk), *g2 = static_cast<uint16_t*>(pv);
    const lora_status s =
        r.n_axes ? lora_qk_norm_rope_axes_backward(x.p, x.ld, r.pos, r.n_axes, r.pair_axes, g0, g1, g2, T, n_q, n_kv, D, r.table,
                                                   r.max_pos, r.rot, r.interleaved, r.qw, r.kw, r.eps, d.p, d.ld, gq, gk, word,
                                                   pw, bytes, stream(a[16]))
                 : lora_qk_norm_rope_backward(x.p, x.ld, r.pos, g0, g1, g2, T, n_q, n_kv, D, r.table, r.max_pos, r.rot,
                                              r.interleaved, r.qw, r.kw, r.eps, d.p, d.ld, gq, gk, word, pw, bytes, stream(a[16]));
    if (s != LORA_OK) return status(s);
    if (!r.qw) return Py_BuildValue("(NOO)", THPVariable_Wrap(dqkv), Py_None, Py_None);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dqkv), THPVariable_Wrap(dqw), THPVariable_Wrap(dkw));
  });
}

// qkv, positions, slots, k_cache, v_cache, n_q, cos_sin, q_weight, k_weight, eps, interleaved, k_scale, v_scale, q_out, status,
// pair_axes, stream -> q
PyObject* rope_append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const Tensor& qkv = req(a[0], "qkv");
    const at::Device dev = qkv.device();
    const Cache c = cache(a[3], a[4], a[11], a[12], dev);
    const int32_t T = tokens(qkv, "qkv"), n_q = int32(a[5]);
    const Rows x = rows(qkv, "qkv", ((int64_t)n_q + 2ll * c.n_kv) * c.D, T, dev);
    const Rope r = rope(a[1], a[15], a[6], a[7], a[8], a[9], a[10], T, c.D, dev);
    const void* slots = need(req(a[2], "slots"), "slots", at::kInt, {T}, dev);
    if (n_q < 1 || c.n_kv < 1 || c.D < 1) return status(LORA_ERR_INVALID_ARG);
    const Tensor* qo = opt(a[13], "q_out");
    const Tensor q = qo ? *qo : empty({T, n_q, c.D}, at::kBFloat16, dev);
    const Rows ro = rows(q, "q_out", (int64_t)n_q * c.D, T, dev);
    const int32_t* at = static_cast<const int32_t*>(slots);
    int32_t* word = status_word(a[14], dev);
    const lora_status s =
        r.n_axes ? lora_rope_axes_append_kv(x.p, x.ld, r.pos, r.n_axes, r.pair_axes, at, T, n_q, c.n_kv, c.D, r.table, r.max_pos,
                                            r.rot, r.interleaved, r.qw, r.kw, r.eps, ro.p, ro.ld, c.fmt, c.k, c.v, c.ks, c.vs,
                                            c.n_pages, c.page, word, stream(a[16]))
                 : lora_rope_append_kv(x.p, x.ld, r.pos, at, T, n_q, c.n_kv, c.D, r.table, r.max_pos, r.rot, r.interleaved, r.qw,
                                       r.kw, r.eps, ro.p, ro.ld, c.fmt, c.k, c.v, c.ks, c.vs, c.n_pages, c.page, word,
                                       stream(a[16]));
    if (s != LORA_OK) return status(s);
    return THPVariable_Wrap(q);
  });
}

// parents, q_indptr, max_q, status, stream -> mask
PyObject* tree_mask(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Tensor &par = req(a[0], "parents"), &ip = req(a[1], "q_indptr");
    const int32_t T = tokens(par, "parents"), B = tokens(ip, "q_indptr") - 1, max_q = int32(a[2]);
    const at::Device dev = par.device();
    const void* pp = need(par, "parents", at::kInt, {T}, dev);
    const void* pi = need(ip, "q_indptr", at::kInt, {B + 1}, dev);
    const int32_t words = std::max(1, (int32_t)(((int64_t)max_q + 63) / 64));
    const Tensor mask = empty({T, words}, at::kLong, dev);
    const lora_status s = lora_tree_mask(static_cast<const int32_t*>(pp), static_cast<const int32_t*>(pi), B, T, max_q, words,
                                         static_cast<uint64_t*>(mask.data_ptr()), status_word(a[3], dev), stream(a[4]));
    if (s != LORA_OK) return status(s);
    return THPVariable_Wrap(mask);
  });
}

// q, k_cache, v_cache, page_table, kv_len, q_indptr, max_q, tree_mask, scale, k_scale, v_scale, out, lse, workspace, status,
// stream -> (out, lse)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const Tensor& q = req(a[0], "q");
    if (q.dim() != 3) throw Refused("q must be [tokens, heads, head_dim]");
    const at::Device dev = q.device();
    const int32_t T = tokens(q, "q"), n_q = (int32_t)q.size(1), D = (int32_t)q.size(2);
    const Tensor& kc = req(a[1], "k_cache");
    if (kc.dim() == 4 && kc.size(3) != D)
      throw Refused("q has heads of " + std::to_string(D) + " values, the cache of " + std::to_string(kc.size(3)));
    const Cache c = cache(a[1], a[2], a[9], a[10], dev);
    const Rows x = rows(q, "q", (int64_t)n_q * D, T, dev);
    const Tensor &table = req(a[3], "page_table"), &kv = req(a[4], "kv_len"), &ip = req(a[5], "q_indptr");
    const int32_t B = tokens(kv, "kv_len"), max_q = int32(a[6]);
    if (table.dim() != 2 || table.size(1) > INT32_MAX) throw Refused("page_table must be [sequences, max pages]");
    const int32_t max_pages = (int32_t)table.size(1);
    const Tensor* mask = opt(a[7], "tree_mask");
    int32_t words = 0;
    void* pm = nullptr;
    if (mask) {
      if ((mask->scalar_type() != at::kLong && mask->scalar_type() != at::kUInt64) || mask->dim() != 2 || mask->size(1) > INT32_MAX)
        throw Refused("tree_mask must be int64 or uint64 [tokens, words]");
      words = (int32_t)mask->size(1);
      pm = need(*mask, "tree_mask", mask->scalar_type(), {T, words}, dev);
    }
    const void* pt = need(table, "page_table", at::kInt, {B, max_pages}, dev);
    const void* pl = need(kv, "kv_len", at::kInt, {B}, dev);
    const void* pi = need(ip, "q_indptr", at::kInt, {(int64_t)B + 1}, dev);
    const Tensor *to = opt(a[11], "out"), *tl = opt(a[12], "lse"), *tw = opt(a[13], "workspace");
    const Tensor out = to ? *to : empty({T, n_q, D}, at::kBFloat16, dev), lse = tl ? *tl : empty({T, n_q}, at::kFloat, dev);
    const Tensor ws = tw ? *tw : empty({std::max<int64_t>(16, (int64_t)lora_tree_attention_workspace_bytes(n_q, c.n_kv, D, max_q))}, at::kByte, dev);
    void* po = need(out, "out", at::kBFloat16, {T, n_q, D}, dev);
    void* ps = need(lse, "lse", at::kFloat, {T, n_q}, dev);
    void* pw = need(ws, "workspace", at::kByte, {ws.numel()}, dev);
    const lora_status s = lora_tree_attention(
        x.p, x.ld, c.fmt, c.k, c.v, c.ks, c.vs, c.n_pages, c.page, static_cast<const int32_t*>(pt), max_pages,
        static_cast<const int32_t*>(pl), static_cast<const int32_t*>(pi), B, T, max_q, n_q, c.n_kv, D, static_cast<uint64_t*>(pm),
        words, (float)number(a[8]), static_cast<uint16_t*>(po), static_cast<float*>(ps), status_word(a[14], dev), pw,
        (size_t)ws.numel(), stream(a[15]));
    if (s != LORA_OK) return status(s);
    if (T > 0 && (B == 0 || max_q == 0)) {  // the library does nothing here; what it returns is defined all the same
      out.zero_();
      lse.fill_(-std::numeric_limits<double>::infinity());
      if (const Tensor* word = opt(a[14], "status")) word->bitwise_or_(LORA_ATTN_BAD_LENGTH);
    }
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
  });
}

PyMethodDef methods[] = {ENTRY(qk_norm_rope), ENTRY(qk_norm_rope_backward), ENTRY(rope_append_kv), ENTRY(tree_mask),
                         ENTRY(tree_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn() { return PyModule_Create(&module); }
