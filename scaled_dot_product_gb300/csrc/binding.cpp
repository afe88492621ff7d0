// Argument marshalling of the query/key norm and paged-cache calls, for sdpa.py.
//
// Single-token calls take 2 to 12 us on the GPU; filling the C structs in Python took 12 to 16 us of
// host time a call (strides, pointers and types one attribute at a time).  Here they are read from
// the tensors directly.  Nothing is computed: each function checks types and shapes, allocates the
// outputs the caller left out, fills the struct of include/sdpa.h and calls the entry point whose
// address sdpa.py passes (so that every call goes through the library it loaded).  It returns the
// outputs, or the entry point's non-zero status as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <sstream>
#include <stdexcept>
#include <string>

#include "sdpa.h"

namespace {

using at::Tensor;

struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};

template <typename... A>
[[noreturn]] void bad(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw BadArgument(s.str());
}

std::string shape_text(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

// The positional arguments of one call.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, at = 0;
  PyObject* next() {
    if (at >= n) bad("too few arguments");
    return a[at++];
  }
  const Tensor* tensor(const char* name) {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad(name, " must be a tensor");
    return &THPVariable_Unpack(o);
  }
  const Tensor& needed(const char* name) {
    const Tensor* t = tensor(name);
    if (!t) bad(name, " must be a tensor");
    return *t;
  }
  long long integer(const char* name) {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) bad(name, " must be an integer");
    return v;
  }
  int32_t i32(const char* name) {
    const long long v = integer(name);
    if (v < INT32_MIN || v > INT32_MAX) bad(name, " ", v, " does not fit 32 bits");
    return (int32_t)v;
  }
  double real(const char* name) {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) bad(name, " must be a number");
    return v;
  }
  void* address(const char* name) { return reinterpret_cast<void*>((uintptr_t)integer(name)); }
};

int32_t small(int64_t v, const char* what) {
  if (v > INT32_MAX) bad(what, " ", v, " does not fit 32 bits");
  return (int32_t)v;
}

sdpa_dtype element_type(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return SDPA_F32;
    case at::kHalf: return SDPA_F16;
    case at::kBFloat16: return SDPA_BF16;
    default: bad("unsupported type ", c10::toString(t.scalar_type()));
  }
}

// The device every given tensor must be on; unset while only a struct is wanted.
struct Place {
  bool any = true;
  c10::Device device = c10::kCPU;
  const char* first = "";
  void start(const Tensor& t, const char* name) {
    any = false;
    device = t.device();
    first = name;
    if (!t.is_cuda()) bad(name, " must be a CUDA tensor, got ", device.str());
  }
};

void typed(const Place& pl, const Tensor* t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  if (!t) return;
  if (t->scalar_type() != type) bad(name, " must be ", c10::toString(type), ", got ", c10::toString(t->scalar_type()));
  if (t->sizes() != shape) bad(name, " must have shape ", shape_text(shape), ", got ", shape_text(t->sizes()));
  if (!pl.any && t->device() != pl.device)
    bad(name, " must be a CUDA tensor on the device of ", pl.first, ", got ", t->device().str(), " and ", pl.device.str());
}

void* flat(const Tensor* t, const char* name) {
  if (!t) return nullptr;
  if (!t->is_contiguous()) bad(name, " must be contiguous");
  return t->data_ptr();
}

// (B, N, S, D), or rank 3: (B, S, N*D) with heads of D.
sdpa_view head_view(const Tensor& t, int64_t D, const char* name) {
  const auto st = t.strides();
  if (st.back() != 1 && t.sizes().back() > 1) bad(name, ": the last dimension must be contiguous");
  if (t.dim() == 4) return sdpa_view{t.data_ptr(), st[0], st[1], st[2]};
  return sdpa_view{t.data_ptr(), st[0], D, st[1]};
}

// Packed rows (tokens, heads, dim).
sdpa_view packed(const Tensor& t, const char* name) {
  const auto st = t.strides();
  if (st[2] != 1 && t.size(2) > 1) bad(name, ": the last dimension must be contiguous");
  return sdpa_view{t.data_ptr(), 0, st[1], st[0]};
}

sdpa_view pool_view(const Tensor& t, const char* name) {
  const auto st = t.strides();
  if (st[3] != 1 && t.size(3) > 1) bad(name, ": the last dimension must be contiguous");
  return sdpa_view{t.data_ptr(), st[0], st[1], st[2]};
}

Tensor like(const Place& pl, const Tensor* t, const Tensor& ref, const char* name) {
  if (!t) return at::empty(ref.sizes(), ref.options().requires_grad(false));
  typed(pl, t, name, ref.scalar_type(), ref.sizes());
  return *t;
}

PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// ------------------------------------------------------------------ query/key norm

struct Norm {
  Place place;
  sdpa_qk_norm_params p;
  const Tensor *q, *k, *qw, *kw;
  Tensor pos;                        // keeps a converted copy until the call has been made
};

// q, k, q_weight, k_weight, cos_cache, sin_cache, position_ids, eps, rotary_dim, interleaved, num_heads,
// kv_num_heads (0: not given)
void read_norm(Args& a, Norm& n) {
  n.q = &a.needed("q");
  n.k = &a.needed("k");
  n.qw = &a.needed("q_weight");
  n.kw = &a.needed("k_weight");
  const Tensor *cos = a.tensor("cos_cache"), *sin = a.tensor("sin_cache"), *pos = a.tensor("position_ids");
  std::memset(&n.p, 0, sizeof n.p);
  sdpa_qk_norm_params& p = n.p;
  p.struct_size = sizeof p;
  p.eps = (float)a.real("eps");
  p.rotary_dim = a.i32("rotary_dim");
  p.rotary_interleaved = a.i32("interleaved");
  const int64_t nq = a.integer("num_heads"), nkv = a.integer("kv_num_heads");
  const Tensor &q = *n.q, &k = *n.k;
  n.place.start(q, "q");
  const auto type = q.scalar_type();
  int64_t B, Nq, Nkv, S, D;
  if (q.dim() == 4 && k.dim() == 4) {
    B = q.size(0); Nq = q.size(1); S = q.size(2); D = q.size(3); Nkv = k.size(1);
    typed(n.place, &k, "k", type, {B, Nkv, S, D});
  } else if (q.dim() == 3 && k.dim() == 3) {
    if (nq < 1 || nkv < 1) bad("rank-3 inputs need num_heads and kv_num_heads");
    B = q.size(0); S = q.size(1); Nq = nq; Nkv = nkv; D = q.size(2) / Nq;
    if (D * Nq != q.size(2)) bad("q: ", q.size(2), " channels are no multiple of ", Nq, " heads");
    typed(n.place, &k, "k", type, {B, S, Nkv * D});
  } else {
    bad("q and k must both be rank 3 (B, S, N*D) or both rank 4 (B, N, S, D)");
  }
  p.B = small(B, "B"); p.Nq = small(Nq, "Nq"); p.Nkv = small(Nkv, "Nkv"); p.S = small(S, "S"); p.D = small(D, "D");
  p.dtype = element_type(q);
  typed(n.place, n.qw, "q_weight", type, {D});
  typed(n.place, n.kw, "k_weight", type, {D});
  p.q = head_view(q, D, "q");
  p.k = head_view(k, D, "k");
  p.q_weight = flat(n.qw, "q_weight");
  p.k_weight = flat(n.kw, "k_weight");
  if (!cos != !sin) bad("cos_cache and sin_cache must be given together");
  if (!cos) {
    if (pos) bad("position_ids without cos_cache and sin_cache");
    return;
  }
  const int64_t half = (p.rotary_dim ? p.rotary_dim : D) / 2;
  if (pos) {
    typed(n.place, cos, "cos_cache", type, {cos->dim() ? cos->size(0) : 0, half});
    p.rotary_max_pos = cos->size(0);
    const bool direct = pos->scalar_type() == at::kLong && pos->sizes() == at::IntArrayRef({B, S}) && pos->is_contiguous();
    n.pos = direct ? *pos : pos->to(at::kLong).expand({B, S}).contiguous();
    typed(n.place, &n.pos, "position_ids", at::kLong, {B, S});
    p.position_ids = n.pos.data_ptr<int64_t>();
  } else {
    typed(n.place, cos, "cos_cache", type, {B, S, half});
    p.rotary_max_pos = B * S;
  }
  typed(n.place, sin, "sin_cache", type, cos->sizes());
  p.rotary_cos = flat(cos, "cos_cache");
  p.rotary_sin = flat(sin, "sin_cache");
}

using NormFwd = int (*)(const sdpa_qk_norm_params*, sdpa_view, sdpa_view, sdpa_stream_t);
using NormBwd = int (*)(const sdpa_qk_norm_params*, sdpa_view, sdpa_view, sdpa_view, sdpa_view, void*, void*, void*, size_t,
                        sdpa_stream_t);
using NormSize = size_t (*)(const sdpa_qk_norm_params*);

// entry point, stream, then read_norm's arguments, q_out, k_out -> (q_out, k_out) or a status
PyObject* qk_norm_rotary(Args& a) {
  const auto fn = reinterpret_cast<NormFwd>(a.address("entry"));
  const auto st = static_cast<sdpa_stream_t>(a.address("stream"));
  Norm n;
  read_norm(a, n);
  const Tensor *qo = a.tensor("q_out"), *ko = a.tensor("k_out");
  Tensor q_out = like(n.place, qo, *n.q, "q_out"), k_out = like(n.place, ko, *n.k, "k_out");
  const int rc = fn(&n.p, head_view(q_out, n.p.D, "q_out"), head_view(k_out, n.p.D, "k_out"), st);
  return rc ? PyLong_FromLong(rc) : pack({q_out, k_out});
}

// entry point, size query, stream, read_norm's arguments, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace
PyObject* qk_norm_rotary_bwd(Args& a) {
  const auto fn = reinterpret_cast<NormBwd>(a.address("entry"));
  const auto size = reinterpret_cast<NormSize>(a.address("size"));
  const auto st = static_cast<sdpa_stream_t>(a.address("stream"));
  Norm n;
  read_norm(a, n);
  const Tensor &gq = a.needed("dq_out"), &gk = a.needed("dk_out");
  typed(n.place, &gq, "dq_out", n.q->scalar_type(), n.q->sizes());
  typed(n.place, &gk, "dk_out", n.k->scalar_type(), n.k->sizes());
  const Tensor *pq = a.tensor("dq"), *pk = a.tensor("dk"), *pwq = a.tensor("dq_weight"), *pwk = a.tensor("dk_weight");
  const Tensor* pws = a.tensor("workspace");
  Tensor dq = like(n.place, pq, *n.q, "dq"), dk = like(n.place, pk, *n.k, "dk");
  Tensor dwq = like(n.place, pwq, *n.qw, "dq_weight"), dwk = like(n.place, pwk, *n.kw, "dk_weight");
  Tensor ws = pws ? *pws : at::empty({std::max<int64_t>(1, (int64_t)size(&n.p))}, n.q->options().dtype(at::kByte));
  typed(n.place, &ws, "workspace", ws.scalar_type(), ws.sizes());
  const int64_t D = n.p.D;
  const int rc = fn(&n.p, head_view(gq, D, "dq_out"), head_view(gk, D, "dk_out"), head_view(dq, D, "dq"),
                    head_view(dk, D, "dk"), flat(&dwq, "dq_weight"), flat(&dwk, "dk_weight"), flat(&ws, "workspace"),
                    ws.nbytes(), st);
  return rc ? PyLong_FromLong(rc) : pack({dq, dk, dwq, dwk});
}

// ------------------------------------------------------------------ paged cache

// Channels of a record of `bytes` bytes: 32 of them are 16 bytes of codes and two values of their side.
int64_t record_channels(int64_t bytes, sdpa_dtype dt, const char* name) {
  const int64_t part = dt == SDPA_F32 ? 24 : 20;
  if (bytes < part || bytes % part) bad(name, ": ", bytes, " bytes are no record of whole groups of ", part, " bytes");
  return bytes / part * 32;
}

// k_pages, v_pages, page_table, kv_lens, cu_new, then by the caller: tokens and Nq.  records: the type of
// the rows beside pools of records (bytes), or nullptr for pools in that type.
void read_pages(Args& a, const Place& pl, sdpa_paged_params& p, const Tensor*& kp, const Tensor*& vp,
                const Tensor* records = nullptr) {
  std::memset(&p, 0, sizeof p);
  p.struct_size = sizeof p;
  kp = &a.needed("k_pages");
  vp = &a.needed("v_pages");
  const Tensor &table = a.needed("page_table"), &lens = a.needed("kv_lens");
  const Tensor* cu = a.tensor("cu_new");
  if (kp->dim() != 4 || vp->dim() != 4) bad("k_pages and v_pages are (pages, heads, slots, dim) views");
  const auto type = records ? at::kByte : kp->scalar_type();
  p.dtype = element_type(records ? *records : *kp);
  typed(pl, kp, "k_pages", type, kp->sizes());
  typed(pl, vp, "v_pages", type, {kp->size(0), kp->size(1), kp->size(2), vp->size(3)});
  if (table.dim() != 2) bad("page_table must be (B, max_pages)");
  if (table.stride(1) != 1 && table.size(1) > 1) bad("the rows of page_table must be contiguous");
  const int64_t B = table.size(0);
  typed(pl, &table, "page_table", at::kInt, table.sizes());
  typed(pl, &lens, "kv_lens", at::kInt, {B});
  typed(pl, cu, "cu_new", at::kInt, {B + 1});
  p.B = small(B, "B");
  p.num_pages = small(kp->size(0), "num_pages"); p.Nkv = small(kp->size(1), "Nkv");
  p.page_size = small(kp->size(2), "page_size");
  p.H = small(records ? record_channels(kp->size(3), p.dtype, "k_pages") : kp->size(3), "H");
  p.Hv = small(records ? record_channels(vp->size(3), p.dtype, "v_pages") : vp->size(3), "Hv");
  p.max_pages = small(table.size(1), "max_pages");
  p.k_pages = pool_view(*kp, "k_pages");
  p.v_pages = pool_view(*vp, "v_pages");
  p.page_table = table.data_ptr<int32_t>();
  p.page_table_stride = table.stride(0);
  p.kv_lens = static_cast<const int32_t*>(flat(&lens, "kv_lens"));
  p.cu_new = static_cast<const int32_t*>(flat(cu, "cu_new"));
  p.window = -1;
}

// cos_cache, sin_cache, rotary_dim, interleaved
void read_rotation(Args& a, const Place& pl, sdpa_paged_params& p, at::ScalarType type) {
  const Tensor *cos = a.tensor("cos_cache"), *sin = a.tensor("sin_cache");
  p.rotary_dim = a.i32("rotary_dim");
  p.rotary_interleaved = a.i32("interleaved");
  if (!cos != !sin) bad("cos_cache and sin_cache must be given together");
  if (!cos) return;
  const int64_t half = (p.rotary_dim ? p.rotary_dim : p.H) / 2;
  typed(pl, cos, "cos_cache", type, {cos->dim() ? cos->size(0) : 0, half});
  typed(pl, sin, "sin_cache", type, cos->sizes());
  p.rotary_max_pos = cos->size(0);
  p.rotary_cos = flat(cos, "cos_cache");
  p.rotary_sin = flat(sin, "sin_cache");
}

// scale (None: default), softcap, causal, window, head_sink, max_new
void read_rules(Args& a, const Place& pl, sdpa_paged_params& p, at::ScalarType type) {
  if (a.at < a.n && a.a[a.at] == Py_None) {
    ++a.at;
  } else {
    p.has_scale = 1;
    p.scale = (float)a.real("scale");
  }
  p.softcap = (float)a.real("softcap");
  p.causal = a.i32("causal");
  p.window = a.integer("window");
  const Tensor* sink = a.tensor("head_sink");
  typed(pl, sink, "head_sink", type, {p.Nq});
  p.head_sink = flat(sink, "head_sink");
  p.max_new = a.i32("max_new");
}

using AppendFn = int (*)(const sdpa_paged_params*, sdpa_view, sdpa_view, sdpa_stream_t);
using AttnFn = int (*)(const sdpa_paged_params*, sdpa_view, sdpa_view, void*, size_t, sdpa_stream_t);
using PagedSize = size_t (*)(const sdpa_paged_params*);

// tokens, Nq, read_pages', read_rotation's and read_rules' arguments -> the struct's bytes
PyObject* paged_params(Args& a) {
  const int32_t tokens = a.i32("tokens"), Nq = a.i32("Nq");
  sdpa_paged_params p;
  const Tensor *kp, *vp;
  Place any;
  read_pages(a, any, p, kp, vp);
  p.tokens = tokens;
  p.Nq = Nq;
  read_rotation(a, any, p, kp->scalar_type());
  read_rules(a, any, p, kp->scalar_type());
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&p), sizeof p);
}

// entry point, stream, k, v, read_pages' and read_rotation's arguments -> None or a status
PyObject* paged_append(Args& a) {
  const auto fn = reinterpret_cast<AppendFn>(a.address("entry"));
  const auto st = static_cast<sdpa_stream_t>(a.address("stream"));
  const Tensor &k = a.needed("k"), &v = a.needed("v");
  Place pl;
  pl.start(k, "k");
  if (k.dim() != 3 || v.dim() != 3) bad("k and v must be packed rows (tokens, heads, dim)");
  sdpa_paged_params p;
  const Tensor *kp, *vp;
  read_pages(a, pl, p, kp, vp);
  const auto type = kp->scalar_type();
  typed(pl, &k, "k", type, {k.size(0), p.Nkv, p.H});
  typed(pl, &v, "v", type, {k.size(0), p.Nkv, p.Hv});
  p.tokens = small(k.size(0), "tokens");
  p.Nq = p.Nkv;
  read_rotation(a, pl, p, type);
  const int rc = fn(&p, packed(k, "k"), packed(v, "v"), st);
  if (rc) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
}

// entry point, size query, stream, q, read_pages' and read_rules' arguments, y, workspace -> y or a status
template <bool kRecords>
PyObject* paged_attn(Args& a) {
  const auto fn = reinterpret_cast<AttnFn>(a.address("entry"));
  const auto size = reinterpret_cast<PagedSize>(a.address("size"));
  const auto st = static_cast<sdpa_stream_t>(a.address("stream"));
  const Tensor& q = a.needed("q");
  Place pl;
  pl.start(q, "q");
  if (q.dim() != 3) bad("q must be packed rows (tokens, heads, dim)");
  sdpa_paged_params p;
  const Tensor *kp, *vp;
  read_pages(a, pl, p, kp, vp, kRecords ? &q : nullptr);
  const auto type = kRecords ? q.scalar_type() : kp->scalar_type();
  typed(pl, &q, "q", type, {q.size(0), q.size(1), p.H});
  p.tokens = small(q.size(0), "tokens");
  p.Nq = small(q.size(1), "Nq");
  read_rules(a, pl, p, type);
  const Tensor *py = a.tensor("y"), *pws = a.tensor("workspace");
  const int64_t shape[3] = {q.size(0), q.size(1), p.Hv};
  Tensor y = py ? *py : at::empty(shape, q.options().requires_grad(false));
  typed(pl, &y, "y", type, shape);
  const auto bytes = q.options().dtype(at::kByte).requires_grad(false);
  Tensor ws = pws ? *pws : at::empty({std::max<int64_t>(1, (int64_t)size(&p))}, bytes);
  typed(pl, &ws, "workspace", ws.scalar_type(), ws.sizes());
  const int rc = fn(&p, packed(q, "q"), packed(y, "y"), flat(&ws, "workspace"), ws.nbytes(), st);
  return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(y);
}

// entry point, stream, k, v, k_pages, v_pages, slots, positions, cos_cache, sin_cache, rotary_dim, interleaved, k_held,
// v_held -> None or a status
PyObject* paged4_append(Args& a) {
  using Fn = int (*)(const sdpa_paged4_append_params*, sdpa_view, sdpa_view, sdpa_view, sdpa_view, sdpa_stream_t);
  const auto fn = reinterpret_cast<Fn>(a.address("entry"));
  const auto st = static_cast<sdpa_stream_t>(a.address("stream"));
  const Tensor &k = a.needed("k"), &v = a.needed("v"), &kp = a.needed("k_pages"), &vp = a.needed("v_pages");
  const Tensor &slots = a.needed("slots"), *pos = a.tensor("positions");
  const Tensor *cos = a.tensor("cos_cache"), *sin = a.tensor("sin_cache");
  sdpa_paged4_append_params p;
  std::memset(&p, 0, sizeof p);
  p.struct_size = sizeof p;
  p.rotary_dim = a.i32("rotary_dim");
  p.rotary_interleaved = a.i32("interleaved");
  const Tensor *kh = a.tensor("k_held"), *vh = a.tensor("v_held");
  Place pl;
  pl.start(k, "k");
  const auto type = k.scalar_type();
  p.dtype = element_type(k);
  if (k.dim() != 3 || v.dim() != 3) bad("k and v must be packed rows (tokens, heads, dim)");
  const int64_t tokens = k.size(0), heads = k.size(1), H = k.size(2), Hv = v.size(2);
  typed(pl, &v, "v", type, {tokens, heads, Hv});
  if (kp.dim() != 4 || vp.dim() != 4) bad("k_pages and v_pages are (pages, heads, slots, record) views");
  typed(pl, &kp, "k_pages", at::kByte, {kp.size(0), heads, kp.size(2), kp.size(3)});
  typed(pl, &vp, "v_pages", at::kByte, {kp.size(0), heads, kp.size(2), vp.size(3)});
  if (record_channels(kp.size(3), p.dtype, "k_pages") != H) bad("k_pages: records of ", kp.size(3), " bytes do not hold ", H, " channels");
  if (record_channels(vp.size(3), p.dtype, "v_pages") != Hv) bad("v_pages: records of ", vp.size(3), " bytes do not hold ", Hv, " channels");
  typed(pl, &slots, "slots", at::kLong, {tokens});
  typed(pl, pos, "positions", at::kLong, {tokens});
  p.tokens = small(tokens, "tokens"); p.Nkv = small(heads, "Nkv"); p.H = small(H, "H"); p.Hv = small(Hv, "Hv");
  p.num_pages = small(kp.size(0), "num_pages"); p.page_size = small(kp.size(2), "page_size");
  p.k_pages = pool_view(kp, "k_pages");
  p.v_pages = pool_view(vp, "v_pages");
  p.slots = static_cast<const int64_t*>(flat(&slots, "slots"));
  p.positions = static_cast<const int64_t*>(flat(pos, "positions"));
  if (!cos != !sin) bad("cos_cache and sin_cache must be given together");
  if (cos) {
    const int64_t half = (p.rotary_dim ? p.rotary_dim : H) / 2;
    typed(pl, cos, "cos_cache", type, {cos->dim() ? cos->size(0) : 0, half});
    typed(pl, sin, "sin_cache", type, cos->sizes());
    p.rotary_max_pos = cos->size(0);
    p.rotary_cos = flat(cos, "cos_cache");
    p.rotary_sin = flat(sin, "sin_cache");
  }
  typed(pl, kh, "k_held", type, {tokens, heads, H});
  typed(pl, vh, "v_held", type, {tokens, heads, Hv});
  const sdpa_view none{nullptr, 0, 0, 0};
  const int rc = fn(&p, packed(k, "k"), packed(v, "v"), kh ? packed(*kh, "k_held") : none, vh ? packed(*vh, "v_held") : none, st);
  if (rc) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
}

// entry point, stream, page_table, past_lens, new_lens, free_pages, free_count, page_size, tokens, kv_lens, cu_new, positions,
// slots, free_count_out -> (kv_lens, cu_new, positions, slots, free_count_out) or a status
PyObject* paged_tables(Args& a) {
  using Fn = int (*)(const sdpa_paged_tables_params*, sdpa_stream_t);
  const auto fn = reinterpret_cast<Fn>(a.address("entry"));
  const auto st = static_cast<sdpa_stream_t>(a.address("stream"));
  const Tensor &table = a.needed("page_table"), &past = a.needed("past_lens"), &fresh = a.needed("new_lens");
  const Tensor &pages = a.needed("free_pages"), &count = a.needed("free_count");
  sdpa_paged_tables_params p;
  std::memset(&p, 0, sizeof p);
  p.struct_size = sizeof p;
  p.page_size = a.i32("page_size");
  p.tokens = a.i32("tokens");
  const Tensor *lens = a.tensor("kv_lens"), *cu = a.tensor("cu_new"), *pos = a.tensor("positions"), *slots = a.tensor("slots");
  const Tensor* left = a.tensor("free_count_out");
  Place pl;
  pl.start(table, "page_table");
  if (table.dim() != 2) bad("page_table must be (B, max_pages)");
  if (table.stride(1) != 1 && table.size(1) > 1) bad("the rows of page_table must be contiguous");
  if (p.tokens < 0) bad("tokens ", p.tokens, " is negative");
  const int64_t B = table.size(0);
  typed(pl, &table, "page_table", at::kInt, table.sizes());
  typed(pl, &past, "past_lens", at::kInt, {B});
  typed(pl, &fresh, "new_lens", at::kInt, {B});
  if (pages.dim() != 1) bad("free_pages must be (num_pages,)");
  typed(pl, &pages, "free_pages", at::kInt, pages.sizes());
  typed(pl, &count, "free_count", at::kInt, {1});
  typed(pl, lens, "kv_lens", at::kInt, {B});
  typed(pl, cu, "cu_new", at::kInt, {B + 1});
  typed(pl, pos, "positions", at::kLong, {p.tokens});
  typed(pl, slots, "slots", at::kLong, {p.tokens});
  typed(pl, left, "free_count_out", at::kInt, {1});
  const auto ints = past.options().requires_grad(false), longs = ints.dtype(at::kLong);
  Tensor o_lens = lens ? *lens : at::empty({B}, ints), o_cu = cu ? *cu : at::empty({B + 1}, ints);
  Tensor o_pos = pos ? *pos : at::empty({p.tokens}, longs), o_slots = slots ? *slots : at::empty({p.tokens}, longs);
  Tensor o_left = left ? *left : at::empty({1}, ints);
  p.B = small(B, "B");
  p.max_pages = small(table.size(1), "max_pages");
  p.num_pages = small(pages.size(0), "num_pages");
  p.page_table = table.data_ptr<int32_t>();
  p.page_table_stride = table.stride(0);
  p.past_lens = static_cast<const int32_t*>(flat(&past, "past_lens"));
  p.new_lens = static_cast<const int32_t*>(flat(&fresh, "new_lens"));
  p.free_pages = static_cast<int32_t*>(flat(&pages, "free_pages"));
  p.free_count = static_cast<const int32_t*>(flat(&count, "free_count"));
  p.kv_lens = static_cast<int32_t*>(flat(&o_lens, "kv_lens"));
  p.cu_new = static_cast<int32_t*>(flat(&o_cu, "cu_new"));
  p.positions = static_cast<int64_t*>(flat(&o_pos, "positions"));
  p.slots = static_cast<int64_t*>(flat(&o_slots, "slots"));
  p.free_count_out = static_cast<int32_t*>(flat(&o_left, "free_count_out"));
  const int rc = fn(&p, st);
  return rc ? PyLong_FromLong(rc) : pack({o_lens, o_cu, o_pos, o_slots, o_left});
}

// Runs one of the above; a C++ exception becomes a Python one.
template <PyObject* (*F)(Args&)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    Args a{args, n};
    return F(a);
  } catch (const BadArgument& e) {
    PyErr_Clear();
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*F)(Args&)>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<qk_norm_rotary>("qk_norm_rotary"), method<qk_norm_rotary_bwd>("qk_norm_rotary_bwd"),
                         method<paged_params>("paged_params"), method<paged_append>("paged_append"),
                         method<paged_attn<false>>("paged_attn"), method<paged_attn<true>>("paged4_attn"),
                         method<paged4_append>("paged4_append"), method<paged_tables>("paged_tables"), PyMethodDef{nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
