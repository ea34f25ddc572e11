// Native binding of the packed, paged and rotary entry points (include/fa.h)
// for torch tensors: the checks that the C ABI documents, views, output and
// workspace allocation, stream handling. No arithmetic. These calls are made
// once or more per generated token, where the same marshalling in Python
// (19 us for a call of one kernel) takes longer than the kernels.
//
// Every function takes its outputs and workspace or None; what is None is
// allocated, on the stream of the call. `stream` is a cudaStream_t handle or
// None for the current stream; where it is another stream than the current
// one, the caching allocator is told that the inputs are used on it.

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/stl.h>
#include <torch/csrc/utils/pybind.h>

#include <climits>
#include <cmath>
#include <optional>
#include <string>
#include <vector>

#include "../../include/fa.h"

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;
using Handle = std::optional<uint64_t>;

namespace {

PyObject* g_error = nullptr;  // the class FaError(status, where); held for good

void done(int rc, const char* where) {
  if (rc == FA_OK) return;
  py::object e = py::handle(g_error)(rc, where);
  PyErr_SetObject(g_error, e.ptr());
  throw py::error_already_set();
}

// A size as the C ABI's int.
int size32(const char* name, int64_t n) {
  if (n > INT_MAX || n < INT_MIN) throw py::value_error(std::string(name) + " does not fit 32 bits: " + std::to_string(n));
  return static_cast<int>(n);
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

void on_gpu(const char* name, const Tensor& t) {
  if (!t.is_cuda()) throw std::runtime_error(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
}

// A tensor of this type and shape on device `dev` whose last dimension is contiguous.
void check(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  on_gpu(name, t);
  if (t.get_device() != dev)
    throw py::value_error(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                          " but the current device is cuda:" + std::to_string(dev));
  if (t.scalar_type() != type)
    throw py::type_error(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.sizes() != shape)
    throw py::value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  if (shape.back() > 1 && t.stride(-1) != 1)
    throw py::value_error(std::string(name) + " must be contiguous in its last dimension");
}

void three(const char* name, const Tensor& t) {
  on_gpu(name, t);
  if (t.dim() != 3) throw py::value_error(std::string(name) + " must be a [T, H, d] tensor");
}

// The call's device and stream; `side`: a stream other than the current one.
struct Call {
  int dev;
  c10::cuda::CUDAStream stream;
  bool side;
  explicit Call(const Handle& h)
      : dev(c10::cuda::current_device()), stream(c10::cuda::getCurrentCUDAStream(dev)), side(false) {
    if (!h) return;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(*h);
    if (s == stream.stream()) return;
    stream = s ? c10::cuda::getStreamFromExternal(s, dev) : c10::cuda::getDefaultCUDAStream(dev);
    side = true;
  }
  void* handle() const { return stream.stream(); }
  void used(std::initializer_list<const Tensor*> ts) const {
    if (!side) return;
    for (const Tensor* t : ts)
      if (t && t->defined()) t->record_stream(stream);
  }
  Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) const {
    if (!side) return at::empty(shape, like.options().dtype(type));
    c10::cuda::CUDAStreamGuard guard(stream);
    return at::empty(shape, like.options().dtype(type));
  }
};

const Tensor* ptr(const Opt& t) { return t ? &*t : nullptr; }

fa_rows rows(const char* name, const Tensor& t, at::IntArrayRef shape, const Call& c) {
  check(name, t, at::kBFloat16, shape, c.dev);
  return fa_rows{t.data_ptr(), t.stride(0), t.stride(1)};
}

fa_pages pages(const char* name, const Tensor& t, at::IntArrayRef shape, const Call& c) {
  check(name, t, at::kBFloat16, shape, c.dev);
  return fa_pages{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

template <typename E>
E* flat(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef shape, const Call& c) {
  check(name, t, type, shape, c.dev);
  if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
  return static_cast<E*>(t.data_ptr());
}

struct Work {
  Tensor t;
  void* p;
  size_t bytes;
  Work(const Opt& given, size_t need, const Tensor& like, const Call& c) {
    t = given ? *given : c.empty({static_cast<int64_t>(need < 16 ? 16 : need)}, like, at::kByte);
    if (!t.is_cuda() || !t.is_contiguous()) throw py::value_error("workspace must be a contiguous CUDA tensor");
    if (t.get_device() != c.dev) throw py::value_error("workspace is on another device than the current one");
    p = t.data_ptr();
    bytes = t.nbytes();
  }
};

// Offsets of S sequences; none: one token each.
struct Seqs {
  int S;
  const int* cu;
  Seqs(const Opt& t, int T, const Call& c) {
    if (!t) {
      S = T;
      cu = nullptr;
      return;
    }
    on_gpu("cu_seqlens", *t);
    if (t->dim() != 1 || t->numel() < 1) throw py::value_error("cu_seqlens must be a tensor of S + 1 offsets");
    S = size32("S", t->numel() - 1);
    cu = flat<int>("cu_seqlens", *t, at::kInt, t->sizes(), c);
  }
};

float scale_of(const std::optional<double>& scale, int d) {
  return static_cast<float>(scale ? *scale : 1.0 / std::sqrt(static_cast<double>(d)));
}

Tensor out(const Opt& given, at::IntArrayRef shape, const Tensor& like, at::ScalarType type, const Call& c) {
  return given ? *given : c.empty(shape, like, type);
}

py::object packed_fwd(const Tensor& q, const Tensor& k, const Tensor& v, const Opt& o_, const Opt& lse_,
                      const Opt& resid_, bool residual, const Tensor& cu, bool causal, std::optional<double> scale,
                      const Opt& workspace, Handle stream) {
  three("q", q);
  three("k", k);
  const Call c(stream);
  const int T = size32("T", q.size(0)), Hq = size32("Hq", q.size(1)), Hkv = size32("Hkv", k.size(1)),
            d = size32("d", q.size(2));
  const Seqs s(cu, T, c);
  c.used({&q, &k, &v, &cu, ptr(o_), ptr(lse_), ptr(resid_), ptr(workspace)});
  const Tensor o = out(o_, {T, Hq, d}, q, at::kBFloat16, c);
  const Tensor lse = out(lse_, {Hq, T}, q, at::kFloat, c);
  Tensor resid;
  if (residual || resid_) resid = out(resid_, {T, Hq, d}, q, at::kBFloat16, c);
  const fa_rows rq = rows("q", q, {T, Hq, d}, c), rk = rows("k", k, {T, Hkv, d}, c), rv = rows("v", v, {T, Hkv, d}, c),
                ro = rows("o", o, {T, Hq, d}, c);
  fa_rows rr{};
  if (resid.defined()) rr = rows("o_resid", resid, {T, Hq, d}, c);
  float* la = flat<float>("lse", lse, at::kFloat, {Hq, T}, c);
  const Work w(workspace, fa_packed_fwd_workspace_bytes(s.S, T, Hq, Hkv, d), q, c);
  done(fa_packed_fwd(&rq, &rk, &rv, &ro, resid.defined() ? &rr : nullptr, la, s.cu, s.S, T, Hq, Hkv, d, causal,
                     scale_of(scale, d), w.p, w.bytes, c.handle()),
       "fa_packed_fwd");
  if (resid.defined()) return py::make_tuple(o, lse, resid);
  return py::make_tuple(o, lse);
}

py::object packed_bwd(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Opt& resid,
                      const Tensor& dout, const Tensor& lse, const Opt& dq_, const Opt& dk_, const Opt& dv_,
                      const Tensor& cu, bool causal, std::optional<double> scale, const Opt& workspace, Handle stream) {
  three("q", q);
  three("k", k);
  const Call c(stream);
  const int T = size32("T", q.size(0)), Hq = size32("Hq", q.size(1)), Hkv = size32("Hkv", k.size(1)),
            d = size32("d", q.size(2));
  const Seqs s(cu, T, c);
  c.used({&q, &k, &v, &o, ptr(resid), &dout, &lse, &cu, ptr(dq_), ptr(dk_), ptr(dv_), ptr(workspace)});
  const Tensor dq = out(dq_, {T, Hq, d}, q, at::kBFloat16, c), dk = out(dk_, {T, Hkv, d}, q, at::kBFloat16, c),
               dv = out(dv_, {T, Hkv, d}, q, at::kBFloat16, c);
  const fa_rows rq = rows("q", q, {T, Hq, d}, c), rk = rows("k", k, {T, Hkv, d}, c), rv = rows("v", v, {T, Hkv, d}, c),
                ro = rows("o", o, {T, Hq, d}, c), rg = rows("dout", dout, {T, Hq, d}, c),
                rdq = rows("dq", dq, {T, Hq, d}, c), rdk = rows("dk", dk, {T, Hkv, d}, c),
                rdv = rows("dv", dv, {T, Hkv, d}, c);
  fa_rows rr{};
  if (resid) rr = rows("o_resid", *resid, {T, Hq, d}, c);
  const float* la = flat<float>("lse", lse, at::kFloat, {Hq, T}, c);
  const Work w(workspace, fa_packed_bwd_workspace_bytes(s.S, T, Hq, Hkv, d), q, c);
  done(fa_packed_bwd(&rq, &rk, &rv, &ro, resid ? &rr : nullptr, &rg, la, &rdq, &rdk, &rdv, s.cu, s.S, T, Hq, Hkv, d,
                     causal, scale_of(scale, d), w.p, w.bytes, c.handle()),
       "fa_packed_bwd");
  return py::make_tuple(dq, dk, dv);
}

// A paged cache's arguments.
struct Cache {
  fa_pages k, v;
  int n_pages, page, max_pages;
  const int* table;
  int64_t table_stride;
  const int* lens;
  Cache(const Tensor& kp, const Tensor& vp, const Tensor& bt, const Tensor& sl, int S, int Hkv, int d,
        const Call& c) {
    on_gpu("k_pages", kp);
    on_gpu("block_table", bt);
    if (kp.dim() != 4) throw py::value_error("k_pages must be [n_pages, Hkv, page_size, d]");
    if (bt.dim() != 2) throw py::value_error("block_table must be [S, max_pages]");
    const std::vector<int64_t> shape{kp.size(0), Hkv, kp.size(2), d};
    k = pages("k_pages", kp, shape, c);
    v = pages("v_pages", vp, shape, c);
    n_pages = size32("n_pages", shape[0]);
    page = size32("page_size", shape[2]);
    max_pages = size32("max_pages", bt.size(1));
    check("block_table", bt, at::kInt, {S, bt.size(1)}, c.dev);
    table = static_cast<const int*>(bt.data_ptr());
    table_stride = bt.stride(0);
    lens = flat<int>("seq_lens", sl, at::kInt, {S}, c);
  }
};

py::object paged_fwd(const Tensor& q, const Tensor& k_pages, const Tensor& v_pages, const Opt& o_, const Opt& lse_,
                     const Tensor& table, const Tensor& lens, const Opt& cu, std::optional<int64_t> max_q, bool causal,
                     std::optional<double> scale, const Opt& workspace, Handle stream) {
  three("q", q);
  const Call c(stream);
  const int T = size32("T", q.size(0)), Hq = size32("Hq", q.size(1)), d = size32("d", q.size(2));
  const Seqs s(cu, T, c);
  const int Hkv = k_pages.dim() == 4 ? size32("Hkv", k_pages.size(1)) : 0;
  const Cache ca(k_pages, v_pages, table, lens, s.S, Hkv, d, c);
  const int mq = max_q ? size32("max_q", *max_q) : (cu ? std::max(1, T) : 1);
  c.used({&q, &k_pages, &v_pages, &table, &lens, ptr(cu), ptr(o_), ptr(lse_), ptr(workspace)});
  const Tensor o = out(o_, {T, Hq, d}, q, at::kBFloat16, c);
  const Tensor lse = out(lse_, {Hq, T}, q, at::kFloat, c);
  const fa_rows rq = rows("q", q, {T, Hq, d}, c), ro = rows("o", o, {T, Hq, d}, c);
  float* la = flat<float>("lse", lse, at::kFloat, {Hq, T}, c);
  const Work w(workspace, fa_paged_fwd_workspace_bytes(s.S, T, mq, Hq, Hkv, d, ca.page, ca.max_pages), q, c);
  done(fa_paged_fwd(&rq, &ca.k, &ca.v, &ro, la, ca.n_pages, ca.page, ca.table, ca.table_stride, ca.max_pages, ca.lens,
                    s.cu, s.S, T, mq, Hq, Hkv, d, causal, scale_of(scale, d), w.p, w.bytes, c.handle()),
       "fa_paged_fwd");
  return py::make_tuple(o, lse);
}

// A rotation's arguments.
struct Turn {
  std::vector<int> sections;
  const int* positions = nullptr;
  const double* inv_freq = nullptr;
  Turn(const Opt& pos, const Opt& freq, const std::optional<std::vector<int>>& sec, int T, const Call& c) {
    if (!freq) {
      if (sec && !sec->empty()) throw py::value_error("sections need inv_freq");
      return;
    }
    on_gpu("inv_freq", *freq);
    const int64_t pairs = freq->numel();
    sections = sec ? *sec : std::vector<int>{size32("pairs", pairs)};
    int64_t sum = 0;
    for (int n : sections) sum += n;
    if (sum != pairs)
      throw py::value_error("sections must sum to inv_freq's " + std::to_string(pairs) + " pairs, got " + std::to_string(sum));
    inv_freq = flat<double>("inv_freq", *freq, at::kDouble, {pairs}, c);
    if (pos) positions = flat<int>("positions", *pos, at::kInt, {static_cast<int64_t>(sections.size()), T}, c);
  }
};

py::object rope(const Opt& q, const Opt& k, const Opt& q_out, const Opt& k_out, const Tensor& pos, const Tensor& freq,
                std::optional<std::vector<int>> sections, bool interleaved, bool inverse, Handle stream) {
  if (!q && !k) throw py::value_error("q or k is required");
  if (q) three("q", *q);
  if (k) three("k", *k);
  const Call c(stream);
  const Tensor& x = q ? *q : *k;
  const int T = size32("T", x.size(0)), d = size32("d", x.size(2)), Hq = q ? size32("Hq", q->size(1)) : 0,
            Hkv = k ? size32("Hkv", k->size(1)) : 0;
  const Turn t(pos, freq, sections, T, c);
  c.used({ptr(q), ptr(k), ptr(q_out), ptr(k_out), &pos, &freq});
  fa_rows r[4] = {};
  Tensor qo, ko;
  if (q) {
    r[0] = rows("q", *q, {T, Hq, d}, c);
    qo = out(q_out, {T, Hq, d}, x, at::kBFloat16, c);
    r[2] = rows("q_out", qo, {T, Hq, d}, c);
  }
  if (k) {
    r[1] = rows("k", *k, {T, Hkv, d}, c);
    ko = out(k_out, {T, Hkv, d}, x, at::kBFloat16, c);
    r[3] = rows("k_out", ko, {T, Hkv, d}, c);
  }
  done(fa_rope(&r[0], &r[1], &r[2], &r[3], t.positions, t.inv_freq, t.sections.data(),
               static_cast<int>(t.sections.size()), T, Hq, Hkv, d, interleaved, inverse, c.handle()),
       "fa_rope");
  return py::make_tuple(q ? py::cast(qo) : py::none(), k ? py::cast(ko) : py::none());
}

py::object paged_append(const Opt& q, const Tensor& k, const Tensor& v, const Opt& q_out, const Tensor& k_pages,
                        const Tensor& v_pages, const Tensor& table, const Tensor& lens, const Opt& cu, const Opt& pos,
                        const Opt& freq, std::optional<std::vector<int>> sections, bool interleaved, Handle stream) {
  three("k", k);
  if (q) three("q", *q);
  const Call c(stream);
  const int T = size32("T", k.size(0)), Hkv = size32("Hkv", k.size(1)), d = size32("d", k.size(2)),
            Hq = q ? size32("Hq", q->size(1)) : 0;
  const Seqs s(cu, T, c);
  const Cache ca(k_pages, v_pages, table, lens, s.S, Hkv, d, c);
  const Turn t(pos, freq, sections, T, c);
  c.used({ptr(q), &k, &v, ptr(q_out), &k_pages, &v_pages, &table, &lens, ptr(cu), ptr(pos), ptr(freq)});
  const fa_rows rk = rows("k", k, {T, Hkv, d}, c), rv = rows("v", v, {T, Hkv, d}, c);
  fa_rows rq{}, ro{};
  Tensor qo;
  if (q) {
    rq = rows("q", *q, {T, Hq, d}, c);
    qo = out(q_out, {T, Hq, d}, *q, at::kBFloat16, c);
    ro = rows("q_out", qo, {T, Hq, d}, c);
  }
  done(fa_paged_append(&rq, &rk, &rv, &ro, &ca.k, &ca.v, ca.n_pages, ca.page, ca.table, ca.table_stride, ca.max_pages,
                       ca.lens, s.cu, s.S, T, t.positions, t.inv_freq, t.sections.data(),
                       static_cast<int>(t.sections.size()), Hq, Hkv, d, interleaved, c.handle()),
       "fa_paged_append");
  return q ? py::cast(qo) : py::none();
}

}  // namespace

PYBIND11_MODULE(_fa_torch, m) {
  m.def("set_error", [](py::object e) { g_error = e.release().ptr(); });
  m.def("packed_fwd", &packed_fwd);
  m.def("packed_bwd", &packed_bwd);
  m.def("paged_fwd", &paged_fwd);
  m.def("rope", &rope);
  m.def("paged_append", &paged_append);
}
