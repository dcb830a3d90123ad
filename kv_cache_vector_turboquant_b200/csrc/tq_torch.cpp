// Argument checks, output allocation and calls of the operators around the
// packed cache (tq_qk_norm_rope, tq_attend_window(_paged), tq_pages_*) for
// PyTorch tensors: the part of the Python wrappers that runs on every call. A
// call of a decode step takes 5-10 us on the GPU and takes a dozen tensors;
// checked one by one in Python these took 10-15 us of host time, here below
// one. Computes nothing: every call goes to the C entry point of libtq.so.
//
// Functions take Python objects and raise ValueError ("name: what it has to
// be") before any pointer reaches the library, and the package's TQError for a
// status. Outputs are allocated on the tensors' device, whose current stream
// the call uses.
#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <cstring>
#include <initializer_list>
#include <string>
#include <utility>
#include <vector>

#include "tq.h"

namespace py = pybind11;
using at::ScalarType;
using at::Tensor;

namespace {

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

std::string kind_name(ScalarType t) {
  switch (t) {
    case ScalarType::Half: return "torch.float16";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Bool: return "torch.bool";
    default: return c10::toString(t);
  }
}

std::string shape_name(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// The tensor of a Python object; an undefined one for None where that is allowed.
Tensor tensor(py::handle h, const char* name) {
  if (!THPVariable_Check(h.ptr())) refuse(std::string(name) + ": a torch tensor");
  return THPVariable_Unpack(h.ptr());
}
Tensor maybe(py::handle h, const char* name) { return h.is_none() ? Tensor() : tensor(h, name); }

void check_kind(const Tensor& t, const char* name, std::initializer_list<ScalarType> kinds) {
  std::string all;
  for (ScalarType k : kinds) {
    if (t.scalar_type() == k) return;
  }
  for (ScalarType k : kinds) all += (all.empty() ? "" : " or ") + kind_name(k);
  refuse(std::string(name) + ": dtype " + all + ", got " + kind_name(t.scalar_type()));
}
void check(const Tensor& t, const char* name, std::initializer_list<ScalarType> kinds) {
  check_kind(t, name, kinds);
  if (!t.is_contiguous()) refuse(std::string(name) + ": contiguous");
}
void check_shape(const Tensor& t, const char* name, std::initializer_list<ScalarType> kinds,
                 std::initializer_list<int64_t> shape) {
  check(t, name, kinds);
  if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
    refuse(std::string(name) + ": shape " + shape_name(at::IntArrayRef(shape.begin(), shape.size())) + ", got " +
           shape_name(t.sizes()));
}
void check_numel(const Tensor& t, const char* name, std::initializer_list<ScalarType> kinds, int64_t n) {
  check(t, name, kinds);
  if (t.numel() != n)
    refuse(std::string(name) + ": " + std::to_string(n) + " elements, got " + std::to_string(t.numel()));
}

// The CUDA device that holds all the defined tensors.
int one_device(std::initializer_list<std::pair<const char*, const Tensor*>> all) {
  int dev = -1;
  for (const auto& [name, t] : all) {
    if (!t->defined()) continue;
    if (!t->is_cuda()) refuse(std::string(name) + ": a CUDA tensor");
    if (dev < 0) dev = t->get_device();
    if (t->get_device() != dev)
      refuse(std::string(name) + ": on cuda:" + std::to_string(dev) + " like the other tensors, got cuda:" +
             std::to_string(t->get_device()));
  }
  return dev;
}

// The calls have no backward pass: a tensor whose gradient is being recorded
// would lose it without a word.
void forward_only(std::initializer_list<std::pair<const char*, const Tensor*>> all) {
  if (!c10::GradMode::is_enabled()) return;
  for (const auto& [name, t] : all)
    if (t->defined() && t->requires_grad())
      refuse(std::string(name) + ": requires a gradient, which this call does not compute (detach it, or call under "
             "torch.no_grad())");
}

// First address of a tensor and the first behind it.
std::pair<uintptr_t, uintptr_t> span(const Tensor& t) {
  int64_t n = t.numel() ? 1 : 0;
  if (n)
    for (int64_t i = 0; i < t.dim(); ++i) n += (t.size(i) - 1) * t.stride(i);
  const uintptr_t a = reinterpret_cast<uintptr_t>(t.data_ptr());
  return {a, a + (uintptr_t)(n * t.element_size())};
}
// Same strides, wherever there is a second element to step to.
bool same_strides(const Tensor& a, const Tensor& b) {
  if (a.sizes() != b.sizes()) return false;
  for (int64_t i = 0; i < a.dim(); ++i)
    if (a.size(i) > 1 && a.stride(i) != b.stride(i)) return false;
  return true;
}
// Refuse an output that shares memory with another argument; with `itself`
// only unless it is that very tensor.
void apart(const char* name, const Tensor& out, std::initializer_list<const Tensor*> others, const Tensor* itself) {
  const auto [lo, hi] = span(out);
  auto clash = [&, lo = lo, hi = hi](const Tensor& t) {
    const auto [a, b] = span(t);
    return lo < b && a < hi;
  };
  bool bad = itself && clash(*itself) &&
             !(itself->data_ptr() == out.data_ptr() && same_strides(*itself, out) &&
               itself->scalar_type() == out.scalar_type());
  for (const Tensor* t : others) bad = bad || (t->defined() && clash(*t));
  if (bad) refuse(std::string(name) + ": shares memory with another argument");
}

void raise_status(tq_status st, const char* what) {
  if (st == TQ_OK) return;
  py::object error = py::module_::import("kv_cache_vector_turboquant_b200._binding").attr("TQError");
  py::object e = error((int)st, what);
  PyErr_SetObject(error.ptr(), e.ptr());
  throw py::error_already_set();
}

void* address(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T* address_as(const Tensor& t) {
  return static_cast<T*>(address(t));
}
tq_stream stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
Tensor bytes_on(size_t n, const Tensor& like) {
  return n ? at::empty({(int64_t)n}, like.options().dtype(ScalarType::Byte)) : Tensor();
}
Tensor fresh(const Tensor& like) { return at::empty(like.sizes(), like.options()); }
// An integer of Python (anything with __index__) that is at least `least`.
int64_t whole(py::handle h, const char* name, int64_t least, const char* what) {
  const py::object i = py::reinterpret_steal<py::object>(PyNumber_Index(h.ptr()));
  const int64_t v = i ? PyLong_AsLongLong(i.ptr()) : -1;
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + ": " + what);
  }
  if (v < least) refuse(std::string(name) + ": " + what);
  return v;
}
void check_sizes(std::initializer_list<int64_t> sizes) {
  for (int64_t v : sizes)
    if (v > 0x7fffffff) refuse("sizes: below 2^31");
}

// Allocations and the call itself: made on device `dev` with Python's lock
// released, as either may wait.
template <typename F>
void launching(int dev, const char* what, F&& f) {
  tq_status st;
  {
    py::gil_scoped_release unlocked;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    st = f();
  }
  raise_status(st, what);
}

// Strides of a [T, H, d] view whose rows are dense and 16-byte aligned (0 for a
// dimension of one element, whose stride is never used and may be anything).
std::pair<int64_t, int64_t> head_rows(const Tensor& t, const char* name) {
  const int64_t s0 = t.size(0) > 1 ? t.stride(0) : 0, s1 = t.size(1) > 1 ? t.stride(1) : 0;
  if (t.stride(2) != 1 || ((s0 | s1) & 7) || (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15))
    refuse(std::string(name) + ": dense rows, 16-byte aligned, strides multiples of 8 elements");
  return {s0, s1};
}

// ------------------------------------------------------------------ norm and rotation

py::tuple qk_norm_rope(py::handle q_, py::handle k_, py::handle positions_, py::handle inv_freq_, bool interleaved,
                       double rope_scale, py::handle q_weight_, py::handle k_weight_, double eps, py::handle out_) {
  const Tensor q = tensor(q_, "q"), k = tensor(k_, "k"), positions = tensor(positions_, "positions");
  const Tensor inv_freq = maybe(inv_freq_, "inv_freq");
  const Tensor w[2] = {maybe(q_weight_, "q_weight"), maybe(k_weight_, "k_weight")};
  if (q.dim() != 3 || k.dim() != 3) refuse("q: [T, Hq, d]; k: [T, Hkv, d]");
  const int64_t T = q.size(0), hq = q.size(1), d = q.size(2), hkv = k.size(1);
  if (k.size(0) != T || k.size(2) != d) refuse("q: [T, Hq, d]; k: [T, Hkv, d] with the same T and d");
  if (d != 64 && d != 128 && d != 256) refuse("head_dim: 64, 128 or 256, got " + std::to_string(d));
  if (hq == 0 || hkv == 0) refuse("q, k: at least one head");
  const ScalarType kind = q.scalar_type();
  if ((kind != ScalarType::Half && kind != ScalarType::BFloat16) || k.scalar_type() != kind)
    refuse("q, k: both float16 or both bfloat16, got " + kind_name(kind) + " and " + kind_name(k.scalar_type()));
  const auto qs = head_rows(q, "q"), ks = head_rows(k, "k");
  check_numel(positions, "positions", {ScalarType::Int}, T);
  int64_t rot = 0;
  if (inv_freq.defined()) {
    check(inv_freq, "inv_freq", {ScalarType::Double});
    rot = 2 * inv_freq.numel();
    if (rot > d)
      refuse("inv_freq: at most " + std::to_string(d / 2) + " frequencies, got " + std::to_string(rot / 2));
  }
  for (int i = 0; i < 2; ++i) {
    const char* name = i ? "k_weight" : "q_weight";
    if (!w[i].defined()) continue;
    check_numel(w[i], name, {kind, ScalarType::Float}, d);
    if (reinterpret_cast<uintptr_t>(w[i].data_ptr()) & 15) refuse(std::string(name) + ": 16-byte aligned");
  }
  if (w[0].defined() && w[1].defined() && w[0].scalar_type() != w[1].scalar_type())
    refuse("q_weight, k_weight: the same dtype");
  if (!(eps >= 0.0)) refuse("eps: >= 0");
  Tensor qo, ko;
  if (!out_.is_none()) {
    const py::sequence out = py::reinterpret_borrow<py::sequence>(out_);
    qo = tensor(py::object(out[0]), "out q");
    ko = tensor(py::object(out[1]), "out k");
    check_shape(qo, "out q", {ScalarType::Half}, {T, hq, d});
    check_shape(ko, "out k", {ScalarType::Half}, {T, hkv, d});
    apart("out q", qo, {&k, &ko, &positions, &inv_freq, &w[0], &w[1]}, &q);
    apart("out k", ko, {&q, &qo, &positions, &inv_freq, &w[0], &w[1]}, &k);
  }
  forward_only({{"q", &q}, {"k", &k}, {"inv_freq", &inv_freq}, {"q_weight", &w[0]}, {"k_weight", &w[1]},
                {"out q", &qo}, {"out k", &ko}});
  const int dev = one_device({{"q", &q}, {"k", &k}, {"positions", &positions}, {"inv_freq", &inv_freq},
                              {"q_weight", &w[0]}, {"k_weight", &w[1]}, {"out q", &qo}, {"out k", &ko}});
  check_sizes({hq, hkv});
  launching(dev, "tq_qk_norm_rope", [&] {
    if (!qo.defined()) {
      qo = at::empty({T, hq, d}, q.options().dtype(ScalarType::Half));
      ko = at::empty({T, hkv, d}, q.options().dtype(ScalarType::Half));
    }
    const Tensor& some = w[0].defined() ? w[0] : w[1];
    return tq_qk_norm_rope(q.data_ptr(), k.data_ptr(), kind == ScalarType::Half ? TQ_F16 : TQ_BF16, T, (int)hq,
                           (int)hkv, (int)d, qs.first, qs.second, ks.first, ks.second, address_as<int32_t>(positions),
                           address_as<double>(inv_freq), (int)rot, interleaved, (float)rope_scale, address(w[0]),
                           address(w[1]), some.defined() && some.scalar_type() == ScalarType::Float, (float)eps,
                           qo.data_ptr(), ko.data_ptr(), stream_of(dev));
  });
  return py::make_tuple(qo, ko);
}

// ------------------------------------------------------------------ windowed attention

// Both forms: `table` undefined for contiguous caches. `k_codec`, `v_codec`:
// addresses of the codecs' contexts. With RUN false the arguments are only
// checked.
template <bool RUN>
Tensor attend_window(py::handle q_, uintptr_t k_codec, uintptr_t v_codec, py::handle kc_, py::handle kn_,
                     py::handle vc_, py::handle vn_, bool paged, py::handle table_, py::handle lens_,
                     py::handle window_, py::handle sinks_, py::handle offsets_, py::handle max_q_, py::handle out_,
                     py::handle workspace_) {
  const tq_ctx* ck = reinterpret_cast<const tq_ctx*>(k_codec);
  const tq_ctx* cv = reinterpret_cast<const tq_ctx*>(v_codec);
  const char *k_name = paged ? "k_cache" : "k_packed", *v_name = paged ? "v_cache" : "v_packed";
  const Tensor q = tensor(q_, "q"), kc = tensor(kc_, k_name), kn = tensor(kn_, "k_norms"), vc = tensor(vc_, v_name),
               vn = tensor(vn_, "v_norms"), lens = tensor(lens_, "context_lens");
  const Tensor table = paged ? tensor(table_, "block_tables") : Tensor();
  const Tensor offsets = maybe(offsets_, "q_offsets");
  Tensor out = maybe(out_, "out"), workspace = maybe(workspace_, "workspace");
  if (q.dim() != 3 || kc.dim() != 4 || (paged && table.dim() != 2))
    refuse(paged ? "q: [T, Hq, d]; k_cache: [num_blocks, 16, Hkv, Pk]; block_tables: [B, max_blocks]"
                 : "q: [T, Hq, d]; k_packed: [B, S, Hkv, Pk]");
  const int64_t n0 = kc.size(0), n1 = kc.size(1), hkv = kc.size(2);
  if (paged && n1 != TQ_PAGE_BLOCK) refuse("cache blocks must hold 16 positions");
  const int64_t B = paged ? table.size(0) : n0, s_max = paged ? table.size(1) * TQ_PAGE_BLOCK : n1;
  const int64_t T = q.size(0), hq = q.size(1), d = tq_head_dim(ck);
  check_shape(q, "q", {ScalarType::Half}, {T, hq, d});
  if (tq_head_dim(cv) != d) refuse("k_codec, v_codec: the same head_dim");
  if (hkv <= 0 || hq <= 0 || hq % hkv)
    refuse("q: a multiple of " + std::to_string(hkv) + " heads, got " + std::to_string(hq));
  const int64_t window = window_.is_none() ? 0 : whole(window_, "window", 1, "None or at least 1");
  const int64_t sinks = whole(sinks_, "sinks", 0, "at least 0");
  int64_t max_q = 1;
  if (offsets.defined()) {
    check_numel(offsets, "q_offsets", {ScalarType::Int}, B + 1);
    const char* what = "the largest number of tokens of a sequence";
    if (max_q_.is_none()) refuse(std::string("max_q: ") + what);
    max_q = whole(max_q_, "max_q", 1, what);
  } else if (T != B || !(max_q_.is_none() || whole(max_q_, "max_q", 1, "None or 1 where q_offsets is None") == 1)) {
    refuse("q: one token per sequence where q_offsets is None");
  }
  check_shape(kc, k_name, {ScalarType::Byte}, {n0, n1, hkv, (int64_t)tq_packed_bytes(ck)});
  check_shape(vc, v_name, {ScalarType::Byte}, {n0, n1, hkv, (int64_t)tq_packed_bytes(cv)});
  check_shape(kn, "k_norms", {ScalarType::Float}, {n0, n1, hkv});
  check_shape(vn, "v_norms", {ScalarType::Float}, {n0, n1, hkv});
  if (paged) check(table, "block_tables", {ScalarType::Int});
  check_numel(lens, "context_lens", {ScalarType::Int}, B);
  if (out.defined()) check_shape(out, "out", {ScalarType::Half}, {T, hq, d});
  if (workspace.defined()) check(workspace, "workspace", {ScalarType::Byte});
  if (out.defined()) apart("out", out, {&kc, &kn, &vc, &vn, &table, &lens, &offsets, &workspace}, &q);
  if (workspace.defined()) apart("workspace", workspace, {&q, &kc, &kn, &vc, &vn, &table, &lens, &offsets}, nullptr);
  forward_only({{"q", &q}, {"k_norms", &kn}, {"v_norms", &vn}, {"out", &out}});
  const int dev = one_device({{"q", &q}, {"q_offsets", &offsets}, {"out", &out}, {"workspace", &workspace},
                              {k_name, &kc}, {v_name, &vc}, {"k_norms", &kn}, {"v_norms", &vn},
                              {"block_tables", &table}, {"context_lens", &lens}});
  check_sizes({B, max_q, hq, hkv, paged ? table.size(1) : 0});
  if (!RUN) return q;
  launching(dev, paged ? "tq_attend_window_paged" : "tq_attend_window", [&] {
    if (!out.defined()) out = at::empty({T, hq, d}, q.options());
    if (!workspace.defined())
      workspace = bytes_on(tq_attend_window_workspace_bytes(T, (int)B, (int)max_q, (int)hq, (int)hkv, (int)d, s_max,
                                                            window, sinks),
                           q);
    const size_t ws = workspace.defined() ? (size_t)workspace.numel() : 0;
    if (paged)
      return tq_attend_window_paged(ck, cv, q.data_ptr(), T, (int)B, address_as<int32_t>(offsets), (int)max_q,
                                    (int)hq, (int)hkv, kc.data_ptr(), address_as<float>(kn), vc.data_ptr(),
                                    address_as<float>(vn), n0, address_as<int32_t>(table), (int)table.size(1),
                                    address_as<int32_t>(lens), window, sinks, out.data_ptr(), address(workspace), ws,
                                    stream_of(dev));
    return tq_attend_window(ck, cv, q.data_ptr(), T, (int)B, address_as<int32_t>(offsets), (int)max_q, (int)hq,
                            (int)hkv, kc.data_ptr(), address_as<float>(kn), vc.data_ptr(), address_as<float>(vn),
                            s_max, address_as<int32_t>(lens), window, sinks, out.data_ptr(), address(workspace), ws,
                            stream_of(dev));
  });
  return out;
}

// ------------------------------------------------------------------ pages

// Tables of a paged cache: [rows, max_blocks] entries, lengths (where given)
// and one count per page.
void check_state(const Tensor& table, const Tensor& lens, const Tensor& refs, int64_t num_blocks) {
  check(table, "block_tables", {ScalarType::Int});
  if (table.dim() != 2 || !table.numel()) refuse("block_tables: [rows, max_blocks]");
  if (lens.defined()) check_numel(lens, "context_lens", {ScalarType::Int}, table.size(0));
  check(refs, "refs", {ScalarType::Int});
  if (refs.dim() != 1 || !refs.numel() || (num_blocks >= 0 && refs.numel() != num_blocks))
    refuse("refs: one count per page (" + (num_blocks < 0 ? "None" : std::to_string(num_blocks)) + "), got " +
           shape_name(refs.sizes()));
  if (table.size(0) > 0x7fffffff || table.size(1) > 0x7fffffff) refuse("block_tables: sizes below 2^31");
}

Tensor output(py::handle out, int i, const Tensor& like) {
  const Tensor t = tensor(py::object(py::reinterpret_borrow<py::sequence>(out)[i]), "out");
  check(t, "out", {like.scalar_type()});
  if (t.sizes() != like.sizes()) refuse("out: shape " + shape_name(like.sizes()) + ", got " + shape_name(t.sizes()));
  return t;
}

py::tuple pages_trim(py::handle table_, py::handle lens_, py::handle refs_, py::handle window_, py::handle sinks_,
                     py::handle release_, py::handle out_) {
  const Tensor table = tensor(table_, "block_tables"), lens = tensor(lens_, "context_lens"),
               refs = tensor(refs_, "refs"), release = maybe(release_, "release");
  check_state(table, lens, refs, -1);
  const int64_t window = window_.is_none() ? -1 : whole(window_, "window", 0, "None or at least 0");
  const int64_t sinks = whole(sinks_, "sinks", 0, "at least 0");
  if (release.defined()) check_numel(release, "release", {ScalarType::Bool, ScalarType::Byte}, table.size(0));
  Tensor t, n, r;
  if (!out_.is_none()) {
    t = output(out_, 0, table), n = output(out_, 1, lens), r = output(out_, 2, refs);
    apart("out", t, {&lens, &refs, &n, &r, &release}, &table);
    apart("out", n, {&table, &refs, &t, &r, &release}, &lens);
    apart("out", r, {&table, &lens, &t, &n, &release}, &refs);
  }
  const int dev = one_device({{"block_tables", &table}, {"context_lens", &lens}, {"refs", &refs},
                              {"release", &release}, {"out", &t}, {"out", &n}, {"out", &r}});
  launching(dev, "tq_pages_trim", [&] {
    if (!t.defined()) t = fresh(table), n = fresh(lens), r = fresh(refs);
    return tq_pages_trim(address_as<int32_t>(table), address_as<int32_t>(t), address_as<int32_t>(lens),
                         address_as<int32_t>(n), address_as<int32_t>(refs), address_as<int32_t>(r),
                         (int)table.size(0), (int)table.size(1), refs.numel(), window, sinks,
                         address_as<uint8_t>(release), stream_of(dev));
  });
  return py::make_tuple(t, n, r);
}

void on_pools(int dev, int pool_dev) {
  if (dev != pool_dev)
    refuse("tensors on cuda:" + std::to_string(pool_dev) + " like the pools, got cuda:" + std::to_string(dev));
}

// Refuse tables and workspaces that share memory with a pool, whose pages the
// call moves.
void off_pools(const tq_page_pool* pools, int n_pools, int64_t num_blocks,
               std::initializer_list<std::pair<const char*, const Tensor*>> all) {
  for (const auto& [name, t] : all) {
    if (!t->defined()) continue;
    const auto [lo, hi] = span(*t);
    for (int i = 0; i < n_pools; ++i) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(pools[i].base);
      if (lo < a + (uintptr_t)(pools[i].block_bytes * num_blocks) && a < hi)
        refuse(std::string(name) + ": shares memory with pool " + std::to_string(i));
    }
  }
}

// `pools`: address of `n_pools` tq_page_pool.
py::tuple pages_fork(uintptr_t pools, int n_pools, int64_t num_blocks, int pool_dev, py::handle table_,
                     py::handle lens_, py::handle refs_, py::handle parents_, py::handle children_, py::handle out_,
                     py::handle workspace_) {
  const Tensor table = tensor(table_, "block_tables"), lens = tensor(lens_, "context_lens"),
               refs = tensor(refs_, "refs"), parents = tensor(parents_, "parents"),
               children = tensor(children_, "children");
  Tensor workspace = maybe(workspace_, "workspace");
  check_state(table, lens, refs, num_blocks);
  const int64_t rows = table.size(0), forks = parents.numel();
  check(parents, "parents", {ScalarType::Int});
  check_numel(children, "children", {ScalarType::Int}, forks);
  if (forks > rows || rows > TQ_MAX_PAGE_ROWS)
    refuse("at most " + std::to_string(rows) + " forks of at most " + std::to_string(TQ_MAX_PAGE_ROWS) + " rows");
  if (workspace.defined()) check(workspace, "workspace", {ScalarType::Byte});
  Tensor t, n, r;
  if (!out_.is_none()) {
    t = output(out_, 0, table), n = output(out_, 1, lens), r = output(out_, 2, refs);
    apart("out", t, {&lens, &refs, &n, &r, &parents, &children}, &table);
    apart("out", n, {&table, &refs, &t, &r, &parents, &children}, &lens);
    apart("out", r, {&table, &lens, &t, &n, &parents, &children}, &refs);
  }
  if (workspace.defined())
    apart("workspace", workspace, {&table, &lens, &refs, &parents, &children, &t, &n, &r}, nullptr);
  const tq_page_pool* const of = reinterpret_cast<const tq_page_pool*>(pools);
  off_pools(of, n_pools, num_blocks, {{"block_tables", &table}, {"context_lens", &lens}, {"refs", &refs},
                                      {"parents", &parents}, {"children", &children}, {"workspace", &workspace},
                                      {"out", &t}, {"out", &n}, {"out", &r}});
  const int dev = one_device({{"block_tables", &table}, {"context_lens", &lens}, {"refs", &refs},
                              {"parents", &parents}, {"children", &children}, {"workspace", &workspace}, {"out", &t},
                              {"out", &n}, {"out", &r}});
  on_pools(dev, pool_dev);
  launching(dev, "tq_pages_fork", [&] {
    if (!t.defined()) t = fresh(table), n = fresh(lens), r = fresh(refs);
    if (!workspace.defined()) workspace = bytes_on(tq_pages_fork_workspace_bytes((int)forks), refs);
    return tq_pages_fork(of, n_pools, num_blocks, address_as<int32_t>(table),
                         address_as<int32_t>(t), address_as<int32_t>(lens), address_as<int32_t>(n),
                         address_as<int32_t>(refs), address_as<int32_t>(r), (int)rows, (int)table.size(1),
                         address_as<int32_t>(parents), address_as<int32_t>(children), (int)forks, address(workspace),
                         workspace.defined() ? (size_t)workspace.numel() : 0, stream_of(dev));
  });
  return py::make_tuple(t, n, r);
}

py::tuple pages_compact(uintptr_t pools, int n_pools, int64_t num_blocks, int pool_dev, py::handle table_,
                        py::handle refs_, py::handle out_, py::handle workspace_) {
  const Tensor table = tensor(table_, "block_tables"), refs = tensor(refs_, "refs");
  Tensor workspace = maybe(workspace_, "workspace");
  check_state(table, Tensor(), refs, num_blocks);
  if (table.size(0) > TQ_MAX_PAGE_ROWS)
    refuse("block_tables: at most " + std::to_string(TQ_MAX_PAGE_ROWS) + " rows");
  if (workspace.defined()) check(workspace, "workspace", {ScalarType::Byte});
  Tensor t, r, remap, used;
  if (!out_.is_none()) {
    const py::sequence out = py::reinterpret_borrow<py::sequence>(out_);
    t = output(out_, 0, table), r = output(out_, 1, refs);
    remap = tensor(py::object(out[2]), "out remap");
    used = tensor(py::object(out[3]), "out used");
    check_numel(remap, "out remap", {ScalarType::Int}, num_blocks);
    check_numel(used, "out used", {ScalarType::Int}, 1);
    apart("out", t, {&refs, &r, &remap, &used}, &table);
    apart("out", r, {&table, &t, &remap, &used}, &refs);
    apart("out", remap, {&table, &refs, &t, &r, &used}, nullptr);
    apart("out", used, {&table, &refs, &t, &r, &remap}, nullptr);
  }
  if (workspace.defined()) apart("workspace", workspace, {&table, &refs, &t, &r, &remap, &used}, nullptr);
  const tq_page_pool* const of = reinterpret_cast<const tq_page_pool*>(pools);
  off_pools(of, n_pools, num_blocks, {{"block_tables", &table}, {"refs", &refs}, {"workspace", &workspace},
                                      {"out", &t}, {"out", &r}, {"out remap", &remap}, {"out used", &used}});
  const int dev = one_device({{"block_tables", &table}, {"refs", &refs}, {"workspace", &workspace}, {"out", &t},
                              {"out", &r}, {"out", &remap}, {"out", &used}});
  on_pools(dev, pool_dev);
  launching(dev, "tq_pages_compact", [&] {
    if (!t.defined()) {
      t = fresh(table), r = fresh(refs), remap = fresh(refs);
      used = at::empty({1}, refs.options());
    }
    if (!workspace.defined()) workspace = bytes_on(tq_pages_compact_workspace_bytes(num_blocks), refs);
    return tq_pages_compact(of, n_pools, num_blocks,
                            address_as<int32_t>(table), address_as<int32_t>(t), address_as<int32_t>(refs),
                            address_as<int32_t>(r), (int)table.size(0), (int)table.size(1),
                            address_as<int32_t>(remap), address_as<int32_t>(used), address(workspace),
                            workspace.defined() ? (size_t)workspace.numel() : 0, stream_of(dev));
  });
  return py::make_tuple(t, r, remap, used);
}

}  // namespace

PYBIND11_MODULE(_ops, m) {
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("attend_window", &attend_window<true>);
  m.def("check_attend_window", &attend_window<false>);
  m.def("pages_trim", &pages_trim);
  m.def("pages_fork", &pages_fork);
  m.def("pages_compact", &pages_compact);
}
