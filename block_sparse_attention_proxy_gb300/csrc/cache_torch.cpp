// The torch front end of rotary positions and the paged key-value cache: argument checks, output
// allocation, the autograd node of the rotation.  The computation is in the library's kernels.
#include "torch_front.h"

namespace {

using namespace msa_front;

// Frequencies and layout of a rotation, made once by a program (rotary_plan).
struct Plan {
  std::vector<uint64_t> freq;
  bool interleaved;
  float amplitude;
  int64_t dims() const { return 2 * (int64_t)freq.size(); }
};

constexpr int64_t kMost = std::numeric_limits<int32_t>::max();

Tensor or_none(const std::optional<Tensor>& t) { return t ? *t : Tensor(); }
bool integers(const Tensor& t) {
  return t.scalar_type() == at::kInt || t.scalar_type() == at::kLong;
}
const int32_t* ints_in(const Tensor& t) {
  return t.defined() ? t.const_data_ptr<int32_t>() : nullptr;
}
const void* any_in(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void* any_out(const Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }
void no_grad(const Tensor& t, const char* who) {
  no_tangent(t, who);
  TORCH_CHECK_NOT_IMPLEMENTED(
      !(t.defined() && t.requires_grad() && at::GradMode::is_enabled()), who,
      " has no backward (an input requires a gradient)");
}

// ------------------------------ rotary ------------------------------------------

msa_dtype type_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MSA_BF16;
    case at::kHalf: return MSA_FP16;
    case at::kFloat: return MSA_FP32;
    default: throw py::type_error("q and k must be bf16, fp16 or fp32 tensors");
  }
}

// One launch over q and, if it is defined, k.
void rotate(const Plan& plan, const Tensor& q, const Tensor& k, const Tensor& cu,
            const Tensor& positions, bool inverse, Tensor* q_out, Tensor* k_out) {
  msa_rotary_params p{};
  p.total_tokens = (int32_t)q.size(0);
  p.num_docs = cu.defined() ? (int32_t)(cu.numel() - 1) : 0;
  p.d = (int32_t)q.size(2);
  p.dims = (int32_t)plan.dims();
  p.interleaved = plan.interleaved;
  p.inverse = inverse;
  p.dtype = type_of(q);
  p.position_bytes = positions.defined() ? (int32_t)positions.element_size() : 0;
  p.freq = plan.freq.data();
  p.amplitude = plan.amplitude;
  const auto opt = q.options().requires_grad(false);
  const Tensor q_ = take(q, &p.q_stride);
  Tensor k_;
  p.hq = (int32_t)q.size(1);
  *q_out = at::empty(q.sizes(), opt);
  if (k.defined()) {
    k_ = take(k, &p.k_stride);
    p.hkv = (int32_t)k.size(1);
    *k_out = at::empty(k.sizes(), opt);
  }
  raise_on(msa_rotary(&p, ints_in(cu), any_in(positions), any_in(q_), any_in(k_),
                      any_out(*q_out), any_out(*k_out), current_stream()),
           "msa_rotary");
}

variable_list turn(const std::shared_ptr<Plan>& plan, const variable_list& x, const Tensor& cu,
                   const Tensor& positions, bool inverse);

// The gradient turns by the opposite angles: the same operator again, so that it can be
// differentiated further.
struct RotaryBackward : torch::autograd::Node {
  std::shared_ptr<Plan> plan;
  SavedVariable cu, positions;
  int64_t sizes[2] = {0, 0};  // of cu and positions
  at::ScalarType type = at::kFloat;
  bool inverse = false;

  std::string name() const override { return "RotaryBackward"; }
  void release_variables() override {
    cu.reset_data();
    positions.reset_data();
  }
  variable_list apply(variable_list&& grads) override {
    variable_list g(grads.size()), in;
    std::vector<size_t> at;
    for (size_t i = 0; i < grads.size(); ++i) {
      no_tangent(grads[i], "rotary");
      if (!grads[i].defined() || !task_should_compute_output(i)) continue;
      in.push_back(grads[i].scalar_type() == type ? grads[i] : grads[i].to(type));
      at.push_back(i);
    }
    if (in.empty()) return g;
    try {
      const at::Device device = in[0].device();
      c10::cuda::CUDAGuard guard(device);
      check_capture(*this, "rotary");
      const variable_list y = turn(plan, in, back(cu, device, sizes[0]),
                                   back(positions, device, sizes[1]), !inverse);
      for (size_t i = 0; i < at.size(); ++i) g[at[i]] = y[i];
    } catch (const StatusError& e) {
      throw_to_engine(e);
    }
    return g;
  }
  // A saved tensor may come back from its hooks in another layout, but with the forward's values.
  static Tensor back(const SavedVariable& s, const at::Device& device, int64_t size) {
    Tensor t = s.unpack();
    if (!t.defined()) return t;
    if (!integers(t) || t.dim() != 1 || t.numel() != size || t.device() != device)
      throw StatusError(MSA_ERR_INVALID_ARG, "rotary: a saved tensor");
    return t.contiguous();
  }
};

// Turns one tensor or two of one type, number of rows and device, and remembers how.
variable_list turn(const std::shared_ptr<Plan>& plan, const variable_list& x, const Tensor& cu,
                   const Tensor& positions, bool inverse) {
  variable_list y(2);
  {
    at::NoGradGuard no_grad;
    rotate(*plan, x[0], x.size() > 1 ? x[1] : Tensor(), cu, positions, inverse, &y[0], &y[1]);
  }
  y.resize(x.size());
  bool keep = false;
  for (const Tensor& t : x) keep |= at::GradMode::is_enabled() && t.requires_grad();
  if (keep) {
    std::shared_ptr<RotaryBackward> node(new RotaryBackward(), torch::autograd::deleteNode);
    node->set_next_edges(torch::autograd::collect_next_edges(x));
    node->plan = plan;
    node->type = x[0].scalar_type();
    node->inverse = inverse;
    node->sizes[0] = cu.defined() ? cu.numel() : 0;
    node->sizes[1] = positions.defined() ? positions.numel() : 0;
    node->cu = SavedVariable(cu, false);
    node->positions = SavedVariable(positions, false);
    for (Tensor& t : y) torch::autograd::set_history(t, node);
  }
  return y;
}

std::tuple<Tensor, Tensor> rotary(const Tensor& q, const std::optional<Tensor>& k_,
                                  const std::shared_ptr<Plan>& plan,
                                  const std::optional<Tensor>& cu_,
                                  const std::optional<Tensor>& positions_) {
  const Tensor k = or_none(k_), cu = or_none(cu_), positions = or_none(positions_);
  for (const Tensor* t : {&q, &k}) {
    if (!t->defined()) continue;
    no_tangent(*t, "rotary");
    if (!t->is_cuda()) throw py::type_error("q and k must be CUDA tensors");
    if (t->dim() != 3 || t->size(0) != q.size(0) || t->size(2) != q.size(2) ||
        t->device() != q.device())
      throw py::value_error("q [T, Hq, d] and k [T, Hkv, d] on one device expected");
    if (t->scalar_type() != q.scalar_type()) throw py::type_error("q and k must have one type");
    if (t->size(0) > kMost || t->size(1) > kMost || t->size(2) > kMost)
      throw py::value_error("sizes beyond 32 bits");
  }
  type_of(q);
  if (cu.defined() == positions.defined())
    throw py::value_error("either cu_seqlens or positions expected");
  const Tensor& where = cu.defined() ? cu : positions;
  if (!integers(where)) throw py::type_error("cu_seqlens and positions must be integers");
  if (where.dim() != 1 || where.device() != q.device() ||
      (cu.defined() ? cu.numel() < 2 || cu.numel() > kMost : positions.numel() != q.size(0)))
    throw py::value_error(
        "cu_seqlens must be [num_docs + 1], positions [T], on the device of q");
  if (plan->dims() > q.size(2)) throw py::value_error("the plan rotates more than a head has");
  c10::cuda::CUDAGuard guard(q.device());
  const variable_list y = turn(plan, k.defined() ? variable_list{q, k} : variable_list{q},
                               cu.defined() ? ints(cu).contiguous() : Tensor(),
                               positions.defined() ? positions.contiguous() : Tensor(), false);
  return {y[0], y.size() > 1 ? y[1] : Tensor()};
}

// ------------------------------ cache -------------------------------------------

// The cache's tensors and a page table, checked and described for the library.
struct Pages {
  msa_cache cache{};
  msa_table table{};
  Tensor k, v, weight, position, pages, lens;

  Pages(const char* who, const Tensor& k_, const Tensor& v_, const std::optional<Tensor>& weight_,
        const std::optional<Tensor>& position_, const Tensor& table_, const Tensor& lens_)
      : k(k_), v(v_), weight(or_none(weight_)), position(or_none(position_)) {
    for (const Tensor* t : {&k, &v}) {
      if (t->scalar_type() != at::kBFloat16 || !t->is_cuda())
        throw py::type_error("the cache's k and v must be bf16 CUDA tensors");
      no_grad(*t, who);
    }
    if (k.dim() != 4 || k.sizes() != v.sizes() || k.device() != v.device())
      throw py::value_error("the cache's k and v must be [pages, page size, Hkv, d] on one device");
    for (int i = 0; i < 4; ++i)
      if (k.size(i) > kMost) throw py::value_error("sizes beyond 32 bits");
    if (k.size(3) > 1 && (k.stride(3) != 1 || v.stride(3) != 1))
      throw py::value_error("the elements of a head must be contiguous");
    meta(weight, at::kFloat, "weight must be fp32 [pages, Hkv, page size], contiguous");
    meta(position, at::kInt, "position must be int32 [pages, Hkv, page size], contiguous");
    if (!integers(table_) || !integers(lens_))
      throw py::type_error("table and lens must be integers");
    if (table_.dim() != 2 || lens_.dim() != 1 || table_.size(0) != lens_.size(0) ||
        table_.device() != k.device() || lens_.device() != k.device())
      throw py::value_error(
          "table must be [sequences, pages] and lens [sequences], on the device of the cache");
    if (table_.size(0) > kMost || table_.size(1) > kMost)
      throw py::value_error("sizes beyond 32 bits");
  }
  void meta(const Tensor& t, at::ScalarType type, const char* what) {
    if (!t.defined()) return;
    if (t.scalar_type() != type) throw py::type_error(what);
    if (t.device() != k.device() || t.dim() != 3 || t.size(0) != k.size(0) ||
        t.size(1) != k.size(2) || t.size(2) != k.size(1) || !t.is_contiguous())
      throw py::value_error(what);
  }
  // after the device has been made current
  void describe(const Tensor& table_, const Tensor& lens_) {
    pages = ints(table_);
    if (pages.size(1) > 1 && pages.stride(1) != 1) pages = pages.contiguous();
    if (pages.size(0) > 1 && pages.stride(0) < pages.size(1)) pages = pages.contiguous();
    lens = ints(lens_).contiguous();
    cache.k = out(k);
    cache.v = out(v);
    cache.weight = weight.defined() ? weight.mutable_data_ptr<float>() : nullptr;
    cache.position = position.defined() ? position.mutable_data_ptr<int32_t>() : nullptr;
    cache.num_pages = (int32_t)k.size(0);
    cache.page_size = (int32_t)k.size(1);
    cache.hkv = (int32_t)k.size(2);
    cache.d = (int32_t)k.size(3);
    cache.k_page_stride = k.stride(0);
    cache.k_slot_stride = k.stride(1);
    cache.k_head_stride = k.stride(2);
    cache.v_page_stride = v.stride(0);
    cache.v_slot_stride = v.stride(1);
    cache.v_head_stride = v.stride(2);
    table.pages = ints_in(pages);
    table.lens = ints_in(lens);
    table.num_seqs = (int32_t)pages.size(0);
    table.max_pages = (int32_t)pages.size(1);
    table.stride = pages.stride(0);
  }
  // What a call writes in place; said before it does, so that a tensor that must not be written
  // is refused.
  void changed(bool rows, bool position_too) {
    if (rows) {
      torch::autograd::impl::bump_version(k);
      torch::autograd::impl::bump_version(v);
    }
    if (weight.defined()) torch::autograd::impl::bump_version(weight);
    if (position_too && position.defined()) torch::autograd::impl::bump_version(position);
  }
};

void rows(const Tensor& t, const Pages& c, int64_t tokens, int64_t heads, const char* what) {
  if (t.scalar_type() != at::kBFloat16) throw py::type_error(what);
  if (t.device() != c.k.device() || t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads ||
      t.size(2) != c.k.size(3))
    throw py::value_error(what);
}

std::optional<Tensor> cache_append(const Tensor& ck, const Tensor& cv,
                                   const std::optional<Tensor>& weight,
                                   const std::optional<Tensor>& position, const Tensor& k,
                                   const Tensor& v, const Tensor& table, const Tensor& lens,
                                   const std::optional<Tensor>& cu_,
                                   const std::optional<Tensor>& positions_,
                                   const std::optional<std::shared_ptr<Plan>>& plan,
                                   const std::optional<Tensor>& q_) {
  constexpr const char* who = "cache_append";
  Pages c(who, ck, cv, weight, position, table, lens);
  const Tensor cu = or_none(cu_), positions = or_none(positions_), q = or_none(q_);
  for (const Tensor& t : {k, v, q, c.weight}) no_grad(t, who);
  if (k.dim() != 3 || k.size(0) > kMost)
    throw py::value_error("k and v must be [T, Hkv, d] as in the cache, on its device");
  const int64_t T = k.size(0);
  for (const Tensor* t : {&k, &v})
    rows(*t, c, T, ck.size(2), "k and v must be bf16 [T, Hkv, d] as in the cache, on its device");
  if (q.defined()) {
    if (q.dim() != 3 || q.size(1) > kMost) throw py::value_error("q must be [T, Hq, d]");
    rows(q, c, T, q.size(1), "q must be bf16 [T, Hq, d], d as in the cache, on its device");
  }
  if (q.defined() && !plan) throw py::value_error("q is for a rotation: plan expected");
  if (plan && (*plan)->dims() > ck.size(3))
    throw py::value_error("the plan rotates more than a head has");
  if (cu.defined()) {
    if (!integers(cu)) throw py::type_error("cu_seqlens must be integers");
    if (cu.dim() != 1 || cu.numel() != lens.size(0) + 1 || cu.numel() < 2 ||
        cu.device() != ck.device())
      throw py::value_error("cu_seqlens must be [sequences + 1] on the device of the cache");
  } else if (T != lens.size(0)) {
    throw py::value_error("without cu_seqlens there is one token a sequence");
  }
  if (positions.defined()) {
    if (!integers(positions)) throw py::type_error("positions must be integers");
    if (positions.dim() != 1 || positions.numel() != T || positions.device() != ck.device())
      throw py::value_error("positions must be [T] on the device of the cache");
  }
  c10::cuda::CUDAGuard guard(ck.device());
  at::NoGradGuard no_grad;
  c.describe(table, lens);
  msa_rotary_params p{};
  p.total_tokens = (int32_t)T;
  p.num_docs = cu.defined() ? (int32_t)(cu.numel() - 1) : 0;
  p.hkv = c.cache.hkv;
  p.d = c.cache.d;
  p.dtype = MSA_BF16;
  p.amplitude = 1.f;
  if (plan) {
    p.dims = (int32_t)(*plan)->dims();
    p.interleaved = (*plan)->interleaved;
    p.freq = (*plan)->freq.data();
    p.amplitude = (*plan)->amplitude;
  }
  Tensor cu32, at_, q__, qo;
  if (cu.defined()) cu32 = ints(cu).contiguous();
  if (positions.defined()) {
    at_ = positions.contiguous();
    p.position_bytes = (int32_t)at_.element_size();
  }
  int64_t v_stride = 0;
  const Tensor k_ = take(k, &p.k_stride), v_ = take(v, &v_stride);
  if (q.defined()) {
    q__ = take(q, &p.q_stride);
    p.hq = (int32_t)q.size(1);
    qo = at::empty(q.sizes(), q.options().requires_grad(false));
  }
  c.changed(true, true);
  raise_on(msa_cache_append(&c.cache, &c.table, &p, v_stride, ints_in(cu32), any_in(at_), in(q__),
                            in(k_), in(v_), out(qo), current_stream()),
           "msa_cache_append");
  if (!qo.defined()) return std::nullopt;
  return qo;
}

Tensor paged_attention(const Tensor& q, const Tensor& ck, const Tensor& cv,
                       const std::optional<Tensor>& weight, const std::optional<Tensor>& position,
                       const Tensor& table, const Tensor& lens, double softmax_scale,
                       bool accumulate) {
  constexpr const char* who = "paged_attention";
  Pages c(who, ck, cv, weight, position, table, lens);
  no_grad(q, who);
  if (q.dim() != 3 || q.size(1) > kMost) throw py::value_error("q must be [sequences, Hq, d]");
  rows(q, c, lens.size(0), q.size(1),
       "q must be bf16 [sequences, Hq, d], d as in the cache, on its device");
  if (accumulate && !c.weight.defined())
    throw py::value_error("the cache keeps no weights to add to");
  if (accumulate) no_grad(c.weight, who);
  c10::cuda::CUDAGuard guard(ck.device());
  at::NoGradGuard no_grad;
  c.describe(table, lens);
  msa_paged_params p{};
  p.hq = (int32_t)q.size(1);
  p.accumulate = accumulate;
  p.softmax_scale = (float)softmax_scale;
  const Tensor q_ = take(q, &p.q_stride);
  const auto opt = q.options().requires_grad(false);
  Tensor o = at::empty(q.sizes(), opt);
  const size_t need = msa_paged_attention_workspace_size(&c.cache, &c.table, &p);
  Tensor ws;
  if (need > 256) ws = at::empty({(int64_t)need}, opt.dtype(at::kByte));
  if (accumulate) c.changed(false, false);
  raise_on(msa_paged_attention(&c.cache, &c.table, &p, in(q_), out(o), any_out(ws), need,
                               current_stream()),
           "msa_paged_attention");
  return o;
}

Tensor cache_evict(const Tensor& ck, const Tensor& cv, const std::optional<Tensor>& weight,
                   const std::optional<Tensor>& position, const Tensor& table, const Tensor& lens,
                   int64_t keep, int64_t recent) {
  constexpr const char* who = "cache_evict";
  Pages c(who, ck, cv, weight, position, table, lens);
  if (!c.weight.defined()) throw py::value_error("the cache keeps no weights to go by");
  no_grad(c.weight, who);
  if (keep < 1 || keep > kMost || recent < 0 || recent > keep)
    throw py::value_error("keep >= 1 and 0 <= recent <= keep expected");
  if (recent > 0 && !c.position.defined())
    throw py::value_error("the cache keeps no positions: recent must be 0");
  c10::cuda::CUDAGuard guard(ck.device());
  at::NoGradGuard no_grad;
  c.describe(table, lens);
  Tensor left = at::empty(c.lens.sizes(), c.lens.options());
  const size_t need = msa_cache_evict_workspace_size(&c.cache, &c.table, (int32_t)keep);
  Tensor ws;
  if (need > 256) ws = at::empty({(int64_t)need}, c.lens.options().dtype(at::kByte));
  c.changed(true, true);
  raise_on(msa_cache_evict(&c.cache, &c.table, (int32_t)keep, (int32_t)recent,
                           left.mutable_data_ptr<int32_t>(), any_out(ws), need, current_stream()),
           "msa_cache_evict");
  return left;
}

}  // namespace

void bind_cache(py::module_& m) {
  py::class_<Plan, std::shared_ptr<Plan>>(m, "RotaryPlan")
      .def(py::init([](std::vector<uint64_t> freq, bool interleaved, double amplitude) {
        return std::make_shared<Plan>(Plan{std::move(freq), interleaved, (float)amplitude});
      }))
      .def_property_readonly("dims", &Plan::dims)
      .def_readonly("frequencies", &Plan::freq)
      .def_readonly("interleaved", &Plan::interleaved)
      .def_readonly("amplitude", &Plan::amplitude);
  m.def("rotary", [](const Tensor& q, const std::optional<Tensor>& k,
                     const std::shared_ptr<Plan>& plan, const std::optional<Tensor>& cu,
                     const std::optional<Tensor>& positions) {
    auto [a, b] = rotary(q, k, plan, cu, positions);
    return std::make_tuple(a, b.defined() ? std::optional<Tensor>(b) : std::nullopt);
  });
  m.def("cache_append", &cache_append);
  m.def("paged_attention", &paged_attention);
  m.def("cache_evict", &cache_evict);
}
