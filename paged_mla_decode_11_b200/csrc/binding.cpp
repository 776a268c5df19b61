// Native argument marshalling for the operators called every layer of a decode step, where the
// interpreter's checks cost several times the kernel: the tensors are checked and handed to the C
// ABI here, in C++, on the tensors' device and its current stream.  What is checked and raised is
// what the Python functions of ops.py document; the checks of shapes, strides and types come before
// the one of the device.
#include <dlfcn.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "pagedmla.h"

namespace {

struct Api {
  decltype(&mla_rope) rope;
  decltype(&mla_cache_slots) cache_slots;
  decltype(&mla_cache_write) cache_write;
  decltype(&mla_cache_write_fp8) cache_write_fp8;
  decltype(&mla_cache_read) cache_read;
  decltype(&mla_cache_read_fp8) cache_read_fp8;
  decltype(&mla_verify_draft) verify_draft;
  decltype(&mla_decode_paged_fp8_rows) decode_fp8_rows;
  decltype(&mla_last_error_string) last_error;
} api;
PyObject *mla_error = nullptr;  // ops.MlaError

constexpr int64_t kLatent = MLA_D_V, kRope = MLA_D_QK - MLA_D_V, kRow = MLA_D_QK;

// Raised as a Python exception of `type`.
struct Refused {
  PyObject *type;
  std::string message;
};

[[noreturn]] void refuse_value(std::string message) { throw Refused{PyExc_ValueError, std::move(message)}; }
[[noreturn]] void refuse_type(std::string message) { throw Refused{PyExc_TypeError, std::move(message)}; }

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void need_type(const at::Tensor &t, const char *name, at::ScalarType type) {
  if (t.scalar_type() != type)
    refuse_type(std::string(name) + " must be " + c10::toString(type) + " (got " + c10::toString(t.scalar_type()) + ")");
}

int element_type(const at::Tensor &t, const char *name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MLA_DTYPE_BF16;
    case at::kHalf: return MLA_DTYPE_F16;
    case at::kFloat: return MLA_DTYPE_F32;
    default: refuse_type(std::string(name) + " must be bf16, fp16 or fp32 (got " + c10::toString(t.scalar_type()) + ")");
  }
}

void need_vector(const at::Tensor &t, const char *name, const char *what, int64_t n) {
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse_value(std::string(name) + " must be a contiguous [" + what + "] tensor");
}

// Contiguous last dimension (of any stride where it has one element).
bool rows_contiguous(const at::Tensor &t) { return t.stride(-1) == 1 || t.size(-1) <= 1; }

// Stride of a dimension; one of a single element is never stepped over, whatever its stride says.
int64_t step(const at::Tensor &t, int64_t i) { return t.size(i) > 1 ? t.stride(i) : 0; }

// No element of a [T, H, D] tensor with contiguous rows is reached twice.
void need_rows_apart(const at::Tensor &t, const char *name) {
  int64_t st[2] = {t.stride(0), t.stride(1)}, n[2] = {t.size(0), t.size(1)};
  const int small = (n[0] > 1 && (n[1] <= 1 || st[0] < st[1])) ? 0 : 1;
  int64_t need = t.size(2);
  for (int i : {small, 1 - small}) {
    if (n[i] <= 1) continue;
    if (st[i] < need) refuse_value(std::string("rows of ") + name + " must not overlap");
    need += (n[i] - 1) * st[i];
  }
}

// Whether the bytes from first to last element of two tensors meet.
bool overlap(const at::Tensor &a, const at::Tensor &b) {
  auto end = [](const at::Tensor &t) {
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    return static_cast<const char *>(t.const_data_ptr()) + (last + 1) * t.element_size();
  };
  if (a.numel() == 0 || b.numel() == 0) return false;
  const char *a0 = static_cast<const char *>(a.const_data_ptr()), *b0 = static_cast<const char *>(b.const_data_ptr());
  return a0 < end(b) && b0 < end(a);
}

// Whether a tensor is being differentiated: it needs a gradient or carries a tangent (forward mode).
bool differentiated(const at::Tensor &t) {
  return (c10::GradMode::is_enabled() && t.requires_grad()) ||
         (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined());
}

// A caller's tensor that the call writes: no derivative goes through that write ...
void need_writable(const at::Tensor &t, const char *name) {
  if (differentiated(t))
    refuse_value(std::string(name) + " must not require a gradient or carry a tangent: the call writes it");
}

// ... and autograd is told of it, so that a backward pass that saved the tensor raises.
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The device of a call: that of its first tensor, which the others must share.
struct Place {
  c10::Device device;
  Place(const at::Tensor &t, const char *name) : device(t.device()) {
    if (!device.is_cuda()) refuse_value(std::string(name) + " must be a CUDA tensor");
  }
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::detail::empty_cuda(sizes, type, device, std::nullopt);
  }
  void same(const at::Tensor &t, const char *name) const {
    if (t.device() != device)
      refuse_value(std::string(name) + " must be a CUDA tensor on device " + std::to_string(device.index()));
  }
};

// Calls a C entry point with the device current, on its current stream.
template <typename F>
void launch(const Place &place, F &&call) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != place.device.index()) guard.set_device(place.device);
  const int rc = call(reinterpret_cast<mla_stream_t>(c10::cuda::getCurrentCUDAStream(place.device.index()).stream()));
  if (rc == MLA_OK) return;
  PyObject *e = PyObject_CallFunction(mla_error, "is", rc, api.last_error());
  if (e) {
    PyErr_SetObject(mla_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

int position_flag(const at::Tensor &t, int64_t tokens) {
  if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
    refuse_type(std::string("positions must be int32 or int64 (got ") + c10::toString(t.scalar_type()) + ")");
  need_vector(t, "positions", "tokens", tokens);
  return t.scalar_type() == at::kLong ? MLA_ROPE_POS64 : 0;
}

void need_arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse_type("wrong number of arguments");
}

bool given(PyObject *o) { return o != Py_None; }

float to_float(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

int64_t to_int(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// rope_recorded(x, inv_freq, out) -> whether autograd is to record the call, as x is differentiated.
// Derivatives by the frequencies are refused, and an output where the call is recorded.
PyObject *rope_recorded(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 3);
  auto wanted = [](PyObject *o) { return THPVariable_Check(o) && differentiated(THPVariable_Unpack(o)); };
  if (wanted(a[1])) refuse_value("the derivative by inv_freq is not formed: detach it");
  if (!wanted(a[0])) Py_RETURN_FALSE;
  if (given(a[2])) refuse_value("out cannot be given for an x that needs a gradient");
  Py_RETURN_TRUE;
}

// rope(x, positions, inv_freq, interleaved, magnitude, inverse, out)
PyObject *rope(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 7);
  const at::Tensor &x = tensor(a[0], "x"), &positions = tensor(a[1], "positions"), &freq = tensor(a[2], "inv_freq");
  const int type = element_type(x, "x");
  if (x.dim() != 3) refuse_value("x must be [tokens, heads, width]");
  const int64_t T = x.size(0), H = x.size(1), D = x.size(2);
  if (!rows_contiguous(x)) refuse_value("x's last dimension must be contiguous");
  need_type(freq, "inv_freq", at::kDouble);
  if (freq.dim() != 1 || !freq.is_contiguous() || freq.size(0) < 1 || freq.size(0) > D / 2)
    refuse_value("inv_freq must be a contiguous vector of at most width / 2 frequencies");
  if (H > INT32_MAX || D > INT32_MAX) refuse_value("x has too many heads or columns");
  const unsigned flags = position_flag(positions, T) | (truth(a[3]) ? 0 : MLA_ROPE_HALF) | (truth(a[5]) ? MLA_ROPE_INVERSE : 0);
  const float magnitude = to_float(a[4]);
  at::Tensor fresh;
  const at::Tensor *out = &fresh;
  if (given(a[6])) {
    out = &tensor(a[6], "out");
    need_type(*out, "out", x.scalar_type());
    if (out->sizes() != x.sizes() || !rows_contiguous(*out))
      refuse_value("out must have x's shape, its last dimension contiguous");
    const bool in_place = out->const_data_ptr() == x.const_data_ptr() && out->strides() == x.strides();
    if (!in_place && overlap(x, *out)) refuse_value("out must be x itself or must not overlap it");
    need_rows_apart(*out, "out");
    need_writable(*out, "out");
  }
  const Place place(x, "x");
  place.same(positions, "positions");
  place.same(freq, "inv_freq");
  if (given(a[6]))
    place.same(*out, "out");
  else
    fresh = place.empty({T, H, D}, x.scalar_type());
  if (out->numel() > 0) {
    const int64_t xs[2] = {step(x, 0), step(x, 1)}, os[2] = {step(*out, 0), step(*out, 1)};
    launch(place, [&](mla_stream_t stream) {
      return api.rope(x.const_data_ptr(), xs, type, T, int(H), int(D), int(freq.size(0)), positions.const_data_ptr(),
                      static_cast<const double *>(freq.const_data_ptr()), magnitude, flags, out->data_ptr(), os, stream);
    });
  }
  if (given(a[6])) {
    written(*out);
    return Py_NewRef(a[6]);
  }
  return THPVariable_Wrap(std::move(fresh));
}

// cache_slots(block_table, cache_seqlens, row_ptr, num_pages, tokens, slots, positions)
PyObject *cache_slots(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 7);
  const at::Tensor &table = tensor(a[0], "block_table"), &lens = tensor(a[1], "cache_seqlens"), &ptr = tensor(a[2], "row_ptr");
  need_type(table, "block_table", at::kInt);
  need_type(lens, "cache_seqlens", at::kInt);
  need_type(ptr, "row_ptr", at::kInt);
  if (table.dim() != 2 || table.size(1) < 1 || !rows_contiguous(table))
    refuse_value("block_table must be [batch, max_pages] with contiguous rows");
  const int64_t b = table.size(0), pages = to_int(a[3]), tokens = to_int(a[4]);
  need_vector(lens, "cache_seqlens", "batch", b);
  need_vector(ptr, "row_ptr", "batch + 1", b + 1);
  if (tokens < 0) refuse_value("tokens must not be negative");
  if (b > INT32_MAX || table.size(1) > INT32_MAX) refuse_value("block_table is too large");
  at::Tensor fresh[2];
  const at::Tensor *out[2] = {&fresh[0], &fresh[1]};
  const char *names[2] = {"slots", "positions"};
  const at::ScalarType types[2] = {at::kLong, at::kInt};
  for (int i = 0; i < 2; ++i)
    if (given(a[5 + i])) {
      out[i] = &tensor(a[5 + i], names[i]);
      need_type(*out[i], names[i], types[i]);
      need_vector(*out[i], names[i], "tokens", tokens);
      // one thread's results may be another's arguments
      if (overlap(*out[i], table) || overlap(*out[i], lens) || overlap(*out[i], ptr))
        refuse_value(std::string(names[i]) + " must not overlap the arguments");
    }
  if (given(a[5]) && given(a[6]) && overlap(*out[0], *out[1])) refuse_value("slots and positions must not overlap");
  const Place place(table, "block_table");
  place.same(lens, "cache_seqlens");
  place.same(ptr, "row_ptr");
  for (int i = 0; i < 2; ++i)
    if (given(a[5 + i]))
      place.same(*out[i], names[i]);
    else
      fresh[i] = place.empty({tokens}, types[i]);
  launch(place, [&](mla_stream_t stream) {
    return api.cache_slots(static_cast<const int32_t *>(ptr.const_data_ptr()), static_cast<const int32_t *>(lens.const_data_ptr()),
                           int(b), static_cast<const int32_t *>(table.const_data_ptr()), table.stride(0), int(table.size(1)),
                           pages, tokens, static_cast<int64_t *>(out[0]->data_ptr()),
                           static_cast<int32_t *>(out[1]->data_ptr()), stream);
  });
  for (int i = 0; i < 2; ++i)
    if (given(a[5 + i])) written(*out[i]);
  PyObject *first = given(a[5]) ? Py_NewRef(a[5]) : THPVariable_Wrap(std::move(fresh[0]));
  PyObject *second = given(a[6]) ? Py_NewRef(a[6]) : THPVariable_Wrap(std::move(fresh[1]));
  return Py_BuildValue("(NN)", first, second);
}

// The pool of either cache; scale: k_scale of the FP8 one, else nullptr.
void need_pool(const at::Tensor &pool, const at::Tensor *scale) {
  const bool codes = pool.scalar_type() == at::kByte || pool.scalar_type() == at::kFloat8_e4m3fn;
  if (scale ? !codes : pool.scalar_type() != at::kBFloat16)
    refuse_type(std::string(scale ? "k8 must be uint8 or float8_e4m3fn (got " : "k_cache must be bf16 (got ") +
                c10::toString(pool.scalar_type()) + ")");
  if (pool.dim() != 4 || pool.size(1) != MLA_PAGE_SIZE || pool.size(3) != kRow || !pool.is_contiguous())
    refuse_value("the cache must be a contiguous [pages, 64, h_kv, 576] tensor");
  if (scale) {
    need_type(*scale, "k_scale", at::kFloat);
    if (scale->dim() != 3 || scale->size(0) != pool.size(2) || scale->size(1) != pool.size(0) ||
        scale->size(2) != pool.size(1) || !scale->is_contiguous())
      refuse_value("k_scale must be a contiguous [h_kv, num_pages, page] tensor");
  }
}

// cache_write(latent, rope, slots, pool, k_scale, norm_weight, eps, positions, inv_freq, interleaved, magnitude)
PyObject *cache_write(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 11);
  const at::Tensor &latent = tensor(a[0], "latent"), &rp = tensor(a[1], "rope"), &slots = tensor(a[2], "slots"),
                   &pool = tensor(a[3], "the cache");
  const at::Tensor *scale = given(a[4]) ? &tensor(a[4], "k_scale") : nullptr;
  const at::Tensor *weight = given(a[5]) ? &tensor(a[5], "norm_weight") : nullptr;
  const at::Tensor *positions = given(a[7]) ? &tensor(a[7], "positions") : nullptr;
  const at::Tensor *freq = given(a[8]) ? &tensor(a[8], "inv_freq") : nullptr;
  const int type = element_type(latent, "latent");
  need_type(rp, "rope", latent.scalar_type());
  need_type(slots, "slots", at::kLong);
  if (latent.dim() != 3 || latent.size(2) != kLatent) refuse_value("latent must be [tokens, h_kv, 512]");
  const int64_t T = latent.size(0), h_kv = latent.size(1);
  if (rp.dim() != 3 || rp.size(0) != T || rp.size(1) != h_kv || rp.size(2) != kRope)
    refuse_value("rope must be [tokens, h_kv, 64]");
  if (latent.stride(2) != 1 || rp.stride(2) != 1) refuse_value("the last dimensions of latent and rope must be contiguous");
  need_vector(slots, "slots", "tokens", T);
  need_pool(pool, scale);
  if (pool.size(2) != h_kv) refuse_value("the cache and latent disagree on h_kv");
  if (overlap(pool, latent) || overlap(pool, rp)) refuse_value("latent and rope must not overlap the cache");
  need_writable(pool, "the cache");
  if (scale) need_writable(*scale, "k_scale");
  if (weight) {
    need_type(*weight, "norm_weight", latent.scalar_type());
    need_vector(*weight, "norm_weight", "512", kLatent);
  }
  if (!positions != !freq) refuse_value(freq ? "inv_freq needs positions" : "positions need inv_freq");
  unsigned flags = 0;
  if (freq) {
    need_type(*freq, "inv_freq", at::kDouble);
    need_vector(*freq, "inv_freq", "32", kRope / 2);
    flags = position_flag(*positions, T) | (truth(a[9]) ? 0 : MLA_ROPE_HALF);
  }
  const float eps = to_float(a[6]), magnitude = to_float(a[10]);
  const Place place(latent, "latent");
  place.same(rp, "rope");
  place.same(slots, "slots");
  place.same(pool, "the cache");
  if (scale) place.same(*scale, "k_scale");
  if (weight) place.same(*weight, "norm_weight");
  if (freq) {
    place.same(*positions, "positions");
    place.same(*freq, "inv_freq");
  }
  if (T == 0) Py_RETURN_NONE;
  const int64_t ls[2] = {step(latent, 0), step(latent, 1)}, rs[2] = {step(rp, 0), step(rp, 1)};
  const void *w = weight ? weight->const_data_ptr() : nullptr, *pos = freq ? positions->const_data_ptr() : nullptr;
  const double *f = freq ? static_cast<const double *>(freq->const_data_ptr()) : nullptr;
  const int64_t *at = static_cast<const int64_t *>(slots.const_data_ptr());
  launch(place, [&](mla_stream_t stream) {
    return scale ? api.cache_write_fp8(latent.const_data_ptr(), ls, rp.const_data_ptr(), rs, type, T, int(h_kv), w, eps, pos, f,
                                       magnitude, flags, at, pool.data_ptr(), static_cast<float *>(scale->data_ptr()),
                                       pool.size(0), int(pool.size(1)), stream)
                 : api.cache_write(latent.const_data_ptr(), ls, rp.const_data_ptr(), rs, type, T, int(h_kv), w, eps, pos, f,
                                   magnitude, flags, at, pool.data_ptr(), pool.size(0), int(pool.size(1)), stream);
  });
  written(pool);
  if (scale) written(*scale);
  Py_RETURN_NONE;
}

// cache_read(pool, k_scale, slots, out)
PyObject *cache_read(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 4);
  const at::Tensor &pool = tensor(a[0], "the cache"), &slots = tensor(a[2], "slots");
  const at::Tensor *scale = given(a[1]) ? &tensor(a[1], "k_scale") : nullptr;
  need_pool(pool, scale);
  need_type(slots, "slots", at::kLong);
  if (slots.dim() != 1 || !slots.is_contiguous()) refuse_value("slots must be a contiguous 1-D tensor");
  const int64_t T = slots.size(0), h_kv = pool.size(2);
  at::Tensor fresh;
  const at::Tensor *out = &fresh;
  if (given(a[3])) {
    out = &tensor(a[3], "out");
    need_type(*out, "out", at::kBFloat16);
    if (out->dim() != 3 || out->size(0) != T || out->size(1) != h_kv || out->size(2) != kRow || out->stride(2) != 1)
      refuse_value("out must be [tokens, h_kv, 576] with contiguous rows");
    need_rows_apart(*out, "out");
    if (overlap(pool, *out)) refuse_value("out must not overlap the cache");
    need_writable(*out, "out");
  }
  const Place place(pool, "the cache");
  place.same(slots, "slots");
  if (scale) place.same(*scale, "k_scale");
  if (given(a[3]))
    place.same(*out, "out");
  else
    fresh = place.empty({T, h_kv, kRow}, at::kBFloat16);
  if (out->numel() > 0) {
    const int64_t os[2] = {step(*out, 0), step(*out, 1)};
    const int64_t *at = static_cast<const int64_t *>(slots.const_data_ptr());
    launch(place, [&](mla_stream_t stream) {
      return scale ? api.cache_read_fp8(pool.const_data_ptr(), static_cast<const float *>(scale->const_data_ptr()), pool.size(0),
                                        int(pool.size(1)), int(h_kv), at, T, out->data_ptr(), os, stream)
                   : api.cache_read(pool.const_data_ptr(), pool.size(0), int(pool.size(1)), int(h_kv), at, T, out->data_ptr(),
                                    os, stream);
    });
  }
  if (given(a[3])) {
    written(*out);
    return Py_NewRef(a[3]);
  }
  return THPVariable_Wrap(std::move(fresh));
}

// verify_draft(target_probs, draft_tokens, uniform, uniform_new, draft_probs, num_drafts)
PyObject *verify_draft(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 6);
  const at::Tensor &target = tensor(a[0], "target_probs"), &tokens = tensor(a[1], "draft_tokens"),
                   &uniform = tensor(a[2], "uniform"), &uniform_new = tensor(a[3], "uniform_new");
  const at::Tensor *draft = given(a[4]) ? &tensor(a[4], "draft_probs") : nullptr;
  const at::Tensor *num = given(a[5]) ? &tensor(a[5], "num_drafts") : nullptr;
  const int type = element_type(target, "target_probs");
  need_type(tokens, "draft_tokens", at::kInt);
  need_type(uniform, "uniform", at::kFloat);
  need_type(uniform_new, "uniform_new", at::kFloat);
  if (target.dim() != 3 || target.size(1) < 2 || target.size(2) < 1)
    refuse_value("target_probs must be [batch, drafts + 1, vocab] with at least one draft");
  const int64_t b = target.size(0), s = target.size(1) - 1, V = target.size(2);
  if (!rows_contiguous(target)) refuse_value("target_probs' last dimension must be contiguous");
  for (const auto &[t, name] : {std::pair<const at::Tensor &, const char *>{tokens, "draft_tokens"}, {uniform, "uniform"}})
    if (t.dim() != 2 || t.size(0) != b || t.size(1) != s || !t.is_contiguous())
      refuse_value(std::string(name) + " must be a contiguous [batch, drafts] tensor");
  need_vector(uniform_new, "uniform_new", "batch", b);
  if (draft) {
    need_type(*draft, "draft_probs", target.scalar_type());
    if (draft->dim() != 3 || draft->size(0) != b || draft->size(1) != s || draft->size(2) != V || !rows_contiguous(*draft))
      refuse_value("draft_probs must be [batch, drafts, vocab], its last dimension contiguous");
  }
  if (num) {
    need_type(*num, "num_drafts", at::kInt);
    need_vector(*num, "num_drafts", "batch", b);
  }
  if (b > INT32_MAX || s > INT32_MAX || V > INT32_MAX) refuse_value("target_probs is too large");
  const Place place(target, "target_probs");
  place.same(tokens, "draft_tokens");
  place.same(uniform, "uniform");
  place.same(uniform_new, "uniform_new");
  if (draft) place.same(*draft, "draft_probs");
  if (num) place.same(*num, "num_drafts");
  at::Tensor accepted = place.empty({b}, at::kInt), made = place.empty({b, s + 1}, at::kInt);
  if (b > 0) {
    const int64_t ts[2] = {step(target, 0), step(target, 1)};
    const int64_t ds[2] = {draft ? step(*draft, 0) : 0, draft ? step(*draft, 1) : 0};
    launch(place, [&](mla_stream_t stream) {
      return api.verify_draft(target.const_data_ptr(), ts, draft ? draft->const_data_ptr() : nullptr, ds, type,
                              static_cast<const int32_t *>(tokens.const_data_ptr()),
                              static_cast<const float *>(uniform.const_data_ptr()),
                              static_cast<const float *>(uniform_new.const_data_ptr()),
                              num ? static_cast<const int32_t *>(num->const_data_ptr()) : nullptr, int(b), int(s), int(V),
                              static_cast<int32_t *>(accepted.data_ptr()), static_cast<int32_t *>(made.data_ptr()), stream);
    });
  }
  PyObject *first = THPVariable_Wrap(std::move(accepted)), *second = THPVariable_Wrap(std::move(made));
  return Py_BuildValue("(NN)", first, second);
}

// decode_fp8_rows(q, k8, k_scale, block_table, cache_seqlens, dv, tile_metadata, num_splits, softmax_scale,
//                 causal, workspace, out, lse, skip_combine)
PyObject *decode_fp8_rows(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 14);
  const at::Tensor &q = tensor(a[0], "q"), &k8 = tensor(a[1], "k8"), &scale = tensor(a[2], "k_scale"),
                   &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "cache_seqlens"),
                   &tile = tensor(a[6], "tile_metadata"), &splits = tensor(a[7], "num_splits");
  need_type(q, "q", at::kBFloat16);
  need_type(table, "block_table", at::kInt);
  need_type(lens, "cache_seqlens", at::kInt);
  need_type(tile, "tile_metadata", at::kInt);
  need_type(splits, "num_splits", at::kInt);
  if (q.dim() != 4 || table.dim() != 2) refuse_value("q must be 4-D, block_table 2-D");
  need_pool(k8, &scale);
  const int64_t b = q.size(0), s_q = q.size(1), h_q = q.size(2), d = q.size(3), dv = to_int(a[5]), h_kv = k8.size(2);
  if (d != kRow) refuse_value("q and k8 disagree on the latent width");
  if (q.stride(3) != 1) refuse_value("q's last dimension must be contiguous");
  if (table.size(0) != b || !rows_contiguous(table)) refuse_value("block_table must be [batch, max_pages] with contiguous rows");
  need_vector(lens, "cache_seqlens", "batch", b);
  if (tile.dim() != 2 || tile.size(1) != MLA_TILE_FIELDS || !tile.is_contiguous())
    refuse_value("tile_metadata must be a contiguous [num_parts, 8] tensor");
  need_vector(splits, "num_splits", "batch + 1", b + 1);
  if (b > INT32_MAX || s_q > INT32_MAX || h_q > INT32_MAX || h_kv > INT32_MAX || tile.size(0) > INT32_MAX || dv < 0 || dv > 4096)
    refuse_value("a dimension is out of range");
  const float softmax_scale = given(a[8]) ? to_float(a[8]) : 1.f / std::sqrt(float(d));
  const bool causal = truth(a[9]);
  at::Tensor fresh_out, fresh_lse;
  const at::Tensor *out = &fresh_out, *lse = &fresh_lse;
  if (given(a[11])) {
    out = &tensor(a[11], "out");
    if (out->sizes() != at::IntArrayRef({b, s_q, h_q, dv}) || out->scalar_type() != at::kBFloat16 || !out->is_contiguous())
      refuse_value("out must be a contiguous bf16 [b, s_q, h_q, dv] tensor");
    need_writable(*out, "out");
  }
  if (given(a[12])) {
    lse = &tensor(a[12], "lse");
    if (lse->sizes() != at::IntArrayRef({b, h_q, s_q}) || lse->scalar_type() != at::kFloat || !lse->is_contiguous())
      refuse_value("lse must be a contiguous fp32 [b, h_q, s_q] tensor");
    need_writable(*lse, "lse");
  }
  // a sequence's results are written while others still read
  for (const auto &[t, name] : {std::pair<const at::Tensor &, const char *>{*out, "out"}, {*lse, "lse"}})
    if (t.defined() && (overlap(t, q) || overlap(t, k8) || overlap(t, scale) || overlap(t, table) || overlap(t, lens) ||
                        overlap(t, tile) || overlap(t, splits)))
      refuse_value(std::string(name) + " must not overlap the arguments");
  if (out->defined() && lse->defined() && overlap(*out, *lse)) refuse_value("out and lse must not overlap");
  const Place place(q, "q");
  place.same(k8, "k8");
  place.same(scale, "k_scale");
  place.same(table, "block_table");
  place.same(lens, "cache_seqlens");
  place.same(tile, "tile_metadata");
  place.same(splits, "num_splits");
  const at::Tensor &workspace = tensor(a[10], "workspace");
  need_type(workspace, "workspace", at::kByte);
  if (!workspace.is_contiguous()) refuse_value("workspace must be contiguous");
  place.same(workspace, "workspace");
  if (given(a[11])) place.same(*out, "out");
  if (given(a[12])) place.same(*lse, "lse");
  if (!given(a[11])) fresh_out = place.empty({b, s_q, h_q, dv}, at::kBFloat16);
  if (!given(a[12])) fresh_lse = place.empty({b, h_q, s_q}, at::kFloat);
  const int64_t qs[3] = {q.stride(0), q.stride(1), q.stride(2)};
  const unsigned flags = truth(a[13]) ? MLA_FLAG_SKIP_COMBINE : 0;
  launch(place, [&](mla_stream_t stream) {
    return api.decode_fp8_rows(
        q.const_data_ptr(), qs, int(b), int(s_q), int(h_q), int(d), k8.const_data_ptr(),
        static_cast<const float *>(scale.const_data_ptr()), k8.size(0), int(k8.size(1)), int(h_kv),
        static_cast<const int32_t *>(table.const_data_ptr()), table.stride(0),
        static_cast<const int32_t *>(lens.const_data_ptr()), int(dv), static_cast<const int32_t *>(tile.const_data_ptr()),
        int(tile.size(0)), static_cast<const int32_t *>(splits.const_data_ptr()), softmax_scale, causal, out->data_ptr(),
        static_cast<float *>(lse->data_ptr()), workspace.data_ptr(), size_t(workspace.numel()), flags, stream);
  });
  if (given(a[11])) written(*out);
  if (given(a[12])) written(*lse);
  PyObject *first = given(a[11]) ? Py_NewRef(a[11]) : THPVariable_Wrap(std::move(fresh_out));
  PyObject *second = given(a[12]) ? Py_NewRef(a[12]) : THPVariable_Wrap(std::move(fresh_lse));
  return Py_BuildValue("(NN)", first, second);
}

// bind(handle of libpagedmla.so, ops.MlaError): the library whose entry points are called.
PyObject *bind(PyObject *const *a, Py_ssize_t n) {
  need_arguments(n, 2);
  void *lib = reinterpret_cast<void *>(static_cast<uintptr_t>(to_int(a[0])));
  auto find = [&](auto &fn, const char *name) {
    void *p = dlsym(lib, name);
    if (!p) throw Refused{PyExc_ImportError, std::string(name) + " is missing from the library"};
    fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(p);
  };
  Api found;
  find(found.rope, "mla_rope");
  find(found.cache_slots, "mla_cache_slots");
  find(found.cache_write, "mla_cache_write");
  find(found.cache_write_fp8, "mla_cache_write_fp8");
  find(found.cache_read, "mla_cache_read");
  find(found.cache_read_fp8, "mla_cache_read_fp8");
  find(found.verify_draft, "mla_verify_draft");
  find(found.decode_fp8_rows, "mla_decode_paged_fp8_rows");
  find(found.last_error, "mla_last_error_string");
  api = found;
  Py_INCREF(a[1]);
  Py_XSETREF(mla_error, a[1]);
  Py_RETURN_NONE;
}

// No C++ exception leaves an entry of the module.
template <PyObject *(*f)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return f(args, n);
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.message.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*f)(PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<f>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),
                         method<rope_recorded>("rope_recorded"),
                         method<rope>("rope"),
                         method<cache_slots>("cache_slots"),
                         method<cache_write>("cache_write"),
                         method<cache_read>("cache_read"),
                         method<verify_draft>("verify_draft"),
                         method<decode_fp8_rows>("decode_fp8_rows"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
