// Python binding of the calls around the decode step (drafted trees, rotary
// writes, pages, compaction), of the 8-bit cache and of scored decode attention
// to the C ABI of libdcp.so.
//
// These calls last a few microseconds on the GPU, and what Python spends on
// checking their tensors one attribute at a time was several times that (28 us
// for a tree or a rotary write on 8 ranks through ctypes, on a Grace core).
// Here a tensor's type, shape, device and address are read directly.  Only
// arguments are handled; every step runs in the library's kernels.
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "dcp.h"

namespace {

PyObject* g_error = nullptr;   // DcpError

// The library's entry points, from the library that the package has loaded.
struct Lib {
  decltype(&dcp_strerror) strerror;
  decltype(&dcp_tree_workspace_size) tree_workspace_size;
  decltype(&dcp_tree_decode_gqa) tree_decode_gqa;
  decltype(&dcp_tree_partial_gqa) tree_partial_gqa;
  decltype(&dcp_rope_write_gqa) rope_write_gqa;
  decltype(&dcp_rope_write_mla) rope_write_mla;
  decltype(&dcp_pages_init) pages_init;
  decltype(&dcp_pages_workspace_size) pages_workspace_size;
  decltype(&dcp_pages_resize) pages_resize;
  decltype(&dcp_pages_fork) pages_fork;
  decltype(&dcp_pages_copy) pages_copy;
  decltype(&dcp_cache_compact) cache_compact;
  decltype(&dcp_q8_append_gqa) q8_append_gqa;
  decltype(&dcp_q8_gather_gqa) q8_gather_gqa;
  decltype(&dcp_q8_decode_gqa) q8_decode_gqa;
  decltype(&dcp_q8_partial_gqa) q8_partial_gqa;
  decltype(&dcp_scored_decode_gqa) scored_decode_gqa;
  decltype(&dcp_scored_partial_gqa) scored_partial_gqa;
  decltype(&dcp_scored_workspace_size) scored_workspace_size;
} g_lib;

// A refusal on its way to Python (the error is set).
struct Refused {};

[[noreturn]] void refuse(const std::string& why) {
  PyErr_SetString(g_error, why.c_str());
  throw Refused{};
}

[[noreturn]] void python_error() { throw Refused{}; }

void check(int rc) {
  if (rc == DCP_OK) return;
  refuse("libdcp error " + std::to_string(rc) + ": " + g_lib.strerror(rc));
}

// A new reference that is dropped with its scope.
struct Ref {
  PyObject* o;
  explicit Ref(PyObject* x) : o(x) {
    if (!o) python_error();
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_DECREF(o); }
};

Ref attr(PyObject* o, PyObject* name) { return Ref(PyObject_GetAttr(o, name)); }
// An attribute's name, made once.
#define NAME(s) ([]() -> PyObject* { static PyObject* const n = PyUnicode_InternFromString(s); return n; }())

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) python_error();
  return v;
}
int64_t integer_attr(PyObject* o, PyObject* name) { return integer(attr(o, name).o); }

// Into an int32 argument; what does not fit is refused here.
int32_t small(int64_t v, const char* what) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + " is out of range");
  return (int32_t)v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) python_error();
  return v != 0;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string said(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

void shaped(const at::Tensor& t, const char* what, at::ScalarType type, at::IntArrayRef shape,
            int dev) {
  if (t.scalar_type() != type || t.layout() != at::kStrided || t.sizes() != shape ||
      !t.is_cuda() || t.get_device() != dev)
    refuse(std::string(what) + " must be a " + c10::toString(type) + " tensor of shape " +
           said(shape) + " on cuda:" + std::to_string(dev) + ", got " +
           c10::toString(t.scalar_type()) + " " + said(t.sizes()) + " on " + t.device().str());
}

// Address of a contiguous tensor of this type and shape on this device.
void* ptr(const at::Tensor& t, const char* what, at::ScalarType type, at::IntArrayRef shape,
          int dev) {
  shaped(t, what, type, shape, dev);
  if (!t.is_contiguous()) refuse(std::string(what) + " must be contiguous");
  return t.data_ptr();
}
void* ptr(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return ptr(tensor(o, what), what, type, shape, dev);
}
void* opt(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return o == Py_None ? nullptr : ptr(o, what, type, shape, dev);
}

int32_t* err_ptr(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "err");
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != dev || t.numel() < 1)
    refuse("err must be an int32 tensor on the call's device");
  return (int32_t*)t.data_ptr();
}

// A tensor's device, which has to be the current one: the kernels launch there.
int device_of(const at::Tensor& t, const char* what) {
  if (!t.is_cuda()) refuse(std::string(what) + " must be a CUDA tensor");
  const int dev = t.get_device(), cur = c10::cuda::current_device();
  if (dev != cur)
    refuse(std::string(what) + " is on cuda:" + std::to_string(dev) +
           ", but the current device is cuda:" + std::to_string(cur));
  return dev;
}

// The stream that a call runs on.  What the call allocates is allocated for that
// stream too: memory of another one may still be in use by work queued there.
struct OnStream {
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  dcp_stream_t st;
  OnStream(PyObject* o, int dev) {
    if (o == Py_None) {
      st = (dcp_stream_t)c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    if (PyObject_HasAttr(o, NAME("device_index")) && integer_attr(o, NAME("device_index")) != dev)
      refuse("the stream is on another device than the tensors");
    st = (dcp_stream_t)(uintptr_t)integer_attr(o, NAME("cuda_stream"));
    guard.emplace(c10::cuda::getStreamFromExternal((cudaStream_t)st, dev));
  }
};

dcp_dtype_t dtype_of(at::ScalarType t) {
  if (t == at::kFloat) return DCP_F32;
  if (t == at::kBFloat16) return DCP_BF16;
  refuse(std::string("unsupported dtype ") + c10::toString(t));
}

dcp_layout_t layout_of(PyObject* o) {
  return dcp_layout_t{small(integer_attr(o, NAME("dcp_size")), "dcp_size"),
                      small(integer_attr(o, NAME("block_size")), "block_size"),
                      small(integer_attr(o, NAME("interleave")), "interleave")};
}

// Memory of the caching allocator, without the way through the dispatcher.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, dev), std::nullopt));
}

// Elements [at, ...) of a buffer as a tensor of its own (a fresh one, no view of
// anything a caller has).
at::Tensor part(const at::Tensor& all, int64_t from, at::IntArrayRef shape, int dev) {
  if (!all.defined()) return fresh(shape, at::kInt, dev);   // nothing in it
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()),
                                                          all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  t.unsafeGetTensorImpl()->set_storage_offset(from);
  return t;
}

// Two tensors of their own in one piece of memory (the second is small beside the
// first, and a piece takes the allocator 2 us).
void fresh_two(at::IntArrayRef s0, at::ScalarType t0, at::Tensor& a, at::IntArrayRef s1,
               at::ScalarType t1, at::Tensor& b, int dev) {
  const int64_t n0 = c10::multiply_integers(s0) * (int64_t)c10::elementSize(t0),
                n1 = c10::multiply_integers(s1) * (int64_t)c10::elementSize(t1);
  const int64_t from = (n0 + 255) / 256 * 256;
  const at::Tensor all = fresh({from + n1}, at::kByte, dev);
  auto make = [&](at::IntArrayRef shape, at::ScalarType type, int64_t at_byte) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(at_byte / (int64_t)c10::elementSize(type));
    return t;
  };
  a = make(s0, t0, 0);
  b = make(s1, t1, from);
}

// The call's workspace: the caller's, or one for this call alone (the caching
// allocator keeps it for the work already in its stream).
struct Workspace {
  void* own = nullptr;
  void* p;
  size_t bytes;
  Workspace(PyObject* o, size_t need, int dev) {
    if (o == Py_None) {
      own = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(
          need > 0 ? need : 1, c10::cuda::getCurrentCUDAStream(dev).stream());
      p = own;
      bytes = need;
      return;
    }
    const at::Tensor& t = tensor(o, "workspace");
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
      refuse("the workspace must be a contiguous tensor on the call's device");
    p = t.data_ptr();
    bytes = t.nbytes();
  }
  Workspace(const Workspace&) = delete;
  ~Workspace() {
    if (own) c10::cuda::CUDACachingAllocator::raw_delete(own);
  }
};

// A sequence of one pool per rank.
dcp_rank_ptrs_t rank_list(const dcp_layout_t& L, PyObject* pools, const char* what,
                          at::ScalarType type, at::IntArrayRef shape, int dev) {
  Ref seq(PySequence_Fast(pools, "pools must be a sequence of tensors, one per rank"));
  const int64_t have = PySequence_Fast_GET_SIZE(seq.o);
  if (L.dcp_size < 1 || L.dcp_size > DCP_MAX_RANKS || have < L.dcp_size)
    refuse(std::string(what) + ": " + std::to_string(have) + " pools for " +
           std::to_string(L.dcp_size) + " ranks");
  dcp_rank_ptrs_t r = {};
  for (int i = 0; i < L.dcp_size; ++i)
    r.ptr[i] = ptr(PySequence_Fast_GET_ITEM(seq.o, i), what, type, shape, dev);
  return r;
}

PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}

void arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    throw Refused{};
  }
}

// Runs a call and hands its error to Python: refusals are set already, torch's
// exceptions (out of memory among them) are translated.
template <typename F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// tree(partial, layout, q, kv, q_start, ctx_lens, tree_mask, scale, max_tree, sink, out_dtype,
//      out, out_lse, workspace, err, stream)
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 16);
    const bool partial = truth(a[0]);
    const dcp_layout_t L = layout_of(a[1]);
    const at::Tensor& q = tensor(a[2], "q");
    const int dev = device_of(q, "q");
    const OnStream on(a[15], dev);
    if (q.dim() != 3) refuse("q must be [tokens, heads, head_dim]");
    const int64_t N = q.size(0), Hq = q.size(1), d = q.size(2);
    const at::ScalarType type = q.scalar_type();
    const dcp_dtype_t dt = dtype_of(type);
    const at::Tensor& ctx = tensor(a[5], "ctx_lens");
    if (ctx.dim() != 1) refuse("ctx_lens must be [requests]");
    const int64_t B = ctx.size(0);
    // the cache
    PyObject* kv = a[3];
    Ref kp(attr(kv, NAME("k_pools"))), vp(attr(kv, NAME("v_pools"))), bto(attr(kv, NAME("block_table")));
    if (vp.o == Py_None) refuse("the cache has no value pools");
    const int64_t nb = integer_attr(kv, NAME("num_blocks"));
    Ref kseq(PySequence_Fast(kp.o, "k_pools must be a sequence of tensors"));
    if (PySequence_Fast_GET_SIZE(kseq.o) < 1) refuse("the cache has no pools");
    const at::Tensor& first = tensor(PySequence_Fast_GET_ITEM(kseq.o, 0), "k_pools");
    if (first.dim() != 4) refuse("pools must be [blocks, heads, block_size, head_dim]");
    const int64_t Hkv = first.size(1);
    const int64_t shape[4] = {nb, Hkv, L.block_size, d};
    dcp_paged_kv_t c = {};
    c.k = rank_list(L, kp.o, "k_pools", type, shape, dev);
    c.v = rank_list(L, vp.o, "v_pools", type, shape, dev);
    const at::Tensor& bt = tensor(bto.o, "block_table");
    const int64_t dim = bt.dim();
    if (dim != 2 && dim != 3) refuse("block_table must be [requests, blocks] or [ranks, ...]");
    c.block_table = (const int32_t*)ptr(bt, "block_table", at::kInt, bt.sizes(), dev);
    c.num_blocks = nb;
    c.max_vblocks = small(bt.size(dim - 1), "max_vblocks");
    const bool each = dim == 3 && bt.size(0) != 1;   // one for each rank, not one for all
    c.bt_rank_stride = each ? bt.size(1) * bt.size(2) : 0;
    if (each && bt.size(0) < L.dcp_size)
      refuse(std::to_string(bt.size(0)) + " block tables for " + std::to_string(L.dcp_size) +
             " ranks");
    if (bt.size(dim - 2) < B)
      refuse("a block table of " + std::to_string(bt.size(dim - 2)) + " requests, " +
             std::to_string(B) + " are needed");
    if (Hkv < 1 || Hq % Hkv)
      refuse(std::to_string(Hq) + " query heads over " + std::to_string(Hkv) + " key/value heads");
    const int32_t most = small(integer(a[8]), "max_tree"), n32 = small(N, "tokens"),
                  b32 = small(B, "requests"), hq = small(Hq, "heads"), hkv = small(Hkv, "heads"),
                  d32 = small(d, "head_dim");
    size_t need = 0;
    check(g_lib.tree_workspace_size(L, b32, most, hq, hkv, d32, dt, &need));
    const void* pq = ptr(q, "q", type, q.sizes(), dev);
    const int32_t* start = (const int32_t*)ptr(a[4], "q_start", at::kInt, {B + 1}, dev);
    const int32_t* pctx = (const int32_t*)ptr(ctx, "ctx_lens", at::kInt, {B}, dev);
    const uint64_t* mask = (const uint64_t*)ptr(a[6], "tree_mask", at::kLong, {N}, dev);
    const float scale = (float)number(a[7]);
    const float* sink = (const float*)opt(a[9], "sink", at::kFloat, {Hq}, dev);
    const int64_t R = L.dcp_size;
    std::vector<int64_t> os, ls;
    if (partial) {
      os = {R, N, Hq, d};
      ls = {R, N, Hq};
    } else {
      os = {N, Hq, d};
      ls = {N, Hq};
    }
    at::ScalarType odt = type;
    if (partial)
      odt = at::kFloat;
    else if (a[11] != Py_None)
      odt = tensor(a[11], "out").scalar_type();
    else if (a[10] != Py_None) {
      if (!THPDtype_Check(a[10])) refuse("out_dtype must be a torch dtype");
      odt = ((THPDtype*)a[10])->scalar_type;
    }
    const dcp_dtype_t codt = dtype_of(odt);
    Workspace ws(a[13], need, dev);
    int32_t* err = err_ptr(a[14], dev);
    at::Tensor out, lse;
    if (a[11] == Py_None) out = fresh(os, odt, dev);
    if (a[12] == Py_None) lse = fresh(ls, at::kFloat, dev);
    const char* oname = partial ? "part_o" : "out";
    const char* lname = partial ? "part_lse" : "out_lse";
    void* po = a[11] == Py_None ? out.data_ptr() : ptr(a[11], oname, odt, os, dev);
    float* pl =
        (float*)(a[12] == Py_None ? lse.data_ptr() : ptr(a[12], lname, at::kFloat, ls, dev));
    check(partial ? g_lib.tree_partial_gqa(L, pq, start, n32, b32, most, hq, hkv, d32, scale, dt, c,
                                           pctx, mask, (float*)po, pl, ws.p, ws.bytes, err, on.st)
                  : g_lib.tree_decode_gqa(L, pq, start, n32, b32, most, hq, hkv, d32, scale, dt, c,
                                          pctx, mask, sink, po, codt, pl, ws.p, ws.bytes, err,
                                          on.st));
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, a[11] == Py_None ? THPVariable_Wrap(out) : given(a[11]));
    PyTuple_SET_ITEM(both, 1, a[12] == Py_None ? THPVariable_Wrap(lse) : given(a[12]));
    return both;
  });
}

// Address and elements between tokens of a tensor [tokens, ...] whose tokens
// are each in one piece (a slice of a wider projection).
const void* tokens(const at::Tensor& t, const char* what, at::ScalarType type,
                   at::IntArrayRef shape, int dev, int64_t& stride) {
  shaped(t, what, type, shape, dev);
  int64_t inner = 1;
  for (int64_t i = t.dim() - 1; i > 0; --i) {
    if (t.size(i) > 1 && t.stride(i) != inner)
      refuse(std::string(what) + ": the heads of a token must be in one piece");
    inner *= t.size(i);
  }
  stride = t.size(0) > 1 ? t.stride(0) : inner;
  return t.data_ptr();
}

// rope(latent, layout, q, k, v, positions, inv_freq, slot, k_pools, v_pools, num_blocks, axis,
//      interleaved, scaling, q_out, k_out, err, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 18);
    const bool latent = truth(a[0]);
    const dcp_layout_t L = layout_of(a[1]);
    const char* kn = latent ? "kv" : "k";
    const at::Tensor& k = tensor(a[3], kn);
    const int dev = device_of(k, kn);
    const OnStream on(a[17], dev);
    const at::ScalarType type = k.scalar_type();
    const dcp_dtype_t dt = dtype_of(type);
    if (k.dim() != (latent ? 2 : 3))
      refuse(latent ? "kv must be [tokens, kv_dim]" : "k must be [tokens, heads, head_dim]");
    const int64_t T = k.size(0), Hkv = latent ? 1 : k.size(1), d = k.size(k.dim() - 1);
    const int64_t nb = integer(a[10]);
    int64_t sq = 0, sk = 0, sv = 0, Hq = 0;
    const void* pk = tokens(k, kn, type, k.sizes(), dev, sk);
    const void* pv = latent ? nullptr : tokens(tensor(a[4], "v"), "v", type, k.sizes(), dev, sv);
    const void* pq = nullptr;
    void* pqo = nullptr;
    at::Tensor own;
    PyObject* q_out = a[14];
    if (a[2] != Py_None) {
      const at::Tensor& q = tensor(a[2], "q");
      if (q.dim() != 3) refuse("q must be [tokens, heads, head_dim]");
      Hq = q.size(1);
      const int64_t shape[3] = {T, Hq, d};
      pq = tokens(q, "q", type, shape, dev, sq);
      if (q_out == Py_None) {
        own = fresh(shape, type, dev);
        pqo = own.data_ptr();
      } else {
        pqo = ptr(q_out, "q_out", type, shape, dev);
      }
    }
    const at::Tensor& pos = tensor(a[5], "positions");
    const at::Tensor& inv = tensor(a[6], "inv_freq");
    if (pos.dim() != 1 && pos.dim() != 2) refuse("positions must be [tokens] or [axes, tokens]");
    if (inv.dim() != 1) refuse("inv_freq must be [rot_dim / 2]");
    const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1, half = inv.size(0);
    if (pos.size(pos.dim() - 1) != T)
      refuse("positions of " + std::to_string(pos.size(pos.dim() - 1)) + " tokens for " +
             std::to_string(T));
    if (a[11] == Py_None && axes > 1)
      refuse("several axes of positions need `axis`, the axis of each pair");
    const int64_t* ppos = (const int64_t*)ptr(pos, "positions", at::kLong, pos.sizes(), dev);
    const float* pinv = (const float*)ptr(inv, "inv_freq", at::kFloat, {half}, dev);
    const int32_t* pax = (const int32_t*)opt(a[11], "axis", at::kInt, {half}, dev);
    const int64_t* slot = (const int64_t*)ptr(a[7], "slot", at::kLong, {L.dcp_size, T}, dev);
    const int32_t rot = small(2 * half, "rot_dim"), hq = small(Hq, "heads"),
                  d32 = small(d, "head_dim"), ax32 = small(axes, "axes");
    const int32_t inter = truth(a[12]) ? 1 : 0;
    const float scaling = (float)number(a[13]);
    int32_t* err = err_ptr(a[16], dev);
    if (latent) {
      const int64_t shape[3] = {nb, L.block_size, d};
      check(g_lib.rope_write_mla(L, pq, sq, pk, sk, T, hq, d32, dt, ppos, ax32, pinv, pax, rot,
                                 inter, scaling, slot, nb,
                                 rank_list(L, a[8], "pools", type, shape, dev), pqo, err, on.st));
    } else {
      const int64_t shape[4] = {nb, Hkv, L.block_size, d};
      check(g_lib.rope_write_gqa(
          L, pq, sq, pk, sk, pv, sv, T, hq, small(Hkv, "heads"), d32, dt, ppos, ax32, pinv, pax,
          rot, inter, scaling, slot, nb, rank_list(L, a[8], "k_pools", type, shape, dev),
          rank_list(L, a[9], "v_pools", type, shape, dev), pqo,
          opt(a[15], "k_out", type, k.sizes(), dev), err, on.st));
    }
    if (a[2] == Py_None) return given(Py_None);
    return q_out == Py_None ? THPVariable_Wrap(own) : given(q_out);
  });
}

// The pages' state, from the tensors of a Pages object.
dcp_pages_t pages_of(PyObject* o, const dcp_layout_t& L, int& dev, int64_t& tables) {
  Ref bto(attr(o, NAME("block_table"))), sqo(attr(o, NAME("seq_lens"))), rfo(attr(o, NAME("ref_count"))),
      fbo(attr(o, NAME("free_bits")));
  const at::Tensor& bt = tensor(bto.o, "block_table");
  dev = device_of(bt, "block_table");
  if (bt.dim() != 3) refuse("block_table must be [tables, requests, max_vblocks]");
  tables = bt.size(0);
  const int64_t B = bt.size(1), VB = bt.size(2), nb = integer_attr(o, NAME("num_blocks"));
  if (B * VB == 0) refuse("block_table has no entries");
  if (tables != 1 && tables != L.dcp_size)
    refuse(std::to_string(tables) + " block tables for " + std::to_string(L.dcp_size) + " ranks");
  dcp_pages_t p = {};
  p.block_table = (int32_t*)ptr(bt, "block_table", at::kInt, bt.sizes(), dev);
  p.seq_lens = (int32_t*)ptr(sqo.o, "seq_lens", at::kInt, {B}, dev);
  p.ref_count = (int32_t*)ptr(rfo.o, "ref_count", at::kInt, {tables, nb}, dev);
  p.free_bits = (uint32_t*)ptr(fbo.o, "free_bits", at::kInt, {tables, (nb + 31) / 32}, dev);
  p.num_reqs = small(B, "requests");
  p.max_vblocks = small(VB, "max_vblocks");
  p.bt_rank_stride = tables == L.dcp_size ? B * VB : 0;
  p.num_blocks = nb;
  return p;
}

// pages_init(layout, pages, stream)
PyObject* pages_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 3);
    const dcp_layout_t L = layout_of(a[0]);
    int dev;
    int64_t tables;
    const dcp_pages_t p = pages_of(a[1], L, dev, tables);
    check(g_lib.pages_init(L, p, OnStream(a[2], dev).st));
    return given(Py_None);
  });
}

// pages(fork, layout, pages, a, b, copy_src, copy_dst, workspace, err, stream)
PyObject* pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 10);
    const bool fork = truth(a[0]);
    const dcp_layout_t L = layout_of(a[1]);
    int dev;
    int64_t tables;
    const dcp_pages_t p = pages_of(a[2], L, dev, tables);
    const OnStream on(a[9], dev);
    const at::Tensor& x = tensor(a[3], "the list");
    if (x.dim() != 1) refuse("the list must have one dimension");
    const int64_t N = x.size(0);
    const int32_t* px = (const int32_t*)ptr(x, "the list", at::kInt, {N}, dev);
    const int32_t* py = (const int32_t*)ptr(a[4], "the list", at::kInt, {N}, dev);
    const int32_t n32 = small(N, "entries");
    size_t need = 0;
    check(g_lib.pages_workspace_size(L, p, n32, &need));
    int32_t* err = err_ptr(a[8], dev);
    // what the caller did not bring comes in one allocation
    const int64_t shape[2] = {tables, N}, each = tables * N;
    const bool own_s = a[5] == Py_None, own_d = a[6] == Py_None, own_w = a[7] == Py_None;
    const int64_t ints = (own_w ? (int64_t)need / 4 : 0) + (own_s ? each : 0) + (own_d ? each : 0);
    at::Tensor all, src, dst;
    if (ints > 0) all = fresh({ints}, at::kInt, dev);
    int64_t from = own_w ? (int64_t)need / 4 : 0;
    if (own_s) src = part(all, from, shape, dev);
    if (own_s) from += each;
    if (own_d) dst = part(all, from, shape, dev);
    std::optional<Workspace> given_ws;
    if (!own_w) given_ws.emplace(a[7], need, dev);
    void* const pw = own_w ? all.data_ptr() : given_ws->p;
    const size_t bytes = own_w ? need : given_ws->bytes;
    int32_t* ps = (int32_t*)(own_s ? src.data_ptr() : ptr(a[5], "copy_src", at::kInt, shape, dev));
    int32_t* pd = (int32_t*)(own_d ? dst.data_ptr() : ptr(a[6], "copy_dst", at::kInt, shape, dev));
    check((fork ? g_lib.pages_fork : g_lib.pages_resize)(L, p, px, py, n32, ps, pd, pw, bytes, err,
                                                         on.st));
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, a[5] == Py_None ? THPVariable_Wrap(src) : given(a[5]));
    PyTuple_SET_ITEM(both, 1, a[6] == Py_None ? THPVariable_Wrap(dst) : given(a[6]));
    return both;
  });
}

// What a PoolSet holds: the device array of addresses and the pools' shape.
dcp_pool_set_t pools_of(PyObject* o, const dcp_layout_t& L, int& dev) {
  Ref po(attr(o, NAME("ptr")));
  const at::Tensor& t = tensor(po.o, "the pool set");
  dev = device_of(t, "the pool set");
  const int64_t ranks = integer_attr(o, NAME("ranks")), bs = integer_attr(o, NAME("block_size"));
  if (ranks != L.dcp_size || bs != L.block_size)
    refuse("pools of " + std::to_string(ranks) + " ranks and " + std::to_string(bs) +
           "-token pages for another layout");
  dcp_pool_set_t p = {};
  p.num_pools = small(t.size(0), "pools");
  p.ptr = (const uint64_t*)ptr(t, "the pool set", at::kLong, {t.size(0), ranks}, dev);
  p.num_heads = small(integer_attr(o, NAME("num_heads")), "heads");
  p.row_bytes = small(integer_attr(o, NAME("row_bytes")), "row_bytes");
  p.num_blocks = integer_attr(o, NAME("num_blocks"));
  return p;
}

// pages_copy(layout, pools, copy_src, copy_dst, err, stream)
PyObject* pages_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 6);
    const dcp_layout_t L = layout_of(a[0]);
    int dev;
    const dcp_pool_set_t p = pools_of(a[1], L, dev);
    const at::Tensor& s = tensor(a[2], "copy_src");
    if (s.dim() != 2) refuse("copy_src must be [tables, n]");
    const int32_t* ps = (const int32_t*)ptr(s, "copy_src", at::kInt, s.sizes(), dev);
    const int32_t* pd = (const int32_t*)ptr(a[3], "copy_dst", at::kInt, s.sizes(), dev);
    check(g_lib.pages_copy(L, p, ps, pd, small(s.size(0), "tables"), small(s.size(1), "copies"),
                           err_ptr(a[4], dev), OnStream(a[5], dev).st));
    return given(Py_None);
  });
}

// cache_compact(layout, pools, block_table, num_blocks, ctx_lens, path, path_len, new_lens, err,
//               stream)
PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 10);
    const dcp_layout_t L = layout_of(a[0]);
    int dev;
    const dcp_pool_set_t p = pools_of(a[1], L, dev);
    const OnStream on(a[9], dev);
    if (integer(a[3]) != p.num_blocks)
      refuse("num_blocks is not that of the pools, " + std::to_string(p.num_blocks));
    const at::Tensor& ctx = tensor(a[4], "ctx_lens");
    if (ctx.dim() != 1) refuse("ctx_lens must be [requests]");
    const int64_t B = ctx.size(0);
    const at::Tensor& path = tensor(a[5], "path");
    if (path.dim() != 2) refuse("path must be [requests, max_path]");
    const int64_t most = path.size(1);
    const at::Tensor& bt = tensor(a[2], "block_table");
    const int64_t dim = bt.dim();
    if ((dim != 2 && dim != 3) || bt.size(dim - 2) < B ||
        (dim == 3 && bt.size(0) != 1 && bt.size(0) != L.dcp_size))
      refuse("block_table " + said(bt.sizes()) + " for " + std::to_string(B) + " requests and " +
             std::to_string(L.dcp_size) + " ranks");
    const int64_t stride = dim == 3 && bt.size(0) == L.dcp_size ? bt.size(1) * bt.size(2) : 0;
    const int32_t* pb = (const int32_t*)ptr(bt, "block_table", at::kInt, bt.sizes(), dev);
    const int32_t* pc = (const int32_t*)ptr(ctx, "ctx_lens", at::kInt, {B}, dev);
    const int32_t* pp = (const int32_t*)ptr(path, "path", at::kInt, {B, most}, dev);
    const int32_t* pn = (const int32_t*)ptr(a[6], "path_len", at::kInt, {B}, dev);
    int32_t* err = err_ptr(a[8], dev);
    at::Tensor own;
    if (a[7] == Py_None) own = fresh({B}, at::kInt, dev);
    int32_t* out = (int32_t*)(a[7] == Py_None ? own.data_ptr()
                                              : ptr(a[7], "new_lens", at::kInt, {B}, dev));
    check(g_lib.cache_compact(L, p, pb, small(B, "requests"), small(bt.size(dim - 1), "max_vblocks"),
                              stride, pc, pp, pn, small(most, "max_path"), out, err, on.st));
    return a[7] == Py_None ? THPVariable_Wrap(own) : given(a[7]);
  });
}

// A paged cache: its pools are [num_blocks, heads, block_size, head_dim] of `type`,
// e4m3 with scales where `eight`, and its table has rows for B requests.
struct PagedCache {
  dcp_paged_kv_t kv = {};
  dcp_paged_kv8_t kv8 = {};
  int64_t Hkv, d;

  PagedCache(PyObject* o, const dcp_layout_t& L, bool eight, at::ScalarType type, int64_t B,
             int dev) {
    if (PyObject_HasAttr(o, NAME("scales")) != eight)
      refuse(eight ? "a 16- or 32-bit cache, where one in 8 bits (PagedKV8) is needed"
                   : "a cache in 8 bits: the q8_ calls read it");
    Ref kp(attr(o, NAME("k_pools"))), vp(attr(o, NAME("v_pools"))),
        bto(attr(o, NAME("block_table")));
    if (vp.o == Py_None) refuse("the cache has no value pools");
    const int64_t nb = integer_attr(o, NAME("num_blocks"));
    Ref kseq(PySequence_Fast(kp.o, "k_pools must be a sequence of tensors"));
    if (PySequence_Fast_GET_SIZE(kseq.o) < 1) refuse("the cache has no pools");
    const at::Tensor& first = tensor(PySequence_Fast_GET_ITEM(kseq.o, 0), "k_pools");
    if (first.dim() != 4) refuse("pools must be [blocks, heads, block_size, head_dim]");
    Hkv = first.size(1);
    d = first.size(3);
    if (Hkv < 1) refuse("pools without heads");
    const int64_t shape[4] = {nb, Hkv, L.block_size, d}, scales[3] = {nb, Hkv, 4};
    const at::ScalarType pool = eight ? at::kFloat8_e4m3fn : type;
    kv8.k = kv.k = rank_list(L, kp.o, "k_pools", pool, shape, dev);
    kv8.v = kv.v = rank_list(L, vp.o, "v_pools", pool, shape, dev);
    if (eight) {
      Ref sc(attr(o, NAME("scales")));
      kv8.scale = rank_list(L, sc.o, "scales", at::kFloat, scales, dev);
    }
    const at::Tensor& bt = tensor(bto.o, "block_table");
    const int64_t dim = bt.dim();
    if (dim != 2 && dim != 3) refuse("block_table must be [requests, blocks] or [ranks, ...]");
    kv.block_table = (const int32_t*)ptr(bt, "block_table", at::kInt, bt.sizes(), dev);
    kv.num_blocks = nb;
    kv.max_vblocks = small(bt.size(dim - 1), "max_vblocks");
    const bool each = dim == 3 && bt.size(0) != 1;   // one for each rank, not one for all
    kv.bt_rank_stride = each ? bt.size(1) * bt.size(2) : 0;
    if (each && bt.size(0) < L.dcp_size)
      refuse(std::to_string(bt.size(0)) + " block tables for " + std::to_string(L.dcp_size) +
             " ranks");
    if (bt.size(dim - 2) < B)
      refuse("a block table of " + std::to_string(bt.size(dim - 2)) + " requests, " +
             std::to_string(B) + " are needed");
    kv8.num_blocks = kv.num_blocks;
    kv8.block_table = kv.block_table;
    kv8.max_vblocks = kv.max_vblocks;
    kv8.bt_rank_stride = kv.bt_rank_stride;
  }
};

// q8_append(layout, k, v, kv, q_start, ctx_lens, err, stream)
PyObject* q8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 8);
    const dcp_layout_t L = layout_of(a[0]);
    const at::Tensor& k = tensor(a[1], "k");
    const int dev = device_of(k, "k");
    const OnStream on(a[7], dev);
    if (k.dim() != 3) refuse("k must be [tokens, heads, head_dim]");
    const at::ScalarType type = k.scalar_type();
    const dcp_dtype_t dt = dtype_of(type);
    const at::Tensor& ctx = tensor(a[5], "ctx_lens");
    if (ctx.dim() != 1) refuse("ctx_lens must be [requests]");
    const int64_t B = ctx.size(0), N = k.size(0);
    const PagedCache c(a[3], L, true, type, B, dev);
    const int64_t shape[3] = {N, c.Hkv, c.d};
    int64_t ks, vs;
    const void* pk = tokens(k, "k", type, shape, dev, ks);
    const void* pv = tokens(tensor(a[2], "v"), "v", type, shape, dev, vs);
    const int32_t* start = (const int32_t*)ptr(a[4], "q_start", at::kInt, {B + 1}, dev);
    const int32_t* pc = (const int32_t*)ptr(ctx, "ctx_lens", at::kInt, {B}, dev);
    check(g_lib.q8_append_gqa(L, pk, ks, pv, vs, small(N, "tokens"), start, pc,
                              small(B, "requests"), small(c.Hkv, "heads"), small(c.d, "head_dim"),
                              dt, c.kv8, err_ptr(a[6], dev), on.st));
    return given(Py_None);
  });
}

// q8_gather(layout, kv, req_idx, positions, dtype, k_out, v_out, err, stream)
PyObject* q8_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 9);
    const dcp_layout_t L = layout_of(a[0]);
    const at::Tensor& req = tensor(a[2], "req_idx");
    const int dev = device_of(req, "req_idx");
    const OnStream on(a[8], dev);
    if (req.dim() != 1) refuse("req_idx must be [tokens]");
    const int64_t N = req.size(0);
    if (!THPDtype_Check(a[4])) refuse("dtype must be a torch dtype");
    at::ScalarType type = ((THPDtype*)a[4])->scalar_type;
    if (a[5] != Py_None) type = tensor(a[5], "k_out").scalar_type();
    const dcp_dtype_t dt = dtype_of(type);
    const PagedCache c(a[1], L, true, type, 0, dev);
    Ref bto(attr(a[1], NAME("block_table")));
    const at::Tensor& bt = tensor(bto.o, "block_table");
    const int64_t shape[3] = {N, c.Hkv, c.d};
    const int32_t* pr = (const int32_t*)ptr(req, "req_idx", at::kInt, {N}, dev);
    const int64_t* pp = (const int64_t*)ptr(a[3], "positions", at::kLong, {N}, dev);
    int32_t* err = err_ptr(a[7], dev);
    at::Tensor k, v;
    if (a[5] == Py_None) k = fresh(shape, type, dev);
    if (a[6] == Py_None) v = fresh(shape, type, dev);
    void* pk = a[5] == Py_None ? k.data_ptr() : ptr(a[5], "k_out", type, shape, dev);
    void* pv = a[6] == Py_None ? v.data_ptr() : ptr(a[6], "v_out", type, shape, dev);
    check(g_lib.q8_gather_gqa(L, c.kv8, small(bt.size(bt.dim() - 2), "requests"),
                              small(c.Hkv, "heads"), small(c.d, "head_dim"), pr, pp, N, pk, pv, dt,
                              err, on.st));
    Ref ko(a[5] == Py_None ? THPVariable_Wrap(k) : given(a[5])),
        vo(a[6] == Py_None ? THPVariable_Wrap(v) : given(a[6]));
    return PyTuple_Pack(2, ko.o, vo.o);
  });
}

// scored(eight, partial, layout, q, kv, seq_lens, scale, scores, sink, out_dtype, out, out_lse,
//        workspace, err, stream)
PyObject* scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 15);
    const bool eight = truth(a[0]), partial = truth(a[1]);
    const dcp_layout_t L = layout_of(a[2]);
    const at::Tensor& q = tensor(a[3], "q");
    const int dev = device_of(q, "q");
    const OnStream on(a[14], dev);
    if (q.dim() != 3) refuse("q must be [requests, heads, head_dim]");
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2);
    const at::ScalarType type = q.scalar_type();
    const dcp_dtype_t dt = dtype_of(type);
    const PagedCache c(a[4], L, eight, type, B, dev);
    if (c.d != d)
      refuse("q with head_dim " + std::to_string(d) + " over a cache with " + std::to_string(c.d));
    if (Hq % c.Hkv)
      refuse(std::to_string(Hq) + " query heads over " + std::to_string(c.Hkv) +
             " key/value heads");
    const void* pq = ptr(q, "q", type, q.sizes(), dev);
    const int32_t* lens = (const int32_t*)ptr(a[5], "seq_lens", at::kInt, {B}, dev);
    const float scale = (float)number(a[6]);
    dcp_scores_t f = {};
    std::optional<Ref> slopes, first;
    if (a[7] != Py_None) {
      f.cap = (float)number(attr(a[7], NAME("cap")).o);
      f.window = small(integer_attr(a[7], NAME("window")), "window");
      f.prefix = small(integer_attr(a[7], NAME("prefix")), "prefix");
      slopes.emplace(PyObject_GetAttr(a[7], NAME("slopes")));
      first.emplace(PyObject_GetAttr(a[7], NAME("first")));
      f.slopes = (const float*)opt(slopes->o, "slopes", at::kFloat, {Hq}, dev);
      f.first = (const int32_t*)opt(first->o, "first", at::kInt, {B}, dev);
    }
    const float* sink = (const float*)opt(a[8], "sink", at::kFloat, {Hq}, dev);
    const int32_t b32 = small(B, "requests"), hq = small(Hq, "heads"), hkv = small(c.Hkv, "heads"),
                  d32 = small(d, "head_dim");
    size_t need = 0;
    check(g_lib.scored_workspace_size(L, b32, hq, hkv, d32, partial, &need));
    const int64_t R = L.dcp_size;
    std::vector<int64_t> os, ls;
    if (partial) {
      os = {R, B, Hq, d};
      ls = {R, B, Hq};
    } else {
      os = {B, Hq, d};
      ls = {B, Hq};
    }
    at::ScalarType odt = type;
    if (partial)
      odt = at::kFloat;
    else if (a[10] != Py_None)
      odt = tensor(a[10], "out").scalar_type();
    else if (a[9] != Py_None) {
      if (!THPDtype_Check(a[9])) refuse("out_dtype must be a torch dtype");
      odt = ((THPDtype*)a[9])->scalar_type;
    }
    const dcp_dtype_t codt = dtype_of(odt);
    int32_t* err = err_ptr(a[13], dev);
    at::Tensor o, l;
    if (a[10] == Py_None && a[11] == Py_None)
      fresh_two(os, odt, o, ls, at::kFloat, l, dev);
    else if (a[10] == Py_None)
      o = fresh(os, odt, dev);
    else if (a[11] == Py_None)
      l = fresh(ls, at::kFloat, dev);
    void* po = a[10] == Py_None ? o.data_ptr() : ptr(a[10], "out", odt, os, dev);
    float* pl = (float*)(a[11] == Py_None ? l.data_ptr() : ptr(a[11], "out_lse", at::kFloat, ls, dev));
    const Workspace ws(a[12], need, dev);
    int rc;
    if (eight)
      rc = partial ? g_lib.q8_partial_gqa(L, pq, b32, hq, hkv, d32, scale, dt, c.kv8, lens, f,
                                          (float*)po, pl, ws.p, ws.bytes, err, on.st)
                   : g_lib.q8_decode_gqa(L, pq, b32, hq, hkv, d32, scale, dt, c.kv8, lens, f, sink,
                                         po, codt, pl, ws.p, ws.bytes, err, on.st);
    else
      rc = partial ? g_lib.scored_partial_gqa(L, pq, b32, hq, hkv, d32, scale, dt, c.kv, lens, f,
                                              (float*)po, pl, ws.p, ws.bytes, err, on.st)
                   : g_lib.scored_decode_gqa(L, pq, b32, hq, hkv, d32, scale, dt, c.kv, lens, f,
                                             sink, po, codt, pl, ws.p, ws.bytes, err, on.st);
    check(rc);
    Ref oo(a[10] == Py_None ? THPVariable_Wrap(o) : given(a[10])),
        ol(a[11] == Py_None ? THPVariable_Wrap(l) : given(a[11]));
    return PyTuple_Pack(2, oo.o, ol.o);
  });
}

// init(path of libdcp.so, DcpError)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 2);
    const char* path = PyUnicode_AsUTF8(a[0]);
    if (!path) return nullptr;
    Py_INCREF(a[1]);
    Py_XSETREF(g_error, a[1]);
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) refuse(dlerror());
    auto get = [&](auto& fn, const char* name) {
      fn = (std::remove_reference_t<decltype(fn)>)dlsym(h, name);
      if (!fn) refuse(std::string("the library has no ") + name);
    };
    get(g_lib.strerror, "dcp_strerror");
    get(g_lib.tree_workspace_size, "dcp_tree_workspace_size");
    get(g_lib.tree_decode_gqa, "dcp_tree_decode_gqa");
    get(g_lib.tree_partial_gqa, "dcp_tree_partial_gqa");
    get(g_lib.rope_write_gqa, "dcp_rope_write_gqa");
    get(g_lib.rope_write_mla, "dcp_rope_write_mla");
    get(g_lib.pages_init, "dcp_pages_init");
    get(g_lib.pages_workspace_size, "dcp_pages_workspace_size");
    get(g_lib.pages_resize, "dcp_pages_resize");
    get(g_lib.pages_fork, "dcp_pages_fork");
    get(g_lib.pages_copy, "dcp_pages_copy");
    get(g_lib.cache_compact, "dcp_cache_compact");
    get(g_lib.q8_append_gqa, "dcp_q8_append_gqa");
    get(g_lib.q8_gather_gqa, "dcp_q8_gather_gqa");
    get(g_lib.q8_decode_gqa, "dcp_q8_decode_gqa");
    get(g_lib.q8_partial_gqa, "dcp_q8_partial_gqa");
    get(g_lib.scored_decode_gqa, "dcp_scored_decode_gqa");
    get(g_lib.scored_partial_gqa, "dcp_scored_partial_gqa");
    get(g_lib.scored_workspace_size, "dcp_scored_workspace_size");
    return given(Py_None);
  });
}

#define DCP_METHOD(name) \
  {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {DCP_METHOD(init),       DCP_METHOD(tree),  DCP_METHOD(rope),
                           DCP_METHOD(pages_init), DCP_METHOD(pages), DCP_METHOD(pages_copy),
                           DCP_METHOD(cache_compact), DCP_METHOD(q8_append),
                           DCP_METHOD(q8_gather), DCP_METHOD(scored), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
