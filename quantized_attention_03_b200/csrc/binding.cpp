// The rotary and 4-bit cache calls for Python, where a call's cost on the host counts: a decode
// step makes them once per layer and their kernels take a few microseconds. Checks the tensors,
// allocates outputs, takes torch's current stream and calls the C ABI (sage.h). Each function
// returns its outputs, or the library's status code as an int when the call was refused.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/sage.h"

namespace {

using at::Tensor;

decltype(&sage_rope) p_rope;
decltype(&sage_kv4_append) p_append;
decltype(&sage_kv4_gather) p_gather;
decltype(&sage_attn_kv4) p_attn;
decltype(&sage_attn_kv4_workspace_size) p_attn_workspace;

// A refusal that becomes a ValueError.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

// A function's arguments in their fixed order, None where a tensor may be left out.
struct Args {
    PyObject *const *v;

    bool none(int i) const { return v[i] == Py_None; }
    const Tensor &tensor(int i, const char *name) const
    {
        if (!THPVariable_Check(v[i]))
            throw Refused(std::string(name) + " is a tensor");
        return THPVariable_Unpack(v[i]);
    }
    int64_t integer(int i) const
    {
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred())
            throw std::invalid_argument("");           // Python's own error is set
        return x;
    }
    int size(int i, const char *name) const
    {
        const int64_t x = integer(i);
        if (x < INT32_MIN || x > INT32_MAX)
            throw Refused(std::string(name) + " does not fit 32 bits");
        return (int)x;
    }
    double real(int i) const
    {
        const double x = PyFloat_AsDouble(v[i]);
        if (x == -1.0 && PyErr_Occurred())
            throw std::invalid_argument("");
        return x;
    }
    bool truth(int i) const
    {
        const int x = PyObject_IsTrue(v[i]);
        if (x < 0)
            throw std::invalid_argument("");
        return x != 0;
    }
};

std::string described(const Tensor &x)
{
    std::string s = std::string(c10::toString(x.scalar_type())) + " [";
    for (int64_t i = 0; i < x.dim(); i++)
        s += (i ? ", " : "") + std::to_string(x.size(i));
    s += "] with strides [";
    for (int64_t i = 0; i < x.dim(); i++)
        s += (i ? ", " : "") + std::to_string(x.stride(i));
    return s + "] on " + x.device().str();
}

void want(bool ok, const Tensor &x, const char *what)
{
    if (!ok)
        throw Refused(std::string(what) + ", got " + described(x));
}

int half_type(const Tensor &x, const char *what)
{
    want(x.scalar_type() == at::kHalf || x.scalar_type() == at::kBFloat16, x, what);
    return x.scalar_type() == at::kHalf ? SAGE_F16 : SAGE_BF16;
}

bool same(const Tensor &x, const Tensor &y) { return x.device() == y.device() && x.scalar_type() == y.scalar_type(); }

int to32(int64_t x, const Tensor &t, const char *what)
{
    want(x <= INT32_MAX, t, what);
    return (int)x;
}

// Outputs that the caller gives. Kernels write an output while they read inputs and write other
// outputs, so its elements lie apart from each other and from those, but that an output may be
// its input itself (same address, same strides), where each element is read before it is written.

// A dimension with more than one place, its step in elements.
struct Dim {
    int64_t step, a, b;                                // sizes in two tensors of the same steps
};

// Whether some difference of two places, i in (-d.b, d.a) along each of n dimensions, is `at`
// elements. Steps ascend and each is at least the extent of those before it, so that at most two
// i of a dimension leave a rest within their reach.
bool reaches(const Dim *d, int n, int64_t at)
{
    if (n == 0)
        return at == 0;
    const Dim &x = d[n - 1];
    const int64_t i = at >= 0 ? at / x.step : -((-at + x.step - 1) / x.step);      // floor
    for (int64_t j = i; j <= i + 1; j++)
        if (j > -x.b && j < x.a && reaches(d, n - 1, at - j * x.step))
            return true;
    return false;
}

// Dimensions of x and y (y with other sizes but the same steps, else x twice) by ascending step;
// -1 where steps differ, -2 where places of one tensor can coincide.
int dims_of(const Tensor &x, const Tensor &y, Dim (&d)[4])
{
    int n = 0;
    for (int64_t i = 0; i < x.dim(); i++) {
        const int64_t a = x.size(i), b = y.size(i);
        if (a == 1 && b == 1)
            continue;
        if (a != 1 && b != 1 && x.stride(i) != y.stride(i))
            return -1;
        int at = n++;
        for (const int64_t step = a != 1 ? x.stride(i) : y.stride(i); at > 0 && d[at - 1].step > step; at--)
            d[at] = d[at - 1];
        d[at] = Dim{a != 1 ? x.stride(i) : y.stride(i), a, b};
    }
    int64_t extent = 1;
    for (int i = 0; i < n; i++) {
        if (d[i].step < extent)
            return -2;
        extent = (std::max(d[i].a, d[i].b) - 1) * d[i].step + extent;
    }
    return n;
}

int64_t extent_of(const Tensor &x)
{
    int64_t n = 1;
    for (int64_t i = 0; i < x.dim(); i++)
        n += (x.size(i) - 1) * x.stride(i);
    return n;
}

// Whether x and y, of one type and number of dimensions (at most 4), are known to share memory.
// `self`: whether that counts where they are the same elements in the same places.
bool meet(const Tensor &x, const Tensor &y, bool self)
{
    if (x.numel() == 0 || y.numel() == 0 || x.device() != y.device())
        return false;
    const int64_t size = x.element_size();
    const char *a = static_cast<const char *>(x.const_data_ptr()), *b = static_cast<const char *>(y.const_data_ptr());
    if (a + extent_of(x) * size <= b || b + extent_of(y) * size <= a)
        return false;
    Dim d[4];
    const int n = dims_of(x, y, d);
    if (a == b)
        return self || n < 0 || x.sizes() != y.sizes();
    if (n >= 0)
        return (b - a) % size != 0 || reaches(d, n, (b - a) / size);
    return x.is_non_overlapping_and_dense() && y.is_non_overlapping_and_dense();
}

void want_apart(const Tensor &out, const Tensor &in, bool same_input, const char *what)
{
    want(!meet(out, in, !same_input), out, what);
}
void want_places(const Tensor &out, const char *what)
{
    Dim d[4];
    want(out.numel() == 0 || dims_of(out, out, d) >= 0, out, what);
}

// Autograd learns that a tensor it may have saved is written over.
void written(const Tensor &x)
{
    if (!x.is_inference())
        x.unsafeGetTensorImpl()->bump_version();
}

// The device of the call's tensors and the stream given (a pointer) made current, so that what
// the call allocates belongs to the stream that uses it: a workspace is free again when the call
// returns, and only that stream's order keeps the kernel's use before the next one's.
struct Where {
    const Tensor &x;
    std::optional<c10::cuda::CUDAGuard> device;
    std::optional<c10::cuda::CUDAStreamGuard> on;
    sage_stream_t given = nullptr;

    Where(const Tensor &x, const Args &a, int stream_arg) : x(x)
    {
        if (!x.is_cuda())
            return;
        if (x.get_device() != c10::cuda::current_device())
            device.emplace(x.device());
        if (a.none(stream_arg))
            return;
        const uintptr_t raw = (uintptr_t)a.integer(stream_arg);
        given = reinterpret_cast<sage_stream_t>(raw);
        on.emplace(raw <= 1 ? c10::cuda::getDefaultCUDAStream(x.get_device())    // 0, cudaStreamLegacy
                            : c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(raw), x.get_device()));
    }
    sage_stream_t stream() const
    {
        want(x.is_cuda(), x, "the tensors are on a CUDA device");
        if (on)
            return given;
        return reinterpret_cast<sage_stream_t>(c10::cuda::getCurrentCUDAStream(x.get_device()).stream());
    }
};

const double *freqs_of(const Args &a, int i, const Tensor &x, int &rot)
{
    rot = 0;
    if (a.none(i))
        return nullptr;
    const Tensor &f = a.tensor(i, "freqs");
    want(f.scalar_type() == at::kDouble && f.dim() == 1 && f.is_contiguous() && f.device() == x.device(), f,
         "freqs is a contiguous float64 vector on the tensors' device");
    rot = to32(2 * f.size(0), f, "freqs is too long");
    return static_cast<const double *>(f.const_data_ptr());
}

// (q, k, freqs, positions, mscale, interleaved, inverse, q_out, k_out, stream); -1 instead of a
// status where a gradient of q or k is wanted: the caller goes through autograd then
PyObject *rope(const Args &a)
{
    const Tensor &q = a.tensor(0, "q");
    if (at::GradMode::is_enabled()) {
        if (!a.none(2) && a.tensor(2, "freqs").requires_grad())
            throw Refused("freqs takes no gradient");
        if (q.requires_grad() || (!a.none(1) && a.tensor(1, "k").requires_grad()))
            return PyLong_FromLong(-1);
        for (int i : {7, 8})
            if (!a.none(i) && a.tensor(i, "q_out and k_out").requires_grad())
                throw Refused("q_out and k_out take no gradient");
    }
    const int type = half_type(q, "q is float16 or bfloat16");
    const bool packed = q.dim() == 3;
    want((packed || q.dim() == 4) && q.stride(-1) == 1, q,
         "q is [B, H, N, d] or [T, H, d], its channels contiguous");
    const int64_t B = packed ? 1 : q.size(0), N = q.size(packed ? 0 : 2), d = q.size(-1);
    const bool has_k = !a.none(1);
    int64_t s[12] = {};
    auto place = [&](int at, const Tensor &x) {
        s[at] = packed ? 0 : x.stride(0);
        s[at + 1] = x.stride(1);
        s[at + 2] = x.stride(packed ? 0 : 2);
    };
    const Where w(q, a, 9);
    Tensor q_out = a.none(7) ? at::empty_like(q) : a.tensor(7, "q_out"), k_out;
    want(q_out.sizes() == q.sizes() && same(q_out, q) && q_out.stride(-1) == 1, q_out,
         "q_out has q's shape, type and device");
    if (!a.none(7)) {
        want_places(q_out, "q_out's elements lie apart, the step of each dimension past what lies within it");
        want_apart(q_out, q, true, "q_out is q itself or lies apart from it");
    }
    place(0, q);
    place(3, q_out);
    const Tensor *k = nullptr;
    if (has_k) {
        k = &a.tensor(1, "k");
        want(k->dim() == q.dim() && same(*k, q) && k->stride(-1) == 1 && k->size(-1) == d &&
                 k->size(packed ? 0 : 2) == N && (packed || k->size(0) == B), *k,
             "k has q's type, device, tokens and head dim, its channels contiguous");
        k_out = a.none(8) ? at::empty_like(*k) : a.tensor(8, "k_out");
        want(k_out.sizes() == k->sizes() && same(k_out, q) && k_out.stride(-1) == 1, k_out,
             "k_out has k's shape, type and device");
        if (!a.none(8)) {
            want_places(k_out, "k_out's elements lie apart, the step of each dimension past what lies within it");
            want_apart(k_out, *k, true, "k_out is k itself or lies apart from it");
            want_apart(k_out, q, false, "k_out lies apart from q");
        }
        if (!a.none(7)) {
            want_apart(q_out, *k, false, "q_out lies apart from k");
            if (!a.none(8))
                want_apart(q_out, k_out, false, "q_out lies apart from k_out");
        }
        place(6, *k);
        place(9, k_out);
    }
    int rot;
    const double *freqs = freqs_of(a, 2, q, rot);
    if (!freqs && rot == 0)
        throw Refused("freqs is a contiguous float64 vector on the tensors' device");
    const int32_t *positions = nullptr;
    int64_t pos_stride = 0;
    if (!a.none(3)) {
        const Tensor &p = a.tensor(3, "positions");
        const bool one = p.dim() == 1 && p.size(0) == N, two = p.dim() == 2 && p.size(0) == B && p.size(1) == N;
        want(p.scalar_type() == at::kInt && p.device() == q.device() && (one || two) && (N < 2 || p.stride(-1) == 1),
             p, "positions is int32 [N], [B, N] or [T] on q's device");
        positions = static_cast<const int32_t *>(p.const_data_ptr());
        pos_stride = two ? p.stride(0) : 0;
    }
    const sage_status_t rc = p_rope(
        q.const_data_ptr(), q_out.mutable_data_ptr(), has_k ? k->const_data_ptr() : nullptr,
        has_k ? k_out.mutable_data_ptr() : nullptr, positions, freqs, type, to32(B, q, "q has too many sequences"),
        to32(N, q, "q has too many tokens"), to32(q.size(1), q, "q has too many heads"),
        has_k ? to32(k->size(1), *k, "k has too many heads") : 0, to32(d, q, "q's head dim is too large"), rot, pos_stride,
        s, a.real(4), (a.truth(5) ? SAGE_ROPE_INTERLEAVED : 0) | (a.truth(6) ? SAGE_ROPE_INVERSE : 0), w.stream());
    if (rc != SAGE_OK)
        return PyLong_FromLong(rc);
    if (!a.none(7))
        written(q_out);
    if (has_k && !a.none(8))
        written(k_out);
    PyObject *qo = THPVariable_Wrap(std::move(q_out));
    PyObject *ko = has_k ? THPVariable_Wrap(std::move(k_out)) : Py_NewRef(Py_None);
    return Py_BuildValue("(NN)", qo, ko);
}

// A cache and its sequences (arguments at..at+3: cache, block_table, kv_lens, cu_seqlens).
struct Seqs {
    const Tensor &cache, &table, &lens;
    const int32_t *cu = nullptr;
    int nseq, Hkv, page_size, num_pages, max_pages;

    Seqs(const Args &a, int at, int64_t d)
        : cache(a.tensor(at, "cache")), table(a.tensor(at + 1, "block_table")), lens(a.tensor(at + 2, "kv_lens"))
    {
        const int64_t bytes = cache.dim() == 3 ? cache.size(2) : 0;
        const int64_t page = d > 0 ? bytes * 8 / (9 * d) : 0;
        want(cache.scalar_type() == at::kByte && cache.dim() == 3 && cache.is_contiguous() && page >= 16 && page <= 256 &&
                 (page & (page - 1)) == 0 && page * 9 * d == bytes * 8, cache,
             "cache is a contiguous uint8 [num_pages, Hkv, page bytes] of kv4_cache for this head dim");
        auto i32 = [&](const Tensor &x) {
            return x.scalar_type() == at::kInt && x.is_contiguous() && x.device() == cache.device();
        };
        want(i32(lens) && lens.dim() == 1, lens, "kv_lens is contiguous int32 [nseq] on the cache's device");
        want(i32(table) && table.dim() == 2 && table.size(0) == lens.size(0), table,
             "block_table is contiguous int32 [nseq, max_pages] on the cache's device");
        if (!a.none(at + 3)) {
            const Tensor &c = a.tensor(at + 3, "cu_seqlens");
            want(i32(c) && c.dim() == 1 && c.size(0) == lens.size(0) + 1, c,
                 "cu_seqlens is contiguous int32 [nseq + 1] on the cache's device");
            cu = static_cast<const int32_t *>(c.const_data_ptr());
        }
        nseq = to32(lens.size(0), lens, "kv_lens is too long");
        Hkv = to32(cache.size(1), cache, "cache has too many heads");
        page_size = (int)page;
        num_pages = to32(cache.size(0), cache, "cache has too many pages");
        max_pages = to32(table.size(1), table, "block_table is too wide");
    }
    const int32_t *table_at() const { return static_cast<const int32_t *>(table.const_data_ptr()); }
    const int32_t *lens_at() const { return static_cast<const int32_t *>(lens.const_data_ptr()); }
};

// (cache, block_table, kv_lens, cu_seqlens, k, v, q, freqs, mscale, interleaved, k_mean, q_out, stream)
PyObject *append(const Args &a)
{
    const Tensor &k = a.tensor(4, "k"), &v = a.tensor(5, "v");
    const int type = half_type(k, "k is float16 or bfloat16");
    want(k.dim() == 3, k, "k is [T, Hkv, d]");
    const Seqs s(a, 0, k.size(2));
    want(k.size(1) == s.Hkv && k.stride(2) == 1 && k.device() == s.cache.device(), k,
         "k is [T, Hkv, d] with the cache's heads and device, its channels contiguous");
    want(v.sizes() == k.sizes() && same(v, k) && v.stride(2) == 1, v, "v has k's shape, type and device");
    const Where w(k, a, 12);
    int64_t st[8] = {k.stride(0), k.stride(1), v.stride(0), v.stride(1), 0, 0, 0, 0};
    const Tensor *q = nullptr;
    Tensor q_out;
    if (!a.none(6)) {
        q = &a.tensor(6, "q");
        want(q->dim() == 3 && q->size(0) == k.size(0) && q->size(2) == k.size(2) && same(*q, k) && q->stride(2) == 1, *q,
             "q is [T, Hq, d] of k's type and device, its channels contiguous");
        q_out = a.none(11) ? at::empty_like(*q) : a.tensor(11, "q_out");
        want(q_out.sizes() == q->sizes() && same(q_out, k) && q_out.stride(2) == 1, q_out,
             "q_out has q's shape, type and device");
        if (!a.none(11)) {
            want_places(q_out, "q_out's elements lie apart, the step of each dimension past what lies within it");
            want_apart(q_out, *q, true, "q_out is q itself or lies apart from it");
            want_apart(q_out, k, false, "q_out lies apart from k");
            want_apart(q_out, v, false, "q_out lies apart from v");
        }
        st[4] = q->stride(0);
        st[5] = q->stride(1);
        st[6] = q_out.stride(0);
        st[7] = q_out.stride(1);
    }
    int rot;
    const double *freqs = freqs_of(a, 7, k, rot);
    const float *mean = nullptr;
    if (!a.none(10)) {
        const Tensor &m = a.tensor(10, "k_mean");
        want(m.scalar_type() == at::kFloat && m.dim() == 2 && m.size(0) == k.size(1) && m.size(1) == k.size(2) &&
                 m.is_contiguous() && m.device() == k.device(), m,
             "k_mean is a contiguous float32 [Hkv, d] on the cache's device");
        mean = static_cast<const float *>(m.const_data_ptr());
    }
    const sage_status_t rc = p_append(
        s.cache.mutable_data_ptr(), s.table_at(), s.lens_at(), s.cu, k.const_data_ptr(), v.const_data_ptr(),
        q ? q->const_data_ptr() : nullptr, q ? q_out.mutable_data_ptr() : nullptr, freqs, mean, type, s.nseq,
        to32(k.size(0), k, "k has too many tokens"), q ? to32(q->size(1), *q, "q has too many heads") : 0, s.Hkv,
        (int)k.size(2), s.page_size, s.num_pages, s.max_pages, rot, st, a.real(8),
        a.truth(9) ? SAGE_ROPE_INTERLEAVED : 0, w.stream());
    if (rc != SAGE_OK)
        return PyLong_FromLong(rc);
    if (q && !a.none(11))
        written(q_out);
    return q ? THPVariable_Wrap(std::move(q_out)) : Py_NewRef(Py_None);
}

// (cache, block_table, kv_lens, cu_seqlens, total, d, bf16, rep, k_out, v_out, stream)
PyObject *gather(const Args &a)
{
    const int total = a.size(4, "total"), d = a.size(5, "d"), rep = a.size(7, "rep");
    const at::ScalarType type = a.truth(6) ? at::kBFloat16 : at::kHalf;
    const Seqs s(a, 0, d);
    if (total < 0 || rep < 1)
        throw Refused("total is not negative and rep is at least 1");
    if ((int64_t)s.Hkv * rep > 65535)                  // before outputs of that size are asked for
        return PyLong_FromLong(SAGE_ERR_UNSUPPORTED);
    const Where w(s.cache, a, 10);
    const int64_t shape[3] = {total, (int64_t)s.Hkv * rep, d};
    auto out = [&](int i, const char *name) -> Tensor {
        if (a.none(i))
            return at::empty(shape, s.cache.options().dtype(type));
        const Tensor &x = a.tensor(i, name);
        want(x.sizes() == at::IntArrayRef(shape, 3) && x.scalar_type() == type && x.is_contiguous() &&
                 x.device() == s.cache.device(), x,
             "k_out and v_out are contiguous [total, Hkv * rep, d] of the dtype asked for, on the cache's device");
        return x;
    };
    Tensor k = out(8, "k_out"), v = out(9, "v_out");
    if (!a.none(8) && !a.none(9))
        want_apart(k, v, false, "k_out lies apart from v_out");
    const sage_status_t rc = p_gather(s.cache.const_data_ptr(), s.table_at(), s.lens_at(), s.cu, k.mutable_data_ptr(),
                                      v.mutable_data_ptr(), type == at::kHalf ? SAGE_F16 : SAGE_BF16, s.nseq, total,
                                      s.Hkv, rep, d, s.page_size, s.num_pages, s.max_pages, w.stream());
    if (rc != SAGE_OK)
        return PyLong_FromLong(rc);
    for (int i : {8, 9})
        if (!a.none(i))
            written(i == 8 ? k : v);
    PyObject *ko = THPVariable_Wrap(std::move(k)), *vo = THPVariable_Wrap(std::move(v));
    return Py_BuildValue("(NN)", ko, vo);
}

// (q, cache, block_table, kv_lens, cu_seqlens, max_q, causal, sm_scale, out, lse, workspace, stream)
PyObject *attn(const Args &a)
{
    const Tensor &q = a.tensor(0, "q");
    const int type = half_type(q, "q is float16 or bfloat16");
    want(q.dim() == 3, q, "q is [T, Hq, d]");
    const Seqs s(a, 1, q.size(2));
    want(q.device() == s.cache.device() && q.stride(2) == 1, q,
         "q is [T, Hq, d] on the cache's device, its channels contiguous");
    const Where w(q, a, 11);
    Tensor out = a.none(8) ? at::empty(q.sizes(), q.options()) : a.tensor(8, "out");
    want(out.sizes() == q.sizes() && same(out, q) && out.is_contiguous(), out,
         "out is contiguous and has q's shape, type and device");
    if (!a.none(8))
        want_apart(out, q, true, "out is q itself or lies apart from it");
    float *lse = nullptr;
    if (!a.none(9)) {
        const Tensor &x = a.tensor(9, "lse");
        want(x.scalar_type() == at::kFloat && x.dim() == 2 && x.size(0) == q.size(0) && x.size(1) == q.size(1) &&
                 x.is_contiguous() && x.device() == q.device(), x, "lse is a contiguous float32 [T, Hq] on q's device");
        lse = static_cast<float *>(x.mutable_data_ptr());
    }
    const int T = to32(q.size(0), q, "q has too many tokens"), Hq = to32(q.size(1), q, "q has too many heads");
    const int max_q = !a.none(5) ? a.size(5, "max_q") : s.cu ? SAGE_DECODE_MAX_Q : T / (s.nseq > 0 ? s.nseq : 1);
    Tensor ws;
    if (a.none(10)) {
        const int64_t need = (int64_t)p_attn_workspace(Hq, s.Hkv, max_q, (int)q.size(2));
        ws = at::empty({need > 16 ? need : 16}, s.cache.options());
    } else {
        ws = a.tensor(10, "workspace");
        want(ws.is_contiguous() && ws.device() == q.device(), ws, "workspace is contiguous and on q's device");
    }
    const int64_t st[2] = {q.stride(0), q.stride(1)};
    const sage_status_t rc =
        p_attn(q.const_data_ptr(), s.cache.const_data_ptr(), s.table_at(), s.lens_at(), s.cu, out.mutable_data_ptr(), lse,
               type, s.nseq, T, max_q, Hq, s.Hkv, (int)q.size(2), s.page_size, s.num_pages, s.max_pages, a.truth(6),
               (float)a.real(7), st, ws.mutable_data_ptr(), ws.nbytes(), w.stream());
    if (rc != SAGE_OK)
        return PyLong_FromLong(rc);
    if (!a.none(8))
        written(out);
    if (lse)
        written(a.tensor(9, "lse"));
    return THPVariable_Wrap(std::move(out));
}

// Argument count and C++ exceptions at the border to Python.
template <PyObject *(*F)(const Args &), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N)
        return PyErr_Format(PyExc_TypeError, "%d arguments, got %zd", N, n);
    try {
        return F(Args{args});
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {                                    // torch's own errors as Python knows them
        if (!PyErr_Occurred())
            torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// The library's entry points, by address.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 5)
        return PyErr_Format(PyExc_TypeError, "5 arguments, got %zd", n);
    void *p[5];
    for (int i = 0; i < 5; i++)
        if (!(p[i] = PyLong_AsVoidPtr(args[i])))
            return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a null entry point");
    p_rope = reinterpret_cast<decltype(p_rope)>(p[0]);
    p_append = reinterpret_cast<decltype(p_append)>(p[1]);
    p_gather = reinterpret_cast<decltype(p_gather)>(p[2]);
    p_attn = reinterpret_cast<decltype(p_attn)>(p[3]);
    p_attn_workspace = reinterpret_cast<decltype(p_attn_workspace)>(p[4]);
    return Py_NewRef(Py_None);
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(bind)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(call<rope, 10>)), METH_FASTCALL, nullptr},
    {"kv4_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(call<append, 13>)), METH_FASTCALL, nullptr},
    {"kv4_gather", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(call<gather, 11>)), METH_FASTCALL, nullptr},
    {"attn_kv4", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(call<attn, 12>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding()
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) {   // the Python and torch, by build.py
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
