// _fastcall: the binding's hot path. Two things that cost a call most of its host time in pure
// Python are done here:
//
//   match(spec, tensor, ...)   the checks of a call's tensors (device, type, shape, layout) in one go:
//                              a tuple of pointers, sizes, strides and type codes, or None if anything
//                              is not as the spec wants it. Then the caller checks step by step in
//                              Python and raises what is wrong; nothing is refused here.
//   bind(name, address)        a C function of the library as a Python callable without ctypes'
//                              conversion of each argument.
//
// The package works without this module (only slower), so nothing but speed depends on it.
#include <Python.h>

#include <cstdint>
#include <cstring>
#include <memory>
#include <new>
#include <string>
#include <tuple>
#include <utility>
#include <vector>

#include <ATen/core/Tensor.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pkv.h"

namespace {

// ------------------------------------------------------------------ specs
// "q:T,Hq,D:rows:X" and so on, one entry a tensor, separated by spaces:
//   name : sizes : layout : type
// sizes: symbols (bound where they first appear), numbers, or symbol+number; layout `c` contiguous or
// `rows` ([tokens, heads, dim], a token's heads contiguous, tokens apart); type i (int32), l (int64),
// f (float32), b (bfloat16), X (float32 or bfloat16, the same for every X), K (a cache's
// type, the same for every K). A leading `?` takes None for a null pointer.
struct Size {
    int symbol;     // -1: a number
    int64_t plus;
};
struct Entry {
    std::vector<Size> sizes;
    bool rows, optional;
    char type;
};
struct Spec {
    std::vector<Entry> entries;
    int symbols = 0, strides = 0;
    bool has_x = false, has_k = false;
};

std::vector<std::string> split(const std::string& s, char by)
{
    std::vector<std::string> out;
    size_t at = 0;
    while (true) {
        const size_t e = s.find(by, at);
        if (e == std::string::npos) {
            if (at < s.size())
                out.push_back(s.substr(at));
            return out;
        }
        if (e > at)
            out.push_back(s.substr(at, e - at));
        at = e + 1;
    }
}

void free_spec(PyObject* capsule) { delete static_cast<Spec*>(PyCapsule_GetPointer(capsule, "pkv.spec")); }

PyObject* make_spec(PyObject*, PyObject* arg)
{
    const char* text = PyUnicode_AsUTF8(arg);
    if (!text)
        return nullptr;
    try {
        auto spec = std::make_unique<Spec>();
        std::vector<std::string> names;
        for (const std::string& e : split(text, ' ')) {
            const std::vector<std::string> f = split(e, ':');
            if (f.size() != 4)
                throw std::runtime_error("a spec's entries are name:sizes:layout:type");
            Entry x;
            x.optional = f[0][0] == '?';
            x.rows = f[2] == "rows";
            x.type = f[3][0];
            spec->strides += x.rows;
            spec->has_x |= x.type == 'X';
            spec->has_k |= x.type == 'K';
            for (const std::string& d : split(f[1], ',')) {
                Size z{-1, 0};
                const size_t p = d.find('+');
                const std::string head = d.substr(0, p);
                if (p != std::string::npos)
                    z.plus = std::stoll(d.substr(p + 1));
                if (head[0] >= '0' && head[0] <= '9') {
                    z.plus = std::stoll(head);
                } else {
                    size_t i = 0;
                    while (i < names.size() && names[i] != head)
                        ++i;
                    if (i == names.size())
                        names.push_back(head);
                    z.symbol = (int)i;
                }
                x.sizes.push_back(z);
            }
            spec->entries.push_back(x);
        }
        spec->symbols = (int)names.size();
        PyObject* c = PyCapsule_New(spec.get(), "pkv.spec", free_spec);
        if (c)
            spec.release();
        return c;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

int code_of(at::ScalarType t)
{
    switch (t) {
    case at::ScalarType::Float: return PKV_F32;
    case at::ScalarType::BFloat16: return PKV_BF16;
    case at::ScalarType::Byte:
    case at::ScalarType::Float8_e4m3fn: return PKV_FP8_E4M3;
    case at::ScalarType::Float8_e5m2: return PKV_FP8_E5M2;
    case at::ScalarType::Char: return PKV_INT8;
    default: return -1;
    }
}

constexpr int kMaxSymbols = 16, kMaxEntries = 24;

// pointers (one an entry), symbols in order of appearance, row strides, the code of X, the code of K,
// the device. Throws for tensors without a storage or with symbolic sizes (vmap's wrappers, fake tensors).
PyObject* match_or_throw(PyObject* const* args, Py_ssize_t n)
{
    const Spec* spec = static_cast<const Spec*>(PyCapsule_GetPointer(args[0], "pkv.spec"));
    if (!spec)
        return nullptr;
    const int E = (int)spec->entries.size();
    if (n != E + 1 || E > kMaxEntries || spec->symbols > kMaxSymbols)
        Py_RETURN_NONE;
    int64_t symbol[kMaxSymbols], stride[kMaxEntries];
    bool bound[kMaxSymbols] = {};
    void* ptr[kMaxEntries];
    int strides = 0, device = -1;
    at::ScalarType x_type = at::ScalarType::Undefined, k_type = at::ScalarType::Undefined;
    for (int e = 0; e < E; ++e) {
        const Entry& want = spec->entries[e];
        PyObject* o = args[e + 1];
        if (o == Py_None) {
            if (!want.optional)
                Py_RETURN_NONE;
            ptr[e] = nullptr;
            continue;
        }
        if (!THPVariable_Check(o))
            Py_RETURN_NONE;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.dim() != (int64_t)want.sizes.size())
            Py_RETURN_NONE;
        if (device < 0)
            device = t.get_device();
        else if (t.get_device() != device)
            Py_RETURN_NONE;
        const at::ScalarType type = t.scalar_type();
        bool ok = true;
        switch (want.type) {
        case 'i': ok = type == at::ScalarType::Int; break;
        case 'l': ok = type == at::ScalarType::Long; break;
        case 'f': ok = type == at::ScalarType::Float; break;
        case 'b': ok = type == at::ScalarType::BFloat16; break;
        case 'X':
            if (x_type == at::ScalarType::Undefined) {
                x_type = type;
                ok = type == at::ScalarType::Float || type == at::ScalarType::BFloat16;
            } else {
                ok = type == x_type;
            }
            break;
        default:
            if (k_type == at::ScalarType::Undefined) {
                k_type = type;
                ok = code_of(type) >= 0;
            } else {
                ok = type == k_type;
            }
        }
        if (!ok)
            Py_RETURN_NONE;
        const auto sizes = t.sizes();
        for (size_t d = 0; d < want.sizes.size(); ++d) {
            const Size z = want.sizes[d];
            if (z.symbol < 0) {
                if (sizes[d] != z.plus)
                    Py_RETURN_NONE;
            } else if (!bound[z.symbol]) {
                bound[z.symbol] = true;
                symbol[z.symbol] = sizes[d] - z.plus;
            } else if (sizes[d] != symbol[z.symbol] + z.plus) {
                Py_RETURN_NONE;
            }
        }
        if (want.rows) {
            const auto st = t.strides();
            const int64_t T = sizes[0], H = sizes[1], D = sizes[2];
            if (T > 0 && (st[2] != 1 || (H > 1 && st[1] != D)))
                Py_RETURN_NONE;
            if (T > 1 && st[0] < H * D)
                Py_RETURN_NONE;
            stride[strides++] = T > 1 ? st[0] : H * D;
        } else if (!t.is_contiguous()) {
            Py_RETURN_NONE;
        }
        ptr[e] = t.data_ptr();
        if (!ptr[e] && t.numel() > 0)   // a fake tensor's
            Py_RETURN_NONE;
    }
    for (int i = 0; i < spec->symbols; ++i)
        if (!bound[i])
            Py_RETURN_NONE;
    if (device < 0 || strides != spec->strides)
        Py_RETURN_NONE;
    // the library launches on the current device
    if (c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index() != device)
        Py_RETURN_NONE;
    const int total = E + spec->symbols + strides + spec->has_x + spec->has_k + 1;
    PyObject* out = PyTuple_New(total);
    if (!out)
        return nullptr;
    int at = 0;
    auto put = [&](PyObject* v) { PyTuple_SET_ITEM(out, at++, v); };
    for (int e = 0; e < E; ++e)
        put(PyLong_FromVoidPtr(ptr[e]));
    for (int i = 0; i < spec->symbols; ++i)
        put(PyLong_FromLongLong(symbol[i]));
    for (int i = 0; i < strides; ++i)
        put(PyLong_FromLongLong(stride[i]));
    if (spec->has_x)
        put(PyLong_FromLong(code_of(x_type)));
    if (spec->has_k)
        put(PyLong_FromLong(code_of(k_type)));
    put(PyLong_FromLong(device));
    for (int i = 0; i < total; ++i)
        if (!PyTuple_GET_ITEM(out, i)) {
            Py_DECREF(out);
            return nullptr;
        }
    return out;
}

// No C++ exception may leave a function that Python calls: what throws is no match, and the caller's
// own checks raise.
PyObject* match(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n < 1) {
        PyErr_SetString(PyExc_TypeError, "match(spec, tensor, ...)");
        return nullptr;
    }
    try {
        return match_or_throw(args, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// ------------------------------------------------------------------ calls

template <class T>
bool convert(PyObject* o, T& v)
{
    if constexpr (std::is_pointer<T>::value) {
        v = nullptr;
        if (o == Py_None)
            return true;
        void* p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred())
            return false;
        v = static_cast<T>(p);
        return true;
    } else if constexpr (std::is_floating_point<T>::value) {
        const double d = PyFloat_AsDouble(o);
        if (d == -1.0 && PyErr_Occurred())
            return false;
        v = (T)d;
        return true;
    } else {
        const long long i = PyLong_AsLongLong(o);
        if (i == -1 && PyErr_Occurred())
            return false;
        v = (T)i;
        if ((long long)v != i || (std::is_unsigned<T>::value && i < 0)) {
            PyErr_SetString(PyExc_OverflowError, "a number does not fit its C argument");
            return false;
        }
        return true;
    }
}

template <class... A, size_t... I>
PyObject* call_with(int (*f)(A...), PyObject* const* args, std::index_sequence<I...>)
{
    std::tuple<A...> v;
    if (!(convert(args[I], std::get<I>(v)) && ...))
        return nullptr;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f(std::get<I>(v)...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

template <class... A>
PyObject* call(int (*f)(A...), PyObject* const* args, Py_ssize_t n)
{
    if (n != (Py_ssize_t)sizeof...(A)) {
        PyErr_Format(PyExc_TypeError, "expected %zu arguments, got %zd", sizeof...(A), n);
        return nullptr;
    }
    return call_with(f, args, std::index_sequence_for<A...>{});
}

#define PKV_FAST(NAME)                                                                     \
    decltype(&::NAME) at_##NAME = nullptr;                                                 \
    PyObject* py_##NAME(PyObject*, PyObject* const* args, Py_ssize_t n)                    \
    {                                                                                      \
        if (!at_##NAME) {                                                                  \
            PyErr_SetString(PyExc_RuntimeError, #NAME " is not bound");                    \
            return nullptr;                                                                \
        }                                                                                  \
        return call(at_##NAME, args, n);                                                   \
    }
PKV_FAST(qk_norm_rope)
PKV_FAST(qk_norm_rope_and_cache)
PKV_FAST(reshape_and_cache_block_scales)
PKV_FAST(paged_attention_decode_block_scales)
PKV_FAST(update_key_bounds)
PKV_FAST(select_blocks)
PKV_FAST(paged_attention_decode_sparse)
PKV_FAST(pkv_stream_recorded)
#undef PKV_FAST

// bind(name, address): the module's function `name` calls the C function at `address` from here on.
PyObject* bind(PyObject*, PyObject* args)
{
    const char* name;
    unsigned long long address;
    if (!PyArg_ParseTuple(args, "sK", &name, &address))
        return nullptr;
#define PKV_BIND(NAME)                                                       \
    if (!std::strcmp(name, #NAME)) {                                         \
        at_##NAME = reinterpret_cast<decltype(at_##NAME)>((uintptr_t)address); \
        Py_RETURN_TRUE;                                                      \
    }
    PKV_BIND(qk_norm_rope)
    PKV_BIND(qk_norm_rope_and_cache)
    PKV_BIND(reshape_and_cache_block_scales)
    PKV_BIND(paged_attention_decode_block_scales)
    PKV_BIND(update_key_bounds)
    PKV_BIND(select_blocks)
    PKV_BIND(paged_attention_decode_sparse)
    PKV_BIND(pkv_stream_recorded)
#undef PKV_BIND
    Py_RETURN_FALSE;
}

#define PKV_METHOD(NAME) {#NAME, (PyCFunction)(void (*)(void))py_##NAME, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"spec", make_spec, METH_O, "A spec of a call's tensors, for match()."},
    {"match", (PyCFunction)(void (*)(void))match, METH_FASTCALL, "The pieces of a call's tensors, or None."},
    {"bind", bind, METH_VARARGS, "Bind a library function's address."},
    PKV_METHOD(qk_norm_rope),
    PKV_METHOD(qk_norm_rope_and_cache),
    PKV_METHOD(reshape_and_cache_block_scales),
    PKV_METHOD(paged_attention_decode_block_scales),
    PKV_METHOD(update_key_bounds),
    PKV_METHOD(select_blocks),
    PKV_METHOD(paged_attention_decode_sparse),
    PKV_METHOD(pkv_stream_recorded),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", "Hot path of the binding.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall()
{
    PyObject* m = PyModule_Create(&module);
    // the torch whose at::Tensor this was compiled against: with another one the package leaves it alone
    if (m && PyModule_AddStringConstant(m, "torch_version", PKV_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
