// packed.cu -- the calls of short kernels with all their arguments in one array of 8-byte words, in the
// order of the C header (pointers and integers as they are, floats as doubles).  For the Python binding: its
// conversion of single arguments costs up to 0.2 us each, more than the rest of a call.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "cp_internal.h"

namespace {

// The words one after the other, each as the type that the call wants.
struct Words {
    const int64_t *at;
    template <typename T>
    operator T *() {
        return reinterpret_cast<T *>(static_cast<uintptr_t>(*at++));
    }
    operator int64_t() { return *at++; }
    operator size_t() { return static_cast<size_t>(*at++); }
    operator cp_dtype() { return static_cast<cp_dtype>(*at++); }
    operator float() {
        double v;
        std::memcpy(&v, at++, sizeof(v));
        return static_cast<float>(v);
    }
};

template <typename... A>
cp_status call(cp_status (*f)(A...), const int64_t *words) {
    Words w{words};
    struct Run {
        cp_status status;
        Run(cp_status (*g)(A...), A... a) : status(g(a...)) {}
    };
    return Run{f, static_cast<A>(w)...}.status;  // (a braced list is evaluated from left to right)
}

}  // namespace

// which: as numbered in the binding.
extern "C" cp_status cp_packed_call(int which, const int64_t *words) {
    if (!words) return CP_ERR_NULL;
    switch (which) {
        case 0: return call(&cp_cache_plan, words);
        case 1: return call(&cp_cache_append_at, words);
        case 2: return call(&cp_cache_keep, words);
        case 3: return call(&cp_tree_plan, words);
        case 4: return call(&cp_tree_attn_fwd, words);
    }
    return CP_ERR_ARGUMENT;
}
