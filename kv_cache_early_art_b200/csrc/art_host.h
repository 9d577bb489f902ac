// art_host.h -- host-side argument-check helpers shared by the entry points.
#pragma once

#include <cstdint>

#include "../../include/art.h"

namespace art_host {

inline bool is_null(const art_tensor_t *t) { return t == nullptr || t->data == nullptr; }

inline int64_t elem_size(int32_t dt) { return dt == ART_BF16 ? 2 : 4; }

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether no two elements of a tensor share an address, as a tensor that is
// written needs it: by strides from the smallest up, each dimension's steps clear
// the span of those before it.  (Every slice or permutation of a dense tensor
// does; layouts that weave two dimensions into one another are turned down.)
inline bool apart(const art_tensor_t &t)
{
    bool done[4] = {false, false, false, false};
    __int128 span = 1;
    for (int n = 0; n < t.ndim; ++n) {
        int least = -1;
        for (int i = 0; i < t.ndim; ++i)
            if (!done[i] && (least < 0 || t.stride[i] < t.stride[least]))
                least = i;
        done[least] = true;
        if (t.shape[least] <= 1)
            continue;
        if (t.stride[least] < span)
            return false;
        span += (__int128)t.stride[least] * (t.shape[least] - 1);
    }
    return true;
}

// The smallest workspace (a ring of 16 block states per unit) with which
// art_decode_attention_ex runs p with merge_cta = 2, whatever p's merge_cta
// and workspace hold; a negative art_status_t when the arguments are invalid
// or that walk is not built for them.  Nothing is launched.
int64_t gr_min_workspace_bytes(const art_params_t *p);

}  // namespace art_host
