// dfc_paged.h - host helpers shared by the paged-cache entry points
// (internal to libdfc).
#pragma once

#include <cstdint>

#include "dfc.h"

namespace dfc {

inline bool is_pow2(uint32_t x) { return x != 0 && (x & (x - 1)) == 0 && x <= (1u << 30); }

inline uint32_t log2_of(uint32_t x) {
    uint32_t s = 0;
    while ((1u << s) < x) ++s;
    return s;
}

// A cache the kernels can address: 16-byte pieces of 8 values everywhere.
inline dfc_status check_cache(const dfc_paged_cache &c) {
    if (!c.k_dev || !c.v_dev) return DFC_EINVAL;
    if ((reinterpret_cast<uintptr_t>(c.k_dev) | reinterpret_cast<uintptr_t>(c.v_dev)) & 15u) return DFC_EINVAL;
    if (!is_pow2(c.page_size) || !c.n_pages || c.n_pages > 0x7fffffffu || !c.kv_heads || c.kv_heads > 65536u)
        return DFC_EINVAL;
    if (!c.head_dim || c.head_dim % 8u) return DFC_EINVAL;
    if (c.dtype != DFC_BF16 && c.dtype != DFC_F16) return DFC_EUNSUPPORTED;
    if (c.head_dim > 256u) return DFC_EUNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (c.k_stride[i] % 8 || c.v_stride[i] % 8 || c.k_stride[i] < 0 || c.v_stride[i] < 0) return DFC_EINVAL;
    return DFC_OK;
}

}  // namespace dfc
