// lmc_internal.h -- the layout object shared by the host builder and the
// store/load launchers inside liblmc (not part of the public ABI).
#pragma once

#include <cstdint>
#include <vector>

#include "lmc.h"

struct lmc_layout {
    int64_t block_size = 0;
    int32_t mode = LMC_LAYOUT_PADDED;
    int32_t num_slabs = 0;
    int64_t page_size = 0;
    int64_t block_stride = 0;
    int64_t num_blocks = 0;
    int64_t pool_bytes = 0;
    std::vector<lmc_layer_spec> specs;      // model order
    std::vector<lmc_layer_desc> desc;       // model order
    std::vector<int32_t> kv_group_kind;
    std::vector<int32_t> kv_group_size;
    std::vector<int32_t> object_group_kind;
    // layers of each object group, in model order
    std::vector<std::vector<int32_t>> object_group_layers;
};

namespace lmc {

// Checked 64-bit arithmetic (false on overflow).
inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
inline bool add_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_add_overflow(a, b, out); }

// The rule lmc_copy_blocks checks on the host copy of its pairs before any
// launch: among the pairs whose two block ids lie in the pool, no block is
// the destination of two pairs, nor the destination of one pair and the
// source of another (KV groups share block ids). LMC_OK or LMC_ERR_OVERLAP
// (LMC_ERR_INVALID_ARG when the host pairs are missing). The batch's group
// count and pair counts are checked by the caller.
int check_copy_pairs(const lmc_layout *L, const lmc_copy_batch *b);

// SMs of the current device (cached per device); -1 when CUDA fails.
int sm_count();

// Bytes of one value of an entry type (LMC_E_*); 0 for an unknown one.
inline int entry_elem_bytes(int32_t dtype) {
    return dtype == LMC_E_BF16 || dtype == LMC_E_F16 ? 2 : dtype == LMC_E_E4M3 ? 1 : 0;
}

// The rules every call on a layer's token entries shares: the layer is a
// paged one, its token_bytes hold entry_dim values of the type, the scale and
// the block table are usable. LMC_OK or LMC_ERR_INVALID_ARG.
int check_entries(const lmc_layout *L, const lmc_entries *e);

// A block table's geometry, and its pointer where it will be read.
inline bool table_ok(const lmc_block_table &t, int64_t num_requests) {
    return t.num_cols >= 0 && t.num_cols <= INT32_MAX && t.row_stride >= t.num_cols &&
           (num_requests == 0 || t.num_cols == 0 || (t.table != nullptr && ((uintptr_t)t.table & 3) == 0));
}

}  // namespace lmc
