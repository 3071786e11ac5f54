// nt_tree.cuh -- what the kernels that verify drafted token trees share.
#pragma once

#include "nt_kernels.cuh"

namespace nt {

constexpr int kTreeMaxNodes = 256;
constexpr int64_t kTreeMaxRows = 1 << 20;  // nodes x query heads of one attention call
constexpr int kFaultTree = 5;              // nt_set_test_fault: nt_tree_attention issues no copies

}  // namespace nt
