// Paged cache: attention of a drafted tree's nodes over their context and their ancestors.
// See include/dspark_tree.h for the contract, attend_core.hpp for the mathematics; kernels
// and splits are those of a sequence, with the nodes' keys seen bit by bit in the tiles that
// hold them.
#include "attend_launch.hpp"

namespace dspark {

hipError_t launch_tree_attend(const dspark_cache& C, const AttendArgs& a, hipStream_t s) {
  return launch_attend<true>(C, a, s);
}

}  // namespace dspark
