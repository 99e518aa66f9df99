// Instances of the chunk attention: softmax, d = 64, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(softmax_d64, kSoftmax, 64)

}  // namespace attend
}  // namespace lssar
