// Instances of the chunk attention: softmax, d = 128, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(softmax_d128, kSoftmax, 128)

}  // namespace attend
}  // namespace lssar
