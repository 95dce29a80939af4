// The decode forward's kernels over caches of different lengths, bf16.
#include "decode_line.cuh"

namespace ffpa {
namespace line {

template cudaError_t run_line<true>(const LineArgs&, const LinePlan&, const CUtensorMap*, cudaStream_t);
template cudaError_t run_join<true>(const LineArgs&, const LinePlan&, cudaStream_t);

}  // namespace line
}  // namespace ffpa
