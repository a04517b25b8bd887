// window.cu -- rows under sinks and a sliding window: the forms of window.cuh.
#include "window.cuh"

namespace sfi {

cudaError_t launch_window(const WindowParams &p, int rows, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                          const CUtensorMap &tm_q, int grid, cudaStream_t stream)
{
    return launch_rows<false>(p, rows, p.n_split > 1, tm_k, tm_v, tm_q, grid, stream);
}

}  // namespace sfi
