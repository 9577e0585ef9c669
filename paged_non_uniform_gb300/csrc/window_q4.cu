// window_q4.cu -- window attention over 4-bit caches (window_mma.cuh).
#include "window_mma.cuh"

namespace kvx {
cudaError_t launch_window_q4(const WindowMmaParams &p, int blocks, cudaStream_t st) {
  return p.w.c.D == 128 ? wmma::launch_rows<128, true>(p, blocks, st)
                        : wmma::launch_rows<64, true>(p, blocks, st);
}
}  // namespace kvx
