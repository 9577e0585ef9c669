// window_bf16.cu -- window attention over bf16 caches (window_mma.cuh).
#include "window_mma.cuh"

namespace kvx {
cudaError_t launch_window_bf16(const WindowMmaParams &p, int blocks, cudaStream_t st) {
  return p.w.c.D == 128 ? wmma::launch_rows<128, false>(p, blocks, st)
                        : wmma::launch_rows<64, false>(p, blocks, st);
}
}  // namespace kvx
