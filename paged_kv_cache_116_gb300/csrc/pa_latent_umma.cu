// pa_latent_umma.cu -- place of the tensor-core form of the latent attention:
// no shape has one so far.
#include "pa_internal.h"

namespace pa {

bool latent_umma_supported(int, int32_t, int32_t, int32_t) { return false; }
size_t latent_umma_workspace(int64_t) { return 0; }
cudaError_t launch_latent_umma(const LatentArgs&, int32_t, void*, std::string*, cudaStream_t) {
    return cudaErrorNotSupported;
}
uint32_t latent_umma_status(bool) { return 0; }

}  // namespace pa
