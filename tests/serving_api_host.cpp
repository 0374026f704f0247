// The serving operators' C entry points (csa_serving_api.cu) for the host, over launchers and CUDA calls that only keep count: what
// an entry point does when a call below it fails.
#include "csa_launch.h"
#include "csa_serving_launch.h"

#include <stdarg.h>
#include <string.h>

namespace {
struct {
    int shared_result, malloc_result;             // what the fakes answer
    int shared, latent, plain, mallocs, frees, cleared;  // calls
    int last;
} g;
char workspace[16];
}  // namespace

extern "C" {
void fake_reset(int shared_result, int malloc_result)
{
    memset(&g, 0, sizeof(g));
    g.shared_result = shared_result;
    g.malloc_result = malloc_result;
}
void fake_counts(int *out)
{
    const int n[7] = {g.shared, g.latent, g.plain, g.mallocs, g.frees, g.cleared, g.last};
    memcpy(out, n, sizeof(n));
}

cudaError_t cudaMallocFromPoolAsync(void **p, size_t, cudaMemPool_t, cudaStream_t)
{
    ++g.mallocs;
    *p = g.malloc_result ? nullptr : workspace;
    if (g.malloc_result)
        g.last = g.malloc_result;
    return (cudaError_t)g.malloc_result;
}
cudaError_t cudaFreeAsync(void *, cudaStream_t) { return ++g.frees, cudaSuccess; }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError()
{
    const int e = g.last;
    g.last = 0;
    return ++g.cleared, (cudaError_t)e;
}
const char *cudaGetErrorName(cudaError_t) { return "name"; }
const char *cudaGetErrorString(cudaError_t) { return "text"; }
}

namespace csa {
int fail_status(int status, const char *, ...) { return status; }
cudaError_t device_facts(int *sms, cudaMemPool_t *pool, unsigned **status)
{
    if (sms)
        *sms = 152;
    if (pool)
        *pool = nullptr;
    if (status)
        *status = nullptr;
    return cudaSuccess;
}
bool latent_mma_supported(const AttnParams &) { return true; }
size_t latent_mma_workspace(const AttnParams &, int) { return 64; }
cudaError_t launch_latent_mma(const AttnParams &, void *, int, unsigned *, cudaStream_t) { return ++g.latent, cudaSuccess; }
cudaError_t launch_shared_mma(const AttnParams &, const int32_t *, const int32_t *, int, int, cudaMemPool_t, unsigned *, cudaStream_t)
{
    g.last = g.shared_result;
    return ++g.shared, (cudaError_t)g.shared_result;
}
cudaError_t launch_attention_plain(const AttnParams &, cudaStream_t) { return ++g.plain, cudaSuccess; }
bool norm_fwd_whole_vectors(const NormFwdParams &) { return true; }
cudaError_t launch_norm_fwd(const NormFwdParams &, cudaStream_t) { return cudaSuccess; }
cudaError_t norm_bwd_blocks(const NormBwdParams &, int *) { return cudaSuccess; }
cudaError_t launch_norm_bwd(const NormBwdParams &, float *, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_layer_fwd(const LayerFwdParams &, cudaStream_t) { return cudaSuccess; }
cudaError_t layer_bwd_blocks(const LayerBwdParams &, int *) { return cudaSuccess; }
cudaError_t launch_layer_bwd(const LayerBwdParams &, float *, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_append(const AppendParams &, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_page_tables(const PageParams &, int, cudaStream_t) { return cudaSuccess; }
}  // namespace csa
