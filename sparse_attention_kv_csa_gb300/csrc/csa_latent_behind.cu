// The attention by requests (csa_latent_mma.cu) for the rows behind a shared prefix, whose items all leave parts.
#define CSA_BEHIND_PREFIX
#include "csa_latent_mma.cu"

namespace csa {

int latent_behind_slots(const AttnParams &p, int num_sms) { return (int)own_items(prefix_call(p, 0)) + make_plan(p, num_sms).blocks; }

cudaError_t launch_latent_behind(const AttnParams &p, const SharedPlan &s, int num_sms, unsigned *status, cudaStream_t st)
{
    static_assert(kTile == kOwnRows, "");
    return launch_mma<true, 2>(p, s, nullptr, num_sms, status, st);  // (prefixes: values of 128 columns or more)
}

}  // namespace csa
