// The rings of a shared prefix's rows and who fills their slots (csa_latent_cuts.h) for the host.
#include "csa_latent_cuts.h"

extern "C" {
void rings_split(int slots, int k_units, int v_units, int least, int *out)
{
    const csa::PairRings r = csa::pair_rings(slots, k_units, v_units, least);
    out[0] = r.k;
    out[1] = r.v;
}
int rings_filler(int slot) { return csa::ring_filler(slot); }
}
