// The attention's division of work (csa_latent_cuts.h) for the host.
#include "csa_latent_cuts.h"

extern "C" {
long long cuts_cut(long long total, int c, int g) { return csa::cut(total, c, g); }
int cuts_holder(long long unit, long long total, int g) { return csa::holder(unit, total, g); }
int cuts_sharing(long long total, int blocks) { return csa::sharing(total, blocks); }
int cuts_head() { return csa::kHead; }
int cuts_least() { return csa::kMinUnits; }
// take, t0, t1; returns whether the item falls to the block
int cuts_segment(int nt, int off, long long left, int *out)
{
    const csa::Segment s = csa::segment_of(nt, off, left);
    out[0] = s.take;
    out[1] = s.t0;
    out[2] = s.t1;
    return s.some;
}
unsigned cuts_quotient(unsigned n, unsigned d) { return csa::Divider(d).quotient(n); }
unsigned cuts_remainder(unsigned n, unsigned d) { return csa::Divider(d).remainder(n); }
}
