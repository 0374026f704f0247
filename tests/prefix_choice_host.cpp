// Which way a call with shared prefixes takes (csa_latent_cuts.h) for the host.
#include "csa_latent_cuts.h"

extern "C" {
static csa::PrefixCall call(long long n_tokens, const int *a, long long n_pages)
{
    return csa::PrefixCall{n_tokens, a[0], a[1], a[2], a[3], a[4], a[5] != 0, n_pages, a[6], a[7]};
}
int choice_apart(long long n_tokens, const int *a, long long n_pages, int sms) { return csa::prefix_apart(call(n_tokens, a, n_pages), sms); }
int choice_image_rows(long long n_tokens, const int *a, long long n_pages) { return csa::image_rows(call(n_tokens, a, n_pages)); }
}
