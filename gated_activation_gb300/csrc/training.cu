// Argument checks shared by the training operators.
#include "training.cuh"

namespace gact {

int check_regions(Region *r, int n) {
    for (int i = 0; i < n; ++i)
        if (r[i].bytes && !r[i].p)
            return GATED_ACT_ERR_NULL;
    for (int i = 0; i < n; ++i)
        if (r[i].bytes && !aligned(r[i].p, r[i].align))
            return GATED_ACT_ERR_ALIGN;
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if ((r[i].write || r[j].write) &&
                ranges_overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes))
                return GATED_ACT_ERR_OVERLAP;
    for (int i = 0; i < n; ++i) {
        r[i].dev = nullptr;
        r[i].host = false;
        if (!r[i].bytes)
            continue;
        const int rc = resolve_ptr(r[i].p, &r[i].dev, &r[i].host);
        if (rc != GATED_ACT_OK)
            return rc;
    }
    return GATED_ACT_OK;
}

}  // namespace gact
