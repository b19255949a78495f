// paged_geom.h -- host-side checks of a paged cache shared by the writers and
// the attention entry points (definitions in dsa_paged_cache_api.cu).
#pragma once

#include "dsa_paged_cache.h"
#include "paged_cache.cuh"

namespace dsa_host {

dsa_status_t check_paged_cache(const dsa_paged_cache_t *c);
// A pool's data and scale pointers against the cache's type.
dsa_status_t check_pool(const dsa_paged_cache_t *c, const void *data, const uint8_t *scale);
dsa::PagedGeom paged_geom(const dsa_paged_cache_t *c);

}  // namespace dsa_host
