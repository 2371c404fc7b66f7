// The stand-in library of step_host.cc with the cache's entry points.
#include "step_host.cc"

extern "C" {
dvl_status dvl_qk_norm_rope(const dvl_qk *, void *s)
{
    event("qk_norm_rope", (uintptr_t)s);
    return DVL_OK;
}
dvl_status dvl_cache_keep(const dvl_kv_cache *, const int32_t *, int64_t, int32_t, const int32_t *,
                          const int32_t *, const int32_t *, int64_t, const int32_t *, int32_t, int32_t,
                          int32_t *, void *s)
{
    event("cache_keep", (uintptr_t)s);
    return DVL_OK;
}
}
