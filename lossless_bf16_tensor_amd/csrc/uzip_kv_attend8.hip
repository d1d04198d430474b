// uzip_kv_attend8.hip -- attention of drafted tokens over a KV cache in 8 bits
// with a scale for each block of tokens and head (gfx950, wave64). The C-ABI is
// declared in include/uzip_kv.h.
#include "kv_attend.h"

extern "C" int uzip_kv_attend_scaled(const uzip_kv_cache_t *cache, const uzip_kv_scales_t *scales, const uzip_kv_attend_args_t *a,
                                     void *d_ws, uint64_t ws_bytes, hipStream_t s)
{
    return uzip_kv::attend<true>(cache, scales, a, d_ws, ws_bytes, s);
}
