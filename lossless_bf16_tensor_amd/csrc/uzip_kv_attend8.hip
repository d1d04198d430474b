// uzip_kv_attend8.hip -- attention of drafted tokens over a KV cache in 8 bits
// with a scale for each block of tokens and head (gfx950, wave64). The C-ABI is
// declared in include/uzip_kv.h.
#include "kv_attend.h"

extern "C" {

uint64_t uzip_kv_attend_scaled_workspace_bytes(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens,
                                               uint32_t tokens, uint32_t heads)
{
    return uzip_kv::workspace_bytes(seqs, kv_heads, dim, cache_tokens, tokens, heads, true);
}

int uzip_kv_attend_scaled(const uzip_kv_cache_t *cache, const uzip_kv_scales_t *scales, const uzip_kv_attend_args_t *a,
                          void *d_ws, uint64_t ws_bytes, hipStream_t s)
{
    return uzip_kv::attend<true>(cache, scales, a, d_ws, ws_bytes, s);
}

}  // extern "C"
