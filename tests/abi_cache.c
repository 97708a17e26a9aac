/*
 * The paged cache's part of include/rcodec.h from a plain C99 program (test
 * infrastructure), built and run by tests/test_c_cache.py as tests/abi_consumer.c is:
 * the layout of rc_cache, which other languages fill in as eleven 64-bit words, and
 * the statuses of calls that end before any HIP call.  Exit status 0 = every check held.
 */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "rcodec.h"

static int failures = 0;

static void check(int cond, const char *what)
{
    if (!cond) {
        fprintf(stderr, "FAIL: %s\n", what);
        ++failures;
    }
}

int main(void)
{
    /* never dereferenced: validation rejects the call before any access */
    void *const even = (void *)(uintptr_t)0x1000, *const odd = (void *)(uintptr_t)0x1008;
    const int32_t *const ints = (const int32_t *)even;
    const rc_cache good = {even, even, 4, 16, 2, 128, ints, 2, 4, ints, ints};
    rc_cache bad = good;

    check(sizeof(rc_cache) == 88, "rc_cache: eleven words");
    check(offsetof(rc_cache, k) == 0 && offsetof(rc_cache, v) == 8, "k, v");
    check(offsetof(rc_cache, pages) == 16 && offsetof(rc_cache, page) == 24, "pages, page");
    check(offsetof(rc_cache, kv_heads) == 32 && offsetof(rc_cache, d) == 40, "kv_heads, d");
    check(offsetof(rc_cache, table) == 48 && offsetof(rc_cache, seqs) == 56, "table, seqs");
    check(offsetof(rc_cache, max_pages) == 64 && offsetof(rc_cache, lengths) == 72, "max_pages, lengths");
    check(offsetof(rc_cache, offsets) == 80, "offsets");

    check(rc_mxfp4_cache_append(NULL, RC_DT_BF16, 3, even, 256, even, 256, 0, NULL, 0, NULL, NULL, 0, 0, 0, NULL) ==
              RC_ERR_NULL, "append: null cache");
    check(rc_mxfp4_cache_append(&good, RC_DT_BF16, 0, NULL, 0, NULL, 0, 4, NULL, 0, NULL, NULL, 0, 0, 0, NULL) == RC_OK,
          "append: no tokens");
    check(rc_mxfp4_cache_append(&good, RC_DT_BF16, 3, even, 256, even, 256, 4, even, 512, even, NULL, 0, 0, 0, NULL) ==
              RC_ERR_UNSUPPORTED, "append: in place");
    check(rc_mxfp4_cache_append(&good, RC_DT_BF16, 3, odd, 256, even, 256, 0, NULL, 0, NULL, NULL, 0, 0, 0, NULL) ==
              RC_ERR_ALIGN, "append: misaligned keys");
    check(rc_mxfp4_cache_read(&good, 3, RC_DT_BF16, NULL, even, NULL) == RC_ERR_NULL, "read: null output");
    check(rc_mxfp4_cache_read(&good, 3, (rc_dtype)7, even, even, NULL) == RC_ERR_UNSUPPORTED, "read: dtype");
    check(rc_mxfp4_cache_attention(&good, RC_DT_BF16, 3, 4, even, 512, 0.1f, 0, 5, 0, odd, NULL, even, NULL) ==
              RC_ERR_UNSUPPORTED, "attention: a window without causal");
    check(rc_mxfp4_cache_attention(&good, RC_DT_BF16, 3, 4, even, 512, 0.1f, 1, 5, 0, odd, NULL, even, NULL) ==
              RC_ERR_ALIGN, "attention: misaligned output");
    check(rc_mxfp4_cache_attention(&good, RC_DT_BF16, 3, 5, even, 512, 0.1f, 1, 0, 0, even, NULL, even, NULL) ==
              RC_ERR_RANGE, "attention: heads that the cache's do not divide");
    bad.d = 80;
    check(rc_mxfp4_cache_read(&bad, 3, RC_DT_BF16, even, even, NULL) == RC_ERR_RANGE, "width");
    bad = good;
    bad.page = 24;
    check(rc_mxfp4_cache_read(&bad, 3, RC_DT_BF16, even, even, NULL) == RC_ERR_RANGE, "page");
    bad = good;
    bad.seqs = RC_MAX_SEQS + 1;
    check(rc_mxfp4_cache_read(&bad, 3, RC_DT_BF16, even, even, NULL) == RC_ERR_RANGE, "sequences");
    bad = good;
    bad.lengths = NULL;
    check(rc_mxfp4_cache_read(&bad, 3, RC_DT_BF16, even, even, NULL) == RC_ERR_NULL, "lengths");
    check(rc_mxfp4_cache_attention_workspace(3, 4, 2, 128) > 0, "workspace");
    check(rc_mxfp4_cache_attention_workspace(3, 5, 2, 128) == 0, "workspace: refused sizes");

    if (failures) {
        fprintf(stderr, "%d failures\n", failures);
        return 1;
    }
    printf("C consumer: all checks held\n");
    return 0;
}
