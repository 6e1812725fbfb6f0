/* Host driver for the sanitizer build of the library's argument checks
 * (test_sanitizers.py), as sanitize_abi.c: the operators between the products
 * and those of steps of several tokens, with arguments that must be rejected or
 * that are no-ops, many of them at the ends of their types, so that no call
 * reaches a GPU. Prints "ok" and exits 0 when every status is as expected. */
#include <float.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "w4a16.h"

static int failures = 0;

static void expect(const char *what, int got, int want) {
    if (got != want) {
        printf("FAIL %s: status %d, expected %d (%s)\n", what, got, want, w4a16_last_error());
        ++failures;
    } else if (want != 0 && strlen(w4a16_last_error()) == 0) {
        printf("FAIL %s: no error message\n", what);
        ++failures;
    }
}

enum { OK = 0, INVALID = W4A16_ERR_INVALID_ARG, UNSUPPORTED = W4A16_ERR_UNSUPPORTED, SIZE = W4A16_ERR_SIZE };

/* The calls with one argument or two of interest; the rest are those of 8 kv heads of 128, pages of 64. */
static void *const p = (void *)(uintptr_t)4096; /* never dereferenced */

static int append(int32_t Hq, int64_t ts, int64_t T, int32_t pairs, int64_t pages, int32_t H) {
    return w4a16_kv_append(p, ts, 128, Hq, p, ts, 128, p, ts, 128, p, ts, 128, T, p, p, pairs, 0, p, p, SIZE_MAX, pages, H, 128,
                           64, 0, 0, NULL);
}
static int sinks_size(int64_t B, int64_t width, int64_t window, int64_t sinks, size_t *out) {
    return w4a16_attention_sinks_workspace_size(B, 32, 8, 128, 64, width, window, sinks, 0, out);
}
static int sinks(int64_t B, int64_t width, int64_t ld, int64_t window, int64_t first, float scale, size_t bytes) {
    return w4a16_attention_sinks(p, 4096, 128, B, 32, p, SIZE_MAX, 4, 8, 128, 64, 0, 0, p, width, ld, p, window, first, scale, p,
                                 4096, 128, p, bytes, NULL);
}
static int tokens_size(int64_t T, int64_t B, int32_t Hq, int32_t H, int64_t width, size_t *out) {
    return w4a16_attention_tokens_workspace_size(T, B, Hq, H, 128, 64, width, 1, out);
}
static int tokens(int64_t T, int64_t B, int64_t words, int64_t tree_ld, int64_t window, int64_t first, float scale, size_t bytes) {
    return w4a16_attention_tokens(p, 4096, 128, T, 32, p, B, words ? p : NULL, words, tree_ld, p, SIZE_MAX, 4, 8, 128, 64, 1, 0, p,
                                  2, 2, p, window, first, scale, p, 4096, 128, p, bytes, NULL);
}
static int sample(int64_t M, int64_t V, int64_t ldl, int32_t dtype) {
    return w4a16_sample(p, M, V, ldl, dtype, p, NULL, NULL, NULL, NULL, p, NULL, NULL);
}

int main(void) {
    const int64_t most = INT64_MAX;
    size_t sz = 0, every = 0;
    expect("rmsnorm M=0", w4a16_rmsnorm(p, 0, 64, 64, 0, p, 0.0f, NULL, 0, NULL, 0, p, 64, NULL), OK);
    expect("rmsnorm M", w4a16_rmsnorm(p, INT64_MIN, 64, 64, 0, p, 0.0f, NULL, 0, NULL, 0, p, 64, NULL), INVALID);
    expect("rmsnorm K", w4a16_rmsnorm(p, 2, most, 64, 0, p, 0.0f, NULL, 0, NULL, 0, p, most, NULL), UNSUPPORTED);
    expect("rmsnorm a8 M=0", w4a8_rmsnorm(p, 0, 64, 64, 0, p, 0.0f, NULL, 0, NULL, 0, p, 64, p, NULL), OK);
    expect("rmsnorm a8 dtype", w4a8_rmsnorm(p, 2, 64, 64, 9, p, 0.0f, NULL, 0, NULL, 0, p, 64, p, NULL), INVALID);
    expect("silu_mul M=0", w4a16_silu_mul(p, 0, 64, 128, 0, p, 64, NULL), OK);
    expect("silu_mul ldx", w4a16_silu_mul(p, 2, 64, 127, 0, p, 64, NULL), INVALID);
    expect("silu_mul a8 M=0", w4a8_silu_mul(p, 0, 64, 128, 0, p, 64, p, NULL), OK);
    expect("silu_mul a8 ldx", w4a8_silu_mul(p, 2, 64, 127, 0, p, 64, p, NULL), INVALID);

    expect("cache size", w4a16_kv_cache_size(1000, 8, 128, 64, 1, &sz), OK);
    expect("cache size pages", w4a16_kv_cache_size(most, 8, 128, 64, 0, &sz), UNSUPPORTED);
    expect("cache size all", w4a16_kv_cache_size(((int64_t)1 << 31) - 1, 1 << 16, 256, 1 << 16, 0, &sz), UNSUPPORTED);
    expect("cache size heads", w4a16_kv_cache_size(4, INT32_MIN, 128, 64, 0, &sz), INVALID);
    expect("kv_write T=0", w4a16_kv_write(p, 128, 128, p, 128, 128, 0, p, p, SIZE_MAX, 4, 8, 128, 64, 0, 0, NULL), OK);
    expect("kv_write T", w4a16_kv_write(p, 128, 128, p, 128, 128, most, p, p, SIZE_MAX, 4, 8, 128, 64, 0, 0, NULL), UNSUPPORTED);
    expect("kv_write ts", w4a16_kv_write(p, most, 128, p, 128, 128, 2, p, p, SIZE_MAX, 4, 8, 128, 64, 0, 0, NULL), UNSUPPORTED);
    expect("kv_read T=0", w4a16_kv_read(p, 0, p, SIZE_MAX, 4, 8, 128, 64, 0, 0, p, 128, 128, p, 128, 128, NULL), OK);
    expect("kv_read bytes", w4a16_kv_read(p, 2, p, 16, 4, 8, 128, 64, 0, 0, p, 128, 128, p, 128, 128, NULL), SIZE);

    expect("append T=0", append(32, 6144, 0, 64, 4, 8), OK);
    expect("append T", append(32, 6144, most, 64, 4, 8), UNSUPPORTED);
    expect("append T, heads", append(1 << 20, 6144, (int64_t)1 << 30, 64, 4, 1 << 16), UNSUPPORTED);
    expect("append T < 0", append(32, 6144, INT64_MIN, 64, 4, 8), INVALID);
    expect("append q_heads", append(INT32_MAX, 6144, 4, 64, 4, 8), UNSUPPORTED);
    expect("append pairs", append(32, 6144, 4, INT32_MAX - 7, 4, 8), UNSUPPORTED);
    expect("append pairs < 0", append(32, 6144, 4, INT32_MIN, 4, 8), UNSUPPORTED);
    expect("append ts", append(32, most, 4, 64, 4, 8), UNSUPPORTED);
    expect("append pages", append(32, 6144, 4, 64, most, 8), UNSUPPORTED);

    expect("attention size", w4a16_attention_workspace_size(1, 32, 8, 128, 64, 64, 0, 0, &every), OK);
    expect("attention size B", w4a16_attention_workspace_size(most, 32, 8, 128, 64, 64, 0, 0, &sz), UNSUPPORTED);
    expect("attention size width", w4a16_attention_workspace_size(1, 32, 8, 128, 64, most, 0, 0, &sz), UNSUPPORTED);
    expect("attention workspace", w4a16_attention(p, 4096, 128, 1, 32, p, SIZE_MAX, 4, 8, 128, 64, 0, 0, p, 64, 64, p, most, 0.1f, p,
                                                  4096, 128, p, every - 1, NULL), SIZE);
    expect("sinks size", sinks_size(1, 64, most, 4, &sz), OK);
    expect("sinks size, same", sz == every ? OK : -1, OK);
    expect("sinks size ends", sinks_size(1, 64, most, most, &sz), OK);
    expect("sinks size ends, same", sz == every ? OK : -1, OK);
    expect("sinks size window", sinks_size(1, 64, INT64_MIN, 4, &sz), INVALID);
    expect("sinks size sinks", sinks_size(1, 64, 4, INT64_MIN, &sz), INVALID);
    expect("sinks size NULL", sinks_size(1, 64, 4, 4, NULL), INVALID);
    expect("sinks B=0", sinks(0, 64, 64, most, most, 0.1f, 0), OK);
    expect("sinks workspace", sinks(1, 64, 64, most, most, 0.1f, every - 1), SIZE);
    expect("sinks table_ld", sinks(2, 64, most, 4, 4, 0.1f, SIZE_MAX), UNSUPPORTED);
    expect("sinks scale", sinks(2, 64, 64, 4, 4, 2 * FLT_MAX, SIZE_MAX), INVALID);

    expect("tokens size", tokens_size(100, 2, 32, 8, 64, &every), OK);
    expect("tokens size T=0", tokens_size(0, 2, 32, 8, 64, &sz), OK);
    expect("tokens size T", tokens_size(most, 2, 32, 8, 64, &sz), UNSUPPORTED);
    expect("tokens size rows", tokens_size((int64_t)1 << 31, 2, INT32_MAX, 1, 64, &sz), UNSUPPORTED);
    expect("tokens size T < 0", tokens_size(INT64_MIN, 2, 32, 8, 64, &sz), INVALID);
    expect("tokens size B", tokens_size(100, most, 32, 8, 64, &sz), UNSUPPORTED);
    expect("tokens size heads", tokens_size(100, 2, INT32_MIN, 8, 64, &sz), INVALID);
    expect("tokens size NULL", tokens_size(100, 2, 32, 8, 64, NULL), INVALID);
    expect("tokens T=0", tokens(0, 2, 1, 1, most, most, 0.1f, 0), OK);
    expect("tokens B=0", tokens(100, 0, 0, 0, most, most, 0.1f, 0), OK);
    expect("tokens words", tokens(100, 2, most, most, 4, 4, 0.1f, SIZE_MAX), INVALID);
    expect("tokens words < 0", tokens(100, 2, INT64_MIN, 1, 4, 4, 0.1f, SIZE_MAX), INVALID);
    expect("tokens tree_ld", tokens(100, 2, 2, 1, 4, 4, 0.1f, SIZE_MAX), INVALID);
    expect("tokens window", tokens(100, 2, 0, 0, INT64_MIN, 4, 0.1f, SIZE_MAX), INVALID);
    expect("tokens sinks", tokens(100, 2, 0, 0, 4, INT64_MIN, 0.1f, SIZE_MAX), INVALID);
    expect("tokens scale", tokens(100, 2, 0, 0, 4, 4, -2 * FLT_MAX, SIZE_MAX), INVALID);
    expect("tokens workspace", tokens(100, 2, 1, 1, most, most, 0.1f, 64), SIZE);

    expect("sample M=0", sample(0, 100, 100, 0), OK);
    expect("sample M", sample(most, 100, 100, 0), UNSUPPORTED);
    expect("sample M < 0", sample(INT64_MIN, 100, 100, 0), INVALID);
    expect("sample V", sample(4, most, most, 0), UNSUPPORTED);
    expect("sample V < 0", sample(4, INT64_MIN, 100, 0), INVALID);
    expect("sample ldl", sample(4, 100, most, 0), UNSUPPORTED);
    expect("sample dtype", sample(4, 100, 100, INT32_MIN), INVALID);
    if (failures == 0) printf("ok\n");
    return failures == 0 ? 0 : 1;
}
