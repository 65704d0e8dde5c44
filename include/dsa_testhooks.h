/*
 * dsa_testhooks.h -- the extra entry points of the TEST build of the library,
 * libdsa_testhooks.so (the same sources compiled with -DDSA_TEST_HOOKS).  The product library
 * libdsa.so does not export them.  The pages have no counterpart: they exist so that the
 * failure handling of the kernels can be exercised without faulting or hanging a GPU.
 *
 * In the test build every bounded device-side wait gives up after 20 ms (1 s in the product).
 *
 * dsa_test_inject_stall(kernel): from the next launch on, the MMA-issuing thread (or its warp) of
 * the first CTA of the chosen kernel (1: the indexer, dsa_li_topk; 2: sparse attention,
 * dsa_sfa_decode / dsa_sfa_prefill; 3: dsa_mla_decode; 4: dsa_mla_prefill; 0: none) first waits on
 * an mbarrier that no thread ever arrives on.  That wait runs out, the CTA raises its abort flag, the kernel stores
 * DSA_ERR_TIMEOUT into *status, the other roles of the CTA (and of its cluster) leave their
 * loops through their own bounded waits, every issued copy is drained, tensor memory is
 * freed, and the launch completes: the next call on the same context works.  The output of the
 * stalled launch is unspecified.  Host-side state, not thread-safe; a test setting.
 * With 5 to 9 that CTA leaves a load out instead, so that what waits for its bytes gives up: 5 and 6 the
 * first keys and the first values of dsa_mla_decode over a bf16 cache, 7, 8 and 9 the first keys, the first
 * values and the queries of dsa_mla_prefill.
 *
 * dsa_test_mla_visible_columns(): on the host, with host pointers, the rule by which dsa_mla_decode's
 * softmax decides how many of a page's 64 positions a query row may use, lookup of the page id
 * included.  `pages` is the sequence's row of the page table, pos0 the page's first position.
 */
#ifndef DSA_TESTHOOKS_H
#define DSA_TESTHOOKS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

void dsa_test_inject_stall(int kernel);
int dsa_test_mla_visible_columns(int owned, int seen, int pos0, int check_pages, const int32_t* pages,
                                 int num_pages);

#ifdef __cplusplus
}
#endif

#endif /* DSA_TESTHOOKS_H */
