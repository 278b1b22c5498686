// Shared parts of the 8-bit K/V cache (kv8.cu) and the attention that reads it (kv8_attn.cu).
#pragma once

#include "common.cuh"
#include "fp8.cuh"

namespace tlb {

// Checks a cache's sizes and pointers on the host; `what` names the entry point.
int kv8_check(const tlb_kv8 *cache, const char *what);

// Where the keys of the sequences are.
struct Kv8Pages {
    const int32_t *pages;        // [n_seq, max_pages]
    const int32_t *lengths;      // [n_seq]
    int64_t max_pages;
    int32_t page;
    int32_t max_len;             // min(max_len, max_pages * page): no key from here on
    int32_t shift;               // page = 2^shift, or -1
};

// Keys of sequence b.
__device__ __forceinline__ int kv8_length(const Kv8Pages &p, int64_t b) { return max(0, min(__ldg(p.lengths + b), p.max_len)); }

// Slot of key j of sequence b, or -1 where the cache has none.
__device__ __forceinline__ int64_t kv8_slot(const Kv8Pages &p, int64_t n_slots, int64_t b, int j) {
    const int at = p.shift >= 0 ? j >> p.shift : j / p.page;
    const int64_t slot = int64_t(__ldg(p.pages + b * p.max_pages + at)) * p.page + (j - at * p.page);
    return slot >= 0 && slot < n_slots ? slot : -1;
}

}  // namespace tlb
