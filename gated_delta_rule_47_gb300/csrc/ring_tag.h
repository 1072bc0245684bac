// ring_tag.h -- the words by which the tensor-core scans' CTAs tell one another how
// far a head's ring is: a slot's "ready" is the launch's key + chunk + 1, a head's
// "taken out" the key + the number of chunks.
//
// A key is the launch's number times 2^64 / golden ratio, modulo 2^64.  Multiples
// of that ratio keep apart as far as points on a circle can: the first 2^37 keys
// (seven months of launches of 0.16 ms), and 0, which a cleared word holds, lie 2^25
// or more apart, and no launch has as many chunks.  So none of those launches takes
// another's word or a cleared one for its own.  Of the 2^64 words that memory may
// have held before, one counts in a slot, and as many as there are chunks in a head's
// count.
#pragma once

namespace gdn {

#ifdef __CUDACC__
#define GDN_BOTH __host__ __device__
#else
#define GDN_BOTH
#endif

GDN_BOTH constexpr unsigned long long ring_key(unsigned long long launch) { return launch * 0x9e3779b97f4a7c15ull; }

// Whether word v is one of first .. last, which may pass 2^64.
GDN_BOTH constexpr bool ring_word_in(unsigned long long v, unsigned long long first, unsigned long long last) {
    return v - first <= last - first;
}

#undef GDN_BOTH

}  // namespace gdn
