"""The words that tag a slot of the tensor-core scans' ring: those of different launches
keep apart by more than a launch has chunks, and what memory commonly holds is none
of them."""
import shutil
import subprocess

import pytest

from gated_delta_rule_47_gb300 import build

MAIN = r"""
#include "ring_tag.h"
#include <algorithm>
#include <cstdio>
#include <vector>
using U = unsigned long long;
int main() {
    for (U n : {1ULL, 2ULL, 4194304ULL, 1ULL << 37}) printf("%llu\n", gdn::ring_key(n));
    const U k = gdn::ring_key(7), wrap = ~0ULL - 2;  // a key whose counts pass 2^64
    printf("%d %d %d %d %d %d\n", gdn::ring_word_in(k + 5, k + 5, k + 5), gdn::ring_word_in(k + 6, k + 5, k + 5),
           gdn::ring_word_in(k + 4, k + 5, k + 9), gdn::ring_word_in(k + 9, k + 5, k + 9), gdn::ring_word_in(wrap + 6, wrap + 5, wrap + 9),
           gdn::ring_word_in(wrap + 1, wrap + 5, wrap + 9));
    // four million launches of 1024 chunks
    std::vector<U> keys;
    for (U n = 1; n <= 1ULL << 22; ++n) keys.push_back(gdn::ring_key(n));
    std::sort(keys.begin(), keys.end());
    auto tag = [&](U v) {  // whether some launch takes v for one of its own
        auto it = std::upper_bound(keys.begin(), keys.end(), v - 1);
        return v >= 1 && it != keys.begin() && gdn::ring_word_in(v, *(it - 1) + 1, *(it - 1) + 1024);
    };
    long long hits = tag(0);
    for (U b = 0; b < 256; ++b) hits += tag(b * 0x0101010101010101ULL);          // bytes of one kind
    for (U w : {0x7fffffffULL, 0x7fc00000ULL, 0xffc00000ULL, 0xffffffffULL, 0x7fc07fc0ULL, 0xffc0ffc0ULL, 0x7fff7fffULL, 0x3f800000ULL,
                0x3f803f80ULL})
        for (U lo : {w, U(0), U(1), U(3000)}) hits += tag(w << 32 | lo);          // NaN and 1 of either type
    for (U i = 1; i <= 1ULL << 22; ++i)
        for (U lo : {U(0), U(1), U(3000), i, (0 - i) & 0xffffffffULL}) {
            hits += tag(i << 32 | lo);                                          // whole numbers, negative ones among them
            hits += tag((0 - i) << 32 | lo);
        }
    printf("%lld\n", hits);
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_words(tmp_path):
    src, exe = tmp_path / "words.cpp", tmp_path / "words"
    src.write_text(MAIN)
    subprocess.run(["g++", "-O2", "-std=c++17", f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    assert [int(x) for x in lines[:4]] == [n * KEY % 2 ** 64 for n in (1, 2, 4194304, 1 << 37)]
    assert lines[4] == "1 0 0 1 1 0"
    assert lines[5] == "0"


KEY = 0x9E3779B97F4A7C15


def test_keys_keep_apart():
    """The nearest of n multiples of KEY to 0, modulo 2^64, are at denominators of the convergents of KEY / 2^64.  A
    launch has at most 2^25 chunks: 2^31 rows of 64."""
    a, b, before, q = KEY, 2 ** 64, 1, 0
    seen = 0
    while b:
        whole, (a, b) = a // b, (b, a % b)
        before, q = q, whole * q + before
        if 0 < q < 1 << 37:
            seen += 1
            assert min(q * KEY % 2 ** 64, -q * KEY % 2 ** 64) > 1 << 25, q
    assert seen > 30
