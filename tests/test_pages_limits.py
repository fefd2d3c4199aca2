"""Upkeep of paged caches at the ends of its stated ranges: the arithmetic of
its plans, on the CPU."""
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_softmax_attention_04_b200", "csrc")

# The plan of attn_pages_reserve with the kernel's own functions, a block's sums
# included: lines of "pages free n" and n needs in, what is granted and where out.
PLAN = r"""
#include <cstdio>
#include <vector>
#include "attn_pages_kernel.cuh"
using namespace attn_sm100;
int main()
{
    long pages, free_pages, n;
    while (std::scanf("%ld %ld %ld", &pages, &free_pages, &n) == 3) {
        std::vector<int> need(n), first(n);
        int64_t before = 0;
        for (long base = 0; base < n; base += PLAN_THREADS) {
            int32_t upto = 0;  // as plan_scan: in 32 bits
            for (long i = base; i < n && i < base + PLAN_THREADS; ++i) {
                std::scanf("%d", &need[i]);
                first[i] = reserve_first(before + upto, static_cast<int>(pages));
                upto = static_cast<int32_t>(static_cast<uint32_t>(upto) + reserve_ask(need[i], static_cast<int>(pages)));
            }
            before += upto;
        }
        const int64_t wanted = before < pages ? before : pages;
        const int found = static_cast<int>(wanted < free_pages ? wanted : free_pages);
        for (long i = 0; i < n; ++i) std::printf("%d:%d ", reserve_met(need[i], first[i], found) ? 1 : 0, first[i]);
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from exact_softmax_attention_04_b200 import build_lib
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cu", d / "plan"
    src.write_text(PLAN)
    subprocess.check_call([build_lib._nvcc(), "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I", CSRC,
                           "-o", str(exe), str(src)])

    def run(cases):
        text = "\n".join(f"{p} {f} {len(needs)} " + " ".join(map(str, needs)) for p, f, needs in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [[tuple(map(int, x.split(":"))) for x in line.split()] for line in out.splitlines()]

    return run


def met(free, needs):
    """In whole numbers: a request is met while the free pages suffice for all
    up to it; -1 is a request that is not valid."""
    granted, asked = [], 0
    for n in needs:
        asked += max(n, 0)
        granted.append(int(n == 0 or (n > 0 and asked <= free)))
    return granted


def test_reserve_counts_up_to_the_largest_pool(plan):
    top = (1 << 21) - 1  # pages: the limit
    rng = random.Random(1)
    cases = [(top, top, [top + 1] * 1024 + [1]), (top, top, [1 << 30] * 1024 + [top, 0, 1]),
             (top, top, [top] * 1025), (top, 7, [-1] * 3 + [5, 0, 3, 2, 1, 0]), (top, 0, [0, 1, 0]),
             (1, 1, [1, 1, 0]), (top, top - 1, [top - 1, 1, 0])]
    for _ in range(60):
        p = rng.choice([1, 9, 5000, top])
        n = rng.choice([3, 40, 1024, 3000])
        cases.append((p, rng.randint(0, p), [rng.choice([-1, 0, 1, rng.randint(0, 9), p, p + 1, 2 ** 31 - 1]) if rng.random() < 0.1
                                             else rng.randint(0, 3) for _ in range(n)]))
    for (p, free, needs), got in zip(cases, plan(cases), strict=True):
        want = met(free, needs)
        assert [g for g, _ in got] == want
        at = 0
        for n, (g, first) in zip(needs, got):
            if g and n > 0:  # its pages lie in the list
                assert first == at and 0 <= first and first + n <= free
            at += max(n, 0)


FAKE = 0x10000  # 16-byte aligned, never dereferenced
MANY = (1 << 30) + 1


@pytest.fixture(scope="module")
def attn():
    from exact_softmax_attention_04_b200 import build_lib
    build_lib.build()
    import exact_softmax_attention_04_b200 as pkg
    return pkg


@pytest.mark.parametrize("n,rows,width", [(MANY, 8, 8), (4, MANY, 8), (4, 8, MANY), (4, 8, 2 ** 31 - 1)])
def test_sizes_that_32_bit_loops_cannot_count_are_refused(attn, n, rows, width):
    """The kernels step through requests, rows and a row's entries in strides of
    up to 1024, in 32 bits."""
    lib = attn.lib()
    p, big = FAKE, 1 << 50
    assert lib.attn_pages_reserve(p, p, p, p, p, p, big, n, rows, 64, 16, width, None) == 2
    assert lib.attn_pages_fork(p, p, None, p, p, p, p, p, p, p, p, big, n, rows, 2, 64, 16, width, 128, None) == 2
    assert lib.attn_pages_free(p, p, p, p, n, rows, 64, width, None) == 2
    if width == 8:
        with pytest.raises(ValueError):
            attn.pages_workspace_bytes(n, rows, 64)


def test_compacting_has_no_limit_on_rows(attn):
    assert attn.pages_workspace_bytes(0, MANY, 64) > 4 * MANY
