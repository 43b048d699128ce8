"""The rule of csrc/prefix_rule.h, compiled for the host: prefixes are read by every sequence
only where that reads little again, whatever the groups hold."""

import os
import random
import shutil
import subprocess

import pytest

from pass_attention_gb300 import build_lib

CSRC = os.path.join(os.path.dirname(build_lib.__file__), "csrc")
LITTLE = 80 << 20   # where no group is empty
MOST = 256 << 20    # wherever the sequences are
PROBE = r"""
#include <cstdio>
#include "prefix_rule.h"
int main() {
  long long batch, groups, blocks, tokens, bytes;
  while (std::scanf("%lld %lld %lld %lld %lld", &batch, &groups, &blocks, &tokens, &bytes) == 5)
    std::printf("%d\n", oss::read_by_every_sequence(batch, groups, blocks, tokens, bytes) ? 1 : 0);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    d = tmp_path_factory.mktemp("rule")
    (d / "probe.cpp").write_text(PROBE)
    exe = str(d / "probe")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-result", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, str(d / "probe.cpp"), "-o", exe], check=True, capture_output=True, text=True)

    def ask(cases):
        r = subprocess.run([exe], input="".join(" ".join(map(str, c)) + "\n" for c in cases), capture_output=True, text=True,
                           timeout=60)
        assert r.returncode == 0, r.stderr
        return [x == "1" for x in r.stdout.split()]
    return ask


def draw(r):
    batch = r.choice((1, 2, 3, 5, 16, 37, 64, 256, 65535))
    return (batch, r.choice((1, 1, 2, 5, 16, 64, 65, 65535)), r.choice((1, 1, 1, 2, 4, 8, 4096)),
            r.choice((16, 128, 1000, 5024, 65536, 2 ** 20, 2 ** 30)) // r.choice((1, 3)) // 16 * 16 or 16,
            4 * r.choice((1, 2, 8, 16, 65535)) * r.choice((64, 128)))


def again(sizes, blocks, tokens, token_bytes):
    """Bytes that groups of these sizes read a second time and more."""
    return sum(max(n * blocks - 1, 0) for n in sizes) * tokens * token_bytes


def test_groups_that_all_hold_a_sequence(rule):
    r = random.Random(1)
    cases = [c for c in (draw(r) for _ in range(2000)) if c[1] <= c[0]]
    for c, pairs in zip(cases, rule(cases)):
        batch, groups, blocks, tokens, token_bytes = c
        if pairs:
            assert again([1] * (groups - 1) + [batch - groups + 1], blocks, tokens, token_bytes) <= LITTLE, c


def test_groups_of_which_all_but_one_are_empty(rule):
    # slots for 64 groups, one of them in use: 64 sequences behind 65536 tokens of 8 key heads read 17 GB
    assert rule([(64, 64, 1, 65536, 4096), (16, 16, 1, 4000, 4096), (16, 16, 1, 16000, 4096)]) == [False, True, False]
    r = random.Random(2)
    cases = [draw(r) for _ in range(2000)]
    for c, pairs in zip(cases, rule(cases)):
        batch, groups, blocks, tokens, token_bytes = c
        if pairs:
            assert again([batch] + [0] * (min(groups, 9) - 1), blocks, tokens, token_bytes) <= MOST, c


def test_a_block_of_query_heads_reads_by_itself(rule):
    # 16 sequences of 128 query heads over one key head read 4000 tokens of 512 bytes 128 times
    assert rule([(16, 1, 8, 4000, 512), (16, 1, 1, 4000, 512)]) == [False, True]
    assert rule([(1, 1, 8, 65536, 512), (1, 1, 1, 65536, 512), (1, 1, 8, 16000, 512)]) == [False, True, True]


def test_no_size_overflows(rule):
    assert rule([(65535, 1, 4096, 2 ** 30, 4 * 65535 * 128), (65535, 65535, 1, 2 ** 30, 256), (1, 1, 1, 2 ** 30, 512)]) == [False, False, True]
