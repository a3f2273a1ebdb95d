"""How attention cuts a long context into spans, on the host from the header that both sides share: enough spans for all keys, none
without keys, no more than the workspace has room for, up to the most keys that a call takes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
MOST = (1 << 31) - 1025
KEYS = sorted({1, 2, 511, 512, 513, 1024, 1025, 20000, 70001, 131072, 1 << 30, (1 << 30) + 1, 2113929215, 2113929216, 2113929217, MOST - 1, MOST}
              | {(512 << i) + e for i in range(22) for e in (-1, 0, 1)})
DRIVER = r"""
#include <cstdio>
#include "gdn_attention_internal.h"
int main() {
    int rows; long long keys;
    while (std::scanf("%d %lld", &rows, &keys) == 2) {
        const int span = gdn::span_keys(rows, (int)keys);
        std::printf("%d %d %d %d\n", gdn::least_span(rows), span, gdn::span_count((int)keys, span), gdn::most_spans(rows, keys));
    }
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")),
                    reason="g++ or the HIP headers not found")
def test_spans(tmp_path):
    src, exe = tmp_path / "spans.cpp", tmp_path / "spans"
    src.write_text(DRIVER)
    built = subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"), "-I", "include", "-I",
                            "gated_deltanet_rule_amd/csrc", str(src), "-o", str(exe)], capture_output=True, text=True, cwd=ROOT)
    assert built.returncode == 0, built.stderr
    asked = [(rows, keys) for rows in (1, 16, 64, 65, 128, 4096) for keys in KEYS]
    ran = subprocess.run([str(exe)], input="\n".join("%d %d" % a for a in asked), capture_output=True, text=True, timeout=60)
    got = [tuple(map(int, line.split())) for line in ran.stdout.splitlines()]
    assert len(got) == len(asked)
    before = {}
    for (rows, keys), (least, span, spans, most) in zip(asked, got):
        assert span >= least and span % least == 0, (rows, keys)
        assert 1 <= spans <= most <= 64, (rows, keys, spans, most)
        assert (spans - 1) * span < keys <= spans * span, (rows, keys, span, spans)
        assert most == min(64, -(-keys // least)), (rows, keys, most)
        assert most >= before.get(rows, 0)
        before[rows] = most
