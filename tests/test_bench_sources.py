"""bench.py's source hashes cover the kernels that its operators launch (CPU only)."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "rotation_int4_weight_amd", "csrc")
# entry points of the attention benchmarks and the file of their kernel
KERNEL_OF = {"paro_attention_prompt": "attention_prompt.hip", "paro_attention_decode": "attention_decode.hip",
             "paro_kv_append": "kv_pages.hip"}


def test_hashed_files_exist():
    for op, files in bench.KERNEL_FILES.items():
        assert all(os.path.exists(os.path.join(CSRC, f)) for f in files), op


def test_attention_hashes_cover_the_kernels_of_their_steps():
    with open(os.path.join(bench.ROOT, "bench.py")) as f:
        body = re.search(r"def bench_attention\(.*?(?=\ndef )", f.read(), re.S).group(0)
    prompt, decode = body.split("\n    else:\n", 1)
    for op, part in (("attention", prompt), ("attention_decode", decode)):
        called = set(re.findall(r"paro\.(paro_\w+)\(", part)) & set(KERNEL_OF)
        assert called and {KERNEL_OF[c] for c in called} <= set(bench.KERNEL_FILES[op]), (op, called)


def test_included_headers_are_hashed():
    for op in ("attention", "attention_decode"):
        for name in bench.KERNEL_FILES[op]:
            with open(os.path.join(CSRC, name)) as f:
                used = set(re.findall(r'#include "(\w+\.hpp)"', f.read()))
            assert used <= set(bench.KERNEL_FILES[op]), (op, name, used)
