"""A tcgen05.ld writes its registers until tcgen05.wait::ld: both stand in one asm statement, since arithmetic that
reads only the registers may be scheduled between two (CPU: the sources are read)."""
import os
import re

import paged_kv_cache_121_gb300 as pa


def test_every_load_from_tensor_memory_waits_in_its_own_statement():
    csrc = os.path.join(os.path.dirname(pa.__file__), "csrc")
    found = 0
    for name in sorted(os.listdir(csrc)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
            depth, end = 1, m.end()
            while depth:                       # to the statement's closing parenthesis
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            body = text[m.end():end]
            if "tcgen05.ld." in body:
                found += 1
                assert body.find("tcgen05.wait::ld") > body.find("tcgen05.ld."), (name, text[:m.start()].count("\n") + 1)
    assert found >= 3
