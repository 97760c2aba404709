"""The kernel sources that bench.py's profile digests cover: a header that a
kernel family includes is among them, so that editing it makes older captures
stale."""
import os
import re

import bench

CSRC = "serving_attention_paged_b200/csrc/"
# declarations of the host side, which no kernel's code comes from
HOST_ONLY = {CSRC + "pa_internal.h"}


def _included(path, seen):
    text = open(os.path.join(bench.ROOT, path)).read()
    for name in re.findall(r'^#include "([^"]+)"', text, re.M):
        p = CSRC + name
        if os.path.exists(os.path.join(bench.ROOT, p)) and p not in seen | HOST_ONLY:
            seen.add(p)
            _included(p, seen)
    return seen


def test_digests_cover_every_included_header():
    for family, sources in bench.KERNEL_SOURCES.items():
        # a cascade run's digest covers the decode kernel's sources, too
        covered = set(sources) | set(bench.KERNEL_SOURCES["decode"] if family == "cascade" else ())
        needed = set()
        for s in sources:
            _included(s, needed)
        assert needed <= covered, f"{family}: {sorted(needed - covered)}"
