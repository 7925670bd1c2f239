"""The attention side's header and sources stay apart from the FFN's: the FFN's
committed traffic counts go by a hash of the sources they were taken under,
and must not go stale where the attention side alone changes."""

import glob
import json
import os
import re

import bench
from activation_sparse_rank_amd import _lib as L


def _text(*path):
    with open(os.path.join(bench.ROOT, *path)) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def test_exports_match_header():
    declared = sorted(set(re.findall(r"\b(pi_[a-z0-9_]+)\s*\(", _text("include", "pi_attn.h"))))
    assert declared == sorted(L.ATTN_EXPORTS)
    lib = L.load()
    for name in declared:
        assert hasattr(lib, name), name
    assert '#include "pi_attn.h"' in _text("include", "pi.h")


def test_ffn_sources_hold_nothing_of_the_attention_side():
    files = {("include", "pi.h")}
    for path in glob.glob(os.path.join(bench.ROOT, "profiles", "*_traffic.md")):
        data = json.loads(re.search(r"```json\n(.*?)\n```", open(path).read(), re.S).group(1))
        for k in data["kernels"]:
            files |= {("activation_sparse_rank_amd", "csrc", f) for f in bench.kernel_sources(k)}
    for f in sorted(files):
        text = _text(*f)
        for name in (*L.ATTN_EXPORTS, "pi_kv_cache", "AttendArgs", "EvictArgs", "CacheArgs", "RopeArgs"):
            assert not re.search(r"\b%s\b" % name, text), (f, name)
