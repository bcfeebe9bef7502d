"""Every kernel file that checks computed indexes in the debug build has its flag read by
kvzip_debug_bounds_status, and the files that index through tables and offsets do check."""
import os
import re

from attention_score_reduction_b200 import build

CHECKED = {"score_tc.cu", "select.cu", "select_fused.cu", "compact.cu", "decode.cu", "cache.cu",
           "cache_attention.cu", "cache_attention_tc.cu", "cache_attention_merge.cu"}


def text(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return f.read()


def with_headers(name):
    """The file and the headers it includes, but not in_bounds' own definition."""
    seen, todo, out = set(), [name], ""
    while todo:
        n = todo.pop()
        if n in seen or n == "kvzip_internal.h" or not os.path.exists(os.path.join(build.CSRC, n)):
            continue
        seen.add(n)
        body = text(n)
        out += body
        todo += re.findall(r'#include "([\w.]+)"', body)
    return out


def test_flags_are_set_somewhere_and_read():
    api = text("kvzip_api.cu")
    read = set(re.findall(r"kvzip::(bounds_flag_\w+)", api))
    for name in CHECKED:
        assert name in build.SOURCES
        assert "in_bounds(" in with_headers(name), name
        flag = re.search(r"cudaError_t (bounds_flag_\w+)\(unsigned int\* out\) \{ return take_bounds_flag", text(name))
        assert flag, name
        assert flag.group(1) in read, name
    assert len(read) == len(CHECKED)
