"""The status word's site names one place in the kernels' sources (host only)."""
import glob
import os
import re

import vlm_zigzag_head_gb300

CSRC = os.path.join(os.path.dirname(vlm_zigzag_head_gb300.__file__), "csrc")


def _calls(text, name):
    """The arguments of every call of a function or macro, split at their commas."""
    for m in re.finditer(r"\b%s\(" % name, text):
        depth, at, args = 1, m.end(), [""]
        while depth:
            c = text[at]
            depth += {"(": 1, ")": -1}.get(c, 0)
            if c == "," and depth == 1:
                args.append("")
            elif depth:
                args[-1] += c
            at += 1
        yield [a.strip() for a in args]


def test_every_site_is_one_place():
    """A wait that gave up, or an index outside its tensor, can be traced to its kernel."""
    seen = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        name, text = os.path.basename(path), re.sub(r"//.*", "", open(path).read())
        if name == "check.cuh":     # the definitions
            continue
        for what, where in (("record_timeout", 2), ("CP_IN_RANGE", 4)):
            for args in _calls(text, what):
                for site in re.findall(r"\b\d+\b", args[where]):
                    assert site not in seen, "site %s: %s and %s" % (site, seen[site], name)
                    seen[site] = name
    files = set(seen.values())
    assert {"tc_fwd.cuh", "tc_bwd_q128.cuh", "gemm_bf16.cu", "gemm_split.cu", "ffn_tokens.cu"} <= files
