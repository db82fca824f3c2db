"""CPU check of the kernels that begin while the one before on their stream ends:
none of them reads or writes global memory before its wait for that kernel.

A kernel on which another one waits may itself have begun early, so that a write
two kernels back can still be under way when a kernel begins: only its own wait
says that everything before it is there."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gaussian_splatting_differentiable_gs_gb300", "csrc")
WAIT = "wait_for_previous();"


def _source(path):
    text = open(path).read()
    return re.sub(r"//[^\n]*", "", text)


def _block(text, at):
    """End of the brace block that opens at or after `at`."""
    i = text.index("{", at)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return i, j + 1
    raise AssertionError("unbalanced braces")


def _kernels():
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = _source(path)
        if "launch_overlapped" not in text:
            continue
        for m in re.finditer(r"__global__", text):
            head, end = _block(text, m.start())
            sig = text[m.start():head]
            names = re.findall(r"(\w+_kernel)\s*\(", sig)
            assert len(names) == 1, sig
            out.append((os.path.basename(path), names[0], sig, text[head + 1:end - 1]))
    return out


def _reads(code, pointers):
    """Places of `code` that go through a pointer to global memory."""
    found = []
    for p in pointers:
        found += re.findall(r"(?<![\w.>])%s\s*\[[^\]]*\]" % p, code)
        found += re.findall(r"\*\s*%s\b" % p, code)
    found += re.findall(r"\bk\.(?:w_pre|w_post|scale|offsets)\s*\[[^\]]*\]", code)
    found += re.findall(r"\(const [\w]+\*\)\s*k\.gate\)\s*\[[^\]]*\]", code)
    found += re.findall(r"\b(?:group_weight|find_group)\b", code)
    found += re.findall(r"\.(?:fetch|load)\s*\(", code)
    return found


KERNELS = _kernels()


def test_kernels_are_found():
    names = {k[1] for k in KERNELS}
    assert {"rope_kernel", "norm_fwd_kernel", "norm_bwd_kernel", "norm_sums_kernel", "wgrad_kernel",
            "wgrad_join_kernel", "wgrad_terms_kernel", "encode_kernel", "decode_kernel",
            "glu_fwd_kernel", "glu_bwd_kernel"} <= names


@pytest.mark.parametrize("file,name,sig,body", KERNELS, ids=[k[1] for k in KERNELS])
def test_nothing_is_read_before_the_wait(file, name, sig, body):
    if "each_unit(" in body:  # the wait is in there, before the first unit
        inside = _source(os.path.join(CSRC, file))
        at = inside.index("void each_unit(")
        head, end = _block(inside, at)
        assert inside[head:end].index(WAIT) < inside[head:end].index("f(row0")
        body_before = body[:body.index("each_unit(")]
    else:
        assert WAIT in body, "%s does not wait" % name
        # up to the last wait: no path may read before the one that it takes
        body_before = body[:body.rindex(WAIT)]
    pointers = re.findall(r"\*\s*(\w+)\s*[,)]", sig)
    # functions that are only defined so far: what they read counts where they are called
    lazy = {}
    code = body_before
    while True:
        m = re.search(r"auto (\w+) = \[&\]", code)
        if not m:
            break
        head, end = _block(code, m.end())
        lazy[m.group(1)] = code[head:end]
        code = code[:m.start()] + code[end:]
    found = _reads(code, pointers)
    for fn, text in lazy.items():
        if re.search(r"\b%s\s*\(" % fn, code) and _reads(text, pointers):
            found.append("%s()" % fn)
    assert not found, "%s touches global memory before its wait: %s" % (name, found)


@pytest.mark.parametrize("file", sorted({k[0] for k in KERNELS} | {"net_common.cuh"}))
def test_no_loads_of_data_that_never_changes(file):
    """Such loads (__ldg, ld.global.nc, const __restrict__) are for data that nobody writes
    while the kernel runs; what the kernel before writes is not, as that may still run."""
    found = re.findall(r"__ldg|\.nc\b|__restrict__|__ldcs|__ldlu", _source(os.path.join(CSRC, file)))
    assert not found, (file, found)
