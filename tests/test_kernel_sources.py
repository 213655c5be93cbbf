"""Rules of the device sources that no run can show: what they guard against reads or writes memory
that belongs to nobody, which seldom faults and changes no result."""

import os
import re

import pytest

import chunked_gated_delta_amd as kda

CSRC = os.path.join(os.path.dirname(kda.__file__), "csrc")


def calls(source, name):
    """The argument lists of all calls of a builtin whose name matches, split at their top-level commas."""
    for m in re.finditer(name + r"\(", source):
        depth, args, start = 1, [], m.end()
        for i in range(m.end(), len(source)):
            c = source[i]
            depth += c in "([{"
            depth -= c in ")]}"
            if (depth == 1 and c == ",") or depth == 0:
                args.append(source[start:i].strip())
                start = i + 1
            if depth == 0:
                break
        yield args


@pytest.mark.parametrize("name,soffset", [("kda_glr.hip", {"load": 2, "store": 3})])
def test_checked_accesses_have_no_scalar_offset(name, soffset):
    """These kernels rely on their descriptors' ends: rows behind the last one are read as zeros and not
    written.  A raw buffer access checks the lane's offset, not the scalar one, against the end."""
    with open(os.path.join(CSRC, name)) as f:
        source = f.read()
    seen = 0
    for kind, at in soffset.items():
        for args in calls(source, rf"__builtin_amdgcn_raw_buffer_{kind}_b\d+"):
            assert args[at] == "0", (name, kind, args)
            seen += 1
    assert seen == 4


def test_a_wait_that_gives_up_leaves_no_number():
    """The search for an entering state is bounded.  Where it ends without one it sets the fault word and
    returns NaN: a zero would be taken for a state."""
    with open(os.path.join(CSRC, "kda_glr.hip")) as f:
        body = re.search(r"float look_back\(.*?\n}\n", f.read(), re.S).group(0)
    fault = body.index("atomicOr(a.faults, FAULT_WAIT_TIMEOUT)")
    assert re.findall(r"return (.*?);", body[fault:]) == ['__builtin_nanf("")']
