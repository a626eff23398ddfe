"""Loads of the weight streams that are switched off read nothing, on the CPU.

A switched-off load goes through a descriptor of no bytes. The buffer range check
compares the lane's offset with num_records - scalar offset, in 32 bits: with a
scalar offset beyond num_records the difference may wrap, and every lane would be in
range, the lanes without a token 2^31 bytes past the base. So the scalar offset has to
be zero wherever the descriptor is empty. This evaluates the scalar offset of every
such load as the sources write it, at the step a switched-off load has (0)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "combine_moe_route_03_amd", "csrc")
FILES = ["layer.hip", "gemm_fp8_stream.hip"]
OUTSIDE = 0x80000000


def calls(text):
    """(descriptor, lane offset, scalar offset) of every load16 / load16_stream call."""
    for m in re.finditer(r"\bload16(?:_stream)?\(", text):
        depth, arg, args, i = 1, "", [], m.end()
        while depth:
            ch = text[i]
            depth += (ch in "([{") - (ch in ")]}")
            if depth == 0 or (ch == "," and depth == 1):
                args.append(arg.strip())
                arg = ""
            else:
                arg += ch
            i += 1
        yield tuple(args)


def in_range(lane, scalar, num_records, wraps):
    limit = (num_records - scalar) % (1 << 32) if wraps else max(num_records - scalar, 0)
    return lane < limit


@pytest.mark.parametrize("name", FILES)
def test_switched_off_loads_are_out_of_range(name):
    with open(os.path.join(CSRC, name)) as f:
        found = list(calls(f.read()))
    assert len(found) >= 2
    for desc, lane, scalar in found:
        assert re.search(r"\.at\(", desc), desc
        switch = re.search(r"\.at\((.*)\)$", desc).group(1)
        chosen = re.fullmatch(r"(.+?) \? .+ : (.+)", scalar)  # C's choice by the same switch
        if chosen:
            assert chosen.group(1) == switch
        expr = (chosen.group(2) if chosen else scalar).replace("Step<kFp8>::kCols", "128")
        for p in range(2):  # the pieces of a step
            off = eval(expr, {"__builtins__": {}}, {"s": 0, "p": p})
            for voff in (0, 16, 4096, OUTSIDE):
                for wraps in (False, True):
                    assert not in_range(voff, off, 0, wraps), (desc, lane, scalar)
