"""Copies from memory into LDS through buffer resources that end with the data (source check, no
GPU).  What lies past the end is kept out by the range check, which is sure to count the vector
offset alone: with a place in the scalar or the immediate offset a copy at the edge can read past
its array, which no result shows."""
import glob
import os

import dense_fp32_matrix_f32_amd as sg

CSRC = os.path.join(os.path.dirname(sg.__file__), "csrc")
COPY = "__builtin_amdgcn_raw_ptr_buffer_load_lds("


def arguments(text, start):
    """The arguments of the call whose first one begins at `start`."""
    parts, depth, at = [], 0, start
    for i in range(start, len(text)):
        c = text[i]
        if c == ")" and depth == 0:
            return parts + [text[at:i].strip()]
        depth += (c in "([{") - (c in ")]}")
        if c == "," and depth == 0:
            parts.append(text[at:i].strip())
            at = i + 1
    raise AssertionError("a call that does not end")


def test_a_copys_place_is_its_vector_offset():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            text = f.read()
        at = text.find(COPY)
        while at >= 0:
            resource, to, size, vector, scalar, immediate, _ = arguments(text, at + len(COPY))
            assert (scalar, immediate) == ("0", "0"), (os.path.basename(path), vector, scalar, immediate)
            seen += 1
            at = text.find(COPY, at + 1)
    assert seen >= 4
