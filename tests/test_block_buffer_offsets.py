"""The row kernels leave chunks past a row's end to the buffer's bounds check
(no GPU needed: the source is read).

The check of a raw buffer access counts the vector offset and the
instruction's own, not the scalar offset.  A chunk that lies past the row only
by its scalar offset would pass it: rows of 193 to 256 chunks in a wave's body
of five, and every chunk but the first of a dropped slot's empty row."""
import os
import re

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "sparse_moe_routed_amd", "csrc", "row_device.h")


def _arguments(text, at):
    """The arguments of the call whose '(' is at `at`, split at its own commas."""
    depth, args, start = 0, [], at + 1
    for i in range(at, len(text)):
        c = text[i]
        if c in "([{":
            depth += 1
        elif c in ")]}":
            depth -= 1
            if depth == 0:
                return args + [text[start:i].strip()]
        elif c == "," and depth == 1:
            args.append(text[start:i].strip())
            start = i + 1
    raise AssertionError("unbalanced call")


def test_offsets_are_inside_the_bounds_check():
    with open(HEADER) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    calls = list(re.finditer(r"__builtin_amdgcn_raw_buffer_(load|store)_\w+\(", text))
    assert len(calls) >= 7
    for m in calls:
        args = _arguments(text, m.end() - 1)
        # load: resource, offset, scalar offset, cache bits; store: the data before them
        assert args[-2] == "0", text[m.start():m.start() + 120]
