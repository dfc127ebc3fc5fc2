"""Register splits (setmaxnreg): all warps of a warpgroup have to reach the same
instruction, so every branch around one must depend on the warpgroup alone.
Read off the sources; no GPU needed."""
import glob
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "bit_quantized_kv_decode_gb300", "csrc")
CALL = re.compile(r"\bsetmaxnreg_(?:inc|dec)<")


def strip(text):
    return re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)


def open_brace(text, close):
    depth = 0
    for i in range(close, -1, -1):
        depth += (text[i] == "}") - (text[i] == "{")
        if depth == 0:
            return i
    raise AssertionError("unbalanced braces")


def header(text, brace):
    """What stands between a block's opening brace and the statement before it."""
    start = max(text.rfind(c, 0, brace) for c in ";{}")
    return start, " ".join(text[start + 1:brace].split())


def conditions(text, at):
    """Conditions of the branches around position `at`, those of the branches
    that an else belongs to among them; a branch without braces is its line's."""
    found = re.findall(r"\bif (?:constexpr )?\((.*)\) *$", text[text.rfind("\n", 0, at):at])
    depth, i = 0, at
    while i >= 0:
        i -= 1
        c = text[i]
        if c == "}":
            depth += 1
        elif c == "{" and depth:
            depth -= 1
        elif c == "{":
            start, head = header(text, i)
            if head.startswith(("if", "else")):
                found += re.findall(r"\bif (?:constexpr )?\((.*)\)", head)
                while head.startswith("else"):
                    start, head = header(text, open_brace(text, start))
                    found += re.findall(r"\bif (?:constexpr )?\((.*)\)", head)
            elif head.endswith(")") or "__global__" in head or "__device__" in head:
                if "__global__" in head or "__device__" in head:
                    break
    return set(found)


# Conditions that a warpgroup's four warps evaluate alike: constants of the
# instance, arguments, the CTA's range, and bounds that are multiples of four warps.
ALIKE = {"D <= 128", "tile >= 0", "s1 > s0", "warp < kSoftWarps", "warp >= (NT == 2 ? 8 : 4)", "warp >= kWarpLoad",
         "warp < kWarpSoftmax0"}


def calls():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = strip(open(path).read())
        for m in CALL.finditer(text):
            yield pytest.param(text, m.start(), id=f"{os.path.basename(path)}:{text[:m.start()].count(chr(10)) + 1}")


@pytest.mark.parametrize("text,at", list(calls()))
def test_branches_around_a_register_split(text, at):
    assert conditions(text, at) <= ALIKE


def test_the_bounds_are_whole_warpgroups():
    chunk = open(os.path.join(CSRC, "chunk_attn.cuh")).read()
    assert re.search(r"\bkSoftWarps = 4 \* NT\b", chunk)
    decode = open(os.path.join(CSRC, "decode.cuh")).read()
    values = dict(re.findall(r"constexpr int (kWarp\w+) = (\d+);", decode))
    for name in ("kWarpLoad", "kWarpSoftmax0"):
        assert int(values[name]) % 4 == 0, name


def test_a_split_on_two_paths_is_seen():
    """The checker itself, on a warpgroup whose warps split on two paths."""
    text = "__global__ void k() { if (warp < kSoftWarps) { a(); } else if (dq >= 0) { b(); } else { setmaxnreg_dec<56>(); } }"
    assert conditions(text, text.index("setmaxnreg")) == {"warp < kSoftWarps", "dq >= 0"}
