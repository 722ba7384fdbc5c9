"""The kernels' sources, read: whoever initialises an mbarrier fences it itself.

fence.mbarrier_init covers the barriers that the executing thread initialised.  A thread that initialises some and leaves
the fence to another one has not ordered them before the bulk copies that complete on them.
"""
import os
import re

from dit_resolution_packed_b200 import _build

FENCE = "fence_mbar_init("


def _strip(src):
    return re.sub(r"//[^\n]*", "", src)


def unfenced(src):
    """Positions of the initialisations that no fence follows in the braces, or the statement, that they stand in."""
    src, bad = _strip(src), []
    for m in re.finditer(r"\bmbar_init\(", src):
        if re.search(r"void\s+$", src[:m.start()]):
            continue  # its definition
        head = src[:m.start()]
        i = m.start()
        # `if (...) mbar_init(...)` without braces is a scope of its own
        lone = re.search(r"\bif\s*\([^{};]*\)\s*$", head)
        scope_end = src.index(";", i) if lone else None
        if scope_end is None:
            # the innermost block that an `if` (a thread's condition) opened
            depth, j = 0, i
            while True:
                j -= 1
                if src[j] == "}":
                    depth += 1
                elif src[j] == "{":
                    if depth:
                        depth -= 1
                    elif re.search(r"\bif\s*\([^{};]*\)\s*$", src[:j]):
                        break
            depth, k = 0, j + 1
            while depth >= 0:
                depth += {"{": 1, "}": -1}.get(src[k], 0)
                k += 1
            scope_end = k
        if FENCE not in src[i:scope_end]:
            bad.append(src.count("\n", 0, i) + 1)
    return bad


def test_the_reading():
    assert unfenced("if (t < n) mbar_init(b + t, 1);\nif (t == 0) {\n fence_mbar_init();\n}") == [1]
    assert unfenced("if (t < n) {\n mbar_init(b + t, 1);\n fence_mbar_init();\n}") == []
    assert unfenced("if (t == 0) {\n for (int s = 0; s < n; ++s) {\n mbar_init(b + s, 1);\n }\n fence_mbar_init();\n}") == []
    assert unfenced("if (t == 0) {\n fence_mbar_init();\n mbar_init(b, 1);\n}") == [3]


def test_every_barrier_is_fenced_by_its_initialiser():
    seen = 0
    for name in _build.SOURCES + _build.HEADERS:
        with open(os.path.join(_build.CSRC, name)) as f:
            src = f.read()
        seen += len(re.findall(r"\bmbar_init\(", _strip(src)))
        assert unfenced(src) == [], name
    assert seen > 20
