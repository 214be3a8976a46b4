"""Kernels that split their registers anew between warpgroups (CPU, static): setmaxnreg is one
instruction for all four warps of a warpgroup, so a kernel may branch on the warpgroup before it and
on the warp only behind it; and what the warpgroups hold afterwards fits what the block was
launched with, or the last of them would wait for ever."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_90_gb300", "csrc")
CALL = re.compile(r"\b(less|more)_registers<(\w+)>\(\)")


def sources():
    out = []
    for name in ("tree_e2m1.cu", "tree_i8.cu"):
        with open(os.path.join(CSRC, name)) as f:
            out.append((name, f.read()))
    return out


def constant(text, name):
    return int(re.search(rf"\b{name} = (\d+)", text).group(1))


@pytest.mark.parametrize("name, text", sources(), ids=lambda x: x if x.endswith(".cu") else "")
def test_a_warpgroup_takes_its_registers_together(name, text):
    """The outermost branches over the roles, evaluated for every warp: each of those that are taken
    sets its registers first, and the warps of a warpgroup take the same one."""
    warps = constant(text, "kThreads") // 32
    lines = text.splitlines()
    branches, calls = [], 0   # (condition or None for the else, the registers it sets)
    for i, line in enumerate(lines):
        head = re.match(r"^  (?:} else )?if \((.*)\) {$", line)
        call = CALL.search(lines[i + 1]) if i + 1 < len(lines) else None
        if call and "void" not in lines[i + 1]:
            assert head or line == "  } else {", f"{name}:{i + 2}: registers are not the first thing of a role"
            branches.append((head.group(1) if head else None, call.group(2)))
            calls += 1
    assert calls == len([m for m in CALL.finditer(text)])   # (none elsewhere)

    def taken(w):
        for k, (cond, _) in enumerate(branches):
            if cond is None or eval(cond.replace("||", " or ").replace("&&", " and "), {}, {"warp": w}):
                return k
        return None
    for w0 in range(0, warps, 4):
        roles = {taken(w) for w in range(w0, w0 + 4)}
        assert len(roles) == 1 and None not in roles, f"{name}: warps {w0} to {w0 + 3} set their registers apart"
    held = [constant(text, branches[taken(w)][1]) for w in range(0, warps, 4)]
    launched = int(re.search(r"launched with (\d+) each", text).group(1))
    assert sum(held) <= launched * len(held)
    assert all(r % 8 == 0 and 24 <= r <= 256 for r in held + [launched])
