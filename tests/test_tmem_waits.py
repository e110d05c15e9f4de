"""Loads from Tensor Memory fill their registers some time after the instruction: each has to be waited for, and the wait has to name the
registers, or the compiler may move what uses them ahead of it.  Checked in the sources: on the GPU such a move shows only if it
happens."""
import glob
import os
import re

import pytest

from attention_tensor_cores_gb300 import build as B

FILES = sorted(glob.glob(os.path.join(B.CSRC, "*.cu*")))
CALL = re.compile(r"(?<![\w(])(tmem_ld(?:16|32p?|_wait)?(?:<[^;<>]*>)?)\(([^;{}]*)\);")


def code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def register(expression):
    """The array of `ov`, or of `su + c4 * 32`."""
    return re.match(r"\s*(\w+)", expression).group(1)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_waits_name_the_registers(path):
    loaded = set()
    for name, args in CALL.findall(code(path)):
        if re.match(r"tmem_ld_wait", name):
            named = {register(a) for a in args.split(",")} if args.strip() else set()
            assert loaded <= named and named, f"{name}({args}) does not name {loaded - named or 'any register'}"
            loaded = set()
        elif not args.startswith(("uint32_t ", "taddr,")):     # not a definition, nor tmem_ld's own branches
            loaded.add(register(args.rsplit(",", 1)[1]))
    assert not loaded, f"no wait for {loaded}"


def test_one_wait_instruction():
    """No other place waits for such loads, and none can without registers."""
    assert {os.path.basename(p): code(p).count("tcgen05.wait::ld") for p in FILES if "tcgen05.wait::ld" in code(p)} == {"ptx.cuh": 1}
    assert "tmem_ld_wait()" not in "".join(map(code, FILES))
