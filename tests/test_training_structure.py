"""The training kernels as they were compiled: loads that go straight into LDS are waited for on every way through a kernel.

A block's LDS is given to the next one when it ends; what is still under way to it then would arrive in the other's."""
import glob
import os
import re
import shutil
import subprocess

import pytest

import broadcast_gemm_amd as bga

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump")) if p and os.path.exists(p)), None)


def kernels(tmp):
    """name -> [(address, instruction, address it jumps to or None)] of the library's training kernels."""
    shutil.copy(bga.LIB_PATH, tmp / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp, check=True, stdout=subprocess.DEVNULL)
    found = {}
    for part in sorted(glob.glob(str(tmp / "lib.so.*gfx950"))):
        names = subprocess.run([OBJDUMP, "--syms", part], check=True, capture_output=True, text=True).stdout
        if "train_" not in names:
            continue
        code = None
        for line in subprocess.run([OBJDUMP, "-d", part], check=True, capture_output=True, text=True).stdout.splitlines():
            head = re.match(r"([0-9a-f]+) <(\S+)>:", line)
            if head:
                code = found.setdefault(head[2], []) if "train_" in head[2] else None
                start = int(head[1], 16)
            elif code is not None and "//" in line:
                text, rest = line.strip().split("//", 1)
                to = re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>", rest)
                code.append((int(rest.split(":")[0], 16), text.strip(), start + int(to[1] or "0", 16) if to else None))
    return found


def ends_before_a_wait(code):
    """Whether a way from the start to an end passes a load into LDS and no wait for all loads after it."""
    at = {a: i for i, (a, _, _) in enumerate(code)}
    seen, todo = set(), [(0, False)]
    while todo:
        i, loaded = todo.pop()
        if (i, loaded) in seen:
            continue
        seen.add((i, loaded))
        _, text, to = code[i]
        name = text.split()[0]
        if name.startswith("s_endpgm"):
            if loaded:
                return True
            continue
        if loaded and name == "s_waitcnt" and "vmcnt(0)" in text:
            continue   # every later load stands in a loop whose turns begin with a wait
        loaded = loaded or name.startswith("global_load_lds")
        if name.startswith(("s_branch", "s_cbranch")):
            assert to in at, text
            todo.append((at[to], loaded))
        if name != "s_branch":
            todo.append((i + 1, loaded))
    return False


def test_the_search_finds_a_way_without_a_wait():
    code = [(0, "s_cbranch_scc0 2", 12), (4, "global_load_lds_dwordx4 v[0:1], off", None), (8, "s_cbranch_vccz 1", 16), (12, "s_waitcnt vmcnt(0)", None),
            (16, "s_endpgm", None)]
    assert ends_before_a_wait(code)
    code[2] = (8, "s_cbranch_vccz 0", 12)
    assert not ends_before_a_wait(code)


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_no_block_ends_with_loads_into_lds_under_way(tmp_path):
    if not os.path.exists(bga.LIB_PATH):
        from broadcast_gemm_amd import build
        build.build()
    code = kernels(tmp_path)
    # Not dQ's: the search does not know that a turn loads nothing if it is the last one.
    staged = [k for k in code if "train_fwd_kernel" in k or "train_dkv_kernel" in k]
    assert len(staged) == 16 and all(any(text.startswith("global_load_lds") for _, text, _ in code[k]) for k in staged)
    assert not [k for k in staged if ends_before_a_wait(code[k])]
