"""The tiled 4-bit product's sums, in the library as it is built.  Its matrix instructions
stand in inline assembly, so the compiler does not know how long their results take: on no way
through the kernel may another instruction touch a sum's register before that."""
import os
import re
import shutil
import subprocess

import pytest

import draft_verification_spec_amd as sv

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
# wait states from a matrix instruction to another's touch of its results: the longest that any
# of the target's asks for is 19 (16 passes), this one's shape takes at most 8 passes
STATES = 20
TOUCH = re.compile(r"\ba(?:\[(\d+):(\d+)\]|(\d+))")


def registers(text):
    out = set()
    for lo, hi, one in TOUCH.findall(text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def too_soon(code):
    """Instructions (address, text) of [(address, text, target or None)] that touch a register
    of sums in fewer than STATES states after a matrix instruction wrote it, over all ways."""
    at = {a: i for i, (a, _, _) in enumerate(code)}
    state = {0: {}}                       # before instruction i: register -> fewest states since its product
    todo, found = [0], set()
    while todo:
        i = todo.pop()
        live = dict(state[i])
        while True:
            a, text, target = code[i]
            op = text.split()[0]
            product = op.startswith("v_mfma")
            regs = registers(text)
            if not product:
                found |= {(a, text) for r in regs if r in live}
            n = int(text.split()[1], 0) + 1 if op == "s_nop" else 1
            live = {r: s + n for r, s in live.items() if s + n < STATES}
            if product:
                live.update((r, 0) for r in registers(text.split(",")[0]))
            ways = [at[target]] if target is not None else []
            if op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                ways.append(i + 1)
            ways = [w for w in ways if w < len(code)]
            if len(ways) == 1 and target is None and ways[0] not in state:
                i = ways[0]
                continue
            for w in ways:
                old = state.get(w)
                new = dict(live) if old is None else {r: min(old.get(r, STATES), live.get(r, STATES)) for r in old.keys() | live.keys()}
                if old != new:
                    state[w] = new
                    todo.append(w)
            break
    return sorted(found)


def kernels(folder):
    """{name: code} of the tiled product's kernels in the built library."""
    lib = os.path.join(folder, "library.so")
    shutil.copy(sv.LIB_PATH, lib)
    subprocess.check_call([OBJDUMP, "--offloading", lib], stdout=subprocess.DEVNULL, cwd=folder)
    out = {}
    for f in sorted(os.listdir(folder)):
        if not f.endswith("gfx950"):
            continue
        text = subprocess.check_output([OBJDUMP, "-d", "--mcpu=gfx950", os.path.join(folder, f)], text=True)
        if "v_mfma_scale" not in text:
            continue
        for part in re.split(r"^(?=[0-9a-f]{16} <)", text, flags=re.M):
            head = re.match(r"([0-9a-f]{16}) <(\w*tile_kernel\w*)>:\n", part)
            if not head:
                continue
            start, code = int(head.group(1), 16), []
            for line in part[head.end():].splitlines():
                m = re.match(r"\s+(\w.*?)\s*// ([0-9A-F]{12}):[^<]*(?:<\w+(?:\+0x([0-9a-f]+))?>)?", line)
                if m:
                    jump = "branch" in m.group(1).split()[0]
                    code.append((int(m.group(2), 16), m.group(1), start + int(m.group(3) or "0", 16) if jump else None))
            out[head.group(2)] = code
    return out


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    sv.load_library()
    return kernels(str(tmp_path_factory.mktemp("code")))


def test_no_sum_is_touched_too_soon(built):
    assert len(built) == 4
    for name, code in built.items():
        assert sum(t.startswith("v_mfma_scale") for _, t, _ in code) >= 64, name
        assert not too_soon(code), name


def test_the_check_sees_a_read_before_the_wait(built):
    """The same listings with a sum read among the products, and behind the wait."""
    for name, code in built.items():
        last = max(i for i, (_, t, _) in enumerate(code) if t.startswith("v_mfma_scale"))
        read = (-1, f"v_accvgpr_read_b32 v0, a{min(registers(code[last][1].split(',')[0]))}", None)
        assert too_soon([*code[:last + 1], read, *code[last + 1:]]) == [read[:2]], name
        wait = max(i for i, (_, t, _) in enumerate(code) if t == "s_nop 3")
        assert wait > last and not too_soon([*code[:wait + 1], read, *code[wait + 1:]]), name
