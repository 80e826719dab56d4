"""The device code that the compiler makes of the sources, as text (no GPU):
rules of the machine that it keeps for its own instructions but not inside an
asm string."""
import glob
import os
import re
import subprocess

import pytest

from markov_draft_sampling_amd import build


def _sources_with(text):
    out = []
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.hip"))):
        with open(path) as f:
            if text in f.read():
                out.append(os.path.basename(path))
    return out


_done = {}


def _kernels(source, tmp):
    """{kernel name: its instructions in order, comments, labels and directives left out} of a source; those of an asm
    string start with "asm "."""
    if source not in _done:
        asm = os.path.join(str(tmp), source + ".s")
        subprocess.run([build._hipcc(), *build.FLAGS, "-w", "-S", "--offload-device-only", "-I",
                        os.path.join(build.HERE, "..", "include"), os.path.join(build.CSRC, source), "-o", asm], check=True)
        kernels, cur, inside = {}, None, ""
        with open(asm) as f:
            for line in f:
                m = re.match(r"(_Z\w+):", line)
                if m:
                    cur = kernels.setdefault(m.group(1), [])
                if "#ASM" in line:
                    inside = "asm " if "#ASMSTART" in line else ""
                line = line.split(";")[0].strip()
                if cur is not None and line and not line.endswith(":") and not line.startswith((".", "#")):
                    cur.append(inside + line)
                if line.startswith(".end_amdhsa_kernel"):
                    cur = None
        _done[source] = kernels
    return _done[source]


def _is_copy(ins):
    """A load straight into LDS, at the address in m0."""
    return bool(re.match(r"(asm )?(global_load_lds_|buffer_load_\S+ .*\blds$)", ins))


@pytest.mark.parametrize("source", _sources_with("s_mov_b32 m0"))
def test_copies_into_lds_wait_for_their_address(source, tmp_path):
    # a scalar write of m0 needs one wait state before a load into LDS reads it: the compiler keeps to that where it
    # places both, not within an asm string
    copies = 0
    for name, code in _kernels(source, tmp_path).items():
        written = [i for i, ins in enumerate(code) if re.match(r"(asm )?s_\w+ m0\b", ins)]
        copies += sum(map(_is_copy, code))
        for i in written:
            assert not _is_copy(code[i + 1]), f"{name}: {code[i]} then {code[i + 1]}"
    assert copies > 0


@pytest.mark.parametrize("source", _sources_with("s_mov_b32 m0"))
def test_nothing_but_copies_uses_m0_where_asm_writes_it(source, tmp_path):
    # the asm strings cannot declare that they write m0 (a reserved register): a kernel that has them has no other use
    for name, code in _kernels(source, tmp_path).items():
        uses = [ins for ins in code if re.search(r"\bm0\b", ins)]
        if any(ins.startswith("asm ") for ins in uses):
            assert all(ins.startswith("asm ") for ins in uses), name


def _scalars(operands):
    out = {"vcc"} if "vcc" in operands else set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", operands):
        out |= {int(m.group(3))} if m.group(3) else set(range(int(m.group(1)), int(m.group(2)) + 1))
    return out


@pytest.mark.parametrize("source", _sources_with("s_mov_b32 m0"))
def test_copies_into_lds_wait_for_their_base(source, tmp_path):
    # a scalar register that the vector unit wrote is there for a load five wait states later
    for name, code in _kernels(source, tmp_path).items():
        for i, ins in enumerate(code):
            if not (ins.startswith("asm ") and _is_copy(ins)):
                continue
            states, j = 0, i - 1
            while j >= 0 and states < 5:
                before = code[j].removeprefix("asm ")
                if before.startswith("v_"):
                    written = before.split(None, 1)[1].split(",")[0]
                    assert not _scalars(written) & _scalars(ins), f"{name}: {before} then {ins}"
                nop = re.match(r"s_nop (\d+)", before)
                states += int(nop.group(1)) + 1 if nop else 1
                j -= 1


def test_lm_head_fp8_barriers_count_nothing_but_copies(tmp_path):
    # A wait for all but the newest N operations before a barrier holds if each of those N is one that the source counted:
    # a copy into LDS written as assembly, of which there are as many in every chunk. A plain load may be dropped by the
    # compiler, or become a scalar one, which the wait does not count.
    few = 0
    for name, code in _kernels("lm_head_fp8.hip", tmp_path).items():
        copies = [i for i, ins in enumerate(code) if _is_copy(ins)]
        waits = [re.search(r"vmcnt\((\d+)\)", code[i - 1]) for i, ins in enumerate(code) if ins == "s_barrier" and i]
        counts = {int(m.group(1)) for m in waits if m}
        if not copies:
            continue
        assert all(waits), name
        for i, ins in enumerate(code):
            if re.match(r"(buffer|global|flat|scratch)_load", ins.removeprefix("asm ")):
                assert i < copies[0] or ins.startswith("asm ") and _is_copy(ins), (name, ins)
        if counts - {0}:
            few += 1
            ring = 4  # chunks; the copies of each but the last are in the code before the loop, of one more in the loop
            assert len(copies) % ring == 0 and counts == {0, len(copies) // ring * (ring - 2)}, (name, counts)
    assert few == 2
