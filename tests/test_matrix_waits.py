"""CPU test of the built library's machine code: results of matrix instructions
are read only when they are there. The hardware does not wait for them by itself;
the compiler puts wait states between, but where ways of different lengths meet
before the reader it has been seen to count the longer one."""
import os
import re
import shutil
import subprocess

import pytest

from lossless_bf16_tensor_amd import build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

# Wait states that the compiler puts between v_mfma_f32_16x16x32 (four passes)
# and what reads or overwrites its result, other than the accumulation of a
# further product; and those that another such instruction in between takes.
NEED, PASSES = 8, 4
REGISTER = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")
LOAD = re.compile(r"(global|flat|scratch|buffer)_load|ds_(read|bpermute)")


def registers(text):
    found = set()
    for kind, a, b, one in REGISTER.findall(text):
        first = 0 if kind == "v" else 512
        found.update(range(first + int(a), first + int(b) + 1) if a else (first + int(one),))
    return found


def functions(lines):
    """(name, address, [(address, instruction, comment)]) of each function of a disassembly."""
    name, start, body = None, 0, []
    for line in lines:
        head = re.match(r"([0-9a-f]{16}) <(\S+)>:", line)
        if head:
            if body:
                yield name, start, body
            name, start, body = head.group(2), int(head.group(1), 16), []
        elif line.startswith("\t") and "// " in line:
            text, note = line.split("// ", 1)
            body.append((int(note[:12], 16), text.strip(), note))
    if body:
        yield name, start, body


def early(start, body):
    """(matrix instruction, reader, wait states between) along any way that has too few of them."""
    place = {address: i for i, (address, _, _) in enumerate(body)}
    found = []
    for i, (_, text, _) in enumerate(body):
        if not text.startswith("v_mfma"):
            continue
        assert "_16x16x32_" in text, "another number of passes"
        result = registers(text.split(",")[0])
        least, ways = {}, [(i + 1, 0)]
        while ways:
            at, waited = ways.pop()
            if waited >= NEED or at >= len(body) or least.get(at, NEED) <= waited:
                continue
            least[at] = waited
            _, other, note = body[at]
            op, _, rest = other.partition(" ")
            states = 1
            if op == "s_nop":
                states = int(rest) + 1
            elif op in ("s_endpgm", "s_setpc_b64"):
                continue
            elif op == "s_branch" or op.startswith("s_cbranch"):
                offset = re.search(r"\+0x([0-9a-f]+)>", note)
                ways.append((place[start + (int(offset.group(1), 16) if offset else 0)], waited + 1))
                if op == "s_branch":
                    continue
            elif op.startswith("v_mfma"):
                to, a, b, c = re.split(r",\s*(?![^\[]*\])", rest)[:4]
                if (registers(a) | registers(b)) & result or (registers(c) & result and registers(c) != result):
                    found.append((text, other, waited))
                    continue
                if registers(to) == result:       # accumulated further or replaced, in order
                    continue
                states = PASSES
            elif op.startswith(("v_", "ds_", "global_", "flat_", "scratch_", "buffer_")):
                if registers(rest.split(",", 1)[1] if LOAD.match(op) and "," in rest else rest) & result:
                    found.append((text, other, waited))
                    continue
            ways.append((at + 1, waited + states))
    return found


def test_the_scan_itself():
    def way(*middle):
        lines = ["0000000000000100 <f>:", "\tv_mfma_f32_16x16x32_bf16 v[4:7], v[0:1], v[2:3], 0 // 000000000100: 0 0",
                 *(f"\t{m} // {0x108 + 4 * i:012X}: 0{n}" for i, (m, n) in enumerate(middle)), "\ts_endpgm // 000000000200: 0"]
        (_, start, body), = functions(lines)
        return early(start, body)
    reads, nops = ("v_max_f32_e32 v9, v5, v5", ""), lambda n: (f"s_nop {n}", "")  # noqa: E731
    assert not way(nops(7), reads) and len(way(nops(6), reads)) == 1
    assert len(way(nops(6), ("v_mov_b32_e32 v7, v9", ""))) == 1 and not way(nops(6), ("v_mov_b32_e32 v8, v9", ""))
    assert not way(nops(3), ("v_mfma_f32_16x16x32_bf16 v[12:15], v[0:1], v[2:3], 0", ""), reads)
    # taken, the branch leaves four wait states out
    skips = ("s_cbranch_vccnz 1", " <f+0x10>"), nops(3)
    assert not way(*skips, nops(6), reads) and [w for _, _, w in way(*skips, nops(2), reads)] == [4]
    assert len(way(("global_store_dword v[0:1], v6, off", ""))) == 1 and not way(("global_load_dword v6, v[0:1], off", ""))


def test_results_of_matrix_instructions_are_waited_for(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    if not os.path.exists(build.LIB):
        build.build()
    lib = shutil.copy(build.LIB, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950"))
    assert objects
    matrix, bad = 0, []
    for f in objects:
        with subprocess.Popen([OBJDUMP, "-d", "--no-show-raw-insn", f], cwd=tmp_path, stdout=subprocess.PIPE, text=True) as p:
            for name, start, body in functions(p.stdout):
                matrix += sum(t.startswith("v_mfma") for _, t, _ in body)
                bad += [(name, *e) for e in early(start, body)]
        assert p.returncode == 0
    assert matrix > 1000
    assert not bad, "\n".join(f"{name}: {text} -> {reader}: {waited} of {NEED} wait states" for name, text, reader, waited in bad)
