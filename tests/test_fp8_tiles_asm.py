"""The LDS DMA statement of the block-scaled FP8 tiles, in the assembly that
the compiler makes of it. The statement writes m0 and reads scalar registers
where the compiler sees neither its register use nor its hazards, so the test
looks at the code around every one: nothing else may use m0, and no scalar
register that the load reads may have been written by a vector instruction
within the five wait states that such a read needs."""
import os
import re
import subprocess

import pytest

from int4_weight_quantized_amd import build as B

SOURCE = os.path.join(B.CSRC, "fp8_block_gemm.hip")


@pytest.fixture(scope="module")
def compiled():
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    flags = [f for f in B.HIPCC_FLAGS if f != "-shared"]
    res = subprocess.run([hipcc, *flags, "--cuda-device-only", "-S", "-o", "-", SOURCE], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    kernels = re.findall(r"\.amdhsa_kernel (\S+)", res.stdout)
    code = [re.sub(r"\s*[;/]+.*", "", line).strip() for line in res.stdout.split("\n")]
    return [c for c in code if c and not c.startswith(".")], res.stderr, kernels


def scalar_registers(text):
    m = re.match(r"s\[(\d+):(\d+)\]$", text)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"s(\d+)$", text)
    return {int(m[1])} if m else set()


def written(instruction):
    """The scalar registers that a vector instruction writes: its first operand, or the carry-out after that."""
    if not instruction.startswith("v_"):
        return set()
    name, rest = instruction.split(None, 1)
    ops = [o.strip() for o in rest.split(",")]
    return scalar_registers(ops[0]) | (scalar_registers(ops[1]) if "_co_" in name else set())


def test_no_warnings(compiled):
    assert "warning" not in compiled[1], compiled[1][:2000]


def test_dma_statements(compiled):
    code = compiled[0]
    loads = [i for i, c in enumerate(code) if re.match(r"buffer_load_dword\S*\s.*\blds$", c)]
    assert len(loads) > 100
    for i in loads:
        assert code[i - 1] == "s_nop 0" and re.match(r"s_mov_b32 m0, s\d+$", code[i - 2]), code[i - 3:i + 1]
    assert sum(bool(re.search(r"\bm0\b", c)) for c in code) == len(loads)
    for i in loads:
        ops = [o.strip() for o in code[i].split(None, 1)[1].replace("offen lds", "").split(",")]
        read = scalar_registers(ops[1]) | scalar_registers(ops[2])
        assert len(read) >= 4
        wait, j = 0, i - 1
        while wait < 5:
            assert not written(code[j]) & read, (code[j], code[i])
            nop = re.match(r"s_nop (\d+)", code[j])
            wait += int(nop[1]) + 1 if nop else not code[j].endswith(":")
            j -= 1


def test_instances(compiled):
    """Every tile kernel that is built is one that a call reaches: (rows and columns of 16 a wave, waves, grouped,
    fp16 operands, output type)."""
    built = set()
    for name in compiled[2]:
        m = re.search(r"fp8_tile_kernelILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb(\d)ELb(\d)ELi(\d)E", name)
        if m:
            built.add(tuple(int(v) for v in m.groups()))
    small = {(mi, 4, 2, 2, 0, f16, out) for mi in (2, 4) for f16, out in ((0, 0), (0, 1), (0, 2), (1, 2))}
    large = {(8, 4, 2, 4, 0, 0, out) for out in (0, 1)}
    grouped = {(mi, 4, 2, wn, 1, 0, out) for mi, wn in ((4, 2), (8, 4)) for out in (0, 1)}
    assert built == small | large | grouped
