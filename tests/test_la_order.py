"""The order of steps in the decayed linear attention's tensor-core kernel that no run can show,
read from its source (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_43_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def statements(code):
    """The outermost statements and blocks of a piece of code, in order."""
    depth, parts = 0, [""]
    for c in code:
        parts[-1] += c
        depth += (c == "{") - (c == "}")
        if depth == 0 and c in ";}":
            parts.append("")
    return parts


def test_the_tensor_memory_address_is_read_before_its_word_is_used_again():
    """The slot that tcgen05.alloc writes shares a word with the decay of a chunk: a barrier of
    all warps, in every call, stands between the last read of one and the roles, which write
    the other."""
    code = source("la_chunk_tc.cu")
    assert "uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + M::kTot)" in code
    start = code.index("const uint32_t tmem = *tslot;")
    setup = code[start:code.index("if (warp < kRowWarps)", start)]
    steps = statements(setup)
    last_read = max(i for i, x in enumerate(steps) if "*tslot" in x)
    assert "__syncthreads();" in [x.strip() for x in steps[last_read + 1:]]
