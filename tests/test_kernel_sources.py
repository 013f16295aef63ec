"""Rules that the kernels' sources keep."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_decode_amd", "csrc")


def test_no_instruction_is_written_in_an_asm_statement():
    """The compiler counts the wait states before and after a matrix instruction between its own instructions alone: one in
    an asm statement that writes a matrix operand, or a register that the matrix cores still read, is not waited for.
    Empty statements, which only hide a value from the optimizer, are fine."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if not path.endswith((".hip", ".hpp", ".cpp")):
            continue
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\b\s*(?:volatile\s*)?\(\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)*)", text):
            if m.group(1).strip() != '""':
                found.append((os.path.basename(path), m.group(1)[:60]))
    assert not found, found
