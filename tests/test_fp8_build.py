"""What the 8-bit sources and their build have to keep to, checked without a GPU."""
import glob
import os
import re

import w4a4_rotated_quantized_gb300 as q

CSRC = os.path.join(os.path.dirname(q.__file__), "csrc")


def test_no_bulk_load_writes_another_cta():
    """The library runs as replicas on several GPUs too: every CTA loads its own tiles into its own shared memory."""
    found = []
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = re.sub(r'"\s*"', "", f.read())  # asm strings that the source breaks over lines, joined
        for ins in re.findall(r"cp\.async\.bulk[\w.:]*", text):
            if "multi" + "cast" in ins:
                found.append((os.path.basename(path), ins))
    assert found == []
