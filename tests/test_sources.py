"""Rules the kernel sources keep that no run on one GPU can show."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_multicast_copies():
    """The library also runs with one process a GPU: its tensor copies load into their own CTA's shared memory only."""
    paths = glob.glob(os.path.join(ROOT, "*_gb300", "csrc", "*.cu*"))
    assert len(paths) > 10
    for path in paths:
        with open(path) as f:
            text = f.read()
        # an instruction may be spread over adjacent string literals
        for asm in re.findall(r'"[^"]*cp\.async\.bulk[^"]*"(?:\s*"[^"]*")*', text):
            assert "multicast" not in asm, (os.path.basename(path), asm)
