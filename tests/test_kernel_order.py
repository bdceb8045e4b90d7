"""Orders inside the kernels that no run can show without hanging or faulting a
GPU, read from their source."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_linear_06_gb300", "csrc")


def kernels():
    """(file, name, body without comments) of every kernel."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__\b[^{;]*?(\w+_kernel\w*|\w+_join)\s*\(", src):
            at = src.index("{", src.index(")", m.end()))
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                end += 1
                if depth == 0:
                    break
            yield os.path.basename(path), m.group(1), src[at:end]


def test_tensor_memory_is_taken_after_the_kernel_before_is_done():
    # A kernel launched under the one before it that holds tensor memory and waits for
    # that one, which may itself still wait for tensor memory, would never end.
    seen = 0
    for path, name, body in kernels():
        wait = re.search(r"griddepcontrol\.wait|wait_before\(\)", body)
        alloc = re.search(r"tcgen05\.alloc|tmem_alloc", body)
        if wait and alloc:
            seen += 1
            assert wait.start() < alloc.start(), (path, name)
    assert seen >= 1
