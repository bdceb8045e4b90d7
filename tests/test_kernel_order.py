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


def test_no_copy_is_asked_for_after_a_wait_that_gave_up():
    # A stage whose copy did not arrive in time is still armed: arming it again for another
    # copy would be an arrival too many.  Every loop that fills stages asks for `ok` first.
    seen = 0
    for path, name, body in kernels():
        for m in re.finditer(r"const auto fill = \[&\]\(\) \{\s*while \(([^{]*)\) \{", body):
            seen += 1
            assert m.group(1).startswith("ok && "), (path, name, m.group(1))
            assert re.search(r"bool ok = true;", body[:m.start()]), (path, name)
    assert seen == 2
    # ... and the lanes of a warp agree on `ok`
    src = open(os.path.join(CSRC, "gdn_moe.cu")).read()
    wait = src[src.index("bool moe_wait("):]
    wait = wait[:wait.index("\n}")]
    assert re.search(r"__all_sync\(0xffffffffu, tc::mbar_wait\(", wait) and "__all_sync(0xffffffffu, done)" in wait
