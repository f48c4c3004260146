"""What the kernel of the 4-bit products by tiles holds while it waits, read from its
source.  Its wait for columns of tensor memory has no limit, so it may hold none while it
waits for anything that another CTA, launch or kernel has to do: two kernels on an SM
could otherwise wait for each other for ever (which no test brings about)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def kernel():
    path = os.path.join(ROOT, "normalization_token_split_gb300", "csrc", "gemv_tile.cuh")
    with open(path) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    start = code.index("gemv_tile_kernel(const __grid_constant__")
    return code[start:code.index("\n}\n", start)]


def test_tensor_memory_is_held_between_the_waits():
    code = kernel()

    def only(what):
        at = [m.start() for m in re.finditer(re.escape(what), code)]
        assert len(at) == 1, what
        return at[0]

    taken, given = only("tmem_alloc<"), only("tmem_free<")
    assert only("grid_dependency_wait(") < taken
    # the launch behind starts when every CTA of this one has its columns: a barrier of the
    # CTA lies between
    assert "__syncthreads" in code[taken:only("allow_dependent_launch(")]
    meetings = [m.start() for m in re.finditer(r"cluster_(arrive|wait)\w*\(", code)]
    assert meetings and all(at < taken or at > given for at in meetings)
    # what is read from the other CTAs is read after they have met
    assert re.search(r"ld\.shared::cluster", code).start() > given


def test_waits_while_it_is_held_are_bounded():
    code = kernel()
    held = code[code.index("tmem_alloc<"):code.index("tmem_free<")]
    assert not re.search(r"mbar_wait\(|try_wait", held)
    waits = re.findall(r"\b(?:mbar_wait_bounded|bar_wait)\([^;]*;", held)
    assert len(waits) >= 8
    assert all("p.wait_limit_ns" in w for w in waits)
