"""What no run shows of the 8-bit cache's kernels, checked from their source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "self_speculative_sparse_paged_gb300", "csrc")


def test_loads_from_tensor_memory_are_named_behind_their_wait():
    """The wait for tcgen05.ld names no register, so the compiler may move a use of what was loaded ahead
    of it unless the registers are named behind the wait."""
    with open(os.path.join(CSRC, "verify_kv8.cu")) as f:
        text = f.read()
    kernel = text[text.index("verify_kv8_kernel("):]
    loads = [(m.end(), m.group(1)) for m in re.finditer(r"tmem_ld8\([^;]*?, (\w+)\);", kernel)]
    loads += [(m.end(), m.group(1)) for m in re.finditer(r"load_o\(\d, c, (\w+)\);", kernel)]
    assert len(loads) == 4
    for at, name in loads:
        rest = kernel[at:]
        wait = min(rest.index(w) for w in ("tmem_ld_wait();", "load_all(tl") if w in rest)
        used = re.search(r"\b%s\b" % name, rest[wait:])
        assert re.match(r"%s(\[k\])?\);" % name, rest[wait + used.start():]), name
        assert re.search(r"loaded(<\S+>)?\($", rest[:wait + used.start()]), name
