"""The query and key norm's kernels in the built library are those that a call can select (CPU: their names are read, nothing runs)."""
import re

from chunkwise_weight_recurrence_amd import binding as B


def test_no_kernel_is_built_that_nothing_selects():
    with open(B.LIB_PATH, "rb") as f:
        built = set(re.findall(rb"qk_(fwd|bwd)_kernelI(\w)Li(\d+)ELi(\d+)ELi(\d+)ELb([01])EE", f.read()))
    want = set()
    for elem, wide in (("t", 8), ("f", 4)):   # t: bf16's 16 bits
        for half in (0, 1):
            for d in range(1, 513):
                for rot in range(0, d + 1, 2):
                    for V in (wide, 1):
                        if d % V or half and V > 1 and (rot // 2 % V or rot % V):
                            continue
                        nr = rot // 2 // V if half else 0
                        units = nr + -(-(d - 2 * nr * V) // (2 * V))
                        lanes = next(n for n in (4, 8, 16, 32, 64) if units <= n) if V > 1 else 64
                        want |= {(way, elem, V, lanes, 1 if units <= lanes else 4, half) for way in ("fwd", "bwd")}
    assert {(w.decode(), e.decode(), *map(int, rest)) for w, e, *rest in built} == want
