"""The layer norm kernels in the built library are those that a plan can select (CPU: their names are read, nothing runs)."""
import itertools
import re

from chunkwise_weight_recurrence_amd import binding as B


def test_no_layer_norm_kernel_is_built_that_nothing_selects():
    with open(B.LIB_PATH, "rb") as f:
        built = set(re.findall(rb"ln_(fwd|bwd)_kernelI(\w)Li(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb([01])EE", f.read()))
    want = set()
    for way, (elem, wide) in itertools.product(("fwd", "bwd"), (("t", 8), ("f", 4))):   # t: bf16's 16 bits
        several = 4 if way == "fwd" else 2   # rows a slot takes at once where rows are narrow
        plans = [(1, 8, 1, 1), (1, 8, 1, several)]   # fewer columns than a piece has
        plans += [(wide, lanes, 1, rows) for lanes in (8, 16, 32, 64) for rows in (1, several)]
        plans += [(wide, 0, 1, 1), (wide, 0, 1, 2), (wide, 0, 2, 1), (wide, 0, 3, 1)]   # whole waves a row
        plans += [(wide, 0, 5, 1)] if elem == "f" else []
        want |= {(way, elem, *p, res) for p in plans for res in (0, 1)}
    assert {(w.decode(), e.decode(), *map(int, rest)) for w, e, *rest in built} == want
