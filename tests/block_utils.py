"""Shared helpers of the recurrence and layer norm tests."""
import numpy as np

# half a step of each type, relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
# below the smallest normal number results may be flushed or lose digits
TINY = 2.0 ** -126


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def rounded(rng, shape, dtype, mean=0.0, std=1.0):
    """Values of a normal distribution as a tensor of ``dtype`` (on the CPU) holds them."""
    import torch
    return torch.from_numpy((rng.standard_normal(shape) * std + mean).astype(np.float32)).to(torch_dtype(dtype))


def f64(t):
    import torch
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def worst(got, ref, bound, dtype):
    """max |got - ref| over what it may be: the fp32 bound and half a step of the output's type.  Above 1 is wrong."""
    got = f64(got) if hasattr(got, "detach") else np.asarray(got, dtype=np.float64)
    ref = np.asarray(ref, dtype=np.float64).reshape(got.shape)
    bound = np.broadcast_to(np.asarray(bound, dtype=np.float64).reshape(-1) if np.ndim(bound) else bound,
                            (got.size,)).reshape(got.shape)
    if got.size == 0:
        return 0.0
    if not np.array_equal(np.isfinite(got), np.isfinite(ref)):
        return float("inf")
    at = np.isfinite(ref)
    room = bound[at] + HALF[dtype] * (np.abs(ref[at]) + bound[at]) + TINY
    return float((np.abs(got[at] - ref[at]) / room).max()) if at.any() else 0.0
