"""Shared by the GPU tests of the operators on rows of logits."""

import numpy as np
import torch

from .gpu_helpers import DEV

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def rows(seed, n, v, dtype="fp32", scale=2.2, head=12.0, masked=0.0, pad=0, lead=0):
    """Logits [n, v] on the device, in a buffer of row stride v + pad whose
    first row starts `lead` elements in, and the same values in fp64. What
    lies around the rows is NaN: nothing may read it."""
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(n, v)) * scale
    for i in range(n):
        at = rng.integers(0, v, min(v, 24))
        z[i, at] += head * rng.random() * rng.random(at.size) ** 2
        if masked:
            z[i, rng.random(v) < masked] = -np.inf
    return place(z, dtype, pad, lead)


def place(z, dtype="fp32", pad=0, lead=0):
    z = np.asarray(z, np.float64)
    n, v = z.shape
    buf = torch.full((lead + n * (v + pad) + 8,), float("nan"), dtype=TYPES[dtype], device=DEV)
    t = buf[lead:lead + n * (v + pad)].view(n, v + pad)[:, :v]
    t.copy_(torch.from_numpy(z).to(DEV).to(torch.float32).to(TYPES[dtype]))
    return t, t.double().cpu().numpy()


def dev(a, dtype):
    return torch.as_tensor(np.asarray(a), dtype=dtype).to(DEV)
