"""Device-side helpers of the mixture-of-experts GPU tests: tensors with sentinel
bytes around every output, checked untouched after the call."""
from __future__ import annotations

import numpy as np
import torch

from gpu_util import require_gpu

PAD = 512  # sentinel bytes on both sides of an output


def moe():
    require_gpu()
    from lossless_bf16_exponent_amd import zc_moe
    return zc_moe


class Out:
    """An output of `shape` and `dtype` inside a byte buffer filled with 0xA5."""

    def __init__(self, shape, dtype, offset=0):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n + 2 * PAD + offset,), 0xA5, dtype=torch.uint8, device="cuda")
        self.lo, self.n = PAD + offset, n
        self.t = self.raw[self.lo:self.lo + n].view(dtype).view(*shape)

    def data_ptr(self):
        return self.raw.data_ptr() + self.lo

    def numpy(self):
        """The values (BF16 as 64-bit floats), after a check of the sentinels."""
        torch.cuda.synchronize()
        assert bool((self.raw[:self.lo] == 0xA5).all()), "written before the output"
        assert bool((self.raw[self.lo + self.n:] == 0xA5).all()), "written past the output"
        return to_numpy(self.t)


def to_numpy(t):
    t = t.detach()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def device(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def bf16_device(x, stride=None, offset=0):
    """64-bit values (already BF16 numbers) as a BF16 tensor with rows `stride` apart, `offset` elements into its buffer."""
    m, k = x.shape
    stride = stride or k
    buf = torch.full((offset + m * stride,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = buf[offset:].view(m, stride)
    view[:, :k] = torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(torch.bfloat16).cuda()
    return view


def close(got, want, tol, what=""):
    """|got - want| <= tol everywhere; NaN and infinities at the same places."""
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN at other places"
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), what + ": other infinities"
    off = np.abs(got[fin] - want[fin]) - np.broadcast_to(tol, want.shape)[fin]
    assert off.size == 0 or off.max() <= 0, "%s: off by %.3g more than the tolerance, %d of %d" % (
        what, off.max(), int((off > 0).sum()), off.size)
