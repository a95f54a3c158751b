"""Shared by the tests of the operators that write gradients: views of
larger buffers (offsets, strides, guard elements) and error bounds."""

import torch

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
# half a step, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GUARD = 7.0


def guarded(shape, dtype, dev, offset=0, ld=None):
    """A [rows, cols] view with row stride ld, ``offset`` elements into a
    buffer filled with GUARD, and a function that checks that every element
    of the buffer outside the view still holds GUARD."""
    rows, cols = shape
    ld = cols if ld is None else ld
    buf = torch.full((offset + rows * ld + 64,), GUARD, dtype=dtype, device=dev)
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols] if rows else \
        buf[offset:offset].view(0, cols)

    def check():
        rest = torch.ones_like(buf, dtype=torch.bool)
        if rows:
            rest[offset:offset + rows * ld].view(rows, ld)[:, :cols] = False
        assert bool((buf[rest] == GUARD).all()), "written outside the view"

    return view, check


def fill_normal(view, std, gen):
    view.copy_(torch.randn(view.shape, generator=gen, device=view.device) * std)
    return view


def assert_within(got, want, bound):
    """|got - want| <= bound elementwise (float64 tensors), NaN nowhere."""
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} elements off, worst ratio "
        f"{float((d / bound.clamp(min=1e-300)).max())}, first at {bad.nonzero()[0].tolist()}")


def same_bits(a, b):
    it = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.contiguous().view(it), b.contiguous().view(it))
