"""What the ctypes binding takes as a device pointer."""
import pytest

from depthwise_convolution_dwconv2d_gb300 import binding as B


class Buffer:
    """A buffer of another library: an address, no notion of strides."""

    def data_ptr(self):
        return 0x1000


class Strided(Buffer):
    def __init__(self, contiguous):
        self.contiguous = contiguous

    def is_contiguous(self):
        return self.contiguous


class Broken:
    """An error of the object's own is not a wrong type."""

    def data_ptr(self):
        return self.missing


def test_pointers():
    assert B._ptr(None) is None and B._ptr(0x2000) == 0x2000
    assert B._ptr(Buffer()) == 0x1000
    assert B._ptr(Strided(True)) == 0x1000
    with pytest.raises(ValueError):
        B._ptr(Strided(False))
    for bad in ("x", 1.5, object()):
        with pytest.raises(TypeError):
            B._ptr(bad)
    with pytest.raises(AttributeError, match="missing"):
        B._ptr(Broken())
