"""The structures that calls pack in one step lie as the ctypes classes of the same C structures do:
sizes, and every field at its place."""
import ctypes
import math
import struct

import pytest

import exact_causal_gqa_gb300 as atlas

PAIRS = [(atlas._pack_launch, atlas._Launch), (atlas._pack_shared, atlas._Shared), (atlas._pack_rope, atlas._Rope),
         (atlas._pack_norm, atlas._Norm), (atlas._pack_resize, atlas._Resize)]


def leaves(cls):
    """(field, index or None, type) of every value that is packed, in order."""
    for name, kind in cls._fields_:
        if issubclass(kind, ctypes.Array):
            yield from ((name, i, kind._type_) for i in range(kind._length_))
        else:
            yield name, None, kind


def value(kind, k):
    """The k-th value: another for each field, the whole of its type's bytes in use."""
    if kind in (ctypes.c_float, ctypes.c_double):
        return (k + 1) * 0.37 if kind is ctypes.c_double else struct.unpack("f", struct.pack("f", (k + 1) * 0.37))[0]
    size = ctypes.sizeof(kind)
    signed = kind(-1).value is not None and kind(-1).value < 0
    return int.from_bytes(bytes(7 * k + i + 1 & 0x7f for i in range(size)), "little", signed=signed)


@pytest.mark.parametrize("pack,cls", PAIRS, ids=[c.__name__ for _, c in PAIRS])
def test_packed_as_the_class(pack, cls):
    fields = list(leaves(cls))
    values = [value(kind, k) for k, (_, _, kind) in enumerate(fields)]
    packed = pack(*values)
    assert len(packed) == ctypes.sizeof(cls)   # (the library copies whole structures)
    filled = cls()
    for (name, i, _), v in zip(fields, values):
        if i is None:
            setattr(filled, name, v)
        else:
            getattr(filled, name)[i] = v
    read = cls.from_buffer_copy(packed)
    for name, i, _ in fields:
        a, b = ((getattr(x, name) if i is None else getattr(x, name)[i]) for x in (read, filled))
        assert a == b and not (isinstance(a, float) and math.isnan(a)), (name, i)


def test_too_few_values_are_noticed():
    for pack, cls in PAIRS:
        with pytest.raises(struct.error):
            pack(*[0] * (len(list(leaves(cls))) - 1))
