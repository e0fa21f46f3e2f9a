"""What libtss.so holds for the GPU, read from the symbol tables of its own code
objects: kernels only where the host launches them, and the bytes of scratch
memory that a kernel's lanes take (registers that do not fit)."""
import os
import struct

import pytest

import tile_size_selection_amd as tss

LIB = os.path.join(os.path.dirname(os.path.abspath(tss.__file__)), "libtss.so")


def symbols(image):
    """(name, value) of every symbol of a 64-bit ELF image."""
    at, = struct.unpack_from("<Q", image, 40)
    size, n = struct.unpack_from("<HH", image, 58)
    sections = [struct.unpack_from("<IIQQQQIIQQ", image, at + i * size) for i in range(n)]
    for s in sections:
        if s[1] != 2:  # a symbol table
            continue
        names = sections[s[6]]
        for k in range(s[4], s[4] + s[5], 24):
            name, _, _, _, value, _ = struct.unpack_from("<IBBHQQ", image, k)
            first = names[4] + name
            yield image[first:image.index(b"\0", first)].decode(), value


@pytest.fixture(scope="module")
def objects():
    """The symbols of each code object, one for each source."""
    data = open(LIB, "rb").read()
    found, at = [], data.find(b"\x7fELF\x02\x01\x01\x40")  # an ELF image for the GPU
    while at >= 0:
        end = data.find(b"\x7fELF\x02\x01\x01\x40", at + 1)
        found.append(dict(symbols(data[at:end if end >= 0 else len(data)])))
        at = end
    assert len(found) > 10
    return found


def scratch(objects, *parts):
    """Bytes of scratch a lane of the kernels whose names hold all of these."""
    tail = ".private_seg_size"
    got = {n[:-len(tail)]: v for o in objects for n, v in o.items() if n.endswith(tail) and all(p in n for p in parts)}
    assert got, parts
    return got


def test_wide_norms_keep_their_registers(objects):
    """Rows of more than 16384 columns, four chunks a thread.  The gradients hold both weights' sums as well, which are
    spilled: 288 to 360 bytes cost 381 us at 2000 x 32768 where 460 to 496 cost 529."""
    assert all(v <= 320 for v in scratch(objects, "layer_norm_backward_kernel", "Li4ELi0ELi64E").values())
    assert all(v == 0 for v in scratch(objects, "layer_norm_kernel", "Lb0ELi4ELi64E").values())
    # up to 16384 columns nothing is spilled
    for chunks in ("Li1ELi1E", "Li2ELi0E"):
        assert all(v == 0 for v in scratch(objects, "layer_norm_backward_kernel", chunks).values())
    assert all(v == 0 for v in scratch(objects, "layer_norm_kernel", "Li2ELi64E").values())
    assert all(v == 0 for v in scratch(objects, "layer_norm_backward_few_kernel").values())


def kernels(objects):
    return [n[:-3] for o in objects for n in o if n.endswith(".kd")]


def test_a_headers_kernels_are_not_in_every_unit(objects):
    """A kernel of a unit's own in a header is copied into whatever includes it, launched or not.  (Templates are made
    where they are launched.)"""
    names = [n for n in kernels(objects) if n.startswith("_ZN3tssL")]
    assert not names, f"of internal linkage, from a header: {sorted(names)}"


def test_the_host_knows_every_kernel(objects):
    """A kernel without the handle that the host launches it by is one that nothing reaches."""
    handles = {n for n, _ in symbols(open(LIB, "rb").read())}
    assert sorted(set(kernels(objects)) - handles) == []
