"""What the built library holds of the serving kernels, by the metadata of its
own code objects.  Runs on the CPU."""

import re
import struct

import pytest

from reduce_rank_buffers_amd import _lib as L

msgpack = pytest.importorskip("msgpack")


@pytest.fixture(scope="module")
def kernels(librrb):
    """{mangled name: metadata} of every kernel in librrb.so: the notes named
    AMDGPU, of type 32, of the code objects in it."""
    with open(L.LIB_PATH, "rb") as f:
        data = f.read()
    out, at = {}, data.find(b"AMDGPU\0\0")
    while at >= 0:
        name, size, kind = struct.unpack("<III", data[at - 12:at])
        if name == 7 and kind == 32:
            for k in msgpack.unpackb(data[at + 8:at + 8 + size]).get("amdhsa.kernels", []):
                out[k[".name"]] = k
        at = data.find(b"AMDGPU\0\0", at + 8)
    assert len(out) > 100
    return out


def _of(kernels, name):
    """{template arguments: metadata} of the kernels of that name: integers and
    truth values, and types by their mangled letter."""
    out = {}
    for mangled, k in kernels.items():
        m = re.search(rf"\d{name}I((?:L[ib]\d+E|[a-z])+)E", mangled)
        if m:
            args = re.findall(r"L[ib](\d+)E|([a-z])", m.group(1))
            out[tuple(int(n) if n else t for n, t in args)] = k
    return out


@pytest.mark.parametrize("name", ["decode_up_kernel", "decode_down_kernel", "decode_up_direct_kernel",
                                  "decode_down_direct_kernel", "quantize_kernel", "product_kernel",
                                  "product_direct_kernel", "product_turns_kernel"])
def test_no_kernel_spills(kernels, name):
    """None keeps vector registers in memory."""
    found = _of(kernels, name)
    assert found
    spilled = {a: k[".private_segment_fixed_size"] for a, k in found.items()
               if k[".private_segment_fixed_size"] or k[".vgpr_spill_count"]}
    assert not spilled, f"{name}: bytes of scratch a lane: {spilled}"


def test_integer_products_built(kernels):
    """The tile shapes that launch_integers chooses among, linear and gated, and
    no others: of product_kernel and product_direct_kernel BM, BN, waves down and
    across, stages (the second), form, gated, elements (a: int8), once."""
    both = (0, 1)
    of = lambda name: {a for a in _of(kernels, name) if "a" in a}
    assert of("product_kernel") == {(*t, 0, g, "a") for t in ((128, 128, 2, 4), (64, 64, 2, 2)) for g in both}
    assert of("product_direct_kernel") == {(*t, 0, g, "a", once) for g in both for *t, once in (
        (32, 64, 2, 2, 4, 1), (64, 64, 2, 2, 5, 0), (64, 128, 2, 2, 3, 0), (128, 256, 2, 4, 3, 0))}
    assert of("product_turns_kernel") == {(0, g, "a") for g in both}


def test_quantisations_built(kernels):
    """What launch_quantize's rule on widths and rows can come to, for bf16 (t)
    and fp32 (f): lanes, turns held (0: any), rows of at least eight."""
    want = {(64, 0, 0)} | {(64, n, 1) for n in (1, 2, 4, 8)} | {(256, n, 1) for n in (1, 2, 4)}
    want |= {(1024, n, 1) for n in (2, 4, 8, 0)}
    assert set(_of(kernels, "quantize_kernel")) == {(t, *a) for t in "tf" for a in want}
