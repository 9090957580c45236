"""Build-time check of the hand-off inside the second product of the layer for
few tokens, on the AMD assembly of this repository's own build (gfx950): a
block stores its sums with agent-coherent stores (sc1: written through its
XCD's L2), waits for them, counts itself, and the last block to count
invalidates its caches (buffer_inv sc1) before it reads all of them."""
import re

from test_isa_publish import _asm, _functions


def test_down_projection_publishes_its_sums(tmp_path):
    bodies = _functions(_asm("decode.hip", tmp_path), r"decode_ffn_kernelILi\dELb0ELi\dELi\dELb1E")
    assert bodies
    for body in bodies:
        add = re.search(r"s_waitcnt vmcnt\(0\)(?:(?!s_waitcnt vmcnt).)*?global_atomic_add", body, flags=re.S)
        assert add, "no vmcnt(0) wait ahead of the counter update"
        stores = re.findall(r"^\s*global_store_dword\b.*$", body[:add.end()], flags=re.M)
        assert stores and all(re.search(r"\bsc1\b", s) for s in stores)
        assert not re.search(r"^\s*global_store_dwordx", body[:add.end()], flags=re.M)
        assert re.search(r"^\s*buffer_inv\s+sc1\b", body[add.end():], flags=re.M)


def test_products_load_by_counted_waits(tmp_path):
    """The products keep two steps of loads in flight: no load of theirs may be a flat one, and no
    register may live in scratch memory (both wait for everything that is outstanding)."""
    asm = _asm("decode.hip", tmp_path)
    # up to the end of the function: a kernel may have more than one s_endpgm
    bodies = re.findall(r"^_Z\S*decode_ffn_kernelILi\S*:(.*?)^\.Lfunc_end", asm, flags=re.M | re.S)
    assert bodies
    for body in bodies:
        assert not re.search(r"^\s*(flat|scratch)_", body, flags=re.M)
        loads = [int(n) for n in re.findall(r"s_waitcnt vmcnt\((\d+)\)", body)]
        assert max(loads) >= 8
