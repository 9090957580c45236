"""Build-time check of the hand-off inside the joining launch of the router's losses,
on the AMD assembly of this repository's own build (gfx950): a block stores its
sequence's sums with agent-coherent stores (sc1: written through its XCD's L2),
waits for them, counts itself, and the last block to count invalidates its
caches (buffer_inv sc1) and reads them with agent-coherent loads."""
import re

from test_isa_publish import _asm


def test_joining_launch_publishes_its_sums(tmp_path):
    asm = _asm("balance.hip", tmp_path)
    # up to the end of the function: it has more than one s_endpgm
    bodies = re.findall(r"^_Z\S*balance_join_kernel\S*:(.*?)^\.Lfunc_end", asm, flags=re.M | re.S)
    assert len(bodies) == 1
    body = bodies[0]
    adds = list(re.finditer(r"^\s*global_atomic_add\b.*$", body, flags=re.M))
    assert len(adds) == 1
    # the block's balance sum, squared log-sum-exp and number of tokens, then the wait, then the count
    wait = body.rfind("s_waitcnt vmcnt(0)", 0, adds[0].start())
    assert wait > 0
    shared = [m for m in re.finditer(r"^\s*global_store_dword\b.*\bsc1\b.*$", body, flags=re.M)]
    assert len(shared) == 3 and all(m.end() < wait for m in shared)
    # nothing between the wait and the count writes memory
    assert not re.search(r"^\s*(global|flat|buffer)_store", body[wait:adds[0].start()], flags=re.M)
    after = body[adds[0].end():]
    inv = re.search(r"^\s*buffer_inv\s+sc1\b", after, flags=re.M)
    assert inv
    # one load of each of the three by the last block, unrolled or not, and none of them ahead of the invalidate
    loads = list(re.finditer(r"^\s*global_load_dword\b.*\bsc1\b.*$", after, flags=re.M))
    assert len(loads) >= 3 and all(m.start() > inv.start() for m in loads)
