"""Host-side checks of the serving operators, no GPU: what a kernel's source must
order, and what the wrappers refuse and why."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_evict_select_waits_for_its_cluster_before_remote_shared_memory():
    """A cluster's CTAs may touch one another's shared memory only after a barrier of
    the whole cluster.  The first one stands before the first remote access on every
    path: outside every block of the kernel's body."""
    src = open(os.path.join(ROOT, "fsq_latent_decode_b200", "csrc", "evict.cu")).read()
    body = src[src.index("evict_select(SelectParams p, int per) {"):]
    body = re.sub(r"//[^\n]*", "", body[body.index("{"):])
    arrive, wait = body.index("cl.barrier_arrive()"), body.index("cl.barrier_wait()")
    remote = body.index("map_shared_rank")
    assert arrive < wait < remote
    for at in (arrive, wait):
        assert body[:at].count("{") - body[:at].count("}") == 1
        assert re.search(r"if \(CS > 1\) $", body[:at])
