"""A block may touch a peer's shared memory only once the whole cluster is known to
run: in the kernels whose text runs straight through, a cluster barrier comes
before the first access to a peer."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_151_gb300", "csrc")


def kernel_text(name, kernel):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    return text[re.search(r"\b%s\(const __grid_constant__" % kernel, text).start():]


@pytest.mark.parametrize("name,kernel", [("pa_verify.cu", "verify_drafts_kernel"),
                                         ("pa_prefill_f8.cuh", "prefill_f8_kernel")])
def test_a_cluster_barrier_comes_before_the_first_access_to_a_peer(name, kernel):
    text = kernel_text(name, kernel)
    peer = re.search(r"\b(?:map_to_rank|map_rank|st_dsmem\w*|ld_dsmem\w*)\(", text).start()
    met = re.search(r"\bcluster_(?:wait|sync)\(\)", text).start()
    assert met < peer
    waits, arrivals = (len(re.findall(r"\bcluster_%s\(\)" % x, text)) for x in ("wait", "arrive"))
    assert waits == arrivals
