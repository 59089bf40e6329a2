"""Orders that no run can show to be missing, shown on the source: memory written by some threads and read
or written again by others, with what has to stand between."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_row_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name,call", [("latent_attn.cu", "attend_again<"), ("latent_pair.cu", "attend_again<"),
                                       ("latent_prompt.cu", "attend_row<D>(p,")])
def test_rows_that_are_stored_again_wait_for_the_lanes_that_stored_them_first(name, call):
    src = source(name)
    calls = [m.start() for m in re.finditer(re.escape(call), src)]
    assert calls
    for at in calls:
        assert "__syncwarp();" in src[at - 160:at], src[at - 160:at]


def between(src, start, end):
    at = src.index(start)
    return src[at:src.index(end, at)]


def test_shared_memory_that_the_peers_products_read_is_released_to_the_cluster_and_acquired_from_it():
    """Ordinary stores of one CTA that a product of both reads: a proxy fence of the storing threads, an arrival
    with a release to the cluster, a wait with an acquire from it."""
    ptx = source("ptx.cuh")
    body = between(ptx, "void mbar_arrive_remote_shared(", "\n}")
    assert body.index("fence.release.sync_restrict::shared::cta.cluster;") < body.index("mbarrier.arrive.relaxed.cluster.")
    assert "fence.acquire.sync_restrict::shared::cluster.cluster;" in between(ptx, "void fence_acquire_shared_cluster(", "\n}")
    for name in ("bool mbar_wait_cluster(", "bool mbar_test_wait_cluster("):
        body = between(ptx, name, "\n}")
        assert body.rindex("fence_acquire_shared_cluster();") > max(body.rfind("mbar_try_wait_relaxed("), body.rfind(".relaxed.cluster."))
    # pairs: probabilities and zeroed values of every page
    src = source("latent_pair.cu")
    stores = src[src.index("// ---- P into shared memory"):]
    fence, arrive = stores.index("fence_proxy_async_smem();"), stores.index("mbar_arrive_remote_shared(pfull0")
    assert stores.index("= make_uint4(0u, 0u, 0u, 0u);") < fence < arrive
    assert re.findall(r"mbar_arrive\w*\(pfull0", src) == ["mbar_arrive_remote_shared(pfull0"]
    issuer = between(src, "// ======================= products' issuer", "// ============================== softmax")
    assert "mbar_test_wait_cluster(bar, parity)" in between(issuer, "auto done =", "};") and "done(pfull" in issuer
    # prompts: zeroed values of a tile's last step (probabilities are in tensor memory)
    src = source("latent_prompt.cu")
    step = src[src.index("if (ok && partial) {"):]
    assert step.index("= make_uint4(0u, 0u, 0u, 0u);") < step.index("fence_proxy_async_smem();") < step.index("mbar_arrive_remote_shared(pfull0)")
    assert "if (hh == 0 && partial) mbar_arrive_remote_shared(pfull0);" in step
    issuer = between(src, "issuer (rank 0)", "// ============================== softmax")
    assert "mbar_wait_cluster(b2, p2" in between(issuer, "auto wait2 =", "};") and "wait2(vfull, js & 1, pfull, js & 1)" in issuer


def test_the_paged_prompt_kernel_acquires_zeroed_values_from_the_cluster():
    src = source("chunk.cu")
    assert "if (partial) mbar_arrive_cluster(pfull0" in src
    issuer = between(src, "// ========================= P.V issuer (rank 0)", "// ============================== softmax")
    assert "mbar_wait_cluster(smem_addr(pfull + b)" in issuer
