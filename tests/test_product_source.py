"""What no run can show without a wait that runs out inside a product (CPU only): the outcome of a wait is each lane's own,
and a warp whose lanes disagree about it must not part, for barriers of the warp and of the cluster follow."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_v4_engram_hash_gb300", "csrc")


def test_a_vote_on_the_waits_is_kept():
    for name in ("product.cu", "product_rows.cu"):
        with open(os.path.join(CSRC, name)) as f:
            source = f.read()
        votes = re.findall(r"(\S+ \S+) ?__all_sync\(0xFFFFFFFFu, ok\)", source)
        assert all(v == "ok =" for v in votes), (name, votes)
