"""Arrivals that cross from one CTA pair to the other in the attention over a prefix: each has a wait before the receiver
may leave its cluster (an arrival that comes later writes into shared memory that may be another kernel's).  A missing
wait shows on no GPU run, so the source is what is checked."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_kv_skv_gb300", "csrc", "skv_prefix.cu")


def test_commits_to_the_whole_cluster_are_waited_for():
    with open(SOURCE) as f:
        lines = f.read().splitlines()
    commits = {}
    for line in lines:
        m = re.search(r"mma2_commit_warp\(&c\.(\w+)(?:\[[^\]]*\])?, 15\)", line)
        if m:
            commits.setdefault(m[1], []).append(line)
    assert set(commits) == {"pv_done", "item_done"}
    # a block's last product: the softmax of every CTA waits for it at its item's end
    assert any(re.search(r"wait\(&c\.pv_done\[\(g - 1\) & 1\]", line) for line in lines)
    # an item's: the next item's key loads wait for it, so it is committed only where there is a next item
    waits = [line for line in lines if re.search(r"wait_phase\(&c\.item_done,", line)]
    assert len(waits) == 1
    assert all("i + ncl < pieces" in line for line in commits["item_done"])
