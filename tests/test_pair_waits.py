"""What the pair's kernel (paged_pair.cu) hands from one CTA to the other goes by
arrivals and waits at cluster scope.  By default both are of the CTA's scope:
nothing then orders what was written in one CTA before what the other's issuer
starts on it."""
import os
import re

from fp4_kv_cache_sparse_gb300 import build as lib_build


def source():
    text = open(os.path.join(lib_build.CSRC, "paged_pair.cu")).read()
    return re.sub(r"//[^\n]*", "", text)


def function(text, name):
    at = re.search(r"\bvoid %s\(" % name, text).start()
    return text[at:text.index("\n}", at)]


def across(text):
    """The barriers that the other CTA's arrivals, or products over both CTAs, complete."""
    return set(re.findall(r"(?:arrive_at|hand_at|release_at)\((?:lead|other)\(L::(b\w+)", text)) | set(
        re.findall(r"commit_both\(bar\(L::(b\w+)", text))


def test_arrivals_across_the_pair_are_of_cluster_scope():
    text = source()
    remote = re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster\.b64 _", text)
    assert remote
    for form in remote:
        assert re.match(r"mbarrier\.arrive\.(relaxed|release)\.cluster\.shared::cluster", form), form
    # What lies in shared memory goes behind a release; only tensor memory, ordered by its own fences, without.
    assert "fence.release.sync_restrict::shared::cta.cluster" in function(text, "hand_at")
    assert set(re.findall(r"\barrive_at\(lead\(L::(b\w+)", text)) == {"bKFull", "bSFree", "bOFree"}
    assert not re.search(r"\barrive_at\(other\(", text)


def test_waits_for_the_other_cta_are_of_cluster_scope():
    text = source()
    there = across(text)
    assert {"bKFull", "bVFull", "bPFull", "bQFull", "bSFull", "bKFree", "bVFree", "bPFree", "bVote", "bXchg"} <= there
    near = set(re.findall(r"\bwait\((?:own \? )?L::(b\w+)", text)) | set(re.findall(r": L::(b\w+) \+ slot,", text))
    assert near and not near & there
    assert there - {"bDrain"} <= set(re.findall(r"\bwait2\(L::(b\w+)", text))


def block(text, at):
    """From a brace to the one that closes it."""
    at = text.index("{", at)
    depth, end = 1, at + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at:end]


def test_nobody_follows_barriers_that_do_not_wait_for_them():
    """A wait by phase parity cannot tell a phase from the one two before, so who follows a barrier from item to item has
    to hold it up: scores of an item are not written again before the softmax warps have arrived, and nobody else has.
    The second CTA's warp that issues nothing there followed them too: held up for two items, it ran out of its wait."""
    text = source()
    # The score issuer's role: all of its waits are the first CTA's.
    role = block(text, text.index("warp == kScoreWarp) {"))
    lead = block(role, role.index("if (c == 0)"))
    assert "wait2(L::bSFree" in lead
    assert not re.search(r"\b(wait2?|drain_at)\(", role.replace(lead, ""))
    # The end of all products is a barrier of one phase; both CTAs wait for it once their softmax warps are through.
    assert text.count("drain_at(bar(L::bDrain)") == 1
    roles_end = text.rindex("named_bar_sync(1, kSoftmaxThreads);")
    assert text.index("__syncthreads();", roles_end) < text.index("drain_at(bar(L::bDrain)")
