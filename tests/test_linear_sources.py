"""Rules of the chunked linear attention kernel that no run shows to be broken: a barrier whose phases can complete
twice before a role has waited for the first leaves that role waiting for a third."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_13_gb300", "csrc")
TEXT = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "linear_kernel.cuh")).read())


def test_the_store_warp_waits_stage_by_stage():
    """The output's warps may be two chunks ahead of a slow store, but not in one stage: it is loaded again
    only when the store has released it.  So each stage has its own barrier."""
    store = TEXT[TEXT.index("warp == C::W_STORE"):]
    store = store[:store.index("} else if (warp < 8)")]
    assert "w.wait(&sm.stage_full[n % C::NV], (n / C::NV) & 1" in store
    assert store.index("bulk_wait_read()") < store.index("mbar_arrive(&sm.v_empty[n % C::NV])")
    assert "mbar_arrive(&sm.stage_full[n % C::NV])" in TEXT and "stage_full[C::NV]" in TEXT


def test_named_barriers_are_reached_by_all_or_none():
    """A warp that gives up still comes to the next named barrier of its group (they count threads and have no limit):
    no early return stands between a failed wait and the barrier, and what follows it leaves together."""
    for name, ident in (("auto weights = [&](int n) -> bool {", "named_bar_or(2 + wq, 64, !ok)"),
                        ("auto state = [&](int n) -> bool {", "named_bar_or(1, 256, !ok)")):
        body = TEXT[TEXT.index(name):]
        before = body[:body.index(ident)]
        assert re.findall(r"return[^;]*;", before) in ([], ["return false;"]), name
        if "return false;" in before:
            assert "if (BF16 && !ok) return false;" in before
        after = body[body.index(ident):]
        assert re.match(r"named_bar_or\([^;]*;", after) and "if (!ok) return false;" in after[:900], name
    assert TEXT.count("named_bar") == 2
