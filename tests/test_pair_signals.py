"""Order between the CTAs of the 4-bit decode's clusters, by the source: a signal on
whose strength another CTA reads memory that threads have stored must be a release
at cluster scope or the completion of an asynchronous store or bulk copy, which is
one.  (A missing release shows in no result that a run could be asked for.)
"""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "mla_latent_decode_gb300", "csrc", "mla_tc_fp4.cu")


def body(text, name):
    """The function `name`, from its name to the end of its block."""
    at = text.index(f" {name}(")
    i = text.index("{", at)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[at:j + 1]
    raise AssertionError(name)


def code():
    return re.sub(r"//[^\n]*", "", open(SRC).read())


def test_stored_operands_are_published():
    made, p, corrected = (body(code(), f) for f in ("relay_made", "relay_o", "correct_and_store"))
    for f in (made, p, corrected):
        assert ".relaxed." not in f and "signal_leader" not in f
    # the fence to the async proxy stands between the wait and the store that signals
    assert made.index("mbar_test_wait") < made.index("fence_proxy_async_smem") < made.index("st_async_u32")
    assert "mbar_arrive_cluster" in p and "arrive_leader" in corrected


def test_relaxed_arrives_report_reads_only():
    """One relaxed arrive is left, in signal_leader, whose one caller has read TMEM."""
    text = code()
    assert text.count(".relaxed.") == 1 and ".relaxed." in body(text, "signal_leader")
    callers = re.findall(r"signal_leader\(smem_u32\(&s\.(\w+)", text)
    assert callers == ["sempty"]
