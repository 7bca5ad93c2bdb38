"""A team's exchange, read in the source (no GPU needed).  The CTAs of a cluster send
their maps into each other's shared memory by st.async, whose arrival at the reader's
mbarrier releases at cluster scope.  The reader has to acquire at cluster scope too; a
wait of the default (CTA) scope gives no order between the sender's data and the reads
after it, although it may return the right values on a given run."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_attn_b200", "csrc")


def source(name):
    return open(os.path.join(CSRC, name)).read()


def function(text, name):
    """The text of the first definition of `name`, from its template line to its closing brace."""
    at = text.index(f" {name}(")
    return text[text.rindex("\n}\n", 0, at) + 2:text.index("\n}\n", at)]


def test_waits_have_a_form_that_acquires_at_cluster_scope():
    text = source("device.cuh")
    for name, op in (("mbar_try_wait", "try_wait"), ("mbar_test", "test_wait")):
        body = function(text, name)
        assert "template <bool CLUSTER = false>" in body
        yes, no = body.split("if constexpr (CLUSTER)")[1].split("else\n")
        assert f"mbarrier.{op}.parity.acquire.cluster.shared::cta.b64" in yes
        assert f"mbarrier.{op}.parity.shared::cta.b64" in no
    # the bounded waits pass their scope on to every test they make
    for name in ("mbar_wait_for", "mbar_wait", "mbar_drain"):
        body = function(text, name)
        calls = re.findall(r"\b(mbar_(?:try_wait|test|wait_for))(<CLUSTER>)?\(bar", body)
        assert calls and all(scope for _, scope in calls), (name, calls)


def test_messages_of_the_cluster_are_waited_for_at_cluster_scope():
    text = source("scan.cuh")
    waits = re.findall(r"\bwait\(std::(true|false)_type\{\}, &(\w+)\[", text)
    assert len(waits) == len(re.findall(r"[^_]\bwait\((?=[^\[])", text)) >= 2, waits
    assert all((scope == "true") == (bar == "heard") for scope, bar in waits)
    assert {bar for _, bar in waits} == {"heard", "full"}
    assert "mbar_wait<C>(" in text and "mbar_drain<C>(" in text
    assert not re.search(r"mbar_(wait|drain|try_wait|test)\(", text)
