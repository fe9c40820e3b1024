"""Waits in the CUDA sources.

A bounded wait that ran out ends its role.  A role keeps the outcome of its waits in `ok`.  Where the next wait overwrites it before anything has looked at it, a role whose
first wait ran out goes on as if it had not (a completed phase answers yes whatever has happened elsewhere).

A CTA stores into the shared memory of its cluster's others only when all of them are known to have started.
"""
import os
import re

import pytest

import rotated_codebook_quantized_gb300 as tq

CSRC = os.path.join(os.path.dirname(tq.__file__), "csrc")


def _lost(source):
    """Lines whose outcome of a wait is assigned to `ok` and assigned over by the next statement that names it."""
    text = re.sub(r"//[^\n]*", "", source)
    uses = list(re.finditer(r"\bok\b(?P<set>\s*=(?!=))?", text))
    lost = []
    for use, after in zip(uses, uses[1:]):
        end = text.index(";", use.end())
        # (the next use in the text; the other branch of the same condition does not run behind this one)
        if use["set"] and "_wait" in text[use.end():end] and after["set"] and "} else {" not in text[end:after.start()]:
            lost.append(text.count("\n", 0, use.start()) + 1)
    return lost


def test_a_lost_outcome_is_found():
    assert _lost("ok = mbar_wait(a);\nfor (;;) {\n ok = mbar_wait(b);\n if (!ok) break;\n}") == [1]
    assert _lost("ok = mbar_wait(a);\nif (!ok) break;\nok = mbar_wait(b);\nreturn ok;") == []
    assert _lost("if (x) {\n ok = mbar_wait(a);\n} else {\n ok = mbar_wait(b);\n}\nif (!ok) break;") == []
    assert _lost("ok = mbar_wait(a);\nfor (; i < n && ok; ++i) ok = mbar_wait(b) && mbar_wait(c);\nreturn ok;") == []


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_the_outcome_of_a_wait_is_looked_at(name):
    assert _lost(open(os.path.join(CSRC, name)).read()) == []


def test_a_cluster_has_started_before_its_shared_memory_is_written():
    """In the verification kernel an arrival and a wait that every thread passes, on any road through it, come before the first store."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "verify.cu")).read())
    body = text[text.index("verify_tree_kernel(const __grid_constant__"):]
    body = body[body.index("{"):body.index("store_remote(")]
    depth, unconditional = 0, []
    for part in re.finditer(r"[{}]|\bcluster_(?:arrive|wait|sync)\(\);|\breturn\b", body):
        if part[0] in "{}":
            depth += 1 if part[0] == "{" else -1
        elif depth == 1:
            unconditional.append(part[0])
    assert unconditional in (["cluster_arrive();", "cluster_wait();"], ["cluster_sync();"])
