"""Branches in inline assembly.  The compiler does not see which lanes take them, and a
`.uni` one is undefined where the warp's lanes disagree, as they may on what mbarrier.try_wait
gives each of them: so a `.uni` branch goes by a vote of the whole warp, and a lane's own
result is never a counter in place of what it has seen."""
import glob
import os
import re

import pytest

from weight_rnn_gb300 import build as wbuild

FILES = sorted(glob.glob(os.path.join(wbuild.CSRC, "*.cu")) + glob.glob(os.path.join(wbuild.CSRC, "*.cuh")))
BLOCK = re.compile(r"\basm\b(?:\s+volatile)?\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)")


def instructions(text):
    """each inline assembly's instructions"""
    for m in BLOCK.finditer(text):
        body = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))
        yield [i.strip() for i in re.split(r"\\n|\\t|;|\{|\}", body) if i.strip()]


def unvoted(code):
    """guards of .uni branches that something other than a vote writes"""
    bad = []
    for line in code:
        m = re.match(r"@!?(\S+)\s+bra\.uni\b", line)
        if m:
            writers = [i for i in code if re.match(rf"(?:@\S+\s+)?[a-z][\w.:]*\s+{re.escape(m.group(1))}\b", i)]
            if not writers or not all(re.match(r"(?:@\S+\s+)?vote\.sync", i) for i in writers):
                bad.append(line)
    return bad


def test_the_check_itself():
    lane = ["mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2", "@p bra.uni DONE", "DONE:"]
    voted = lane[:1] + ["vote.sync.all.pred a, p, 0xffffffff", "@a bra.uni DONE"]
    assert unvoted(lane) == ["@p bra.uni DONE"] and unvoted(voted) == []
    assert list(instructions('asm volatile(\n "{\\n\\t.reg .pred p;\\n\\t"\n "a.b p;\\n\\t}" : "=r"(x));')) == [[".reg .pred p", "a.b p"]]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_uniform_branches_go_by_a_vote(path):
    with open(path) as f:
        text = f.read()
    for code in instructions(text):
        assert not unvoted(code)
