"""The count of finished CTAs (kCtrlDone) that the losses and the gradient norm share: a launch leaves it at zero
only when every CTA that counts does so, also one whose waits ran out.  Each place that counts is found in the
sources, with the conditions around it; the count is then run over launches of which CTAs fail."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "overlapped_tensor_gemm_gb300", "csrc")
SOURCES = ["fo_loss_rows.cu", "fo_loss.cu", "fo_adamw.cu"]


def _conditions(text, at):
    """Conditions of the `if`s whose braces or single statements hold position `at`, inside its kernel."""
    found, depth, i = [], 0, at
    while i > 0:
        i -= 1
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth:
                depth -= 1
                continue
            head = text[max(text.rfind(c, 0, i) for c in ";{}") + 1:i]
            if "__global__" in head or "loss_rows_kernel" in head or "extern __shared__" in head:
                break
            m = re.search(r"\bif (?:constexpr )?\((.*)\)\s*$", head, re.S)
            if m:
                found.append(m.group(1))
    line = text[text.rfind("\n", 0, text.rfind("\n", 0, at)) + 1:at]
    m = re.search(r"\bif \((.*?)\)\s", line)
    return found + ([m.group(1)] if m else [])


def _counts(source):
    with open(os.path.join(CSRC, source)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return text, [m.start() for m in re.finditer(r"atomicInc\(a\.ctrl \+ kCtrlDone", text)]


@pytest.mark.parametrize("source", SOURCES)
def test_what_a_count_depends_on(source):
    """Which CTA, warp or lane it is, and the kind of launch: never how the CTA's waits went."""
    text, places = _counts(source)
    assert len(places) == 1
    conditions = _conditions(text, places[0])
    assert conditions
    for c in conditions:
        names = set(re.findall(r"[A-Za-z_]\w*", c))
        assert names <= {"kMode", "kLossPolicy", "rank", "lane", "warp", "threadIdx", "x"}, c


def _launch(word, teams, counts):
    """(the word behind a launch, how many CTAs took themselves for the last): atomicInc wraps at teams - 1"""
    lasts = 0
    for team in range(teams):
        if counts(team):
            lasts += word == teams - 1
            word = 0 if word >= teams - 1 else word + 1
    return word, lasts


@pytest.mark.parametrize("teams,failed", [(1, {0}), (5, {2}), (152, {0, 7, 151}), (4, {0, 1, 2, 3})])
def test_a_launch_of_which_some_fail(teams, failed):
    """Counted always, the next launch of another size finds its last CTA; left out, it does not."""
    word, lasts = _launch(0, teams, lambda t: True)
    assert lasts == 1 and _launch(word, 608, lambda t: True) == (0, 1)
    word, _ = _launch(0, teams, lambda t: t not in failed)
    assert word == (teams - len(failed)) % teams
    if word:
        assert _launch(word, 608, lambda t: True) != (0, 1)
