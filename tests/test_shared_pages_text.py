"""What a call writes belongs to one sequence of it: the header and the binding say so wherever pages may be shared."""

import os
import re

import quantized_weight_q4_gb300 as q4

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "q4.h")


def text_of(name):
    """The comment of an entry point, on one line."""
    with open(HEADER) as f:
        s = f.read()
    at = s.index(" * %s -- " % name)
    return re.sub(r"\s*\n \*\s*", " ", s[at:s.index("*/", at)])


def test_pages_that_are_written():
    with open(HEADER) as f:
        s = re.sub(r"\s*\n \*\s*", " ", f.read())
    assert "a page whose tokens a call writes (appends, moves, weighs) belongs to one sequence of that call" in s


def test_weights_of_a_shared_page_are_refused():
    said = text_of("q4_kv_weigh")
    assert "where two sequences of a call list one page" in said and "undefined" in said
    assert "calls of their own" in said and "calls of their own" in q4.q4_kv_weigh.__doc__


def test_moving_within_shared_pages_is_refused():
    assert "then belong to one sequence" in text_of("q4_kv_compact")
