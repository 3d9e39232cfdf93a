"""What the kernels promise of their reads and no run shows, looked up in their
sources."""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "draft_token_markov_gb300", "csrc")


def _body(name, begin, end):
    """A source's text between the first occurrences of two lines' beginnings."""
    text = open(os.path.join(CSRC, name)).read()
    at = text.index(begin)
    return text[at:text.index(end, at)]


def test_logits_of_a_row_that_is_left_out_are_not_read():
    """A read of memory that need not be there: the kernel leaves before any of its
    loads of logits."""
    body = _body("logprobs.cu", "uint4 x[kTurn], y[kTurn];", " the stream\n")
    leave = body.index("if (token64 < 0 || token64 >= a.vocab) return;")
    assert leave < body.index("load(x, 0)") and "load" not in body[:leave].replace("before the first load", "")
