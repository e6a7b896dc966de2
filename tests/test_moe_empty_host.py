"""CPU tests of what the expert operators refuse where there are no tokens or no
rows: a tensor without elements has no address, which says nothing then."""
import pytest

from test_moe_host import NULLPTR, OK, P, combine, combine_bwd, gather, gather_bwd, sort


def test_gather_of_no_tokens():
    none = dict(tokens=0, x=0, row_of=0, weight=0)
    assert gather(**none) == OK and gather(**none, prob=None) == OK
    assert gather(**none, y_dtype="e4m3", scale=P) == OK
    assert gather(**none, y=0) == NULLPTR and gather(**none, expert_rows=0) == NULLPTR
    assert gather(**none, y_dtype="e4m3") == NULLPTR and gather(**none, scale=P) == NULLPTR
    assert gather(weight=0) == NULLPTR                      # of tokens


@pytest.mark.parametrize("tokens", [0, 7])
def test_gather_into_no_rows(tokens):
    some = dict(tokens=tokens, m=0, y=0, prob=0)
    assert gather(**some) == OK and gather(**some, weight=None) == OK
    assert gather(**some, y_dtype="e4m3") == OK and gather(**some, y_dtype="e4m3", scale=P) == OK
    assert gather(**some, scale=P) == NULLPTR
    assert gather(prob=0) == NULLPTR


def test_gather_bwd_of_no_tokens():
    none = dict(tokens=0, row_of=0, dx=0)
    assert gather_bwd(**none, dweight=0) == OK and gather_bwd(**none, dweight=0, dprob=None) == OK
    assert gather_bwd(tokens=0, row_of=0, dx=0, dweight=0, dy=None, dprob=None, m=0) == OK
    assert gather_bwd(dx=0, dweight=0) == NULLPTR and gather_bwd(dweight=0) == NULLPTR


def test_gather_bwd_of_no_rows():
    """Every pair is without a row: zeros."""
    assert gather_bwd(m=0, dy=0, dprob=0) == OK and gather_bwd(m=0, dy=0, dprob=0, dx=None) == OK
    assert gather_bwd(m=0, dy=0, dprob=0, dweight=None) == OK
    assert gather_bwd(dprob=0) == NULLPTR


def test_combine_bwd_of_no_tokens_or_rows():
    assert combine_bwd(tokens=0, dout=0, row_of=0, weight=0, dweight=0) == OK
    assert combine_bwd(tokens=0, dout=0, row_of=0, weight=0, dweight=0, dy=None, y=None) == OK
    assert combine_bwd(m=0, y=0, dy=0) == OK and combine_bwd(m=0, y=0, dy=0, dweight=None) == OK
    assert combine_bwd(tokens=0, m=0, dout=0, row_of=0, weight=0, y=0, dy=0, dweight=0) == OK
    assert combine_bwd(dy=0, dweight=0) == NULLPTR


def test_the_others_of_no_tokens():
    assert sort(tokens=0, m=0, expert=0, row_of=0, pair_of=0, workspace=0) == OK
    assert combine(tokens=0, m=0, y=0, row_of=0, weight=0, out=0) == OK
