"""Workspaces and refusals at the far ends of the cross entropy's and the
orthogonalised step's arguments.  Host side only: these run without a GPU."""
import pytest

pytest.importorskip("rank_gradient_compression_amd")
from rank_gradient_compression_amd import binding as B  # noqa: E402
from test_ends_abi import MB, matrix, opts, table, xent  # noqa: E402


@pytest.mark.parametrize("vocab", [1, 5, 32000, 2000000])
def test_scoring_many_tokens_needs_no_more_than_a_block(vocab):
    """Sums of 64 words each for a block of tokens, not for all of them."""
    some = B.psgd_xent_workspace(xent(tokens=1 << 23, vocab=vocab), False)
    many = B.psgd_xent_workspace(xent(tokens=(1 << 31) - 1, vocab=vocab), False)
    assert some == many < (1 << 30) + (1 << 26)


def test_the_workspace_query_refuses_what_the_call_refuses():
    far = xent(ldw=2000008, vocab=2, w=1 << 40)  # (read in place: its row stride is too large)
    for train in (False, True):
        with pytest.raises(B.PsgdError, match="in place") as e:
            B.psgd_xent_workspace(far, train)
        assert e.value.status == B.PSGD_ERR_INVALID_ARG


def test_a_decay_that_is_no_number_is_refused():
    both = opts(lr=1e30, weight_decay=1e30)
    for fn, args in ((B.psgd_muon_workspace, ()), (B.psgd_muon_step, (64 * MB, 1 << 30))):
        with pytest.raises(B.PsgdError, match="weight_decay") as e:
            fn(table(matrix()), both, *args)
        assert e.value.status == B.PSGD_ERR_INVALID_ARG


def test_gradients_that_are_not_wanted_take_no_memory():
    many = dict(tokens=100000, vocab=64, dim=32, ldx=32)
    ask = lambda train=True, **kw: B.psgd_xent_workspace(xent(**many, **kw), train)  # noqa: E731
    copy = 100000 * 64 * 2  # (x's rows, padded, of 16 bits: what dw's product takes)
    assert copy <= ask() - ask(dw=0) <= copy + 256
    assert ask(dx=0, dw=0) == ask(False)


@pytest.mark.parametrize("args,match", [
    ((MB, 3, 8, 2 * MB, 3 * MB), "type"), ((MB, 0, -1, 2 * MB, 3 * MB), "number"), ((MB, 0, 1 << 43, 2 * MB, 3 * MB), "number"),
    ((0, 0, 8, 2 * MB, 3 * MB), "NULL"), ((MB, 0, 8, 0, 3 * MB), "NULL"), ((MB, 0, 8, 2 * MB, 0), "NULL"),
    ((MB + 1, 1, 8, 2 * MB, 3 * MB), "aligned"), ((MB, 0, 8, 2 * MB + 2, 3 * MB), "aligned"),
    ((MB, 0, 8, 2 * MB, 3 * MB + 2), "aligned"), ((MB, 0, 8, 2 * MB, MB + 16), "overlaps"),
    ((MB, 0, 8, MB + 4, MB), "overlaps"),
])
def test_scale_refused(args, match):
    with pytest.raises(B.PsgdError, match=match) as e:
        B.psgd_xent_scale(*args)
    assert e.value.status == B.PSGD_ERR_INVALID_ARG


@pytest.mark.parametrize("args,match", [
    ((MB, 2 * MB, -1, 0, True, 3 * MB), "tokens"), ((MB, 2 * MB, 1 << 31, 0, True, 3 * MB), "tokens"),
    ((0, 2 * MB, 5, 0, True, 3 * MB), "NULL"), ((MB, 0, 5, 0, True, 3 * MB), "NULL"), ((MB, 0, 0, 0, True, 0), "NULL"),
    ((MB + 2, 0, 5, 0, False, 3 * MB), "aligned"), ((MB, 2 * MB + 4, 5, 0, True, 3 * MB), "aligned"),
    ((MB, 0, 5, 0, False, 3 * MB + 1), "aligned"), ((MB, 0, 5, 0, False, MB + 16), "overlaps"),
    ((MB, 2 * MB, 5, 0, True, 2 * MB + 36), "overlaps"),
])
def test_total_refused(args, match):
    with pytest.raises(B.PsgdError, match=match) as e:
        B.psgd_xent_total(*args, 64 * MB, 4096)
    assert e.value.status == B.PSGD_ERR_INVALID_ARG


def test_total_workspace_refused():
    for ws, n in ((0, 4096), (64 * MB + 128, 4096), (64 * MB, 4095)):
        with pytest.raises(B.PsgdError, match="workspace") as e:
            B.psgd_xent_total(MB, 2 * MB, 5, 0, True, 3 * MB, ws, n)
        assert e.value.status == B.PSGD_ERR_WORKSPACE
    with pytest.raises(B.PsgdError, match="overlaps"):
        B.psgd_xent_total(MB, 2 * MB, 5, 0, True, 3 * MB, MB, 4096)
