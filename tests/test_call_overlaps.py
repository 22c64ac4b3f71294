"""Outputs that lie over inputs or over each other, where kernels would read what others of their CTAs have written:
refused on the host, nothing is launched."""

import ctypes

import pytest

from test_pages_host import FAKE, _select, compact, fork, free, reserve, sv   # noqa: F401

SHAPE = -2
MB = 1 << 20


@pytest.mark.parametrize("over", [
    dict(granted=FAKE + MB), dict(granted=FAKE + MB + 396), dict(granted=FAKE + 2 * MB - 4),
    dict(granted=FAKE + 2 * MB + 28)])
def test_reserve(sv, over):   # noqa: F811
    """refs: 400 bytes; the table: 32."""
    assert reserve(sv, refs=FAKE + MB, table=FAKE + 2 * MB, lens=FAKE + 3 * MB, **over) == SHAPE


@pytest.mark.parametrize("at", [0, 4, -4])
def test_free(sv, at):   # noqa: F811
    assert free(sv, lens=FAKE + MB, ended=FAKE + MB + at) == SHAPE


@pytest.mark.parametrize("over", [
    dict(out=FAKE + 5 * MB), dict(out=FAKE + 5 * MB - 44), dict(out=FAKE + 4 * MB + 8), dict(lens_out=FAKE + 4 * MB - 8),
    dict(out=FAKE + MB + 384), dict(lens_out=FAKE + MB), dict(out=FAKE + 3 * MB), dict(lens_out=FAKE + 2 * MB + 28),
    dict(lens_out=FAKE + 6 * MB + 44)])
def test_fork(sv, over):   # noqa: F811
    apart = dict(refs=FAKE + MB, table=FAKE + 2 * MB, lens=FAKE + 3 * MB, parents=FAKE + 4 * MB, lens_out=FAKE + 5 * MB,
                 out=FAKE + 6 * MB)
    assert fork(sv, **{**apart, **over}) == SHAPE


@pytest.mark.parametrize("over", [
    dict(map=FAKE + MB), dict(map=FAKE + MB + 396), dict(live=FAKE + MB + 396), dict(live=FAKE + 3 * MB + 396),
    dict(map=FAKE + 2 * MB + 28), dict(live=FAKE + 2 * MB)])
def test_compact(sv, over):   # noqa: F811
    apart = dict(refs=FAKE + MB, table=FAKE + 2 * MB, map=FAKE + 3 * MB, live=FAKE + 4 * MB)
    assert compact(sv, **{**apart, **over}) == SHAPE


@pytest.mark.parametrize("over", [
    dict(tokens=FAKE + MB), dict(out=FAKE + MB + 15996), dict(parents=FAKE + 4 * MB), dict(out=FAKE + 4 * MB + 60),
    dict(tokens=FAKE + 6 * MB - 60)])
def test_select(sv, over):   # noqa: F811
    """logits: 16000 bytes; the outputs: 64 each."""
    apart = dict(logits=FAKE + MB, scores=FAKE + 2 * MB, tokens=FAKE + 4 * MB, parents=FAKE + 5 * MB, out=FAKE + 6 * MB)
    assert _select(sv, **{**apart, "ws": FAKE + 8, **over}) == sv.SPEC_ERR_ALIGN
    assert _select(sv, **{**apart, **over}) == SHAPE


@pytest.mark.parametrize("at", [0, 12, -255])
def test_reorder_over_parents(sv, at):   # noqa: F811
    states = (sv.SpecState * 1)((FAKE, FAKE + MB + at, 64))
    assert sv.load_library().spec_beam_reorder(ctypes.cast(states, ctypes.POINTER(sv.SpecState)), 1, FAKE + MB, 4, 4,
                                               FAKE + 2 * MB, None) == SHAPE
