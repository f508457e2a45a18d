"""The example's arguments (no GPU)."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def arguments():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_loop
    return decode_loop.arguments


@pytest.mark.parametrize("argv,want", [([], (4, 2)), (["--sequences", "8"], (8, 2)), (["--sequences", "9"], (9, 1)),
                                       (["--sequences", "16"], (16, 1)), (["--sequences", "2", "--samples", "8"], (2, 8))])
def test_samples_fit_the_sequences(arguments, argv, want):
    a = arguments(argv)
    assert (a.sequences, a.samples) == want


@pytest.mark.parametrize("argv", [["--sequences", "17"], ["--sequences", "0"], ["--sequences", "9", "--samples", "2"], ["--samples", "0"]])
def test_what_does_not_fit_is_refused(arguments, argv, capsys):
    with pytest.raises(SystemExit):
        arguments(argv)
    assert "samples in all" in capsys.readouterr().err
