"""CPU checks of the library's status word: its refusals, and that a device
that is not there is an error, not an address."""

import ctypes

import pytest

from learned_optimizer_step_gb300 import build as B

torch = pytest.importorskip("torch")

from learned_optimizer_step_gb300 import train_ops as ops   # noqa: E402


def test_refusals():
    B.build()
    assert ops._load()["lopt_status_word"](None) == -1
    assert ops._load()["lopt_status_take"](None) == -1


@pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")
def test_without_a_device():
    B.build()
    word, flags = ctypes.c_void_p(), ctypes.c_int32(7)
    assert ops._load()["lopt_status_word"](word) == -4 and not word.value
    assert ops._load()["lopt_status_take"](flags) == -4 and flags.value == 0
