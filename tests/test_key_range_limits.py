"""Sizes and windows that do not fit the library's 32-bit arguments are refused,
not cut to their low 32 bits."""
import ctypes

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk


@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(Nk=2 ** 32 + 4), dict(Nq=2 ** 32 + 4),
                                dict(B=2 ** 32 + 1), dict(Nk=2 ** 31)])
def test_sizes_beyond_32_bits_are_refused(kw):
    with pytest.raises(ValueError, match="32"):
        sk.key_ranges(**{**dict(B=1, Nq=4, Nk=4, device="cuda"), **kw})


def test_abi_refuses_more_rows_than_a_launch_counts():
    P = ctypes.c_void_p
    args = (P(0),) * 4 + (0, 0) + (P(256),) * 3 + (P(0),)
    for Nq in (2 ** 31 - 1, 2 ** 31 - 255):
        assert sk.load().streamkl_key_ranges(1, Nq, 4, 1, 0, *args) == sk.ERR_UNSUPPORTED


@pytest.mark.gpu
def test_the_widest_window_is_the_causal_mask():
    want = sk.key_ranges(2, 300, 400, "cuda")
    for window in (2 ** 31 - 1, 400, torch.tensor(400)):
        got = sk.key_ranges(2, 300, 400, "cuda", window=window)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide = sk.key_ranges(1, 5, 2 ** 31 - 1, "cuda", window=3)
    assert wide[1].tolist() == [[2 ** 31 - 1 - 4 + i for i in range(5)]] and (wide[1] - wide[0]).tolist() == [[3] * 5]
